// Sparse decode over a paged cache: an upper bound of every block's query-key products
// (tq_block_scores) and the choice of the blocks that each (sequence, KV head) reads
// (tq_select_blocks).
#include "paged_device.cuh"

namespace {

struct BlockScoreArgs {
  int batch, heads, group, bs, max_blocks, d, step_tokens, max_len;
  int64_t n_blocks;
  const int32_t *table, *lens;
  const void *q, *bounds;
  float *out;
};

// Steps that a row costs a warp beside its own: its queries and its first loads.
constexpr int kRowCost = 2;

// max_c over a box: max(q_c lower_c, q_c upper_c) = min(q_c, 0) lower_c + max(q_c, 0) upper_c, so the
// scores of a step's blocks are two products over d, one with each half of the query.  Bound: 2 d values
// per block, read once for the whole group: HBM.  The loads, the operands' layout and the division of the
// work are those of the paged attention, a step being kTok blocks; every warp works alone.
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, Shape<T, D>::kOcc) block_scores_kernel(BlockScoreArgs a) {
  using S = Shape<T, D>;
  constexpr bool kBf = sizeof(T) == 2;
  constexpr int kH = WIDE ? 2 : 1, kParts = kBf ? 1 : 2, kKg = S::kCh / 4, kT = S::kTok / 8;
  constexpr bool kQInRegs = kKg * kH * kParts * 4 <= 64;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Place place[kWarps];
  __shared__ uint32_t masks[kWarps][S::kStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, r = lane >> 2;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  StepScan scan;
  scan.run(a.lens, a.batch, a.heads, a.max_len, a.step_tokens);
  const int64_t workers = min((int64_t)gridDim.x * kWarps, scan.total);
  const Deal deal(scan.total + (int64_t)a.batch * a.heads * kRowCost, workers);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t id = (int64_t)blockIdx.x * kWarps + w;
    if (id < workers) find_unit(scan, deal.begin(id), kRowCost, a.lens, a.max_len, a.step_tokens, place[w]);
  }
  __syncthreads();
  const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
  if (id >= workers) return;
  const int64_t begin = deal.begin(id), end = deal.begin(id + 1);
  int b = place[warp].seq, steps = row_steps(place[warp].len, a.max_len, a.step_tokens);
  int held = held_blocks(place[warp].len, a.bs, a.max_blocks);
  int h = (int)div64(place[warp].unit, steps + kRowCost);
  int64_t unit = place[warp].unit - (int64_t)h * (steps + kRowCost);  // place in the row, its cost in front
  const unsigned ring = smem_addr(smem) + warp * S::kRing;
  const int row_bytes = a.d * (int)sizeof(T), dch = row_bytes / 16;

  for (int64_t pos = begin; pos < end;) {
    const int64_t span = min(steps + kRowCost - unit, end - pos);
    const int first = (int)max(unit - kRowCost, (int64_t)0), n = (int)max(unit + span - kRowCost, (int64_t)0) - first;
    const int64_t row = (int64_t)b * a.heads + h;
    const int32_t *table = a.table + (int64_t)b * a.max_blocks;
    auto entry = [&](int i) {
      const int j = (first + i) * S::kTok + (lane & (S::kTok - 1));
      return i < n && j < held ? __ldg(table + j) : -1;
    };
    auto issue = [&](int i, int e) {
      const int stage = i % S::kStages;
      const bool ok = e >= 0 && e < a.n_blocks;
      const int64_t off = ok ? ((int64_t)e * a.heads + h) * 2 * row_bytes : 0;
      const uint32_t valid = __ballot_sync(TQ_FULL_MASK, ok) & ((1u << S::kTok) - 1u);
      if (lane == 0) masks[warp][stage] = valid;
      const unsigned lb = ring + stage * S::kStage, ub = lb + S::kTok * S::kRow;
#pragma unroll
      for (int x = 0; x < S::kTok * S::kCh / 32; ++x) {
        const int idx = lane + 32 * x, k = idx / S::kCh, ch = idx % S::kCh;
        const int64_t base = __shfl_sync(TQ_FULL_MASK, off, k);
        const bool in = ((valid >> k) & 1u) && ch < dch;
        const char *src = static_cast<const char *>(a.bounds) + (in ? base + 16 * ch : 0);
        cp16(lb + k * S::kRow + 16 * key_chunk(k, ch), src, in ? 16 : 0);
        cp16(ub + k * S::kRow + 16 * key_chunk(k, ch), src + (in ? row_bytes : 0), in ? 16 : 0);
      }
    };
    int e[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) e[i] = entry(i);
    uint4 raw[kQInRegs ? kKg : 1][kH];  // asked for before the bounds, so that it does not queue behind them
    if constexpr (kQInRegs) {
#pragma unroll
      for (int kg = 0; kg < kKg; ++kg) load_q<T, kH>(raw[kg], a.q, row, a.group, a.d, kg, lane);
    }
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
      if (i < n) issue(i, e[i]);
      cp_commit();
    }
    int next = e[S::kStages - 1];
    uint32_t qf[kQInRegs ? kKg : 1][kH][kParts][4];
    if constexpr (kQInRegs) {
#pragma unroll
      for (int kg = 0; kg < kKg; ++kg) make_q<T, kH>(qf[kg], raw[kg]);
    }
    for (int i = 0; i < n; ++i) {
      cp_wait<S::kStages - 2>();
      __syncwarp();  // this step's copies of every lane have landed; the last step's stage is free
      if (i + S::kStages - 1 < n) issue(i + S::kStages - 1, next);
      cp_commit();
      next = entry(i + S::kStages);
      const int stage = i % S::kStages;
      const unsigned lb = ring + stage * S::kStage;
      const uint32_t valid = masks[warp][stage];
      float s[kT][4];
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[t][x] = 0.f;
#pragma unroll
      for (int kg = 0; kg < kKg; ++kg) {
        if constexpr (!kQInRegs) {
          load_q<T, kH>(raw[0], a.q, row, a.group, a.d, kg, lane);
          make_q<T, kH>(qf[0], raw[0]);
        }
        const auto &f = qf[kQInRegs ? kg : 0];
#pragma unroll
        for (int up = 0; up < 2; ++up) {
          // min(q, 0) for the lower bounds, max(q, 0) for the upper ones
          uint32_t g[kH][kParts][4];
#pragma unroll
          for (int x = 0; x < kH; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              if constexpr (kBf) {
                const __nv_bfloat162 w = reinterpret_cast<const __nv_bfloat162 &>(f[x][0][y]), z = __floats2bfloat162_rn(0.f, 0.f);
                const __nv_bfloat162 v = up ? __hmax2(w, z) : __hmin2(w, z);
                g[x][0][y] = reinterpret_cast<const uint32_t &>(v);
              } else {
                const uint32_t neg = (uint32_t)((int32_t)f[x][0][y] >> 31), on = up ? ~neg : neg;
                g[x][0][y] = f[x][0][y] & on;
                g[x][kParts - 1][y] = f[x][kParts - 1][y] & on;
              }
            }
#pragma unroll
          for (int t = 0; t < kT; ++t) {
            uint32_t k[4];
            lds128(k, lb + up * S::kTok * S::kRow + (8 * t + r) * S::kRow + 16 * key_chunk(r, 4 * kg + c));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if constexpr (kBf) {
                mma_bf16(s[t], g[0][0][2 * u], WIDE ? g[kH - 1][0][2 * u] : 0u, g[0][0][2 * u + 1],
                         WIDE ? g[kH - 1][0][2 * u + 1] : 0u, k[2 * u], k[2 * u + 1]);
              } else {
                uint32_t h0, l0, h1, l1;
                split_tf32(k[2 * u], h0, l0);
                split_tf32(k[2 * u + 1], h1, l1);
                if constexpr (WIDE) {
                  mma_tf32(s[t], g[0][kParts - 1][2 * u], g[kH - 1][kParts - 1][2 * u], g[0][kParts - 1][2 * u + 1],
                           g[kH - 1][kParts - 1][2 * u + 1], h0, h1);
                  mma_tf32(s[t], g[0][0][2 * u], g[kH - 1][0][2 * u], g[0][0][2 * u + 1], g[kH - 1][0][2 * u + 1], l0, l1);
                  mma_tf32(s[t], g[0][0][2 * u], g[kH - 1][0][2 * u], g[0][0][2 * u + 1], g[kH - 1][0][2 * u + 1], h0, h1);
                } else {
                  mma_tf32(s[t], g[0][0][2 * u], 0u, g[0][0][2 * u + 1], 0u, l0, l1);
                  mma_tf32(s[t], g[0][0][2 * u], g[0][kParts - 1][2 * u], g[0][0][2 * u + 1], g[0][kParts - 1][2 * u + 1], h0, h1);
                }
              }
            }
          }
        }
      }
      // the largest over the heads: lane holds heads r (and 8 + r) of blocks 8 t + 2 c, 8 t + 2 c + 1
      float mine = -INFINITY;
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float v = r < a.group ? (WIDE || kBf ? s[t][x] : s[t][x] + s[t][2 + x]) : -INFINITY;
          if (WIDE && r + 8 < a.group) v = fmaxf(v, s[t][2 + x]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(TQ_FULL_MASK, v, o));
          if (r == 2 * t + x) mine = v;
        }
      const int k = 8 * (r >> 1) + 2 * c + (r & 1), j = (first + i) * S::kTok + k;
      if (r < 2 * kT && j < a.max_blocks) a.out[row * a.max_blocks + j] = (valid >> k) & 1u ? mine : -INFINITY;
    }
    cp_wait<0>();
    __syncwarp();
    if (n > 0 && first + n == steps)  // behind the row's last step
      for (int64_t j = (int64_t)steps * S::kTok + lane; j < a.max_blocks; j += 32) a.out[row * a.max_blocks + j] = -INFINITY;
    pos += span;
    unit = 0;
    if (pos < end && ++h == a.heads) {
      h = 0;
      ++b;
      steps = row_steps(a.lens[b], a.max_len, a.step_tokens);
      held = held_blocks(a.lens[b], a.bs, a.max_blocks);
    }
  }
}

template <typename T, int D>
cudaError_t launch_scores_d(BlockScoreArgs a, int device, cudaStream_t st) {
  using S = Shape<T, D>;
  const int64_t step = (int64_t)S::kTok * a.bs;
  a.step_tokens = (int)(step < INT32_MAX ? step : INT32_MAX);
  a.max_len = a.max_blocks * a.bs;
  auto kern = a.group > 8 ? block_scores_kernel<T, D, true> : block_scores_kernel<T, D, false>;
  cudaError_t e = tq_smem_limit(reinterpret_cast<const void *>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t want = ((int64_t)a.batch * a.heads * ((a.max_blocks - 1) / S::kTok + 1) + kWarps - 1) / kWarps;
  const int64_t most = (int64_t)S::kOcc * tq_device_sms(device);
  tq_prof_begin(TQK_BLOCK_SCORES, st);
  e = tq_launch_dependent(kern, dim3((unsigned)(want < most ? want : most)), kThreads, S::kSmem, st, a);
  tq_prof_end(TQK_BLOCK_SCORES, st);
  return e;
}

struct SelectArgs {
  int batch, heads, bs, max_blocks, keep, first, last;
  int64_t n_blocks;
  const int32_t *table, *lens;
  const float *scores;
  int32_t *sel_table, *sel_lens;
};

constexpr int kSelectThreads = 512;

// A float's order as an unsigned integer: larger floats have larger keys, -0 and +0 the same one, and
// NaN the key of -infinity.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f != f ? -INFINITY : f + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums of two counts (each below 2^16 per block) over the block's threads, and their totals.
__device__ __forceinline__ void block_scan(int a, int b, int &ea, int &eb, int &ta, int &tb) {
  __shared__ uint32_t w[kSelectThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t v = (uint32_t)a | ((uint32_t)b << 16);
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(TQ_FULL_MASK, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) w[warp] = s;
  __syncthreads();
  uint32_t p = 0, t = 0;
#pragma unroll
  for (int i = 0; i < kSelectThreads / 32; ++i) {
    const uint32_t x = w[i];
    if (i < warp) p += x;
    t += x;
  }
  __syncthreads();
  p += s - v;
  ea = (int)(p & 0xffffu);
  eb = (int)(p >> 16);
  ta = (int)(t & 0xffffu);
  tb = (int)(t >> 16);
}

// One block per (sequence, KV head).  Radix selection: the key of the last block chosen is found
// eight bits at a time from counts of the keys that share the bits found so far; then one pass in
// index order writes the blocks above that key and the first ones at it.  Each thread holds PER
// consecutive keys, so that index order is thread order; rows longer than a block's PER * 512 keys go
// through in chunks, read again for each pass.
template <int PER>
__global__ void __launch_bounds__(kSelectThreads) select_blocks_kernel(SelectArgs a) {
  constexpr int kChunk = PER * kSelectThreads;
  __shared__ int hist[256];
  __shared__ uint32_t found;
  __shared__ int left;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int64_t row = blockIdx.x;
  const int b = (int)(blockIdx.x / (unsigned)a.heads), h = (int)(blockIdx.x - (unsigned)b * (unsigned)a.heads);
  const int len0 = a.lens[b];
  const int n = held_blocks(len0, a.bs, a.max_blocks);
  const int64_t most = (int64_t)n * a.bs;
  const int len = len0 < most ? max(len0, 0) : (int)most;
  const int32_t *table = a.table + (int64_t)b * a.max_blocks;
  int32_t *out = a.sel_table + row * a.keep;
  const float *scores = a.scores + row * a.max_blocks;
  const int kept = n < a.keep ? n : a.keep;
  if (threadIdx.x == 0) a.sel_lens[row] = n > 0 ? (kept - 1) * a.bs + (len - (n - 1) * a.bs) : 0;
  for (int i = kept + threadIdx.x; i < a.keep; i += kSelectThreads) out[i] = -1;
  auto store = [&](int i, int j) {
    const int e = table[j];
    out[i] = e >= 0 && e < a.n_blocks ? e * a.heads + h : -1;
  };
  if (n <= a.keep) {
    for (int j = threadIdx.x; j < n; j += kSelectThreads) store(j, j);
    return;
  }
  const int lo = a.first, hi = n - a.last;  // candidates [lo, hi); the others are always chosen
  uint32_t k[PER];
  auto load = [&](int j0) {  // keys of blocks j0 + PER * thread ..; 0 outside the candidates, below every key
    const int j = j0 + PER * threadIdx.x;
    if ((a.max_blocks & 3) == 0 && j + PER <= n) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(scores + j + i));
        k[i] = order_key(v.x);
        k[i + 1] = order_key(v.y);
        k[i + 2] = order_key(v.z);
        k[i + 3] = order_key(v.w);
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (j + i < lo || j + i >= hi) k[i] = 0;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) k[i] = j + i >= lo && j + i < hi ? order_key(__ldg(scores + j + i)) : 0;
    }
  };
  const bool once = n <= kChunk;
  if (once) load(0);
  uint32_t key = 0xffffffffu;  // above every key, where only the forced blocks are kept
  int equal = 0;               // blocks at exactly `key` to take, the first ones
  int need = a.keep - a.first - a.last;
  if (need > 0) {
    key = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int j0 = 0; j0 < n; j0 += kChunk) {
        if (!once) load(j0);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (k[i] != 0 && (shift == 24 || ((k[i] ^ key) >> ((shift + 8) & 31)) == 0)) atomicAdd(&hist[(k[i] >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x < 32) {  // lane l: digits 255 - 8 l down to 248 - 8 l
        int cnt[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += cnt[i] = hist[255 - 8 * threadIdx.x - i];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(TQ_FULL_MASK, incl, o);
          if ((int)threadIdx.x >= o) incl += u;
        }
        int rest = need - (incl - sum);
        if (rest > 0 && rest <= sum) {
          int i = 0;
#pragma unroll
          for (int x = 0; x < 7; ++x)
            if (i == x && rest > cnt[x]) {
              rest -= cnt[x];
              ++i;
            }
          found = key | ((uint32_t)(255 - 8 * threadIdx.x - i) << shift);
          left = rest;
        }
      }
      __syncthreads();
      key = found;
      need = left;
    }
    equal = need;
  }
  int at = 0, seen = 0;  // blocks written, blocks at `key` passed, before this chunk
  for (int j0 = 0; j0 < n; j0 += kChunk) {
    if (!once) load(j0);
    const int j = j0 + PER * threadIdx.x;
    int above = 0, ties = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool forced = j + i < n && (j + i < lo || j + i >= hi);
      above += forced || k[i] > key;
      ties += k[i] == key;
    }
    int ea, eb, ta, tb;
    block_scan(above, ties, ea, eb, ta, tb);
    // ties before this thread that were taken: the first `equal` of the row
    int t = seen + eb;
    int p = at + ea + min(t, equal) - min(seen, equal);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool forced = j + i < n && (j + i < lo || j + i >= hi);
      const bool tie = k[i] == key;
      if (forced || k[i] > key || (tie && t < equal)) store(p++, j + i);
      t += tie;
    }
    at += ta + min(seen + tb, equal) - min(seen, equal);
    seen += tb;
  }
}

}  // namespace

extern "C" tq_status tq_block_scores(const tq_pages *pages, const int32_t *seq_lens, const void *q, tq_dtype dtype,
                                     int32_t n_q_heads, int32_t d, const void *bounds, float *scores, void *stream) {
  tq_status st = tq_check_pages(pages);
  if (st != TQ_OK) return st;
  st = tq_check_rows(dtype, d);
  if (st != TQ_OK) return st;
  st = tq_check_group(*pages, n_q_heads);
  if (st != TQ_OK) return st;
  if (pages->batch == 0) return TQ_OK;
  if (!seq_lens || !q || !bounds || !scores) return tq_fail(TQ_EINVAL, "seq_lens/q/bounds/scores is NULL");
  if (!tq_aligned(q, 16) || !tq_aligned(bounds, 16) || !tq_aligned(scores, 16))
    return tq_fail(TQ_EINVAL, "q/bounds/scores not 16-byte aligned");
  if (!tq_aligned(seq_lens, 4)) return tq_fail(TQ_EINVAL, "seq_lens not 4-byte aligned");
  DeviceScope dev_scope;
  st = dev_scope.enter(pages->device);
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BlockScoreArgs a{pages->batch, pages->n_kv_heads, n_q_heads / pages->n_kv_heads, pages->block_size, pages->max_blocks,
                   d, 0, 0, pages->n_blocks, pages->block_table, seq_lens, q, bounds, scores};
  cudaError_t e;
  if (dtype == TQ_F32)
    e = d <= 64 ? launch_scores_d<float, 64>(a, pages->device, s) : d <= 128 ? launch_scores_d<float, 128>(a, pages->device, s) : launch_scores_d<float, 256>(a, pages->device, s);
  else
    e = d <= 64    ? launch_scores_d<__nv_bfloat16, 64>(a, pages->device, s)
        : d <= 128 ? launch_scores_d<__nv_bfloat16, 128>(a, pages->device, s)
                   : launch_scores_d<__nv_bfloat16, 256>(a, pages->device, s);
  return tq_cuda_check(e, "block scores launch");
}

extern "C" tq_status tq_select_blocks(const tq_pages *pages, const int32_t *seq_lens, const float *scores,
                                      int32_t n_keep, int32_t n_first, int32_t n_last, int32_t *sel_table,
                                      int32_t *sel_lens, void *stream) {
  tq_status st = tq_check_pages(pages);
  if (st != TQ_OK) return st;
  if (n_keep <= 0 || n_first < 0 || n_last < 1 || n_first > n_keep - n_last)
    return tq_fail(TQ_EINVAL, "n_keep=%d, n_first=%d, n_last=%d: n_first >= 0, n_last >= 1, n_first + n_last <= n_keep",
                   n_keep, n_first, n_last);
  if ((int64_t)n_keep * pages->block_size > INT32_MAX)
    return tq_fail(TQ_EUNSUPPORTED, "n_keep * block_size must be below 2^31");
  if (pages->batch == 0) return TQ_OK;
  if (!seq_lens || !scores || !sel_table || !sel_lens)
    return tq_fail(TQ_EINVAL, "seq_lens/scores/sel_table/sel_lens is NULL");
  if (!tq_aligned(scores, 16)) return tq_fail(TQ_EINVAL, "scores not 16-byte aligned");
  if (!tq_aligned(seq_lens, 4) || !tq_aligned(sel_table, 4) || !tq_aligned(sel_lens, 4))
    return tq_fail(TQ_EINVAL, "int32 arrays must be 4-byte aligned");
  DeviceScope dev_scope;
  st = dev_scope.enter(pages->device);
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  SelectArgs a{pages->batch, pages->n_kv_heads, pages->block_size, pages->max_blocks, n_keep, n_first, n_last,
               pages->n_blocks, pages->block_table, seq_lens, scores, sel_table, sel_lens};
  tq_prof_begin(TQK_SELECT_BLOCKS, s);
  const unsigned grid = (unsigned)(pages->batch * pages->n_kv_heads);
  const cudaError_t e = tq_launch_dependent(pages->max_blocks <= 4 * kSelectThreads ? select_blocks_kernel<4> : select_blocks_kernel<16>,
                                            dim3(grid), kSelectThreads, 0, s, a);
  tq_prof_end(TQK_SELECT_BLOCKS, s);
  return tq_cuda_check(e, "block selection launch");
}
