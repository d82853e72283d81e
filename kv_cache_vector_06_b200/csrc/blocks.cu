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

// max_c over a box: max(q_c lower_c, q_c upper_c) = min(q_c, 0) lower_c + max(q_c, 0) upper_c.
//
// bf16: a step's scores are two products over d, one with each half of the query, on the tensor cores.
// Lane: chunk 4 kg + lane % 4 of heads lane / 4 (+ 8).
template <typename T, int D, bool WIDE>
struct Scorer {
  using S = Shape<T, D>;
  static constexpr int kH = WIDE ? 2 : 1, kKg = S::kCh / 4, kT = S::kTok / 8;
  static constexpr bool kQInRegs = kKg * kH <= 16;
  uint32_t q[kQInRegs ? kKg : 1][2][kH][4];

  static __device__ __forceinline__ int chunk(int row, int ch) { return key_chunk(row, ch); }
  __device__ __forceinline__ void halves(uint32_t (&f)[2][kH][4], const uint4 (&v)[kH]) {
#pragma unroll
    for (int x = 0; x < kH; ++x) {
      const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const __nv_bfloat162 p = reinterpret_cast<const __nv_bfloat162 &>(w[y]), z = __floats2bfloat162_rn(0.f, 0.f);
        const __nv_bfloat162 lo = __hmin2(p, z), hi = __hmax2(p, z);
        f[0][x][y] = reinterpret_cast<const uint32_t &>(lo);
        f[1][x][y] = reinterpret_cast<const uint32_t &>(hi);
      }
    }
  }
  uint4 raw[kQInRegs ? kKg : 1][kH];
  __device__ __forceinline__ void ask(const BlockScoreArgs &a, int64_t row, int lane) {
    if constexpr (kQInRegs) {
#pragma unroll
      for (int kg = 0; kg < kKg; ++kg) load_q<T, kH>(raw[kg], a.q, row, a.group, a.d, kg, lane);
    }
  }
  __device__ __forceinline__ void prepare() {
    if constexpr (kQInRegs) {
#pragma unroll
      for (int kg = 0; kg < kKg; ++kg) halves(q[kg], raw[kg]);
    }
  }
  // The score of block `k` of the step, in the lanes that have one (k >= 0).
  __device__ __forceinline__ float step(const BlockScoreArgs &a, int64_t row, unsigned lower, unsigned upper, int lane, int &k) {
    const int c = lane & 3, r = lane >> 2;
    // chunk 4 kg + c of block r lies at at[kg & 1] + 128 (kg / 2): key_chunk swaps the groups of odd rows
    const unsigned at[2] = {(unsigned)(r * S::kRow + 16 * key_chunk(r, c)), (unsigned)(r * S::kRow + 16 * key_chunk(r, 4 + c))};
    float s[2][kT][4];
#pragma unroll
    for (int x = 0; x < 8 * kT; ++x) s[x / (4 * kT)][x / 4 % kT][x % 4] = 0.f;
#pragma unroll
    for (int kg = 0; kg < kKg; ++kg) {
      if constexpr (!kQInRegs) {
        load_q<T, kH>(raw[0], a.q, row, a.group, a.d, kg, lane);
        halves(q[0], raw[0]);
      }
#pragma unroll
      for (int up = 0; up < 2; ++up) {
        const auto &g = q[kQInRegs ? kg : 0][up];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          uint32_t x[4];
          lds128(x, (up ? upper : lower) + at[kg & 1] + 8 * t * S::kRow + 128 * (kg >> 1));
#pragma unroll
          for (int u = 0; u < 2; ++u)
            mma_bf16(s[up][t], g[0][2 * u], WIDE ? g[kH - 1][2 * u] : 0u, g[0][2 * u + 1], WIDE ? g[kH - 1][2 * u + 1] : 0u,
                     x[2 * u], x[2 * u + 1]);
        }
      }
    }
    // the largest over the heads: lane holds heads r (and 8 + r) of blocks 8 t + 2 c, 8 t + 2 c + 1
    float mine = -INFINITY;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float v = r < a.group ? s[0][t][x] + s[1][t][x] : -INFINITY;
        if (WIDE && r + 8 < a.group) v = fmaxf(v, s[0][t][2 + x] + s[1][t][2 + x]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(TQ_FULL_MASK, v, o));
        if (r == 2 * t + x) mine = v;
      }
    k = r < 2 * kT ? 8 * (r >> 1) + 2 * c + (r & 1) : -1;
    return mine;
  }
};

// fp32: on the CUDA cores, where a term is a select and a multiply-add.  (TF32 parts on the tensor cores took
// 1.4 times the instructions for 4 heads, and a tensor core cuts each sum that it returns: these sums
// grow from term to term, and were 1.2e-6 off instead of 4e-8.)  A row of D / 4 lanes holds four channels
// (D = 256: twice four) of every head; four heads at a time, the lanes' sums over a step's 8 blocks are
// exchanged until each lane has one whole sum.
template <int D, bool WIDE>
struct Scorer<float, D, WIDE> {
  using S = Shape<float, D>;
  static constexpr int kLanes = D == 64 ? 16 : 32;  // lanes of a row
  static constexpr int kAt = 32 / kLanes;           // blocks at once
  static constexpr int kEach = 8 / kAt;             // blocks of a lane, of eight
  static constexpr int kVec = D == 256 ? 2 : 1;
  static constexpr int kHeads = WIDE ? 16 : 8;
  static constexpr bool kQInRegs = kHeads * kVec <= 16;  // else four heads at a time, from the cache
  float4 q[kQInRegs ? kHeads : 4][kVec];

  static __device__ __forceinline__ int chunk(int, int ch) { return ch; }
  __device__ __forceinline__ void load(const BlockScoreArgs &a, int64_t row, int h0, int lane) {
#pragma unroll
    for (int h = 0; h < (kQInRegs ? kHeads : 4); ++h)
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int ch = lane % kLanes + 32 * v;
        q[h][v] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (h0 + h < a.group && 4 * ch < a.d)
          q[h][v] = *(reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + (row * a.group + h0 + h) * a.d) + ch);
      }
  }
  __device__ __forceinline__ void ask(const BlockScoreArgs &a, int64_t row, int lane) {
    if constexpr (kQInRegs) load(a, row, 0, lane);
  }
  __device__ __forceinline__ void prepare() {}
  static __device__ __forceinline__ float pick(float x, float lo, float hi, float s) { return fmaf(x, x >= 0.f ? hi : lo, s); }
  __device__ __forceinline__ float step(const BlockScoreArgs &a, int64_t row, unsigned lower, unsigned upper, int lane, int &k) {
    const int v = lane % kLanes;
    float mine = -INFINITY;
    for (int half = 0; half < S::kTok / 8; ++half, lower += 8 * S::kRow, upper += 8 * S::kRow) {
      const float x = eight(a, row, lower, upper, lane);
      if (v / kEach == half) mine = x;
    }
    k = v < kEach * (S::kTok / 8) ? 8 * (v / kEach) + lane / kLanes + kAt * (v % kEach) : -1;
    return mine;
  }
  // The score of block lane / kLanes + kAt (v % kEach) of eight.
  __device__ __forceinline__ float eight(const BlockScoreArgs &a, int64_t row, unsigned lower, unsigned upper, int lane) {
    const int v = lane % kLanes;
    float best = -INFINITY;
#pragma unroll
    for (int h0 = 0; h0 < kHeads; h0 += 4) {
      if (h0 >= a.group) break;
      if constexpr (!kQInRegs) load(a, row, h0, lane);
      float s[4 * kEach];  // [head][block]
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kVec; ++w) {
          uint32_t l[4], u[4];
          lds128(l, lower + i * kAt * S::kRow + 16 * (lane + 32 * w));
          lds128(u, upper + i * kAt * S::kRow + 16 * (lane + 32 * w));
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float4 x = q[(kQInRegs ? h0 : 0) + h][w];
            t[h] = pick(x.x, __uint_as_float(l[0]), __uint_as_float(u[0]), t[h]);
            t[h] = pick(x.y, __uint_as_float(l[1]), __uint_as_float(u[1]), t[h]);
            t[h] = pick(x.z, __uint_as_float(l[2]), __uint_as_float(u[2]), t[h]);
            t[h] = pick(x.w, __uint_as_float(l[3]), __uint_as_float(u[3]), t[h]);
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) s[h * kEach + i] = t[h];
      }
      // lane v of a row ends with the sum over the row's lanes of s[v]
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const bool high = lane & o;
          const float give = high ? s[i] : s[i + o], keep = high ? s[i + o] : s[i];
          s[i] = keep + __shfl_xor_sync(TQ_FULL_MASK, give, o);
        }
      float x = h0 + v / kEach < a.group ? s[0] : -INFINITY;
#pragma unroll
      for (int o = kEach; o < kLanes; o <<= 1) x = fmaxf(x, __shfl_xor_sync(TQ_FULL_MASK, x, o));
      best = fmaxf(best, x);
    }
    return best;
  }
};

// Bound: 2 d values per block, read once for the whole group: HBM.  The loads and the division of the work
// are those of the paged attention, a step being kTok blocks; every warp works alone.  4 x 128K tokens x 8
// heads of 128 channels in 16-token blocks, bf16 (134 MB): 26.5 us, about 6 of them before the first and after the
// last bounds; a ragged fp32 batch (557 MB): 95 us, 5.8 TB/s.
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(Shape<T, D>::kThreads, Shape<T, D>::kOcc) block_scores_kernel(BlockScoreArgs a) {
  using S = Shape<T, D>;
  using Sc = Scorer<T, D, WIDE>;
  constexpr int kWarps = S::kWarps;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Place place[kWarps];
  __shared__ uint32_t masks[kWarps][S::kStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  StepScan<kWarps> scan;
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
  Sc scorer;

  for (int64_t pos = begin; pos < end;) {
    const int64_t span = min(steps + kRowCost - unit, end - pos);
    const int first = (int)max(unit - kRowCost, (int64_t)0), n = (int)max(unit + span - kRowCost, (int64_t)0) - first;
    const int64_t row = (int64_t)b * a.heads + h;
    const int32_t *table = a.table + (int64_t)b * a.max_blocks;
    auto entry = [&](int i) {
      const int j = (first + i) * S::kTok + (lane & (S::kTok - 1));
      return i < n && j < held ? table[j] : -1;
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
        const int bytes = ((valid >> k) & 1u) && ch < dch ? 16 : 0;
        const char *src = static_cast<const char *>(a.bounds) + (__shfl_sync(TQ_FULL_MASK, off, k) + 16 * min(ch, dch - 1));
        cp16(lb + k * S::kRow + 16 * Sc::chunk(k, ch), src, bytes);
        cp16(ub + k * S::kRow + 16 * Sc::chunk(k, ch), src + row_bytes, bytes);
      }
    };
    int e[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) e[i] = entry(i);
    scorer.ask(a, row, lane);  // before the bounds, so that it does not queue behind them
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
      if (i < n) issue(i, e[i]);
      cp_commit();
    }
    int next = e[S::kStages - 1];
    scorer.prepare();
    for (int i = 0; i < n; ++i) {
      cp_wait<S::kStages - 2>();
      __syncwarp();  // this step's copies of every lane have landed; the last step's stage is free
      if (i + S::kStages - 1 < n) issue(i + S::kStages - 1, next);
      cp_commit();
      next = entry(i + S::kStages);
      const int stage = i % S::kStages;
      const unsigned lb = ring + stage * S::kStage;
      int k;
      const float s = scorer.step(a, row, lb, lb + S::kTok * S::kRow, lane, k);
      const int j = (first + i) * S::kTok + k;
      if (k >= 0 && j < a.max_blocks) a.out[row * a.max_blocks + j] = (masks[warp][stage] >> k) & 1u ? s : -INFINITY;
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
  const int64_t want = ((int64_t)a.batch * a.heads * ((a.max_blocks - 1) / S::kTok + 1) + S::kWarps - 1) / S::kWarps;
  const int64_t most = (int64_t)S::kOcc * tq_device_sms(device);
  tq_prof_begin(TQK_BLOCK_SCORES, st);
  e = tq_launch_dependent(kern, dim3((unsigned)(want < most ? want : most)), S::kThreads, S::kSmem, st, a);
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

constexpr int kSelectList = 2048;  // keys of one leading digit that are put aside

// A float's order as an unsigned integer: larger floats have larger keys, -0 and +0 the same one, and
// NaN the key of -infinity.  Never 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f != f ? -INFINITY : f + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums of two counts (each below 2^16 per block) over the block's threads, and their totals.
template <int THREADS>
__device__ __forceinline__ void block_scan(int a, int b, int &ea, int &eb, int &ta, int &tb) {
  __shared__ uint32_t w[THREADS / 32];
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
  for (int i = 0; i < THREADS / 32; ++i) {
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

// The 2048 counts of `hist`, largest digit first, cut where `need` of them are passed: the digit, and how many
// of its keys are still needed; true if that is all of them.  Leaves the counts at zero.
template <int THREADS>
__device__ __forceinline__ bool cut_digit(int *hist, int need, int &digit, int &rest) {
  __shared__ int wsum[THREADS / 32];
  __shared__ int found, left, held;
  constexpr int kPer = 2048 / THREADS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, top = 2047 - kPer * threadIdx.x;
  int cnt[kPer], sum = 0;  // from the thread's largest digit down
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    int2 *mine = reinterpret_cast<int2 *>(hist + top - 1 - i);
    const int2 v = *mine;
    *mine = make_int2(0, 0);
    cnt[i] = v.y;
    cnt[i + 1] = v.x;
    sum += v.x + v.y;
  }
  int s = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(TQ_FULL_MASK, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  int before = s - sum;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i)
    if (i < warp) before += wsum[i];
  int r = need - before;
  if (r > 0 && r <= sum) {
    int i = 0;
#pragma unroll
    for (int x = 0; x < kPer - 1; ++x)
      if (i == x && r > cnt[x]) {
        r -= cnt[x];
        ++i;
      }
    found = top - i;
    left = r;
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      if (i == x) held = cnt[x];
  }
  __syncthreads();
  digit = found;
  rest = left;
  return left == held;
}

// One block per (sequence, KV head).  Radix selection: the key of the last block chosen is found from
// counts of its digits (11, 11 and 10 bits), the leading one over all keys; the keys that share it are then
// put aside, and the other digits are found among those.  What block_scores_kernel returns lies within a power of
// two or so (200 .. 280 over 8192 blocks of normal keys, where 600 to 8000 keys share that digit, 4700 in the middle
// row; 590 of up to 2048 on a ragged batch), normally distributed scores spread (140; 50).  One
// pass in index order writes the blocks above that key and the first ones at it.  Each thread holds PER
// consecutive keys, so that index order is thread order; rows longer than a block's PER * THREADS keys go
// through in chunks, read again for each pass, and so do those where a digit's keys outgrow the list.
// Latency bounds it: a dozen barriers and scans, so a table takes as few threads as hold its keys (64 sequences x
// 8 heads of 64 .. 2048 blocks: 8.7 us per call in a row of calls with 256 threads, 10.8 with 512, 12.2 with
// 128; 32 rows of 8192: 8.0 with 512, 9.6 with 1024; 16 rows of 16383: 13 with 1024, 24 with 512 in two chunks).
// These are times on normally distributed scores; on scores of blocks the ragged batch takes 9.2 us instead of 8.0, and 32
// rows of 8192, whose digits outgrow the list, 9.9 instead of 8.5.
// A digit whose keys are all taken ends the search (8.7 -> 8.1 us).  The next kernel is let in late: its
// waiting blocks crowd this one's onto fewer SMs (11.1 us).
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) select_blocks_kernel(SelectArgs a) {
  constexpr int kChunk = PER * THREADS;
  __shared__ __align__(16) int hist[2048];
  __shared__ uint32_t list[kSelectList];
  __shared__ int listed;
#pragma unroll
  for (int i = 0; i < 2048 / THREADS; ++i) hist[threadIdx.x + i * THREADS] = 0;
  if (threadIdx.x == 0) listed = 0;
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
  for (int i = kept + threadIdx.x; i < a.keep; i += THREADS) out[i] = -1;
  auto store = [&](int i, int j) {
    const int e = table[j];
    out[i] = e >= 0 && e < a.n_blocks ? e * a.heads + h : -1;
  };
  if (n <= a.keep) {
    for (int j = threadIdx.x; j < n; j += THREADS) store(j, j);
    return;
  }
  const int lo = a.first, hi = n - a.last;  // candidates [lo, hi); the others are always chosen
  uint32_t k[PER];
  const int off = (int)((reinterpret_cast<uintptr_t>(scores) >> 2) & 3);  // the row's place in its 16 bytes
  auto load = [&](int j0) {  // keys of blocks j0 + PER * thread ..; 0 outside the candidates, below every key
    const int j = j0 + PER * threadIdx.x;
    if (j + PER + (off ? 4 : 0) <= n) {
      // whole 16-byte loads from the row's aligned start on, shifted
      float f[PER + 4];
#pragma unroll
      for (int i = 0; i < PER + 4; i += 4) {
        if (i == PER && off == 0) break;
        const float4 v = *(reinterpret_cast<const float4 *>(scores - off + j + i));
        f[i] = v.x;
        f[i + 1] = v.y;
        f[i + 2] = v.z;
        f[i + 3] = v.w;
      }
      if (off == 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) k[i] = order_key(f[i]);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) k[i] = order_key(off == 1 ? f[i + 1] : off == 2 ? f[i + 2] : f[i + 3]);
      }
      if (j < lo || j + PER > hi) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (j + i < lo || j + i >= hi) k[i] = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) k[i] = j + i >= lo && j + i < hi ? order_key(scores[j + i]) : 0;
    }
  };
  const bool once = n <= kChunk;
  if (once) load(0);
  __syncthreads();  // the counts are zero
  uint32_t key = 0xffffffffu;  // above every key, where only the forced blocks are kept
  int equal = 0;               // blocks at exactly `key` to take, the first ones
  const int need = a.keep - a.first - a.last;
  if (need > 0) {
    int digit;
    for (int j0 = 0; j0 < n; j0 += kChunk) {
      if (!once) load(j0);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (k[i] != 0) atomicAdd(&hist[k[i] >> 21], 1);
    }
    __syncthreads();
    bool whole = cut_digit<THREADS>(hist, need, digit, equal);  // all keys of the digit: no further one is needed
    key = (uint32_t)digit << 21;
    if (!whole) {
      for (int j0 = 0; j0 < n; j0 += kChunk) {
        if (!once) load(j0);
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (k[i] != 0 && (k[i] ^ key) < (1u << 21)) {
            const int at = atomicAdd(&listed, 1);
            if (at < kSelectList) list[at] = k[i];
          }
      }
      __syncthreads();
      const int count = listed;
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        const int shift = pass ? 0 : 10, above = pass ? 10 : 21;
        const uint32_t mask = pass ? 1023u : 2047u;
        if (count <= kSelectList) {
          for (int i = threadIdx.x; i < count; i += THREADS)
            if (((list[i] ^ key) >> above) == 0) atomicAdd(&hist[(list[i] >> shift) & mask], 1);
        } else {
          for (int j0 = 0; j0 < n; j0 += kChunk) {
            if (!once) load(j0);
#pragma unroll
            for (int i = 0; i < PER; ++i)
              if (k[i] != 0 && ((k[i] ^ key) >> above) == 0) atomicAdd(&hist[(k[i] >> shift) & mask], 1);
          }
        }
        __syncthreads();
        whole = cut_digit<THREADS>(hist, equal, digit, equal);
        key |= (uint32_t)digit << shift;
        if (whole) break;
      }
    }
    if (whole) {  // every key from here on
      --key;
      equal = 0;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  int at = 0, seen = 0;  // blocks written, blocks at `key` passed, before this chunk
  for (int j0 = 0; j0 < n; j0 += kChunk) {
    if (!once) load(j0);
    const int j = j0 + PER * threadIdx.x;
    uint32_t above = 0, ties = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      above |= (k[i] > key ? 1u : 0u) << i;
      ties |= (k[i] == key ? 1u : 0u) << i;
    }
    if (j < lo || j + PER > hi) {  // the forced ones
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (j + i < n && (j + i < lo || j + i >= hi)) above |= 1u << i;
    }
    int ea, eb, ta, tb;
    block_scan<THREADS>(__popc(above), __popc(ties), ea, eb, ta, tb);
    // of the row's ties the first `equal` are taken: so many of this thread's
    const int first = seen + eb;
    int p = at + ea + min(first, equal) - min(seen, equal);
    int room = max(equal - first, 0);
    while (ties) {
      const uint32_t bit = ties & (0u - ties);
      if (room-- > 0) above |= bit;
      ties ^= bit;
    }
    while (above) {
      store(p++, j + __ffs(above) - 1);
      above &= above - 1;
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
  const int n = pages->max_blocks;
  const cudaError_t e = n <= 512    ? tq_launch_dependent(select_blocks_kernel<128, 4>, dim3(grid), 128, 0, s, a)
                        : n <= 2048 ? tq_launch_dependent(select_blocks_kernel<256, 8>, dim3(grid), 256, 0, s, a)
                        : n <= 8192 ? tq_launch_dependent(select_blocks_kernel<512, 16>, dim3(grid), 512, 0, s, a)
                                    : tq_launch_dependent(select_blocks_kernel<1024, 16>, dim3(grid), 1024, 0, s, a);
  tq_prof_end(TQK_SELECT_BLOCKS, s);
  return tq_cuda_check(e, "block selection launch");
}
