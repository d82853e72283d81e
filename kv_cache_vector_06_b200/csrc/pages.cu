// Paged-cache bookkeeping: block tables, lengths and slot maps from request lengths
// (tq_page_extend), and the append of uncompressed rows with the channel bounds of every block's
// keys (tq_append_kv).
#include <algorithm>
#include <atomic>

#include "paged_device.cuh"

int tq_device_sms(int device) {
  constexpr int kMax = 64;
  static std::atomic<int> known[kMax];
  if (device >= 0 && device < kMax && known[device].load(std::memory_order_relaxed) > 0) return known[device];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  if (device >= 0 && device < kMax) known[device] = n;
  return n;
}

tq_status tq_check_pages(const tq_pages *p) {
  tq_clear_error();
  if (!p) return tq_fail(TQ_EINVAL, "pages is NULL");
  if (p->batch < 0 || p->n_kv_heads <= 0 || p->block_size <= 0 || p->max_blocks <= 0 || p->n_blocks < 0)
    return tq_fail(TQ_EINVAL, "pages: batch=%d n_kv_heads=%d block_size=%d max_blocks=%d n_blocks=%lld", p->batch,
                   p->n_kv_heads, p->block_size, p->max_blocks, (long long)p->n_blocks);
  if (p->batch > 0 && !p->block_table) return tq_fail(TQ_EINVAL, "pages: block_table is NULL");
  if (!tq_aligned(p->block_table, 4)) return tq_fail(TQ_EINVAL, "pages: block_table not 4-byte aligned");
  if ((int64_t)p->batch * p->n_kv_heads > INT32_MAX || p->n_blocks > INT32_MAX / p->n_kv_heads ||
      (int64_t)p->max_blocks * p->block_size > kPagedMaxTokens || p->n_kv_heads > kPagedMaxHeads)
    return tq_fail(TQ_EUNSUPPORTED,
                   "pages: n_kv_heads up to %d, batch * n_kv_heads and n_blocks * n_kv_heads below 2^31, "
                   "max_blocks * block_size up to 2^30", kPagedMaxHeads);
  return TQ_OK;
}

tq_status tq_check_rows(tq_dtype dtype, int32_t d) {
  if (dtype != TQ_F32 && dtype != TQ_BF16) return tq_fail(TQ_EINVAL, "unknown dtype %d", (int)dtype);
  if (d < 8 || d > kPagedMaxD || d % 8 != 0)
    return tq_fail(TQ_EUNSUPPORTED, "d=%d: must be a multiple of 8 in [8, %d]", d, kPagedMaxD);
  return TQ_OK;
}

tq_status tq_check_group(const tq_pages &p, int32_t n_q_heads) {
  if (n_q_heads <= 0 || n_q_heads % p.n_kv_heads != 0)
    return tq_fail(TQ_EINVAL, "n_q_heads=%d: must be a positive multiple of n_kv_heads=%d", n_q_heads, p.n_kv_heads);
  if (n_q_heads / p.n_kv_heads > kPagedMaxGroup)
    return tq_fail(TQ_EUNSUPPORTED, "%d query heads per KV head: at most %d", n_q_heads / p.n_kv_heads, kPagedMaxGroup);
  return TQ_OK;
}

namespace {

constexpr int kExtendThreads = 256;

// Exclusive prefix sum over the block's threads, and the total.  int64: lengths are any int32 values.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t &total) {
  __shared__ int64_t w[kExtendThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(TQ_FULL_MASK, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) w[warp] = s;
  __syncthreads();
  int64_t p = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kExtendThreads / 32; ++i) {
    const int64_t x = w[i];
    if (i < warp) p += x;
    total += x;
  }
  __syncthreads();
  return p + s - v;
}

struct ExtendArgs {
  int batch, heads, bs, max_blocks, n_free;
  int64_t n_blocks, n_rows, rows_each;  // rows of a block of the grid
  int32_t *table;
  const int32_t *lens, *grow, *free_blocks, *free_head;
  int32_t *lens_out, *granted, *free_head_out;
  int64_t *offsets, *slots;
  FastDiv by_parts, by_bs;  // heads / VEC, block_size
};

// What one sequence of the current chunk needs for its slots.
struct Grown {
  int before;  // tokens held
  int have;    // blocks held
  int at;      // entry of the free list of its first new block
  int ok;
};

// Prefix sums of the new rows and of the needed blocks over the batch, a chunk of kExtendThreads
// sequences at a time.  The needed blocks of a sequence that the free list cannot serve stay in the sum,
// so every later one that needs a block is refused too and the blocks taken are a run of the free list.
//
// SLOTS: this block writes the slots and table entries of its equal share of the rows.  A few tokens per
// sequence take one block that does both halves; for whole prompts every block of a large grid repeats
// the scan and writes its share, 8 bytes per (row, head).  (For 64 sequences a launch that scans and writes the state
// alone takes 5.4 us between two events, no longer than a kernel that does next to nothing, 6.2.)  STATE: the first
// block writes the lengths and counters.  Where a large grid would update them in place, they follow in a launch of their
// own, after every block has read them.
//
// A thread writes the slots of VEC neighbouring heads of a row at once, which differ by a block's tokens, and
// takes four rows per look-up: with one slot per look-up the instructions bound this kernel (64 prompts, 70 MB of
// slots: 49 us, with VEC 33, with four rows and 32-byte stores 18.7; a fill of these bytes takes 12.6).  Where the
// other 6 us go was not found; by the figures above it is not the scan.
template <bool SLOTS, bool STATE, int VEC>
__global__ void __launch_bounds__(kExtendThreads) page_extend_kernel(ExtendArgs a) {
  const bool state = STATE && blockIdx.x == 0;
  __shared__ int64_t first_row[kExtendThreads + 1];
  __shared__ Grown grown[kExtendThreads];
  int64_t rows0 = 0, need0 = 0;  // sums before this chunk
  int64_t taken = 0;             // blocks granted, this thread's sequences
  const int64_t most = (int64_t)a.max_blocks * a.bs;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int64_t head = min(max((int64_t)*a.free_head, (int64_t)0), (int64_t)a.n_free);
  const int64_t lo = min(a.rows_each * blockIdx.x, a.n_rows), hi = min(lo + a.rows_each, a.n_rows);
  for (int b0 = 0; b0 < a.batch; b0 += kExtendThreads) {
    const int b = b0 + threadIdx.x;
    const bool in = b < a.batch;
    const int len = in ? max(a.lens[b], 0) : 0, add = in ? max(a.grow[b], 0) : 0;
    const int have = len > 0 ? a.by_bs(len - 1) + 1 : 0;
    // the rows' offsets decide which sequences fit, so they come before the blocks' sum
    int64_t rows_total, need_total;
    const int64_t row = rows0 + block_scan(add, rows_total);
    const bool fits = (int64_t)len + add <= most && row + add <= a.n_rows;
    const int64_t need = in && fits && add > 0 ? a.by_bs(len + add - 1) + 1 - have : 0;
    const int64_t upto = need0 + block_scan(need, need_total);
    const bool ok = fits && (need == 0 || head + upto + need <= a.n_free);
    if (state && in) {
      a.offsets[b] = row;
      a.granted[b] = ok ? add : 0;
      a.lens_out[b] = ok ? len + add : len;
      if (ok) taken += need;
    }
    if (SLOTS && rows0 < hi && rows0 + rows_total > lo) {
      const int count = min(kExtendThreads, a.batch - b0);
      first_row[threadIdx.x] = row;
      if (threadIdx.x == 0) first_row[count] = rows0 + rows_total;
      // a sequence that is not grown is never asked for its other values
      grown[threadIdx.x] = Grown{len, have, (int)(ok ? head + upto : 0), ok && add > 0};
      __syncthreads();
      const int64_t r0 = max(lo, rows0), r1 = min(hi, rows0 + rows_total);
      // rows x heads stays below 2^31 in a pass of this many rows
      const int parts = a.heads / VEC;
      const int64_t pass = max((int64_t)1, (int64_t)(1 << 30) / parts);
      for (int64_t p0 = r0; p0 < r1; p0 += pass) {
        const int n = (int)(min(r1, p0 + pass) - p0) * parts;
        // entry of a sequence's block j, and the slots of heads h .. h + VEC - 1 of token `off` of that block
        auto entry_of = [&](const Grown &g, const int32_t *table, int j) {
          return !g.ok ? -1 : j >= g.have ? a.free_blocks[g.at + (j - g.have)] : table[j];
        };
        auto slots_of = [&](const Grown &g, int32_t *table, int j, int off, int h, int64_t *to, int e) {
          if (off == 0 && h == 0 && g.ok && j >= g.have) table[j] = e;  // a new block begins with a new row
          const bool in = e >= 0 && e < a.n_blocks;
          const int64_t slot = in ? (int64_t)(e * a.heads + h) * a.bs + off : -1, step = in ? a.bs : 0;
          if constexpr (VEC == 1) {
            *to = slot;
          } else if constexpr (VEC == 2) {
            *reinterpret_cast<longlong2 *>(to) = make_longlong2(slot, slot + step);
          } else {
            asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};\n" ::"l"(to), "l"(slot), "l"(slot + step), "l"(slot + 2 * step),
                         "l"(slot + 3 * step)
                         : "memory");
          }
        };
        auto find = [&](int64_t r) {  // first_row[u] <= r < first_row[u + 1]
          int u = 0, v = count;
          while (v - u > 1) {
            const int mid = (u + v) >> 1;
            if (first_row[mid] <= r) u = mid;
            else v = mid;
          }
          return u;
        };
        // where prompts are long, each sequence in turn, a thread keeping its heads and taking four rows at a
        // time, mostly of one block, whose entry is asked for one turn ahead; else a search for each row
        const int s0 = find(p0), s1 = find(min(r1, p0 + pass) - 1), at_once = kExtendThreads / parts;
        if (at_once > 0 && s1 - s0 < n / (4 * kExtendThreads)) {
          const int sub = a.by_parts(threadIdx.x), h = (threadIdx.x - sub * parts) * VEC;
          for (int s = s0; s <= s1 && sub < at_once; ++s) {
            const int64_t s_lo = first_row[s], from = max(s_lo, p0);
            const int rows = (int)(min(first_row[s + 1], min(r1, p0 + pass)) - from);
            const Grown g = grown[s];
            const int pos = g.before + (int)(from - s_lo);
            int32_t *table = a.table + (int64_t)(b0 + s) * a.max_blocks;
            int64_t *to = a.slots + ((from + 4 * sub) * a.heads + h);
            int j = a.by_bs(pos + 4 * sub), next = 4 * sub < rows ? entry_of(g, table, j) : -1;
            for (int i = 4 * sub; i < rows; i += 4 * at_once) {
              int e = next, now = j, off = pos + i - j * a.bs;
              j = a.by_bs(pos + i + 4 * at_once);
              if (i + 4 * at_once < rows) next = entry_of(g, table, j);
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                if (i + x >= rows) break;
                if (off == a.bs) {
                  off = 0;
                  e = entry_of(g, table, ++now);
                }
                slots_of(g, table, now, off++, h, to + x * a.heads, e);
              }
              to += (int64_t)4 * at_once * a.heads;
            }
          }
        } else {
          for (int i = threadIdx.x; i < n; i += kExtendThreads) {
            const int k = a.by_parts(i), s = find(p0 + k), h = (i - k * parts) * VEC;
            const Grown g = grown[s];
            const int pos = g.before + (int)(p0 + k - first_row[s]), j = a.by_bs(pos);
            int32_t *table = a.table + (int64_t)(b0 + s) * a.max_blocks;
            slots_of(g, table, j, pos - j * a.bs, h, a.slots + ((p0 + k) * a.heads + h), entry_of(g, table, j));
          }
        }
      }
      __syncthreads();
    }
    rows0 += rows_total;
    need0 += need_total;
  }
  if (SLOTS)  // behind the last sequence
    for (int64_t i = max(lo, rows0) * a.heads + threadIdx.x; i < hi * a.heads; i += kExtendThreads) a.slots[i] = -1;
  if (state) {
    int64_t total;
    block_scan(taken, total);
    if (threadIdx.x == 0) {
      a.offsets[a.batch] = rows0;
      *a.free_head_out = (int32_t)(head + total);
    }
  }
}

// Slots, in units of VEC, up to which one block does the whole call.
constexpr int64_t kExtendOneBlock = 2048;
constexpr int kExtendBlocksPerSm = 4;

struct AppendArgs {
  int batch, heads, bs, max_blocks, d, per_warp;
  int64_t n_blocks, n_rows, ld, units;
  const int32_t *table, *lens, *granted;
  const int64_t *offsets;
  const void *k, *v;
  void *kc, *vc, *bounds;
};

// Channel minimum and maximum of 16-byte chunks, exact in the rows' own type.
template <typename T>
__device__ __forceinline__ void widen(uint4 &mn, uint4 &mx, const uint4 &v);
template <>
__device__ __forceinline__ void widen<float>(uint4 &mn, uint4 &mx, const uint4 &v) {
  const float *x = reinterpret_cast<const float *>(&v);
  float *l = reinterpret_cast<float *>(&mn), *u = reinterpret_cast<float *>(&mx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l[i] = fminf(l[i], x[i]);
    u[i] = fmaxf(u[i], x[i]);
  }
}
template <>
__device__ __forceinline__ void widen<__nv_bfloat16>(uint4 &mn, uint4 &mx, const uint4 &v) {
  const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&v);
  __nv_bfloat162 *l = reinterpret_cast<__nv_bfloat162 *>(&mn), *u = reinterpret_cast<__nv_bfloat162 *>(&mx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l[i] = __hmin2(l[i], x[i]);
    u[i] = __hmax2(u[i], x[i]);
  }
}
__device__ __forceinline__ uint4 shfl4(const uint4 &v, int src) {
  return make_uint4(__shfl_sync(TQ_FULL_MASK, v.x, src), __shfl_sync(TQ_FULL_MASK, v.y, src), __shfl_sync(TQ_FULL_MASK, v.z, src),
                    __shfl_sync(TQ_FULL_MASK, v.w, src));
}
__device__ __forceinline__ uint4 ld_stream(const uint4 *p) { return __ldcs(p); }

constexpr int kAppendWarps = 8, kAppendAhead = 4;
constexpr int64_t kAppendBytes = 16384;

// A copy with a reduction riding along: bound by HBM (4 rows of d in and out per (token, head), and two per
// block).  A warp takes one KV head of one touched block, whose rows lie together in the cache, or per_warp
// heads where these rows are short (finding the block costs as much as 8 KB of copy); the block's warps take
// neighbouring heads, whose rows lie together in the input.  Lanes hold 16-byte chunks,
// 32 / chunks rows at a time, kAppendAhead loads of each array in flight.  4 x 128K tokens x 8 heads of 128 bf16
// channels (4.4 GB in and out): 676 us, 6.56 TB/s.
//
// Work unit u of sequence b: u - (offsets[b] / bs + 2 b) is the touched block's number; a sequence of n
// rows touches at most n / bs + 2 blocks, so units of different sequences never meet (a few stay empty).
template <typename T>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kv_kernel(AppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * (int64_t)kAppendWarps + (threadIdx.x >> 5);
  const int parts = (a.heads + a.per_warp - 1) / a.per_warp;
  const int64_t u = w / parts;
  const int h0 = (int)(w - u * parts) * a.per_warp, h1 = min(h0 + a.per_warp, a.heads);
  if (u >= a.units) return;
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] / a.bs + 2 * (int64_t)mid <= u) lo = mid;
    else hi = mid;
  }
  const int b = lo;
  const int64_t row0 = a.offsets[b];
  const int add = a.granted[b], len = a.lens[b];
  if (add <= 0 || len < add || len > (int64_t)a.max_blocks * a.bs || row0 < 0 || row0 + add > a.n_rows) return;
  const int before = len - add;
  const int64_t nth = u - (row0 / a.bs + 2 * (int64_t)b);
  if (nth < 0) return;  // in front of the first sequence's rows
  const int64_t j = before / a.bs + nth;
  if (j > (len - 1) / a.bs) return;
  const int e = a.table[(int64_t)b * a.max_blocks + j];
  if (e < 0 || e >= a.n_blocks) return;
  const int64_t begin = j * a.bs;  // the block's first token
  const int t0 = begin > before ? 0 : (int)(before - begin);
  const int t1 = begin + a.bs < len ? a.bs : (int)(len - begin);
  const int chunks = a.d * (int)sizeof(T) / 16;
  const int64_t ld = a.ld * (int64_t)sizeof(T) / 16;
  const int at_once = chunks < 32 ? 32 / chunks : 1;  // rows per pass
  const int sub = chunks < 32 ? lane / chunks : 0;
  for (int h = h0; h < h1; ++h) {
    const int64_t blk = (int64_t)e * a.heads + h;
    const uint4 *k = reinterpret_cast<const uint4 *>(a.k) + (row0 - before + begin) * ld + (int64_t)h * chunks;
    const uint4 *v = reinterpret_cast<const uint4 *>(a.v) + (row0 - before + begin) * ld + (int64_t)h * chunks;
    uint4 *kc = reinterpret_cast<uint4 *>(a.kc) + blk * a.bs * chunks, *vc = reinterpret_cast<uint4 *>(a.vc) + blk * a.bs * chunks;
    uint4 *bound = reinterpret_cast<uint4 *>(a.bounds) + blk * 2 * chunks;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const int c = chunks < 32 ? lane - sub * chunks : c0 + lane;
      const bool on = c < chunks && sub < at_once;
      uint4 mn, mx;
      bool any = false;
      for (int t = t0 + sub; on && t < t1; t += kAppendAhead * at_once) {
        uint4 x[kAppendAhead], y[kAppendAhead];
#pragma unroll
        for (int i = 0; i < kAppendAhead; ++i) {
          const int tt = t + i * at_once;
          if (tt < t1) {
            x[i] = ld_stream(k + tt * ld + c);
            if (a.kc) y[i] = ld_stream(v + tt * ld + c);
          }
        }
#pragma unroll
        for (int i = 0; i < kAppendAhead; ++i) {
          const int tt = t + i * at_once;
          if (tt < t1) {
            if (a.kc) {
              kc[(int64_t)tt * chunks + c] = x[i];
              vc[(int64_t)tt * chunks + c] = y[i];
            }
            if (!any) mn = mx = x[i];
            any = true;
            widen<T>(mn, mx, x[i]);
          }
        }
      }
      if (!a.bounds) continue;
      // the rows of one pass lie `chunks` lanes apart; at most t1 - t0 of them hold anything
      const int parts = min(at_once, t1 - t0);
      for (int i = 1; i < parts; ++i) {
        const int src = (c + i * chunks) & 31;
        const uint4 l = shfl4(mn, src), m = shfl4(mx, src);
        uint4 unused = mx;
        if (sub == 0 && on) {
          widen<T>(mn, unused, l);
          unused = mn;
          widen<T>(unused, mx, m);
        }
      }
      if (sub == 0 && on) {
        if (t0 > 0) {  // begun before: its bounds are widened
          const uint4 l = bound[c], m = bound[chunks + c];
          uint4 unused = mx;
          widen<T>(mn, unused, l);
          unused = mn;
          widen<T>(unused, mx, m);
        }
        bound[c] = mn;
        bound[chunks + c] = mx;
      }
    }
  }
}

template <int VEC>
cudaError_t launch_extend(ExtendArgs a, int64_t n_slots, int device, cudaStream_t st) {
  const int64_t want = n_slots <= kExtendOneBlock * VEC ? 1 : n_slots / (4 * VEC * kExtendThreads) + 1;
  const int64_t most = kExtendBlocksPerSm * (int64_t)tq_device_sms(device);
  const unsigned grid = (unsigned)(want < most ? want : most);
  a.rows_each = (a.n_rows + grid - 1) / grid;
  const bool in_place = a.lens_out == a.lens || a.granted == a.grow || a.free_head_out == a.free_head;
  if (want == 1 || !in_place) {
    tq_prof_begin(TQK_PAGE_EXTEND, st);
    const cudaError_t e =
        tq_launch_dependent(page_extend_kernel<true, true, VEC>, dim3(grid), kExtendThreads, 0, st, a);
    tq_prof_end(TQK_PAGE_EXTEND, st);
    return e;
  }
  tq_prof_begin(TQK_PAGE_SLOTS, st);
  cudaError_t e = tq_launch_dependent(page_extend_kernel<true, false, VEC>, dim3(grid), kExtendThreads, 0, st, a);
  tq_prof_end(TQK_PAGE_SLOTS, st);
  if (e != cudaSuccess) return e;
  tq_prof_begin(TQK_PAGE_EXTEND, st);
  e = tq_launch_dependent(page_extend_kernel<false, true, 1>, dim3(1), kExtendThreads, 0, st, a);
  tq_prof_end(TQK_PAGE_EXTEND, st);
  return e;
}

}  // namespace

extern "C" tq_status tq_page_extend(const tq_pages *pages, const int32_t *seq_lens, const int32_t *new_lens,
                                    const int32_t *free_blocks, int32_t n_free, const int32_t *free_head,
                                    int32_t *seq_lens_out, int32_t *granted, int32_t *free_head_out,
                                    int64_t *row_offsets, int64_t *new_slots, int64_t n_slots, void *stream) {
  tq_status st = tq_check_pages(pages);
  if (st != TQ_OK) return st;
  if (n_free < 0 || n_slots < 0) return tq_fail(TQ_EINVAL, "n_free < 0 or n_slots < 0");
  if (n_slots % pages->n_kv_heads != 0)
    return tq_fail(TQ_EINVAL, "n_slots=%lld: must be a multiple of n_kv_heads=%d", (long long)n_slots, pages->n_kv_heads);
  if (pages->batch > 0 && (!seq_lens || !new_lens || !seq_lens_out || !granted))
    return tq_fail(TQ_EINVAL, "seq_lens/new_lens/seq_lens_out/granted is NULL");
  if (!free_head || !free_head_out || !row_offsets || (n_free > 0 && !free_blocks) || (n_slots > 0 && !new_slots))
    return tq_fail(TQ_EINVAL, "free_blocks/free_head/row_offsets/new_slots is NULL");
  if (!tq_aligned(seq_lens, 4) || !tq_aligned(new_lens, 4) || !tq_aligned(seq_lens_out, 4) || !tq_aligned(granted, 4) ||
      !tq_aligned(free_blocks, 4) || !tq_aligned(free_head, 4) || !tq_aligned(free_head_out, 4) ||
      !tq_aligned(row_offsets, 8) || !tq_aligned(new_slots, 8))
    return tq_fail(TQ_EINVAL, "int32 arrays must be 4-byte and int64 arrays 8-byte aligned");
  if (pages->batch > 0 && (seq_lens_out == new_lens || granted == seq_lens || granted == seq_lens_out ||
                           seq_lens_out == free_blocks || granted == free_blocks))
    return tq_fail(TQ_EINVAL, "seq_lens_out may be seq_lens and granted new_lens; no other arrays may be the same");
  DeviceScope dev_scope;
  st = dev_scope.enter(pages->device);
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ExtendArgs a{pages->batch, pages->n_kv_heads, pages->block_size, pages->max_blocks, n_free, pages->n_blocks,
               n_slots / pages->n_kv_heads, 0, pages->block_table, seq_lens, new_lens, free_blocks, free_head,
               seq_lens_out, granted, free_head_out, row_offsets, new_slots, FastDiv(), FastDiv(pages->block_size)};
  const int vec = pages->n_kv_heads % 4 == 0 && tq_aligned(new_slots, 32)   ? 4
                  : pages->n_kv_heads % 2 == 0 && tq_aligned(new_slots, 16) ? 2
                                                                            : 1;
  a.by_parts = FastDiv(pages->n_kv_heads / vec);
  cudaError_t e = vec == 4 ? launch_extend<4>(a, n_slots, pages->device, s) : vec == 2 ? launch_extend<2>(a, n_slots, pages->device, s) : launch_extend<1>(a, n_slots, pages->device, s);
  return tq_cuda_check(e, "page extend launch");
}

extern "C" tq_status tq_append_kv(const tq_pages *pages, const int32_t *seq_lens, const int32_t *granted,
                                  const int64_t *row_offsets, const void *k_new, const void *v_new, tq_dtype dtype,
                                  int32_t d, int64_t n_rows, int64_t ld, void *k_cache, void *v_cache, void *bounds,
                                  void *stream) {
  tq_status st = tq_check_pages(pages);
  if (st != TQ_OK) return st;
  st = tq_check_rows(dtype, d);
  if (st != TQ_OK) return st;
  if (n_rows < 0) return tq_fail(TQ_EINVAL, "n_rows < 0");
  if (!k_cache != !v_cache) return tq_fail(TQ_EINVAL, "k_cache and v_cache must both be given, or neither");
  if (!k_cache && !bounds) return tq_fail(TQ_EINVAL, "nothing to append to: k_cache, v_cache and bounds are NULL");
  if (pages->batch == 0 || n_rows == 0) return TQ_OK;
  if (!seq_lens || !granted || !row_offsets) return tq_fail(TQ_EINVAL, "seq_lens/granted/row_offsets is NULL");
  if (!k_new || (k_cache && !v_new)) return tq_fail(TQ_EINVAL, "k_new/v_new is NULL");
  if (ld < (int64_t)pages->n_kv_heads * d)
    return tq_fail(TQ_EINVAL, "ld=%lld < n_kv_heads * d = %lld", (long long)ld, (long long)pages->n_kv_heads * d);
  const int esz = dtype == TQ_F32 ? 4 : 2;
  if (!tq_aligned(k_new, 16) || !tq_aligned(v_new, 16) || (ld * esz) % 16 != 0)
    return tq_fail(TQ_EINVAL, "k_new/v_new must be 16-byte aligned with a row stride that is a multiple of 16 bytes");
  if (!tq_aligned(k_cache, 16) || !tq_aligned(v_cache, 16) || !tq_aligned(bounds, 16))
    return tq_fail(TQ_EINVAL, "k_cache/v_cache/bounds not 16-byte aligned");
  if (!tq_aligned(seq_lens, 4) || !tq_aligned(granted, 4) || !tq_aligned(row_offsets, 8))
    return tq_fail(TQ_EINVAL, "int32 arrays must be 4-byte and int64 arrays 8-byte aligned");
  const int64_t units = n_rows / pages->block_size + 2 * (int64_t)pages->batch;
  if (units > INT32_MAX / pages->n_kv_heads)
    return tq_fail(TQ_EUNSUPPORTED, "n_rows=%lld, n_kv_heads=%d: too many", (long long)n_rows, pages->n_kv_heads);
  DeviceScope dev_scope;
  st = dev_scope.enter(pages->device);
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t held = (int64_t)pages->block_size * d * esz * (k_cache ? 4 : 2);  // bytes in and out per (block, head)
  const int per_warp = (int)std::max((int64_t)1, std::min((int64_t)pages->n_kv_heads, kAppendBytes / held));
  AppendArgs a{pages->batch, pages->n_kv_heads, pages->block_size, pages->max_blocks, d, per_warp, pages->n_blocks, n_rows, ld,
               units, pages->block_table, seq_lens, granted, row_offsets, k_new, v_new, k_cache, v_cache, bounds};
  const int parts = (pages->n_kv_heads + per_warp - 1) / per_warp;
  const unsigned grid = (unsigned)((units * parts + kAppendWarps - 1) / kAppendWarps);
  tq_prof_begin(TQK_APPEND_KV, s);
  const cudaError_t e = tq_launch_dependent(dtype == TQ_F32 ? append_kv_kernel<float> : append_kv_kernel<__nv_bfloat16>, dim3(grid),
                                            32 * kAppendWarps, 0, s, a);
  tq_prof_end(TQK_APPEND_KV, s);
  return tq_cuda_check(e, "append launch");
}
