// Paged-cache bookkeeping: block tables, lengths and slot maps from request lengths
// (tq_page_extend), and the append of uncompressed rows with the channel bounds of every block's
// keys (tq_append_kv).
#include "device_common.cuh"

tq_status tq_check_pages(const tq_pages *p) {
  tq_fail(TQ_OK, "%s", "");
  if (!p) return tq_fail(TQ_EINVAL, "pages is NULL");
  if (p->batch < 0 || p->n_kv_heads <= 0 || p->block_size <= 0 || p->max_blocks <= 0 || p->n_blocks < 0)
    return tq_fail(TQ_EINVAL, "pages: batch=%d n_kv_heads=%d block_size=%d max_blocks=%d n_blocks=%lld", p->batch,
                   p->n_kv_heads, p->block_size, p->max_blocks, (long long)p->n_blocks);
  if (p->batch > 0 && !p->block_table) return tq_fail(TQ_EINVAL, "pages: block_table is NULL");
  if (!tq_aligned(p->block_table, 4)) return tq_fail(TQ_EINVAL, "pages: block_table not 4-byte aligned");
  if ((int64_t)p->batch * p->n_kv_heads > INT32_MAX || p->n_blocks > INT32_MAX / p->n_kv_heads ||
      (int64_t)p->max_blocks * p->block_size > INT32_MAX)
    return tq_fail(TQ_EUNSUPPORTED,
                   "pages: batch * n_kv_heads, n_blocks * n_kv_heads and max_blocks * block_size must be below 2^31");
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

constexpr int kExtendThreads = 1024;

// Exclusive prefix sums of two values over the block's threads; totals in every thread.  Sums are
// int64: lengths are arbitrary int32 values.
__device__ __forceinline__ void block_scan2(int64_t a, int64_t b, int64_t &ea, int64_t &eb, int64_t &ta, int64_t &tb) {
  __shared__ int64_t wa[32], wb[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t sa = a, sb = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ua = __shfl_up_sync(TQ_FULL_MASK, sa, o), ub = __shfl_up_sync(TQ_FULL_MASK, sb, o);
    if (lane >= o) {
      sa += ua;
      sb += ub;
    }
  }
  if (lane == 31) {
    wa[warp] = sa;
    wb[warp] = sb;
  }
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = tb = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) {
      pa += wa[w];
      pb += wb[w];
    }
    ta += wa[w];
    tb += wb[w];
  }
  __syncthreads();
  ea = pa + sa - a;
  eb = pb + sb - b;
}

struct ExtendArgs {
  int batch, heads, bs, max_blocks, n_free;
  int64_t n_blocks, n_rows, n_slots;
  int32_t *table;
  const int32_t *lens, *grow, *free_blocks, *free_head;
  int32_t *lens_out, *granted, *free_head_out;
  int64_t *offsets, *slots;
};

// One block: prefix sums of the new rows and of the needed blocks over the batch, a chunk of
// kExtendThreads sequences at a time.  The needed blocks of a sequence that the free list cannot
// serve stay in the sum, so every later one that needs a block is refused too and the blocks taken
// are a run of the free list.
__global__ void __launch_bounds__(kExtendThreads) page_extend_kernel(ExtendArgs a) {
  int64_t rows0 = 0, need0 = 0;  // sums before this chunk
  int64_t taken = 0;             // blocks granted, this thread's sequences
  const int64_t most = (int64_t)a.max_blocks * a.bs;
  const int64_t head = min(max((int64_t)*a.free_head, (int64_t)0), (int64_t)a.n_free);
  for (int b0 = 0; b0 < a.batch; b0 += kExtendThreads) {
    const int b = b0 + threadIdx.x;
    const bool in = b < a.batch;
    const int64_t len = in ? max(a.lens[b], 0) : 0, add = in ? max(a.grow[b], 0) : 0;
    const int64_t have = (len + a.bs - 1) / a.bs;
    int64_t row, rows_total, upto, need_total;
    // the rows' offsets decide which sequences fit, so they come before the blocks' sum
    int64_t unused, unused_total;
    block_scan2(add, 0, row, unused, rows_total, unused_total);
    row += rows0;
    const bool fits = len + add <= most && row + add <= a.n_rows;
    const int64_t need = in && fits ? (len + add + a.bs - 1) / a.bs - have : 0;
    block_scan2(need, 0, upto, unused, need_total, unused_total);
    upto += need0;
    const bool ok = fits && (need == 0 || head + upto + need <= a.n_free);
    if (in) {
      a.offsets[b] = row;
      a.granted[b] = ok ? (int32_t)add : 0;
      a.lens_out[b] = (int32_t)(ok ? len + add : len);
      if (ok) {
        taken += need;
        for (int64_t i = 0; i < need; ++i)
          a.table[(int64_t)b * a.max_blocks + have + i] = a.free_blocks[head + upto + i];
      }
    }
    rows0 += rows_total;
    need0 += need_total;
  }
  int64_t ea, eb, total, unused;
  block_scan2(taken, 0, ea, eb, total, unused);
  if (threadIdx.x == 0) {
    a.offsets[a.batch] = rows0;
    *a.free_head_out = (int32_t)(head + total);
  }
}

// Last sequence whose rows begin at or before `row` and do not end there (row < offsets[batch]).
__device__ __forceinline__ int row_sequence(const int64_t *offsets, int batch, int64_t row) {
  int lo = 0, hi = batch;  // offsets[lo] <= row < offsets[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void page_slots_kernel(ExtendArgs a) {
  const int64_t end = a.offsets[a.batch];
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < a.n_slots; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / a.heads;
    const int h = (int)(i - row * a.heads);
    int64_t slot = -1;
    if (row < end) {
      const int b = row_sequence(a.offsets, a.batch, row);
      const int add = a.granted[b];
      if (add > 0) {
        const int pos = a.lens_out[b] - add + (int)(row - a.offsets[b]);
        const int e = a.table[(int64_t)b * a.max_blocks + pos / a.bs];
        if (e >= 0 && e < a.n_blocks) slot = ((int64_t)e * a.heads + h) * a.bs + pos % a.bs;
      }
    }
    a.slots[i] = slot;
  }
}

struct AppendArgs {
  int batch, heads, bs, max_blocks, d;
  int64_t n_blocks, n_rows, ld;
  const int32_t *table, *lens, *granted;
  const int64_t *offsets;
  const void *k, *v;
  void *kc, *vc, *bounds;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// One block = one KV head of one touched cache block, a thread per channel.  Work unit u of
// sequence b: u - (offsets[b] / bs + 2 b) is the touched block's number; a sequence of n rows touches
// at most n / bs + 2 blocks, so units of different sequences never meet (a few stay empty).
template <typename T>
__global__ void append_kv_kernel(AppendArgs a) {
  const int64_t u = blockIdx.x;
  const int h = blockIdx.y;
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] / a.bs + 2 * (int64_t)mid <= u) lo = mid;
    else hi = mid;
  }
  const int b = lo;
  const int64_t row0 = a.offsets[b];
  const int add = a.granted[b], len = a.lens[b];
  if (add <= 0 || len < add || len > (int64_t)a.max_blocks * a.bs || row0 + add > a.n_rows) return;
  const int before = len - add;
  const int64_t j = before / a.bs + (u - (row0 / a.bs + 2 * (int64_t)b));
  if (j > (len - 1) / a.bs) return;
  const int e = a.table[(int64_t)b * a.max_blocks + j];
  if (e < 0 || e >= a.n_blocks) return;
  const int64_t t0 = j * a.bs > before ? j * a.bs : before;
  const int64_t t1 = (j + 1) * a.bs < len ? (j + 1) * a.bs : len;
  const int64_t blk = (int64_t)e * a.heads + h;
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    T *bound = a.bounds ? static_cast<T *>(a.bounds) + blk * 2 * a.d : nullptr;
    const bool fresh = j * a.bs >= before;
    T mn{}, mx{};
    if (bound && !fresh) {
      mn = bound[c];
      mx = bound[a.d + c];
    }
    for (int64_t t = t0; t < t1; ++t) {
      const int64_t src = (row0 + (t - before)) * a.ld + (int64_t)h * a.d + c;
      const int64_t dst = (blk * a.bs + (t - j * a.bs)) * a.d + c;
      const T kv = static_cast<const T *>(a.k)[src];
      if (a.kc) {
        static_cast<T *>(a.kc)[dst] = kv;
        static_cast<T *>(a.vc)[dst] = static_cast<const T *>(a.v)[src];
      }
      if (t == t0 && fresh) mn = mx = kv;
      if (to_f(kv) < to_f(mn)) mn = kv;
      if (to_f(kv) > to_f(mx)) mx = kv;
    }
    if (bound) {
      bound[c] = mn;
      bound[a.d + c] = mx;
    }
  }
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
  DeviceScope dev_scope;
  st = dev_scope.enter(pages->device);
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ExtendArgs a{pages->batch, pages->n_kv_heads, pages->block_size, pages->max_blocks, n_free, pages->n_blocks,
               n_slots / pages->n_kv_heads, n_slots, pages->block_table, seq_lens, new_lens, free_blocks, free_head,
               seq_lens_out, granted, free_head_out, row_offsets, new_slots};
  tq_prof_begin(TQK_PAGE_EXTEND, s);
  page_extend_kernel<<<1, kExtendThreads, 0, s>>>(a);
  tq_prof_end(TQK_PAGE_EXTEND, s);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && n_slots > 0) {
    const int64_t want = (n_slots + 255) / 256, most = 16 * (int64_t)tq_sm_count();
    tq_prof_begin(TQK_PAGE_SLOTS, s);
    page_slots_kernel<<<(unsigned)(want < most ? want : most), 256, 0, s>>>(a);
    tq_prof_end(TQK_PAGE_SLOTS, s);
    e = cudaGetLastError();
  }
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
  if (units > INT32_MAX || pages->n_kv_heads > 65535)
    return tq_fail(TQ_EUNSUPPORTED, "n_rows=%lld, n_kv_heads=%d: too many", (long long)n_rows, pages->n_kv_heads);
  DeviceScope dev_scope;
  st = dev_scope.enter(pages->device);
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AppendArgs a{pages->batch, pages->n_kv_heads, pages->block_size, pages->max_blocks, d, pages->n_blocks, n_rows, ld,
               pages->block_table, seq_lens, granted, row_offsets, k_new, v_new, k_cache, v_cache, bounds};
  const dim3 grid((unsigned)units, (unsigned)pages->n_kv_heads);
  tq_prof_begin(TQK_APPEND_KV, s);
  if (dtype == TQ_F32) append_kv_kernel<float><<<grid, 128, 0, s>>>(a);
  else append_kv_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
  tq_prof_end(TQK_APPEND_KV, s);
  return tq_cuda_check(cudaGetLastError(), "append launch");
}
