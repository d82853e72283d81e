// Sparse decode over a paged cache: an upper bound of every block's query-key products
// (tq_block_scores) and the choice of the blocks that each (sequence, KV head) reads
// (tq_select_blocks).
#include "device_common.cuh"

namespace {

struct BlockScoreArgs {
  int batch, heads, group, bs, max_blocks, d;
  int64_t n_blocks;
  const int32_t *table, *lens;
  const void *q, *bounds;
  float *out;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// Blocks that hold a sequence's tokens: ceil(len / bs), with the length clamped to the table.
__device__ __forceinline__ int held_blocks(int len, int bs, int max_blocks) {
  if (len <= 0) return 0;
  const int n = (len - 1) / bs + 1;
  return n < max_blocks ? n : max_blocks;
}

// A warp per (sequence, KV head, block), lanes over the channels.
template <typename T>
__global__ void block_scores_kernel(BlockScoreArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t total = (int64_t)a.batch * a.heads * a.max_blocks;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5); i < total; i += step) {
    const int64_t row = i / a.max_blocks;
    const int j = (int)(i - row * a.max_blocks);
    const int b = (int)(row / a.heads), h = (int)(row - (int64_t)b * a.heads);
    float best = -INFINITY;
    if (j < held_blocks(a.lens[b], a.bs, a.max_blocks)) {
      const int e = a.table[(int64_t)b * a.max_blocks + j];
      if (e >= 0 && e < a.n_blocks) {
        const T *bound = static_cast<const T *>(a.bounds) + ((int64_t)e * a.heads + h) * 2 * a.d;
        for (int g = 0; g < a.group; ++g) {
          const T *q = static_cast<const T *>(a.q) + (row * a.group + g) * a.d;
          float s = 0.f;
          for (int c = lane; c < a.d; c += 32) {
            const float x = to_f(q[c]);
            s = fmaf(x, x >= 0.f ? to_f(bound[a.d + c]) : to_f(bound[c]), s);
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(TQ_FULL_MASK, s, o);
          best = fmaxf(best, s);
        }
      }
    }
    if (lane == 0) a.out[i] = best;
  }
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

// Sum over the block and exclusive prefix of one value per thread.
__device__ __forceinline__ int block_scan1(int v, int &total) {
  __shared__ int w[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(TQ_FULL_MASK, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) w[warp] = s;
  __syncthreads();
  int p = 0;
  total = 0;
  for (int i = 0; i < nw; ++i) {
    if (i < warp) p += w[i];
    total += w[i];
  }
  __syncthreads();
  return p + s - v;
}

// One block per (sequence, KV head).  Radix selection: the key of the last block chosen is found
// eight bits at a time from counts of the keys that share the bits found so far; then one pass in
// index order writes the blocks above that key and the first ones at it.
__global__ void __launch_bounds__(kSelectThreads) select_blocks_kernel(SelectArgs a) {
  __shared__ int hist[256];
  __shared__ uint32_t found;
  __shared__ int left;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / a.heads), h = (int)(row - (int64_t)b * a.heads);
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
  const bool all = n <= a.keep;
  const int lo = a.first, hi = n - a.last;  // candidates [lo, hi); the others are always chosen
  uint32_t key = 0;
  int equal = 0;  // blocks at exactly `key` to take, the first ones
  if (!all) {
    int need = a.keep - a.first - a.last;
    if (need == 0) {
      key = 0xffffffffu;  // above every key but NaN's, which none has
    } else {
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int j = lo + threadIdx.x; j < hi; j += kSelectThreads) {
          const uint32_t k = order_key(scores[j]);
          if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
          int d = 255, rest = need;
          while (hist[d] < rest) rest -= hist[d--];
          found = key | ((uint32_t)d << shift);
          left = rest;
        }
        __syncthreads();
        key = found;
        need = left;
        __syncthreads();
      }
      equal = need;
    }
  }
  int at = 0, seen = 0;  // blocks written, blocks at `key` passed
  for (int j0 = 0; j0 < n; j0 += kSelectThreads) {
    const int j = j0 + threadIdx.x;
    bool take = j < n, tie = false;
    if (take && !all && j >= lo && j < hi) {
      const uint32_t k = order_key(scores[j]);
      take = k > key;
      tie = k == key && equal > 0;
    }
    int ties, taken;
    const int before = block_scan1(tie ? 1 : 0, ties);
    if (tie) take = seen + before < equal;
    const int p = at + block_scan1(take ? 1 : 0, taken);
    if (take) {
      const int e = table[j];
      out[p] = e >= 0 && e < a.n_blocks ? e * a.heads + h : -1;
    }
    at += taken;
    seen += ties;
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
                   d, pages->n_blocks, pages->block_table, seq_lens, q, bounds, scores};
  tq_prof_begin(TQK_BLOCK_SCORES, s);
  const unsigned grid = (unsigned)(8 * tq_sm_count());
  if (dtype == TQ_F32) block_scores_kernel<float><<<grid, 256, 0, s>>>(a);
  else block_scores_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  tq_prof_end(TQK_BLOCK_SCORES, s);
  return tq_cuda_check(cudaGetLastError(), "block scores launch");
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
  select_blocks_kernel<<<(unsigned)(pages->batch * pages->n_kv_heads), kSelectThreads, 0, s>>>(a);
  tq_prof_end(TQK_SELECT_BLOCKS, s);
  return tq_cuda_check(cudaGetLastError(), "block selection launch");
}
