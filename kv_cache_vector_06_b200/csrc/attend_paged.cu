// Decode attention over an uncompressed paged cache (tq_attend_paged).
#include "device_common.cuh"

namespace {

struct PagedArgs {
  int batch, heads, group, bs, max_blocks, max_len, d;
  int64_t n_blocks;
  float scale;
  const int32_t *table, *lens;
  const void *q, *k, *v;
  void *out;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float *p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

constexpr int kWarps = 8;

// One block per (sequence, query head); its warps take tokens in turn, each with its own running
// maximum m, sum l and output o of the softmax, joined at the end.
template <typename T, typename O>
__global__ void __launch_bounds__(32 * kWarps) attend_paged_kernel(PagedArgs a) {
  constexpr int kPer = kPagedMaxD / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kPagedMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = blockIdx.x;  // b * n_q_heads + hq
  const int hq = a.heads * a.group;
  const int b = (int)(r / hq), h = (int)(r - (int64_t)b * hq) / a.group;
  const int len = min(max(a.lens[b], 0), a.max_len);
  float q[kPer], o[kPer];
  for (int i = 0; i < kPer; ++i) {
    const int c = lane + 32 * i;
    q[i] = c < a.d ? to_f(static_cast<const T *>(a.q)[r * a.d + c]) * a.scale : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = warp; t < len; t += kWarps) {
    const int e = a.table[(int64_t)b * a.max_blocks + t / a.bs];
    if (e < 0 || e >= a.n_blocks) continue;
    const int64_t base = (((int64_t)e * a.heads + h) * a.bs + t % a.bs) * a.d;
    float s = 0.f;
    for (int i = 0; i < kPer; ++i) {
      const int c = lane + 32 * i;
      if (c < a.d) s = fmaf(q[i], to_f(static_cast<const T *>(a.k)[base + c]), s);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(TQ_FULL_MASK, s, x);
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : __expf(m - mn), p = __expf(s - mn);
    l = l * f + p;
    m = mn;
    for (int i = 0; i < kPer; ++i) {
      const int c = lane + 32 * i;
      if (c < a.d) o[i] = fmaf(p, to_f(static_cast<const T *>(a.v)[base + c]), o[i] * f);
    }
  }
  for (int i = 0; i < kPer; ++i) so[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kWarps; ++w) L += sl[w] > 0.f ? sl[w] * __expf(sm[w] - M) : 0.f;
  for (int c = threadIdx.x; c < a.d; c += 32 * kWarps) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += sl[w] > 0.f ? so[w][c] * __expf(sm[w] - M) : 0.f;
    store(static_cast<O *>(a.out) + r * a.d + c, L > 0.f ? x / L : 0.f);
  }
}

tq_status check_attend(const tq_pages *pages, int32_t max_seq_len, int32_t n_q_heads, int32_t d) {
  tq_status st = tq_check_pages(pages);
  if (st != TQ_OK) return st;
  st = tq_check_rows(TQ_F32, d);
  if (st != TQ_OK) return st;
  st = tq_check_group(*pages, n_q_heads);
  if (st != TQ_OK) return st;
  if (max_seq_len < 0 || max_seq_len > (int64_t)pages->max_blocks * pages->block_size)
    return tq_fail(TQ_EINVAL, "max_seq_len=%d: must be in [0, max_blocks * block_size = %lld]", max_seq_len,
                   (long long)pages->max_blocks * pages->block_size);
  if ((int64_t)pages->batch * n_q_heads > INT32_MAX)
    return tq_fail(TQ_EUNSUPPORTED, "batch * n_q_heads must be below 2^31");
  return TQ_OK;
}

}  // namespace

extern "C" tq_status tq_attend_paged_workspace_size(const tq_pages *pages, int32_t max_seq_len, int32_t n_q_heads,
                                                    int32_t d, size_t *bytes) {
  tq_status st = check_attend(pages, max_seq_len, n_q_heads, d);
  if (st != TQ_OK) return st;
  if (!bytes) return tq_fail(TQ_EINVAL, "bytes is NULL");
  *bytes = 0;
  return TQ_OK;
}

extern "C" tq_status tq_attend_paged(const tq_pages *pages, const int32_t *seq_lens, int32_t max_seq_len,
                                     const void *q, const void *k_cache, const void *v_cache, tq_dtype dtype,
                                     int32_t n_q_heads, int32_t d, float scale, void *out, tq_dtype out_dtype,
                                     void *ws, size_t ws_bytes, void *stream) {
  size_t need = 0;
  tq_status st = tq_attend_paged_workspace_size(pages, max_seq_len, n_q_heads, d, &need);
  if (st != TQ_OK) return st;
  st = tq_check_rows(dtype, d);
  if (st != TQ_OK) return st;
  if (out_dtype != TQ_F32 && out_dtype != dtype)
    return tq_fail(TQ_EINVAL, "out_dtype=%d: must be TQ_F32 or dtype=%d", (int)out_dtype, (int)dtype);
  if (pages->batch == 0) return TQ_OK;
  if (!seq_lens || !q || !k_cache || !v_cache || !out)
    return tq_fail(TQ_EINVAL, "seq_lens/q/k_cache/v_cache/out is NULL");
  if (!tq_aligned(q, 16) || !tq_aligned(k_cache, 16) || !tq_aligned(v_cache, 16) || !tq_aligned(out, 16))
    return tq_fail(TQ_EINVAL, "q/k_cache/v_cache/out not 16-byte aligned");
  if (!tq_aligned(seq_lens, 4)) return tq_fail(TQ_EINVAL, "seq_lens not 4-byte aligned");
  if (need > 0 && (!ws || ws_bytes < need || !tq_aligned(ws, 16)))
    return tq_fail(TQ_EINVAL, "workspace: %zu bytes (16-byte aligned) needed, %zu given", need, ws_bytes);
  DeviceScope dev_scope;
  st = dev_scope.enter(pages->device);
  if (st != TQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PagedArgs a{pages->batch, pages->n_kv_heads, n_q_heads / pages->n_kv_heads, pages->block_size, pages->max_blocks,
              max_seq_len, d, pages->n_blocks, scale != 0.f ? scale : 1.f / sqrtf((float)d), pages->block_table, seq_lens,
              q, k_cache, v_cache, out};
  const unsigned grid = (unsigned)(pages->batch * n_q_heads);
  tq_prof_begin(TQK_ATTEND_PAGED, s);
  if (dtype == TQ_F32) attend_paged_kernel<float, float><<<grid, 32 * kWarps, 0, s>>>(a);
  else if (out_dtype == TQ_F32) attend_paged_kernel<__nv_bfloat16, float><<<grid, 32 * kWarps, 0, s>>>(a);
  else attend_paged_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 32 * kWarps, 0, s>>>(a);
  tq_prof_end(TQK_ATTEND_PAGED, s);
  return tq_cuda_check(cudaGetLastError(), "paged attention launch");
}
