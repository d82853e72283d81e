// Device helpers of the paged-cache kernels: asynchronous copies, tensor-core products and their operands'
// layouts in shared memory, and the equal division of a ragged batch's steps.
#pragma once

#include "device_common.cuh"

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// Rows of d padded to D channels; T the cache's type.  A step's keys and values take 64 D bytes of ring.
template <typename T, int D>
struct Shape {
  static constexpr int kTok = 32 / sizeof(T);             // tokens per step: 16 (bf16) or 8 (fp32)
  static constexpr int kRow = D * (int)sizeof(T);         // bytes of a padded row
  static constexpr int kCh = kRow / 16;                   // 16-byte chunks of a row
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr int kOcc = D == 64 ? 3 : D == 128 ? 2 : 1;  // blocks per SM
  static constexpr int kStage = 2 * kTok * kRow;
  static constexpr int kRing = kStages * kStage;          // per warp
  static constexpr int kSmem = kWarps * kRing;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], unsigned addr) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16-byte asynchronous copy; `bytes` 0 fills with zeros and reads nothing.
__device__ __forceinline__ void cp16(unsigned dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(y) : "f"(x));
  return y;
}
// x = hi + lo to 2^-22 of x: each part rounded to TF32's 11 bits.
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t &hi, uint32_t &lo) {
  hi = tf32(__uint_as_float(x));
  lo = tf32(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return reinterpret_cast<const uint32_t &>(v);
}
// The same, leaving what the rounding dropped in lo and hi.
__device__ __forceinline__ uint32_t take_bf16(float &lo, float &hi) {
  const uint32_t v = pack_bf16(lo, hi);
  lo -= __uint_as_float(v << 16);
  hi -= __uint_as_float(v & 0xffff0000u);
  return v;
}

// Swizzles of a row's 16-byte chunks, so that the accesses below touch every bank once: keys are read as
// four chunks of two rows, bf16 values as one chunk of eight rows, fp32 values as two chunks of every
// other row.
__device__ __forceinline__ int key_chunk(int row, int ch) { return ch ^ ((row & 1) << 2); }
template <typename T>
__device__ __forceinline__ int value_chunk(int row, int ch) {
  return sizeof(T) == 2 ? ch ^ (row & 7) : ch ^ (row & 6);
}

// Chunk 4 kg + lane % 4 of query head lane / 4 (+ 8 x) of row `row`: this lane's part of the left operand, the
// channels in the order in which a key's chunk holds them.  fp32: split into TF32 parts.
template <typename T, int H>
__device__ __forceinline__ void load_q(uint32_t (&f)[H][sizeof(T) == 2 ? 1 : 2][4], const void *q, int64_t row, int group, int d, int kg,
                                       int lane) {
  const int ch = 4 * kg + (lane & 3);
#pragma unroll
  for (int x = 0; x < H; ++x) {
    const int hd = (lane >> 2) + 8 * x;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (hd < group && ch < d * (int)sizeof(T) / 16)
      v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(q) + (row * group + hd) * d) + ch);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) f[x][0][i] = w[i];
      else split_tf32(w[i], f[x][0][i], f[x][1][i]);
    }
  }
}

// Division of 0 <= n < 2^31 by a fixed d >= 1: q = (mulhi(n, mul) + n) >> shift with
// mul = floor(2^32 (2^shift - d) / d) + 1, shift = ceil(log2 d).
struct FastDiv {
  uint32_t mul, shift;
  int32_t d;
  FastDiv() = default;
  explicit FastDiv(int32_t div) : d(div) {
    shift = 0;
    while ((1ull << shift) < (uint64_t)div) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - (uint64_t)div)) / (uint64_t)div + 1);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
};

// Steps of one row: at least one, so that every row has a worker to write it.
__device__ __forceinline__ int row_steps(int len, int max_len, int tok) {
  len = min(len, max_len);
  return len <= tok ? 1 : (len - 1) / tok + 1;
}

// The steps of all (sequence, KV head) rows laid end to end, sequence by sequence: each thread of the
// block sums a run of sequences, then a block scan.  kThreads threads; ends with a block barrier.
struct StepScan {
  int64_t b0, b1;       // this thread's sequences
  int64_t before, mine; // steps before and in them
  int64_t total;
  int heads;
  __device__ __forceinline__ void run(const int32_t *lens, int batch, int n_heads, int max_len, int tok) {
    __shared__ int64_t wsum[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (batch + kThreads - 1) / kThreads;
    heads = n_heads;
    b0 = min((int64_t)threadIdx.x * per, (int64_t)batch);
    b1 = min(b0 + per, (int64_t)batch);
    mine = 0;
    for (int64_t b = b0; b < b1; ++b) mine += row_steps(lens[b], max_len, tok);
    mine *= heads;
    int64_t incl = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int64_t u = __shfl_up_sync(TQ_FULL_MASK, incl, x);
      if (lane >= x) incl += u;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    total = 0;
    before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
  }
  // The thread that holds step `pos` writes its sequence and the step's place in the sequence's rows.
  __device__ __forceinline__ void find(int64_t pos, const int32_t *lens, int max_len, int tok, int &seq, int64_t &place) const {
    if (pos < before || pos >= before + mine) return;
    int64_t left = pos - before, b = b0;
    for (;; ++b) {
      const int64_t n = (int64_t)row_steps(lens[b], max_len, tok) * heads;
      if (left < n) break;
      left -= n;
    }
    seq = (int)b;
    place = left;
  }
};

// Blocks that hold a sequence's tokens: ceil(len / bs), with the length clamped to the table.
__device__ __forceinline__ int held_blocks(int len, int bs, int max_blocks) {
  if (len <= 0) return 0;
  const int n = (len - 1) / bs + 1;
  return n < max_blocks ? n : max_blocks;
}
