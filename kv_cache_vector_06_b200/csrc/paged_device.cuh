// Device helpers of the paged-cache kernels: asynchronous copies, tensor-core products and their operands'
// layouts in shared memory, and the equal division of a ragged batch's steps.
#pragma once

#include "device_common.cuh"

// Rows of d padded to D channels; T the cache's type.  A step's keys and values take 4 to 16 KB of ring.  At
// least two blocks share an SM, so that one streams while the other begins a row or joins its warps, with
// one (256 channels) to three (64 channels, bf16) steps of each warp in flight beside the one that it works on, and
// as many registers as the tiles need.  Measured (32 sequences of
// up to 2000 tokens x 8 heads of 256 channels, bf16): 3 warps x 2 blocks 58 us, 6 x 1 69 us; (up to 4000
// tokens of 128 channels) 4 x 2 50 us, 8 x 1 58 us, 3 x 3 54 us, two stages instead of three 52 us; (up to
// 8000 of 64) 4 x 3 51 us, 4 x 2 54 us; (7 x 9999 tokens of 64, fp32) 4 x 2 24.7 us, 4 x 3
// 27.8 us; steps of 16 tokens there instead of 8 (two independent chains) 96 us instead of 105 for 32 x 8000.
template <typename T, int D>
struct Shape {
  static constexpr int kTok = sizeof(T) == 2 || D == 64 ? 16 : 8;  // tokens per step
  static constexpr int kRow = D * (int)sizeof(T);         // bytes of a padded row
  static constexpr int kCh = kRow / 16;                   // 16-byte chunks of a row
  static constexpr int kStages = D == 64 && sizeof(T) == 2 ? 4 : D <= 128 ? 3 : 2;
  static constexpr int kWarps = D == 256 ? 3 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kOcc = D == 64 && sizeof(T) == 2 ? 3 : 2;  // blocks per SM
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
// The same for the cache's own values, of which there are many, in two instructions: the products read the
// first 11 bits of an operand, so x is its own head and the tail needs no rounding; cut to 11 bits, it
// leaves 2^-20 of x at most.
__device__ __forceinline__ void split_tf32_cut(uint32_t x, uint32_t &hi, uint32_t &lo) {
  hi = x;
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(x & 0xffffe000u));
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
// channels in the order in which a key's chunk holds them.
template <typename T, int H>
__device__ __forceinline__ void load_q(uint4 (&v)[H], const void *q, int64_t row, int group, int d, int kg, int lane) {
  const int ch = 4 * kg + (lane & 3);
#pragma unroll
  for (int x = 0; x < H; ++x) {
    const int hd = (lane >> 2) + 8 * x;
    v[x] = make_uint4(0u, 0u, 0u, 0u);
    if (hd < group && ch < d * (int)sizeof(T) / 16)
      v[x] = *(reinterpret_cast<const uint4 *>(static_cast<const T *>(q) + (row * group + hd) * d) + ch);
  }
}
// The operand itself; fp32: split into TF32 parts.
template <typename T, int H>
__device__ __forceinline__ void make_q(uint32_t (&f)[H][sizeof(T) == 2 ? 1 : 2][4], const uint4 (&v)[H]) {
#pragma unroll
  for (int x = 0; x < H; ++x) {
    const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) f[x][0][i] = w[i];
      else split_tf32(w[i], f[x][0][i], f[x][1][i]);
    }
  }
}

__device__ __forceinline__ void store2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}

// Launch that may begin while the kernel before it on the stream ends: every kernel launched so waits for
// that one with griddepcontrol.wait before it touches memory, and lets its own successor begin at once.  What
// the one before may still write is read with plain loads: a read-only load is for data that no one writes
// while the kernel is there.  `blocks` above 1: in clusters of so many.
// With per-kernel profiling on, an event sits between the two and a plain launch is used.
template <typename... P, typename... A>
cudaError_t tq_launch_clusters(void (*kern)(P...), int blocks, dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (!tq_prof_on()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (blocks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)blocks;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename... P, typename... A>
cudaError_t tq_launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A &...args) {
  return tq_launch_clusters(kern, 1, grid, threads, smem, st, args...);
}

// Division of 0 <= n < 2^31 by a fixed d >= 1 (Granlund and Montgomery's method):
// q = (mulhi(n, mul) + n) >> shift with
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

// a / b for 0 <= a, 0 < b: the 32-bit division where it will do (the 64-bit one takes some 100 instructions).
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// `total` units dealt to `workers` in equal runs, the first `total % workers` of them one longer.
struct Deal {
  int64_t each, more;
  __device__ __forceinline__ Deal(int64_t total, int64_t workers) : each(div64(total, workers)), more(total - each * workers) {}
  __device__ __forceinline__ int64_t begin(int64_t id) const { return each * id + min(id, more); }
  __device__ __forceinline__ int64_t owner(int64_t unit) const {
    const int64_t longer = (each + 1) * more;  // units of the longer runs
    return unit < longer ? div64(unit, each + 1) : more + div64(unit - longer, each);
  }
};

// The steps of all (sequence, KV head) rows laid end to end, sequence by sequence: each thread of the
// block sums a run of sequences, then a block scan.  Has one block barrier.
template <int WARPS>
struct StepScan {
  int b0, b1;           // this thread's sequences
  int len0;             // the first one's length
  int64_t before, mine; // steps before and in them
  int64_t total;
  int heads;
  __device__ __forceinline__ void run(const int32_t *lens, int batch, int n_heads, int max_len, int tok) {
    __shared__ int64_t wsum[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (batch + 32 * WARPS - 1) / (32 * WARPS);
    heads = n_heads;
    b0 = (int)min((int64_t)threadIdx.x * per, (int64_t)batch);
    b1 = (int)min((int64_t)b0 + per, (int64_t)batch);
    len0 = b0 < b1 ? lens[b0] : 0;
    mine = b0 < b1 ? row_steps(len0, max_len, tok) : 0;
    for (int b = b0 + 1; b < b1; ++b) mine += row_steps(lens[b], max_len, tok);
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
    for (int w = 0; w < WARPS; ++w) {
      const int64_t x = wsum[w];
      if (w < warp) before += x;
      total += x;
    }
  }
};

// Where a worker begins: a sequence, its length, and a unit's place in the sequence's rows.
struct Place {
  int seq, len;
  int64_t unit;
};

// With `extra` units of work counted in front of every row's steps (what a row costs beside them): the
// thread that holds unit `pos` of all rows writes where it lies.
template <int WARPS>
__device__ __forceinline__ void find_unit(const StepScan<WARPS> &s, int64_t pos, int extra, const int32_t *lens, int max_len, int tok, Place &out) {
  const int64_t front = s.before + (int64_t)s.b0 * s.heads * extra;
  int64_t left = pos - front;
  if (left < 0 || left >= s.mine + (int64_t)(s.b1 - s.b0) * s.heads * extra) return;
  int b = s.b0, len = s.len0;
  for (;;) {
    const int64_t n = (int64_t)(extra + row_steps(len, max_len, tok)) * s.heads;
    if (left < n) break;
    left -= n;
    len = lens[++b];
  }
  out = Place{b, len, left};
}

// Blocks that hold a sequence's tokens: ceil(len / bs), with the length clamped to the table.
__device__ __forceinline__ int held_blocks(int len, int bs, int max_blocks) {
  if (len <= 0) return 0;
  const int n = (len - 1) / bs + 1;
  return n < max_blocks ? n : max_blocks;
}
