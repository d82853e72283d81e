// Decode attention over an uncompressed paged cache (tq_attend_paged).
//
//   o = sum_t e^{s_t - m} v_t / sum_t e^{s_t - m},  s_t = scale <q, k_t>,  m a running maximum
//
// Bound: 2 d rows of the cache per (token, KV head) against 4 g d flop, a few flop per byte: HBM.  The
// group's query heads share each row read, so the products run on the tensor cores (mma.sync: the
// 128-row tiles of tcgen05 would hold at most 16 query heads), and the loads never wait for them.
//
// Work is counted in steps of 16 tokens (fp32 rows of more than 64 channels: 8) over all (sequence, KV head) rows laid end to end; every worker
// takes an equal run of steps, so a ragged batch ends at one time whatever its lengths.  A worker is a
// block of four warps that share a row's steps (long rows) or a single warp (many short rows).  Each
// warp streams its steps through a ring of its own (cp.async, no block barrier) with its own m, l and o.
// A row that falls to several workers leaves pieces (m, l, o) in the workspace, joined by a second
// kernel.  A ragged batch of 64 sequences of 1024 .. 32768 tokens x 8 KV heads of 128 bf16 channels (4.4 GB):
// 640-670 us, 6.6-6.9 TB/s, where a kernel that only reads reaches 7.3.  Where rows are few and short, a cluster of
// blocks takes each whole, in one launch.
#include <algorithm>
#include "paged_device.cuh"

namespace {

struct PagedArgs {
  int batch, heads, group, bs, max_blocks, max_len, d;
  int64_t n_blocks;
  float scale;
  const int32_t *table, *lens;
  const void *q, *k, *v;
  void *out;
  FastDiv by_bs;
  int2 *owner;   // [rows]: slot of the first piece, and pieces (0: the output is written), negated where they lie a warp apart
  float *piece;  // [workers][2][piece_floats]: [group][d] o, then [group] m, [group] l of each
};

// What a row costs a worker beside its steps (its queries, its first loads, the joining of the warps), in
// steps of the worker: as long as 64 KB (a block) or 16 KB (a warp) of the cache take it.  Without it a block
// that drew several short rows ended last: 7 sequences of 1 to 9999 tokens x 4 heads took 47 us, with it 35.
template <typename T, int D>
constexpr int kTeamRowCost = 65536 / Shape<T, D>::kStage;
template <typename T, int D>
constexpr int kSoloRowCost = 16384 / Shape<T, D>::kStage;

// Floats of one piece, a multiple of four.
__host__ __device__ __forceinline__ int piece_floats(int group, int d) { return (group * (d + 2) + 3) & ~3; }

constexpr float kLog2e = 1.44269504088896340736f;

// One warp's stream over the steps of one row, and its softmax state.
//   WIDE   more than 8 query heads.  Otherwise rows 8 .. 15 of the products' left operand carry the
//          low-order parts of the same heads' weights (fp32: also of the queries), so that the parts
//          cost no products of their own.
//   PARTS  bf16: bf16 parts that a softmax weight is split into, 2 (error 2^-17 of it, under a bf16
//          output's rounding) or 3 (2^-25)
template <typename T, int D, bool WIDE, int PARTS>
struct Stream {
  using S = Shape<T, D>;
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int kKg = S::kCh / 4;                        // 64-byte groups of a row
  static constexpr int kQRegs = kKg * (WIDE ? 8 : 4) * (kBf ? 1 : 2);
  static constexpr bool kQInRegs = kQRegs <= (kBf ? 32 : 64);
  static constexpr int kQ = kQInRegs ? kKg : 1;
  // Queries that the registers do not hold lie in shared memory, once for the block's warps, in the order in
  // which the lanes take them; where a warp works alone, or where they would cost the second block of the SM,
  // each step asks the first-level cache for them (32 x 8 heads of 256 channels, fp32: 138 us, from the cache
  // 172, measured before the sums of add(); with them 160).
  static constexpr int kQBytes = kKg * (WIDE ? 2 : 1) * (kBf ? 1 : 2) * 512;
  static constexpr bool kQInSmem = !kQInRegs && kQBytes <= 16384;
  static constexpr int kSmem = S::kSmem + (kQInSmem ? kQBytes : 0);
  static constexpr int kNt = D / 8;
  static constexpr int kH = WIDE ? 2 : 1;                       // heads per lane: lane / 4 and 8 + lane / 4

  float o[kNt][4], m[kH], l[kH];
  uint32_t qf[kQ][kH][kBf ? 1 : 2][4];

  // A tensor core cuts what it returns: summed there, step after step, o shrank by up to 5e-6 of itself over
  // 20000 tokens.  So each step's products are summed apart and added here, rounded to nearest.
  static __device__ __forceinline__ void add(float (&to)[4], const float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] += x[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
#pragma unroll
    for (int x = 0; x < kH; ++x) {
      m[x] = -INFINITY;
      l[x] = 0.f;
    }
  }

  // This lane's part of group kg in shared memory: parts of 512 bytes.
  static __device__ __forceinline__ unsigned q_at(unsigned qs, int kg, int lane) {
    return qs + (unsigned)(kg * kH * (kBf ? 1 : 2) * 512 + lane * 16);
  }
  static __device__ __forceinline__ void put_q(const PagedArgs &a, int64_t row, unsigned qs, int kg, int lane) {
    uint4 raw[kH];
    uint32_t f[kH][kBf ? 1 : 2][4];
    load_q<T, kH>(raw, a.q, row, a.group, a.d, kg, lane);
    make_q<T, kH>(f, raw);
#pragma unroll
    for (int x = 0; x < kH * (kBf ? 1 : 2); ++x) {
      const auto &v = f[x / (kBf ? 1 : 2)][x % (kBf ? 1 : 2)];
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(q_at(qs, kg, lane) + 512 * x), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                   : "memory");
    }
  }

  // One step: keys at kbase, values at vbase, tokens `valid`; queries at qs where they are in shared memory.
  __device__ __forceinline__ void step(const PagedArgs &a, int64_t row, unsigned qs, unsigned kbase, unsigned vbase, uint32_t valid,
                                       float sc, int lane) {
    constexpr int kT = S::kTok / 8;
    const int c = lane & 3, r = lane >> 2;
    // chunk 4 kg + c of token r lies at at[kg & 1] + 128 (kg / 2): key_chunk swaps the groups of odd rows
    const unsigned at[2] = {(unsigned)(r * S::kRow + 16 * key_chunk(r, c)), (unsigned)(r * S::kRow + 16 * key_chunk(r, 4 + c))};
    float s[kT][4];
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
    for (int kg = 0; kg < kKg; ++kg) {
      if constexpr (!kQInRegs) {
        if (kQInSmem && qs != 0) {
#pragma unroll
          for (int x = 0; x < kH * (kBf ? 1 : 2); ++x) lds128(qf[0][x / (kBf ? 1 : 2)][x % (kBf ? 1 : 2)], q_at(qs, kg, lane) + 512 * x);
        } else {
          uint4 raw[kH];
          load_q<T, kH>(raw, a.q, row, a.group, a.d, kg, lane);
          make_q<T, kH>(qf[0], raw);
        }
      }
      const auto &f = qf[kQInRegs ? kg : 0];
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        uint32_t k[4];
        lds128(k, kbase + at[kg & 1] + 8 * t * S::kRow + 128 * (kg >> 1));
        float acc[4] = {0.f, 0.f, 0.f, 0.f};  // fp32: one group's products, added as in add()
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (kBf) {
            if constexpr (WIDE) mma_bf16(s[t], f[0][0][2 * u], f[1][0][2 * u], f[0][0][2 * u + 1], f[1][0][2 * u + 1], k[2 * u], k[2 * u + 1]);
            else mma_bf16(s[t], f[0][0][2 * u], 0u, f[0][0][2 * u + 1], 0u, k[2 * u], k[2 * u + 1]);
          } else {
            uint32_t h0, l0, h1, l1;
            split_tf32_cut(k[2 * u], h0, l0);
            split_tf32_cut(k[2 * u + 1], h1, l1);
            if constexpr (WIDE) {
              mma_tf32(acc, f[0][1][2 * u], f[1][1][2 * u], f[0][1][2 * u + 1], f[1][1][2 * u + 1], h0, h1);
              mma_tf32(acc, f[0][0][2 * u], f[1][0][2 * u], f[0][0][2 * u + 1], f[1][0][2 * u + 1], l0, l1);
              mma_tf32(acc, f[0][0][2 * u], f[1][0][2 * u], f[0][0][2 * u + 1], f[1][0][2 * u + 1], h0, h1);
            } else {
              mma_tf32(acc, f[0][0][2 * u], 0u, f[0][0][2 * u + 1], 0u, l0, l1);
              mma_tf32(acc, f[0][0][2 * u], f[0][1][2 * u], f[0][0][2 * u + 1], f[0][1][2 * u + 1], h0, h1);
            }
          }
        }
        if constexpr (!kBf) add(s[t], acc);
      }
    }
    // logits in units of log2, masked; lane: head r (+ 8), tokens 8 t + 2 c, 8 t + 2 c + 1
    float p[kH][kT][2];
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = (valid >> (8 * t + 2 * c + i)) & 1u;
        if constexpr (WIDE) {
          p[0][t][i] = in ? s[t][i] * sc : -INFINITY;
          p[kH - 1][t][i] = in ? s[t][2 + i] * sc : -INFINITY;
        } else {
          p[0][t][i] = in ? (kBf ? s[t][i] : s[t][i] + s[t][2 + i]) * sc : -INFINITY;
        }
      }
    // The running maximum moves only when a logit passes it by more than 2^8: weights up to 2^8 above
    // the others' scale cost no precision in fp32, and o is rescaled a few times per row at most.
    float top[kH];
    bool move = false;
#pragma unroll
    for (int x = 0; x < kH; ++x) {
      top[x] = p[x][0][0];
#pragma unroll
      for (int t = 0; t < kT; ++t) top[x] = fmaxf(top[x], fmaxf(p[x][t][0], p[x][t][1]));
      top[x] = fmaxf(top[x], __shfl_xor_sync(TQ_FULL_MASK, top[x], 1));
      top[x] = fmaxf(top[x], __shfl_xor_sync(TQ_FULL_MASK, top[x], 2));
      move = move || top[x] > m[x] + 8.f;
    }
    if (__any_sync(TQ_FULL_MASK, move)) {
      float f[kH];
#pragma unroll
      for (int x = 0; x < kH; ++x) {
        const float to = fmaxf(m[x], top[x]);
        f[x] = m[x] == -INFINITY ? 0.f : exp2a(m[x] - to);
        m[x] = to;
        l[x] *= f[x];
      }
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        o[n][0] *= f[0];
        o[n][1] *= f[0];
        o[n][2] *= f[kH - 1];
        o[n][3] *= f[kH - 1];
      }
    }
#pragma unroll
    for (int x = 0; x < kH; ++x) {
      const float mm = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          p[x][t][i] = exp2a(p[x][t][i] - mm);
          l[x] += p[x][t][i];
        }
    }
    if constexpr (kBf) {
      uint32_t w[PARTS][kH][2];
#pragma unroll
      for (int x = 0; x < kH; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int i = 0; i < PARTS - 1; ++i) w[i][x][t] = take_bf16(p[x][t][0], p[x][t][1]);
          w[PARTS - 1][x][t] = pack_bf16(p[x][t][0], p[x][t][1]);
        }
#pragma unroll
      for (int n = 0; n < kNt; n += 2) {
        uint32_t v[4];
        ldsm4t(v, vbase + (lane & 15) * S::kRow + 16 * value_chunk<T>(lane & 15, n + (lane >> 4)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          if constexpr (WIDE) {
#pragma unroll
            for (int i = PARTS - 1; i >= 0; --i)
              mma_bf16(acc, w[i][0][0], w[i][kH - 1][0], w[i][0][1], w[i][kH - 1][1], v[2 * u], v[2 * u + 1]);
          } else {
            if constexpr (PARTS == 3) mma_bf16(acc, 0u, w[PARTS - 1][0][0], 0u, w[PARTS - 1][0][1], v[2 * u], v[2 * u + 1]);
            mma_bf16(acc, w[0][0][0], w[1][0][0], w[0][0][1], w[1][0][1], v[2 * u], v[2 * u + 1]);
          }
          add(o[n + u], acc);
        }
      }
    } else {
      // left operand of tile t: column c is token 8 t + 2 c, column c + 4 token 8 t + 2 c + 1
      uint32_t ph[kT][kH][2], pl[kT][kH][2];
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int x = 0; x < kH; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i) split_tf32(__float_as_uint(p[x][t][i]), ph[t][x][i], pl[t][x][i]);
#pragma unroll
      for (int g = 0; g < kNt / 4; ++g)
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const int tok = 8 * t + 2 * c;
          uint32_t v0[4], v1[4];  // four channels of tokens 8 t + 2 c and 8 t + 2 c + 1, one per tile of o
          lds128(v0, vbase + tok * S::kRow + 16 * value_chunk<T>(tok, 8 * g + r));
          lds128(v1, vbase + (tok + 1) * S::kRow + 16 * value_chunk<T>(tok + 1, 8 * g + r));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h0, l0, h1, l1;
            split_tf32_cut(v0[i], h0, l0);
            split_tf32_cut(v1[i], h1, l1);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (WIDE) {
              mma_tf32(acc, pl[t][0][0], pl[t][kH - 1][0], pl[t][0][1], pl[t][kH - 1][1], h0, h1);
              mma_tf32(acc, ph[t][0][0], ph[t][kH - 1][0], ph[t][0][1], ph[t][kH - 1][1], l0, l1);
              mma_tf32(acc, ph[t][0][0], ph[t][kH - 1][0], ph[t][0][1], ph[t][kH - 1][1], h0, h1);
            } else {
              mma_tf32(acc, 0u, ph[t][0][0], 0u, ph[t][0][1], l0, l1);
              mma_tf32(acc, ph[t][0][0], pl[t][0][0], ph[t][0][1], pl[t][0][1], h0, h1);
            }
            add(o[4 * g + i], acc);
          }
        }
    }
  }

  __device__ __forceinline__ float value(int n, int i, int x) const {
    return WIDE ? o[n][2 * x + i] : o[n][i] + o[n][2 + i];
  }
  // o of head lane / 4 + 8 x, times f, to d channels at dst.  A lane's columns 2 c, 2 c + 1 of tile n are
  // channels 8 n + 2 c, 8 n + 2 c + 1 (bf16), or, of four tiles, the eight from 32 (n / 4) + 8 c on (fp32).
  template <typename O>
  __device__ __forceinline__ void emit(O *dst, int x, float f, int d, int lane) const {
    const int c = lane & 3;
    if constexpr (kBf) {
#pragma unroll
      for (int n = 0; n < kNt; ++n)
        if (8 * n < d) store2(dst + 8 * n + 2 * c, value(n, 0, x) * f, value(n, 1, x) * f);
    } else {
#pragma unroll
      for (int n = 0; n < kNt; n += 4)
        if (8 * n + 8 * c < d) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float4 *>(dst + 8 * n + 8 * c + 4 * i) =
                make_float4(value(n, i, x) * f, value(n + 1, i, x) * f, value(n + 2, i, x) * f, value(n + 3, i, x) * f);
        }
    }
  }
};

// One warp's steps step0, step0 + apart, ... (n of them) of one row, through its ring: m, l and o of its lanes'
// heads in `st`, l summed over the lanes of a head.
template <typename T, int D, bool WIDE, int PARTS>
__device__ __forceinline__ void stream_row(Stream<T, D, WIDE, PARTS> &st, const PagedArgs &a, int64_t row, const int32_t *table, int h,
                                           int len, int step0, int n, int apart, unsigned ring, uint32_t *masks, unsigned qs, int warp,
                                           int lane) {
  using S = Shape<T, D>;
  using St = Stream<T, D, WIDE, PARTS>;
  const int esz_row = a.d * (int)sizeof(T);  // bytes of a row in the cache
  const int dch = esz_row / 16;
  const bool whole = a.bs % S::kTok == 0;  // a step lies in one block
  const float sc = a.scale * kLog2e;
  // block of this lane's token (of the whole step where it lies in one block)
  auto entry = [&](int i) {
    const int t = (step0 + i * apart) * S::kTok + (whole ? 0 : (lane & (S::kTok - 1)));
    return i < n && t < len ? table[a.by_bs(t)] : -1;
  };
  auto issue = [&](int i, int e) {
    const int stage = i % S::kStages;
    const int t0 = (step0 + i * apart) * S::kTok;
    const bool ok = e >= 0 && e < a.n_blocks;
    const int t = t0 + (whole ? 0 : (lane & (S::kTok - 1)));
    const int64_t off = ok ? (((int64_t)e * a.heads + h) * a.bs + (t - a.by_bs(t) * a.bs)) * esz_row : 0;
    uint32_t valid = __ballot_sync(TQ_FULL_MASK, whole ? ok && t0 + lane < len : ok);
    valid &= (1u << S::kTok) - 1u;
    if (lane == 0) masks[stage] = valid;
    const unsigned kb = ring + stage * S::kStage, vb = kb + S::kTok * S::kRow;
#pragma unroll
    for (int x = 0; x < S::kTok * S::kCh / 32; ++x) {
      const int idx = lane + 32 * x, r = idx / S::kCh, ch = idx % S::kCh;
      const int64_t base = whole ? off + r * esz_row : __shfl_sync(TQ_FULL_MASK, off, r);
      const int64_t src = base + 16 * min(ch, dch - 1);  // inside the cache; read where the token is there
      const int bytes = ((valid >> r) & 1u) && ch < dch ? 16 : 0;
      cp16(kb + r * S::kRow + 16 * key_chunk(r, ch), static_cast<const char *>(a.k) + src, bytes);
      cp16(vb + r * S::kRow + 16 * value_chunk<T>(r, ch), static_cast<const char *>(a.v) + src, bytes);
    }
  };
  int e[S::kStages];
#pragma unroll
  for (int i = 0; i < S::kStages; ++i) e[i] = entry(i);
  uint4 raw[St::kQ][St::kH];  // asked for before the rows, so that it does not queue behind them
  if constexpr (St::kQInRegs) {
#pragma unroll
    for (int kg = 0; kg < St::kKg; ++kg) load_q<T, St::kH>(raw[kg], a.q, row, a.group, a.d, kg, lane);
  }
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) {
    if (i < n) issue(i, e[i]);
    cp_commit();
  }
  int next = e[S::kStages - 1];
  if constexpr (St::kQInRegs) {
#pragma unroll
    for (int kg = 0; kg < St::kKg; ++kg) make_q<T, St::kH>(st.qf[kg], raw[kg]);
  }
  if (qs != 0) {  // the block's warps share a row
    for (int kg = warp; kg < St::kKg; kg += S::kWarps) St::put_q(a, row, qs, kg, lane);
    __syncthreads();
  }
  st.clear();
  for (int i = 0; i < n; ++i) {
    cp_wait<S::kStages - 2>();
    __syncwarp();  // this step's copies of every lane have landed; the last step's stage is free
    if (i + S::kStages - 1 < n) issue(i + S::kStages - 1, next);
    cp_commit();
    next = entry(i + S::kStages);
    const int stage = i % S::kStages;
    const unsigned kb = ring + stage * S::kStage;
    st.step(a, row, qs, kb, kb + S::kTok * S::kRow, masks[stage], sc, lane);
  }
  cp_wait<0>();
  __syncwarp();
#pragma unroll
  for (int x = 0; x < St::kH; ++x) {
    st.l[x] += __shfl_xor_sync(TQ_FULL_MASK, st.l[x], 1);
    st.l[x] += __shfl_xor_sync(TQ_FULL_MASK, st.l[x], 2);
  }
}

// Floats of a head's row in join_warps: padded, so that a warp's stores touch every bank once.
template <typename T, int D>
__host__ __device__ constexpr int padded_row() {
  return D + (sizeof(T) == 2 ? 8 : 4);
}

// The warps' sums of one row joined in shared memory (`buf`, kWarps x 16 padded rows): done(head, channel, o of four
// channels, m, l) for every head and four channels, spread over the block's threads.  Every warp's ring is drained.
template <typename T, int D, bool WIDE, int PARTS, typename F>
__device__ __forceinline__ void join_warps(const Stream<T, D, WIDE, PARTS> &st, const PagedArgs &a, float *buf, float (&mm)[Shape<T, D>::kWarps][16],
                                           float (&ll)[Shape<T, D>::kWarps][16], int warp, int lane, F &&done) {
  using St = Stream<T, D, WIDE, PARTS>;
  constexpr int kWarps = Shape<T, D>::kWarps;
  constexpr int kPad = padded_row<T, D>();
  const int g = a.group;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < St::kH; ++x) {
    const int hd = (lane >> 2) + 8 * x;
    if (hd >= g) continue;
    st.emit(buf + (warp * 16 + hd) * kPad, x, 1.f, D, lane);
    if ((lane & 3) == 0) {
      mm[warp][hd] = st.m[x];
      ll[warp][hd] = st.l[x];
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < g * (D / 4); idx += 32 * kWarps) {
    const int hd = idx / (D / 4), c = 4 * (idx % (D / 4));
    if (c >= a.d) continue;
    float top = -INFINITY, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mm[w][hd]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = mm[w][hd] == -INFINITY ? 0.f : exp2a(mm[w][hd] - top);
      const float4 x = *reinterpret_cast<const float4 *>(buf + (w * 16 + hd) * kPad + c);
      sum = fmaf(f, ll[w][hd], sum);
      v.x = fmaf(f, x.x, v.x);
      v.y = fmaf(f, x.y, v.y);
      v.z = fmaf(f, x.z, v.z);
      v.w = fmaf(f, x.w, v.w);
    }
    done(hd, c, v, top, sum);
  }
}
template <typename O>
__device__ __forceinline__ void put_out(O *out, const float4 &v, float l) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  store2(out, v.x * inv, v.y * inv);
  store2(out + 2, v.z * inv, v.w * inv);
}

template <typename T, int D, bool WIDE, int PARTS, typename O>
__global__ void __launch_bounds__(Shape<T, D>::kThreads, Shape<T, D>::kOcc) attend_paged_kernel(PagedArgs a) {
  using S = Shape<T, D>;
  using St = Stream<T, D, WIDE, PARTS>;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Place place[kWarps];
  __shared__ uint32_t masks[kWarps][S::kStages];
  __shared__ float mm[kWarps][16], ll[kWarps][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  StepScan<kWarps> scan;
  scan.run(a.lens, a.batch, a.heads, a.max_len, S::kTok);
  // ---- workers
  const int64_t rows = (int64_t)a.batch * a.heads;
  const bool solo = rows >= (int64_t)gridDim.x && scan.total < 8 * rows;
  const int team = solo ? 1 : kWarps, extra = solo ? kSoloRowCost<T, D> : kTeamRowCost<T, D>;
  const int64_t workers = max((int64_t)1, min((int64_t)gridDim.x * (solo ? kWarps : 1), scan.total / (solo ? 1 : kWarps)));
  const Deal deal(scan.total + rows * extra, workers);
  for (int w = 0; w < kWarps; w += team) {
    const int64_t id = solo ? (int64_t)blockIdx.x * kWarps + w : (int64_t)blockIdx.x;
    if (id < workers) find_unit(scan, deal.begin(id), extra, a.lens, a.max_len, S::kTok, place[w]);
  }
  __syncthreads();
  const int lead = solo ? warp : 0;  // first warp of the team
  const int slot0 = blockIdx.x * kWarps + lead;
  const int64_t id = solo ? (int64_t)slot0 : (int64_t)blockIdx.x;
  if (id >= workers) return;
  const int64_t begin = deal.begin(id), end = deal.begin(id + 1);
  int b = place[lead].seq, len, steps;
  auto enter = [&](int tokens) {
    len = min(max(tokens, 0), a.max_len);
    steps = row_steps(len, a.max_len, S::kTok);
  };
  enter(place[lead].len);
  int h = (int)div64(place[lead].unit, steps + extra);
  int64_t unit = place[lead].unit - (int64_t)h * (steps + extra);  // place in the row, its cost in front

  const unsigned ring = smem_addr(smem) + warp * S::kRing;
  const int rank = solo ? 0 : warp;
  St st;

  for (int64_t pos = begin; pos < end;) {
    const int64_t span = min(steps + extra - unit, end - pos);
    const int first = (int)max(unit - extra, (int64_t)0), count = (int)max(unit + span - extra, (int64_t)0) - first;
    auto go_on = [&]() {
      pos += span;
      unit = 0;
      if (pos < end && ++h == a.heads) {
        h = 0;
        enter(a.lens[++b]);
      }
    };
    if (count == 0) {  // the worker's run ends in front of the row's first step
      go_on();
      continue;
    }
    const int64_t row = (int64_t)b * a.heads + h;
    const int32_t *table = a.table + (int64_t)b * a.max_blocks;
    const int n = (count - rank + team - 1) / team;
    const unsigned qs = St::kQInSmem && !solo ? smem_addr(smem) + S::kSmem : 0;
    stream_row<T, D, WIDE, PARTS>(st, a, row, table, h, len, first + rank, n, team, ring, masks[warp], qs, warp, lane);

    // ---- the row's end, or the worker's: the output, or a piece of it
    const bool starts = first == 0, ends = first + count == steps;
    const int g = a.group;
    const bool done = starts && ends;
    float *piece = a.piece + ((int64_t)slot0 * 2 + (starts ? 1 : 0)) * piece_floats(g, a.d);
    O *out = static_cast<O *>(a.out) + row * g * a.d;
    if (solo) {
#pragma unroll
      for (int x = 0; x < St::kH; ++x) {
        const int hd = (lane >> 2) + 8 * x;
        if (hd >= g) continue;
        if (done) {
          st.emit(out + hd * a.d, x, st.l[x] > 0.f ? 1.f / st.l[x] : 0.f, a.d, lane);
        } else {
          st.emit(piece + hd * a.d, x, 1.f, a.d, lane);
          if ((lane & 3) == 0) {
            piece[g * a.d + hd] = st.m[x];
            piece[g * a.d + g + hd] = st.l[x];
          }
        }
      }
    } else {
      join_warps<T, D, WIDE, PARTS>(st, a, reinterpret_cast<float *>(smem), mm, ll, warp, lane,
                                    [&](int hd, int c, const float4 &v, float top, float sum) {
                                      if (done) {
                                        put_out(out + hd * a.d + c, v, sum);
                                        return;
                                      }
                                      *reinterpret_cast<float4 *>(piece + hd * a.d + c) = v;
                                      if (c == 0) {
                                        piece[g * a.d + hd] = top;
                                        piece[g * a.d + g + hd] = sum;
                                      }
                                    });
      __syncthreads();
    }
    if (starts && rank == 0 && lane == 0) {
      // the row's last step decides how many workers hold pieces of it
      const int n = done ? 0 : (int)(deal.owner(pos - unit + extra + steps - 1) - id) + 1;
      a.owner[row] = make_int2(slot0, solo ? -n : n);
    }
    go_on();
  }
}

// Few short rows: a cluster of blocks takes one row whole, its warps the row's steps in turn, and joins its
// blocks' sums through distributed shared memory: no scan, no pieces, one launch (8 rows of 1000 tokens: 8.9 us
// per call against 11.0).
template <typename T, int D, bool WIDE, int PARTS, typename O>
__global__ void __launch_bounds__(Shape<T, D>::kThreads, Shape<T, D>::kOcc) attend_paged_rows_kernel(PagedArgs a, int blocks) {
  using S = Shape<T, D>;
  using St = Stream<T, D, WIDE, PARTS>;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t masks[kWarps][S::kStages];
  __shared__ float mm[kWarps][16], ll[kWarps][16];
  __shared__ float2 ml[16];  // the block's m and l of each head
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int rank = blockIdx.x % blocks;
  const int64_t row = blockIdx.x / blocks;
  const int b = (int)(row / a.heads), h = (int)(row - (int64_t)b * a.heads), g = a.group;
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int steps = row_steps(len, a.max_len, S::kTok), step0 = rank * kWarps + warp, team = blocks * kWarps;
  const int n = step0 < steps ? (steps - step0 + team - 1) / team : 0;
  St st;
  stream_row<T, D, WIDE, PARTS>(st, a, row, a.table + (int64_t)b * a.max_blocks, h, len, step0, n, team, smem_addr(smem) + warp * S::kRing,
                                masks[warp], St::kQInSmem ? smem_addr(smem) + S::kSmem : 0, warp, lane);
  float *buf = reinterpret_cast<float *>(smem), *sums = buf + kWarps * 16 * padded_row<T, D>();  // [16][D] behind the warps' rows
  static_assert(sizeof(float) * 16 * (kWarps * padded_row<T, D>() + D) <= S::kSmem, "the block's sums fit behind its warps'");
  O *out = static_cast<O *>(a.out) + row * g * a.d;
  join_warps<T, D, WIDE, PARTS>(st, a, buf, mm, ll, warp, lane, [&](int hd, int c, const float4 &v, float top, float sum) {
    if (blocks == 1) {
      put_out(out + hd * a.d + c, v, sum);
      return;
    }
    *reinterpret_cast<float4 *>(sums + hd * D + c) = v;
    if (c == 0) ml[hd] = make_float2(top, sum);
  });
  if (blocks == 1) return;
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  // each block joins a share of the channels, the blocks' sums in their order
  for (int idx = threadIdx.x * blocks + rank; idx < g * (D / 4); idx += kThreads * blocks) {
    const int hd = idx / (D / 4), c = 4 * (idx % (D / 4));
    if (c >= a.d) continue;
    float m = -INFINITY, l = 0.f;
    float2 pml[8];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f), po[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= blocks) break;
      unsigned at_ml, at_o;
      asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at_ml) : "r"(smem_addr(ml + hd)), "r"(i));
      asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at_o) : "r"(smem_addr(sums + hd * D + c)), "r"(i));
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];\n" : "=f"(pml[i].x), "=f"(pml[i].y) : "r"(at_ml) : "memory");
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                   : "=f"(po[i].x), "=f"(po[i].y), "=f"(po[i].z), "=f"(po[i].w)
                   : "r"(at_o)
                   : "memory");
      m = fmaxf(m, pml[i].x);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= blocks) break;
      const float f = pml[i].x == -INFINITY ? 0.f : exp2a(pml[i].x - m);
      l = fmaf(f, pml[i].y, l);
      o.x = fmaf(f, po[i].x, o.x);
      o.y = fmaf(f, po[i].y, o.y);
      o.z = fmaf(f, po[i].z, o.z);
      o.w = fmaf(f, po[i].w, o.w);
    }
    put_out(out + hd * a.d + c, o, l);
  }
  // no block leaves while another still reads its shared memory
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Joins the pieces of rows that several workers shared: blocks (x, y), rows x, x + gridDim.x, ..., vectors of
// four channels from y * vecs on.  A block holds as many groups of `vecs` threads as it has room for, which
// take pieces in turn, four in flight per thread, and meet in shared memory.  Latency bounds it (a few hundred
// KB in all): with few rows, of many pieces each, the host cuts them into small ranges of vectors (one row of
// 296 pieces, 8 heads of 128 channels: 70 us in one range).
constexpr int kMergeThreads = 256;
template <typename O>
__global__ void __launch_bounds__(kMergeThreads) attend_paged_merge_kernel(PagedArgs a, int warps, int vecs) {
  __shared__ float4 so[kMergeThreads];
  __shared__ float2 ml[kMergeThreads];
  const int g = a.group, tid = threadIdx.x, groups = kMergeThreads / vecs, grp = tid / vecs;
  const int v = blockIdx.y * vecs + tid - grp * vecs;
  const bool on = grp < groups && 4 * v < g * a.d;
  const int hd = on ? 4 * v / a.d : 0;
  const int64_t stride = piece_floats(g, a.d);
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  for (int64_t row = blockIdx.x; row < (int64_t)a.batch * a.heads; row += gridDim.x) {
    const int2 own = a.owner[row];
    if (own.y == 0) continue;
    const int n = abs(own.y), apart = own.y < 0 ? 1 : warps;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](float pm, float pl, const float4 &po) {
      if (pm == -INFINITY && pl == 0.f) return;  // no token; one whose logits are all NaN passes them on
      const float to = fmaxf(m, pm), f0 = exp2a(m - to), f1 = exp2a(pm - to);
      m = to;
      l = l * f0 + pl * f1;
      o.x = o.x * f0 + po.x * f1;
      o.y = o.y * f0 + po.y * f1;
      o.z = o.z * f0 + po.z * f1;
      o.w = o.w * f0 + po.w * f1;
    };
    for (int p0 = grp; on && p0 < n; p0 += 4 * groups) {
      float pm[4], pl[4];
      float4 po[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = p0 + i * groups;
        pm[i] = -INFINITY;
        pl[i] = 0.f;
        if (p < n) {
          // a worker's two pieces: of a row that began before it, and of the row that it begins
          const float *piece = a.piece + ((int64_t)(own.x + p * apart) * 2 + (p == 0 ? 1 : 0)) * stride;
          pm[i] = piece[g * a.d + hd];
          pl[i] = piece[g * a.d + g + hd];
          po[i] = reinterpret_cast<const float4 *>(piece)[v];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) join(pm[i], pl[i], po[i]);
    }
    if (groups > 1) {
      so[tid] = o;
      ml[tid] = make_float2(m, l);
      __syncthreads();
      if (grp == 0 && on)
        for (int i = 1; i < groups; ++i) join(ml[tid + i * vecs].x, ml[tid + i * vecs].y, so[tid + i * vecs]);
      __syncthreads();
    }
    if (grp == 0 && on) put_out(static_cast<O *>(a.out) + row * g * a.d + 4 * v, o, l);
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

// The workspace: the rows' owners, and two pieces for each warp of the largest grid.  One size serves both
// cache types.
size_t owner_bytes(const tq_pages &p) { return (size_t)tq_align_up((int64_t)p.batch * p.n_kv_heads * sizeof(int2), 256); }
template <int D>
int most_workers(int device) {
  return tq_device_sms(device) * std::max(Shape<float, D>::kOcc * Shape<float, D>::kWarps, Shape<__nv_bfloat16, D>::kOcc * Shape<__nv_bfloat16, D>::kWarps);
}
int most_workers(int device, int d) {
  return d <= 64 ? most_workers<64>(device) : d <= 128 ? most_workers<128>(device) : most_workers<256>(device);
}

// Steps of a warp up to which whole rows are taken where they fill less than half of the GPU, and twice as many
// where they fill more.  Beyond, other blocks' bandwidth is worth the deal and the join.  us per call, whole
// rows against dealt: bf16, 128 channels, 8 rows x 2000 tokens (4 steps) 9.8 / 12.0, x 4000 (8) 11.8 / 12.3;
// 256 channels, 8 x 1000 (3) 10.9 / 12.3, x 2000 (6) 15.7 / 12.7; fp32, 128 channels, 8 x 1000 (4)
// 9.9 / 12.0, x 2000 (8) 14.4 / 12.7; more than half full: bf16, 32 x 4096 (8) 16.7 / 19.7; fp32, 128 x 500 (8)
// 18.8 / 26.0; bf16, 256 rows of 1 .. 500 (8) 12.3 / 17.0; 64 channels, 128 x 2000 (16) 19.8 / 20.8, but of
// 1 .. 2000 17.0 / 14.5: whole rows do not even out lengths.
template <typename T, int D>
constexpr int kRowsSteps = sizeof(T) == 2 ? (D < 256 ? 8 : 4) : 32768 / Shape<T, D>::kStage;

template <typename T, int D, bool WIDE, int PARTS, typename O>
cudaError_t launch(const PagedArgs &a, int device, cudaStream_t st) {
  using S = Shape<T, D>;
  constexpr int kSmem = Stream<T, D, WIDE, PARTS>::kSmem;
  const int64_t rows = (int64_t)a.batch * a.heads, row_steps = a.max_len <= S::kTok ? 1 : (a.max_len - 1) / S::kTok + 1;
  const int64_t room_rows = (int64_t)S::kOcc * tq_device_sms(device);
  // whole rows, if each has room for a cluster at once and no warp has too many steps, however the lengths
  // differ
  int blocks = 8;
  while (blocks > 1 && (rows * blocks > room_rows || row_steps <= blocks * S::kWarps / 2)) blocks /= 2;
  const int most = kRowsSteps<T, D> * (2 * rows * blocks > room_rows ? 2 : 1);
  if (rows * blocks <= room_rows && row_steps <= (int64_t)most * blocks * S::kWarps) {
    auto kern = attend_paged_rows_kernel<T, D, WIDE, PARTS, O>;
    cudaError_t e = tq_smem_limit(reinterpret_cast<const void *>(kern), kSmem);
    if (e != cudaSuccess) return e;
    tq_prof_begin(TQK_ATTEND_PAGED, st);
    e = tq_launch_clusters(kern, blocks, dim3((unsigned)(rows * blocks)), S::kThreads, kSmem, st, a, blocks);
    tq_prof_end(TQK_ATTEND_PAGED, st);
    return e;
  }
  auto kern = attend_paged_kernel<T, D, WIDE, PARTS, O>;
  cudaError_t e = tq_smem_limit(reinterpret_cast<const void *>(kern), kSmem);
  if (e != cudaSuccess) return e;
  // as many blocks as fit on the GPU at once, fewer where the rows could not give each warp a step
  const int grid = (int)std::min((rows * row_steps + S::kWarps - 1) / S::kWarps, room_rows);
  tq_prof_begin(TQK_ATTEND_PAGED, st);
  e = tq_launch_dependent(kern, dim3((unsigned)grid), S::kThreads, kSmem, st, a);
  tq_prof_end(TQK_ATTEND_PAGED, st);
  if (e != cudaSuccess) return e;
  // the vectors of a row cut into ranges while all blocks fit on the GPU at once
  const int vecs = a.group * a.d / 4, room = 8 * tq_device_sms(device);
  const int cuts = (int)std::max((int64_t)1, std::min((int64_t)room / rows, (int64_t)(vecs + 15) / 16));
  const int each = std::min(kMergeThreads, (vecs + cuts - 1) / cuts);
  const dim3 mgrid((unsigned)std::min(rows, (int64_t)room), (unsigned)((vecs + each - 1) / each));
  tq_prof_begin(TQK_ATTEND_PAGED_MERGE, st);
  e = tq_launch_dependent(attend_paged_merge_kernel<O>, mgrid, kMergeThreads, 0, st, a, (int)S::kWarps, each);
  tq_prof_end(TQK_ATTEND_PAGED_MERGE, st);
  return e;
}

template <typename T, int PARTS, typename O>
cudaError_t launch_d(const PagedArgs &a, int device, cudaStream_t st) {
  const bool wide = a.group > 8;
  if (a.d <= 64) return wide ? launch<T, 64, true, PARTS, O>(a, device, st) : launch<T, 64, false, PARTS, O>(a, device, st);
  if (a.d <= 128) return wide ? launch<T, 128, true, PARTS, O>(a, device, st) : launch<T, 128, false, PARTS, O>(a, device, st);
  return wide ? launch<T, 256, true, PARTS, O>(a, device, st) : launch<T, 256, false, PARTS, O>(a, device, st);
}

}  // namespace

extern "C" tq_status tq_attend_paged_workspace_size(const tq_pages *pages, int32_t max_seq_len, int32_t n_q_heads,
                                                    int32_t d, size_t *bytes) {
  tq_status st = check_attend(pages, max_seq_len, n_q_heads, d);
  if (st != TQ_OK) return st;
  if (!bytes) return tq_fail(TQ_EINVAL, "bytes is NULL");
  *bytes = owner_bytes(*pages) + sizeof(float) * 2 * (size_t)most_workers(pages->device, d) * piece_floats(n_q_heads / pages->n_kv_heads, d);
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
              q, k_cache, v_cache, out, FastDiv(pages->block_size), nullptr, nullptr};
  a.owner = static_cast<int2 *>(ws);
  a.piece = reinterpret_cast<float *>(static_cast<char *>(ws) + owner_bytes(*pages));
  cudaError_t e = dtype == TQ_F32       ? launch_d<float, 2, float>(a, pages->device, s)
                  : out_dtype == TQ_F32 ? launch_d<__nv_bfloat16, 3, float>(a, pages->device, s)
                                        : launch_d<__nv_bfloat16, 2, __nv_bfloat16>(a, pages->device, s);
  return tq_cuda_check(e, "paged attention launch");
}
