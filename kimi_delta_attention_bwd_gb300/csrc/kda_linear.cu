// Linear attention with one decay per head: per document and head, tokens in
// order, a = exp(A_log[h]),
//   S_t = e^-a S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// its backward, and the single-token step.
//
// Chunk form (C = 64 tokens, entry state S, local index i, exit state S'):
//   o_i = scale (e^{-a(i+1)} S^T q_i + sum_{j<=i} e^{-a(i-j)} (q_i . k_j) v_j)
//   S'  = e^{-an} S + sum_j e^{-a(n-1-j)} k_j v_j^T
// Every gradient is the same operator on other operands, with R the gradient
// of the state:
//   dq: x = dO, y = v, z = k, state S^T, tokens in order
//   dk: x = v, y = dO, z = q, state R^T, tokens in reverse
//   dv: x = k, y = q, z = dO, state R,   tokens in reverse
// (out_i = scale (row_i x_i . S + sum_j e^{-a|i-j|} (x_i . y_j) z_j)).  In reverse
// the chain carries R / scale; a token's own contribution reaches R after its
// decay step, so the row weight is e^{-a i} and the state weight e^{-a(n-j)}.
//
// bf16: the forward's chain keeps every chunk's entry state S and the dv chain
// its exit state's gradient R, so that dq and dk need no chain of their own:
// one kernel over all chunks at once forms both from the pairs
// P = scale e^{-a(i-j)} (dO_i . v_j) that they share (lin_dqk).
//
// Decay gradient: with a exponent per token distance,
//   dL/da = -(A + B + C + D), all sums of products of one sign pattern (no
//   difference of large position sums):
//   A  pairs inside a chunk, sum_{j<i} (i-j) e^{-a(i-j)} scale (dO_i . v_j)(q_i . k_j)
//   B  entry state to row, sum_i (i+1) e^{-a(i+1)} scale q_i . S dO_i
//   C  row to exit state, sum_j (n-1-j) e^{-a(n-1-j)} k_j . R v_j
//   D  entry state to exit state, n e^{-an} <S, R>
//
// The state stays in fp32 registers for a whole chain.  Operands that are not
// inputs are split into bf16 parts: two (off by 2^-16 at most) where the
// product ends in a bf16 output (the pairs and the state's rows), so that its only
// rounding that counts is its own, and three (2^-24) where it enters the fp32
// state or the decay gradient's sums.  The second part of pairs and state rows costs
// the chains 20 to 27% and lin_dqk 2 to 5% (300M prompt's chain 31 -> 37 us); one
// part gave the outputs a 2-norm error of 2.35e-3 instead of 1.66e-3.  (The forms
// compared at the states' layout and at lin_dqk's chains, tiles, prefetch and list
// of pairs were timed with pairs of one part.)  fp32 io: kda_linear_f32.cu.
#include "kda_linear.cuh"

namespace kda {

kda_status check_problem(const kda_problem* p, Dims* d);

namespace lin {
namespace {

constexpr int LIN_SMS = 152;  // SMs of a GB300, for the segment rule
constexpr int SEG_TOK = 256;  // shortest segment (tokens)

// Inclusive scan of x over the 1024-thread block; the block's sum in *total.
__device__ __forceinline__ int block_scan(int x, int* s_w, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_w[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = s_w[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_w[lane] = y;
  }
  __syncthreads();
  x += warp ? s_w[warp - 1] : 0;
  *total = s_w[31];
  __syncthreads();
  return x;
}

// The unit table of packed documents: a document of n tokens has max(1,
// ceil(n / L)) units, of equal length but for the last, and ceil(n / C) chunks.  One CTA; also validates the
// offsets.
__global__ void __launch_bounds__(1024) lin_table_kernel(LinP P) {
  __shared__ int s_bad, s_long, s_w[32];
  const int tid = threadIdx.x, n = P.n_docs;
  pdl_release();
  if (tid == 0) {
    s_bad = P.cu[0] != 0 || P.cu[n] != P.Ntok;
    s_long = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += 1024)
    if (P.cu[i + 1] < P.cu[i]) s_bad = 1;
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      *P.err = KDA_ERR_BAD_SEQLENS;
      *P.wtag = 0;
      P.counts[0] = P.counts[1] = P.counts[2] = 0;
    }
    return;
  }
  int units = 0, chunks = 0;
  for (int base = 0; base < n; base += 1024) {
    const int i = base + tid;
    const int t0 = i < n ? P.cu[i] : 0, len = i < n ? P.cu[i + 1] - t0 : 0;
    // (no document is cut without the kernels that form the pieces' states, whatever the host's offsets said)
    const int L = P.seg ? seg_tokens(P.L, len) : max(len, 1);
    const int ns = i < n ? max(1, (len + L - 1) / L) : 0, nc = (len + C - 1) / C;
    int all;
    const int u0 = units + block_scan(ns, s_w, &all) - ns;
    units += all;
    const int c0 = chunks + block_scan(nc, s_w, &all) - nc;
    chunks += all;
    for (int s = 0; s < ns; s++) {
      P.units[u0 + s] = make_int4(i, t0 + s * L, min(L, len - s * L), s);
      P.unit_at[u0 + s] = make_int2(c0 + s * (L / C), ns);
    }
    if (ns > 1) P.longs[atomicAdd(&s_long, 1)] = make_int2(u0, ns);  // (in any order: they are independent)
  }
  __syncthreads();
  if (tid == 0) {  // units <= n + Ntok / L, chunks <= (Ntok + (C - 1) n) / C, split documents <= Ntok / L
    P.counts[0] = units;
    P.counts[1] = chunks;
    P.counts[2] = s_long;
    *P.err = KDA_OK;
    *P.wtag = P.save ? P.tag : 0;
  }
}

// Turns the segments' own states into their start states, in place and in the
// chain's direction: start_0 = init, start_{s+1} = e^{-a len_s} start_s + own_s.  A
// thread per four elements of a (split document, head)'s state, eight segments'
// loads in flight; the CTAs loop over the pieces, whose number the device alone
// may know (a grid of its bound, mostly empty, took 36 to 62 us).
constexpr int FTH = 128, FCTAS = 8 * LIN_SMS;
__global__ void __launch_bounds__(FTH) lin_fold_kernel(LinP P, float* segc, const float* init, int rev, int N,
                                                       int fwd) {
  pdl_wait();
  pdl_release();
  if (!ready(P, fwd)) return;
  constexpr int F = 8;
  const int pieces = N / (4 * FTH);
  const int64_t total = (int64_t)(P.rows ? P.n_long : P.counts[2]) * P.H * pieces;
  for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
    const int at = ((int)(item % pieces) * FTH + threadIdx.x) * 4, dh = (int)(item / pieces);
    const int d = dh / P.H, h = dh % P.H;
    int u0, ns, doc, len, last;
    if (P.rows) {
      ns = (P.T + P.L - 1) / P.L;
      u0 = d * ns;
      doc = d;
      len = P.L;
      last = P.T - (ns - 1) * P.L;
    } else {
      u0 = P.longs[d].x;
      ns = P.longs[d].y;
      doc = P.units[u0].x;
      len = P.units[u0].z;
      last = P.units[u0 + ns - 1].z;
    }
    const float a = decay_of(P.A_log, h), full = decay_pow(a, len), first = rev ? decay_pow(a, last) : full;
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init) {
      st = *reinterpret_cast<const float4*>(init + ((int64_t)doc * P.H + h) * N + at);
      const float m = rev ? 1.0f / P.scale : 1.0f;
      st.x *= m; st.y *= m; st.z *= m; st.w *= m;
    }
    auto own = [&](int k) -> float4* {  // k-th segment in the chain's direction
      return reinterpret_cast<float4*>(segc + ((int64_t)(u0 + (rev ? ns - 1 - k : k)) * P.H + h) * N + at);
    };
    float4 v[F], nx[F];
#pragma unroll
    for (int e = 0; e < F; e++)
      if (e < ns - 1) v[e] = *own(e);
    *own(0) = st;
    for (int k = 0; k < ns - 1; k += F) {
      // (start k + F goes where own state k + F was: the next F are read first)
#pragma unroll
      for (int e = 0; e < F; e++)
        if (k + F + e < ns - 1) nx[e] = *own(k + F + e);
#pragma unroll
      for (int e = 0; e < F; e++)
        if (k + e < ns - 1) {
          const float g = k + e == 0 ? first : full;
          st.x = fmaf(g, st.x, v[e].x);
          st.y = fmaf(g, st.y, v[e].y);
          st.z = fmaf(g, st.z, v[e].z);
          st.w = fmaf(g, st.w, v[e].w);
          *own(k + e + 1) = st;
        }
#pragma unroll
      for (int e = 0; e < F; e++) v[e] = nx[e];
    }
  }
}

// ------------------------------------------------------------ bf16 chain
constexpr int PART = 10 * 512;  // bytes of a part of a chunk's pairs (pair_at)
// ONLY: state only (a segment's own state), no output rows.
template <int DK, int DVS, bool ONLY>
struct Shape {
  // 16-row tiles of the state per warp: two where the registers hold them, so that every operand
  // fragment read from shared memory serves two products
  static constexpr int MT = DK == 128 ? 1 : 2;
  static constexpr int NW = DVS / (16 * MT), NTH = 32 * NW;
  // bytes of the tiles of a stage (multiples of the swizzle's 1024)
  static constexpr int XB = ONLY ? 0 : 128 * DK, YB = 128 * DK, ZB = 128 * DVS;
  static constexpr int STAGE = XB + YB + ZB;
  static constexpr int STG = DK == 128 || ONLY ? 2 : 1;
  static constexpr int PB = ONLY ? 0 : 2 * PART, OB = ONLY ? 0 : 128 * DVS;
  static constexpr int SMEM = 1024 /* alignment */ + STG * STAGE + PB + OB + 1024 /* lut */ + 272 /* tab */ + 512 + 32;
  static constexpr int NTK = DK / 8;  // 8-key tiles of a warp's state rows
  // resident CTAs: what registers and shared memory allow
  static constexpr int REGS = DK == 32 ? 168 : 255;
  static constexpr int BY_REG = 65536 / (NTH * REGS), BY_SMEM = 227 * 1024 / (SMEM + 1024);
  static constexpr int CTAS = BY_REG < BY_SMEM ? (BY_REG < 1 ? 1 : BY_REG) : BY_SMEM;
};

// Fragments of a 64-row bf16 tile of W columns as TMA's 128-byte (W = 32:
// 64-byte) swizzle lays it out; W = 128 is two tiles of 64 columns.  Pattern 1
// (the 16 x 16 block's rows by bit 0 of the 8 x 8 matrix index, columns by bit
// 1) reads A(m, k) = X[m][k] and, transposed, B(k, n) = X[k][n]; pattern 2 the
// other two.
template <int W, int PAT>
struct Frag {
  uint32_t row, x;  // the lane's row offset and its swizzle term
  __device__ __forceinline__ Frag() {
    const int lane = threadIdx.x & 31, l7 = lane & 7, mi = lane >> 3;
    const int r = PAT == 1 ? mi & 1 : mi >> 1, b = PAT == 1 ? mi >> 1 : mi & 1;
    row = (l7 + 8 * r) * (W == 32 ? 64 : 128);
    x = (uint32_t)(b ^ (W == 32 ? (l7 >> 1) & 3 : l7)) << 4;
  }
  // block of rows r0 .. (a multiple of 8), columns c0 .. (a multiple of 16)
  __device__ __forceinline__ uint32_t at(uint32_t base, int r0, int c0) const {
    if (W == 32) return base + r0 * 64 + row + (((uint32_t)c0 * 2) ^ x);
    return base + (c0 >> 6) * 8192 + r0 * 128 + row + (((uint32_t)(c0 & 63) * 2) ^ x);
  }
};
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// Transposes 8x8 tiles on the way to shared memory (register pairs along rows).
__device__ __forceinline__ void stsm4t(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(mma::smem_u32(p)), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float even(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float odd(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The 16 x 16 blocks (row r, column c <= r) of a chunk's pairs, ten over four
// warps or two: a warp's list, 4 r + c each.  Blocks of a list that share a row
// or a column share that operand's fragments.
template <int... RC>
struct Blocks {
  static constexpr int N = sizeof...(RC);
  static __host__ __device__ constexpr int row(int t) {
    const int rc[N] = {RC...};
    return rc[t] >> 2;
  }
  static __host__ __device__ constexpr int col(int t) {
    const int rc[N] = {RC...};
    return rc[t] & 3;
  }
  static __host__ __device__ constexpr bool has_row(int r) { return ((RC >> 2 == r) || ...); }
  static __host__ __device__ constexpr bool has_col(int c) { return (((RC & 3) == c) || ...); }
};
template <int NW, class F>
__device__ __forceinline__ void for_my_blocks(int warp, F f) {
  if constexpr (NW == 2) {
    if (warp == 0) f(Blocks<12, 13, 14, 15, 0>());
    else f(Blocks<8, 9, 10, 4, 5>());
  } else {
    if (warp == 0) f(Blocks<12, 13, 14>());
    else if (warp == 1) f(Blocks<8, 9, 10>());
    else if (warp == 2) f(Blocks<4, 5, 15>());
    else f(Blocks<0>());
  }
}
// p[t] = block t of x y^T over DK columns; row(r) and col(c) load fragments of a
// 16-row block at column 16 kk.
template <int DK, class B, class FR, class FC>
__device__ __forceinline__ void pair_products(float (&p)[B::N][2][4], FR row, FC col) {
#pragma unroll
  for (int t = 0; t < B::N; t++) mma::zero<2>(p[t]);
#pragma unroll
  for (int kk = 0; kk < DK / 16; kk++) {
    uint32_t fa[4][4], fb[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (B::has_row(i)) row(fa[i], i, kk);
      if (B::has_col(i)) col(fb[i], i, kk);
    }
#pragma unroll
    for (int t = 0; t < B::N; t++) {
      mma::mma_bf16(p[t][0], fa[B::row(t)], fb[B::col(t)][0], fb[B::col(t)][1]);
      mma::mma_bf16(p[t][1], fa[B::row(t)], fb[B::col(t)][2], fb[B::col(t)][3]);
    }
  }
}
// A chunk's pairs in shared memory, two parts of the ten 16 x 16 blocks: rows of
// 32 bytes whose two halves change places in every other group of four, so that
// eight rows of a half lie in different banks.  (Whole 64 x 64 parts take the
// 32/64 kernels' sixth CTA off an SM: 300M prompt 70 us, 57 so.)
__host__ __device__ constexpr int pair_at(int r, int c) { return (r * (r + 1) / 2 + c) * 512; }
// A lane's offset in a block; PAT as Frag's.
template <int PAT>
__device__ __forceinline__ uint32_t pair_lane() {
  const int lane = threadIdx.x & 31, l7 = lane & 7, mi = lane >> 3;
  const int r = PAT == 1 ? mi & 1 : mi >> 1, b = PAT == 1 ? mi >> 1 : mi & 1;
  return (l7 + 8 * r) * 32 + ((b ^ (l7 >> 2)) << 4);
}
// Weights the pairs (lut: weights of a pair of neighbouring columns by distance,
// index 64 at distance 0; sign: +1 where rows come after columns) and stores
// them as two parts in tP, blocks in the chain's order.
template <class B>
__device__ __forceinline__ void pair_store(float (&p)[B::N][2][4], const float2* lut, unsigned char* tP, int sign) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const float2* lp = lut + 64 + sign * (gq - 2 * tq);
  unsigned char* pp = tP + gq * 32 + 4 * tq;
#pragma unroll
  for (int t = 0; t < B::N; t++) {
    const int r = B::row(t), c = B::col(t);
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int k = 0; k < 2; k++) {
        // (in reverse a later block lies before: its distance is positive too)
        const float2 w = lp[16 * (r - c) + sign * (8 * k - 8 * j)];
        p[t][j][2 * k] *= w.x;
        p[t][j][2 * k + 1] *= w.y;
        uint32_t s[2];
        split2<2>(p[t][j][2 * k], p[t][j][2 * k + 1], s);
        unsigned char* at = pp + pair_at(r, c) + 256 * k + ((j ^ (gq >> 2)) << 4);
        *reinterpret_cast<uint32_t*>(at) = s[0];
        *reinterpret_cast<uint32_t*>(at + PART) = s[1];
      }
  }
}

// The tensors of a chain as [Ntok][H d] maps with boxes of 64 tokens.
struct LinMaps {
  CUtensorMap x, y, z, o;
};

// A 64-token x box tile of shared memory (in the map's swizzle) to a tensor.
__device__ __forceinline__ void tma_store_2d(const void* map, int x0, int y0, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(x0),
               "r"(y0), "r"(mma::smem_u32(src))
               : "memory");
}

// Rows n .. of a stage's tiles hold other documents' tokens: zero them, so that
// nothing of them (an infinity) enters a product.  The first A bytes are rows of
// RA bytes, the others of RB; a tile (or 64-column half of one) has 64 rows.
template <int BYTES, int A, int RA, int RB, int NTH>
__device__ __forceinline__ void zero_rows(unsigned char* stg, int n) {
  if (n == C) return;
  for (int b = 16 * threadIdx.x; b < BYTES; b += 16 * NTH) {
    const int row = b < A ? (b / RA) & 63 : ((b - A) / RB) & 63;
    if (row >= n) *reinterpret_cast<uint4*>(stg + b) = make_uint4(0, 0, 0, 0);
  }
}

// A warp's 16 columns (from c0) of an output, accumulator fragments of its
// transpose with token block t at 16 (rev ? 3 - t : t), into a 64 x W tile in the
// maps' swizzle.
template <int W>
__device__ __forceinline__ unsigned char* tile_at(unsigned char* tile, int row, int cg) {
  return W == 32 ? tile + row * 64 + ((cg ^ ((row >> 1) & 3)) << 4) : tile + row * 128 + ((cg ^ (row & 7)) << 4);
}
template <int W>
__device__ __forceinline__ void stage_tile(unsigned char* tile, int c0, const float (&o)[8][4], bool rev) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int p = 0; p < 4; p++) {  // four 8 x 8 tiles: 16 tokens by 16 columns
    const int row = 16 * (rev ? 3 - p : p) + 8 * (lane >> 4) + (lane & 7), cg = c0 / 8 + ((lane >> 3) & 1);
    stsm4t(tile_at<W>(tile, row, cg), pack2(o[2 * p][0], o[2 * p][1]), pack2(o[2 * p][2], o[2 * p][3]),
           pack2(o[2 * p + 1][0], o[2 * p + 1][1]), pack2(o[2 * p + 1][2], o[2 * p + 1][3]));
  }
}
// The warp's NC columns (from c0) of the tile's first n rows to rows ld apart:
// for a chunk that is not full.
template <int W, int NC>
__device__ __forceinline__ void copy_rows(const unsigned char* tile, int c0, bf16* out, int64_t ld, int n) {
  __syncwarp();
  for (int g = threadIdx.x & 31; g < n * (NC / 8); g += 32) {
    const int row = g / (NC / 8), cg = c0 / 8 + g % (NC / 8);
    *reinterpret_cast<uint4*>(out + row * ld + 8 * cg) =
        *reinterpret_cast<const uint4*>(tile_at<W>(const_cast<unsigned char*>(tile), row, cg));
  }
}

// One CTA carries one chain of a DVS-column value slice.  Warp w holds MT x 16
// value rows of S^T as fp32 accumulator fragments for the whole
// chain; per chunk
//   pairs  P = w (x y^T), the ten 16 x 16 blocks on and below the diagonal
//          shared out over the warps, to shared memory
//   o^T    = row weight * (S^T x^T) (S as register fragments) + z^T P^T
//   S^T    = e^{-an} S^T + (weighted z)^T y
// so that the state never leaves its registers and a chunk needs two barriers;
// the state's product comes last, when the output's registers are free.
// Tokens lie in memory order in both directions; in reverse the blocks are
// walked from the other end (blk) and the weights run the other way.
// mma.sync rather than tcgen05: the chain is bound by the instructions around
// its products, and accumulators that are the next product's operands save
// the round trips through TMEM and shared memory (300M layer, 16 x 2048: 37 us,
// the tcgen05 form 87 before the steps that both could take; 128/128, 4 x 8192:
// 315 us at 3.5 TB/s with the chunk states, tensor pipe 60%).
template <int DK, int DVS, bool ONLY, bool rev>
__device__ void chain(const LinP& P, const LinOp& op, const LinMaps& maps, int u, int h, int slice) {
  using SH = Shape<DK, DVS, ONLY>;
  constexpr int NTH = SH::NTH, NW = SH::NW, NTK = SH::NTK, MT = SH::MT;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (mma::smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* tP = smem + SH::STG * SH::STAGE;  // the pairs, blocks in the chain's order
  unsigned char* tO = tP + SH::PB;                 // [64][DVS], the output's rows
  float2* lut = reinterpret_cast<float2*>(tO + SH::OB);
  float* tab = reinterpret_cast<float*>(lut + 128);  // [65] e^{-a m}
  float* sw = tab + 68;                              // [64] weights of the chunk's rows in its state
  float* rwt = sw + 64;                              // [64] weights of the entry state in its rows
  uint64_t* bar = reinterpret_cast<uint64_t*>(rwt + 64);  // [STG]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;

  Unit un;
  if (!unit_of(P, u, un)) return;
  if (ONLY && un.seg == (rev ? 0 : un.nseg - 1)) return;  // the last segment of its direction feeds nobody
  const int H = P.H, DVt = op.DVt, c0 = slice * DVS;
  const int64_t stN = (int64_t)DK * DVt;
  const float a = decay_of(P.A_log, h);
  const int nch = (un.ntok + C - 1) / C;
  auto blk = [&](int t) { return rev ? 3 - t : t; };  // 16-token block t in the chain's direction

  auto load = [&](int c) {  // one thread
    const int t0 = un.tok0 + C * (rev ? nch - 1 - c : c), s = SH::STG == 2 ? c & 1 : 0;
    unsigned char* p = smem + s * SH::STAGE;
    mma::mbar_expect_tx(bar + s, SH::STAGE);
#pragma unroll
    for (int b = 0; b < (DK + 63) / 64; b++) {
      if constexpr (!ONLY) mma::tma_load_2d(p + 8192 * b, &maps.x, h * DK + 64 * b, t0, bar + s);
      mma::tma_load_2d(p + SH::XB + 8192 * b, &maps.y, h * DK + 64 * b, t0, bar + s);
    }
    mma::tma_load_2d(p + SH::XB + SH::YB, &maps.z, h * DVt + c0, t0, bar + s);
  };
  if (tid == 0) {
    for (int s = 0; s < SH::STG; s++) mma::mbar_init(bar + s, 1);
    mma::mbar_init_fence();
    if (nch > 0) load(0);
  }
  for (int i = tid; i < 65; i += NTH) tab[i] = decay_pow(a, i);
  __syncthreads();
  for (int i = tid; i < 128; i += NTH) {  // weights of a pair of neighbouring columns at distances m and m -+ 1
    const int m = i - 64, m2 = rev ? m + 1 : m - 1;
    lut[i] = make_float2(m >= 0 ? P.scale * tab[m] : 0.f, m2 >= 0 ? P.scale * tab[m2] : 0.f);
  }
  int n_w = -1;  // rows for which sw and rwt are set

  float S[MT][NTK][4];
#pragma unroll
  for (int m = 0; m < MT; m++) mma::zero<NTK>(S[m]);
  const int r0 = 16 * MT * warp;  // this warp's first value row
  auto each_at = [&](int tr, auto fn) {
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int j = 0; j < NTK; j++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          fn(S[m][j][e], st_at(tr, c0 + r0 + 16 * m + gq + 8 * (e >> 1), 8 * j + 2 * tq + (e & 1), DK, DVt));
  };
  if (!ONLY) start_state(P, op, un, u, h, stN, [&](auto fn) { each_at(0, fn); });

  const Frag<DK, 1> k1;   // x and y tiles
  const Frag<DK, 2> k2;
  const Frag<DVS, 2> v2;  // z tile
  const uint32_t p2 = mma::smem_u32(tP) + pair_lane<2>();

  bool good = true;
  int out_t0 = -1;  // first token of the output tile that waits in tO
  for (int c = 0; c < nch; c++) {
    const int idx = rev ? nch - 1 - c : c, t0 = un.tok0 + C * idx, n = min(C, un.ntok - C * idx);
    const int st = SH::STG == 2 ? c & 1 : 0;
    unsigned char* stg = smem + st * SH::STAGE;
    const uint32_t tX = mma::smem_u32(stg), tY = tX + SH::XB, tZ = tY + SH::YB;
    if (!ONLY && op.states) {
      // the state where the chain enters the chunk, in tiles of 16 values x 8 keys [value / 8][value % 2]
      // [value % 8 / 2][key]: a word of lin_dqk's operand fragments is 128 bytes of a tile, a pair stored here
      // fills whole sectors (128/128, the two chains and lin_dqk: [dv][dk] 614 + 521 us, the accumulators'
      // own order 569 + 483, this 560 + 484)
      float* p = op.states + ((int64_t)(un.ch0 + idx) * H + h) * stN + (int64_t)(c0 + r0) * DK + 32 * (gq & 1) +
                 8 * (gq >> 1) + 2 * tq;
      const float w = rev ? P.scale : 1.0f;
#pragma unroll
      for (int m = 0; m < MT; m++)
#pragma unroll
        for (int j = 0; j < NTK; j++)
#pragma unroll
          for (int k = 0; k < 2; k++)
            *reinterpret_cast<float2*>(p + 16 * m * DK + 128 * j + 64 * k) =
                make_float2(w * S[m][j][2 * k], w * S[m][j][2 * k + 1]);
      if (!rev && !P.rows && h == 0 && slice == 0 && tid == 0) P.chunks[un.ch0 + idx] = make_int2(t0, n);
    }
    good = mma::mbar_wait(bar + st, (SH::STG == 2 ? c >> 1 : c) & 1);
    if (n != n_w) {  // the first chunk, and the one that is not full
      if (n_w >= 0) __syncthreads();
      for (int i = tid; i < C; i += NTH) {
        sw[i] = i < n ? tab[rev ? i + 1 : n - 1 - i] : 0.f;
        rwt[i] = i < n ? P.scale * tab[rev ? n - 1 - i : i + 1] : 0.f;
      }
      n_w = n;
    }
    zero_rows<SH::STAGE, SH::XB + SH::YB, DK == 32 ? 64 : 128, DVS == 32 ? 64 : 128, NTH>(stg, n);
    mma::fence_async_smem();  // this thread's accesses to the other stage precede the copies into it
    // this chunk's tiles are complete; every reader of the last one is done
    if (__syncthreads_or(!good)) {
      good = false;
      break;
    }
    if (SH::STG == 2 && tid == 0 && c + 1 < nch) load(c + 1);

    if constexpr (!ONLY) {
      if (tid == 0 && out_t0 >= 0) {
        tma_store_2d(&maps.o, h * DVt + c0, out_t0, tO);
        mma::bulk_commit();
      }
      // ---- pairs
      for_my_blocks<NW>(warp, [&](auto blocks) {
        using B = decltype(blocks);
        float p[B::N][2][4];
        pair_products<DK, B>(
            p, [&](uint32_t (&f)[4], int r, int kk) { ldsm(f, k1.at(tX, 16 * blk(r), 16 * kk)); },
            [&](uint32_t (&f)[4], int c, int kk) { ldsm(f, k2.at(tY, 16 * blk(c), 16 * kk)); });
        pair_store<B>(p, lut, tP, rev ? -1 : 1);
      });
      if (tid == 0) mma::bulk_wait_read();  // tO is free again
      __syncthreads();                      // the pairs of every warp
      // ---- the entry state's rows: o^T = S^T x^T
      float o[MT][8][4];
#pragma unroll
      for (int m = 0; m < MT; m++) mma::zero<8>(o[m]);
#pragma unroll
      for (int kk = 0; kk < DK / 16; kk++) {
        uint32_t f[MT][2][4], fb[4][4];
#pragma unroll
        for (int p = 0; p < 4; p++) ldsm(fb[p], k2.at(tX, 16 * blk(p), 16 * kk));
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int q = 0; q < 4; q++) {  // accumulator tiles 2 kk, 2 kk + 1 are the 16 x 16 operand
            const float* st2 = &S[m][2 * kk + (q >> 1)][2 * (q & 1)];
            uint32_t s[2];
            split2<2>(st2[0], st2[1], s);
            f[m][0][q] = s[0];
            f[m][1][q] = s[1];
          }
#pragma unroll
        for (int b = 1; b >= 0; b--)
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int p = 0; p < 4; p++) {
              mma::mma_bf16(o[m][2 * p], f[m][b], fb[p][0], fb[p][1]);
              mma::mma_bf16(o[m][2 * p + 1], f[m][b], fb[p][2], fb[p][3]);
            }
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float2 w = *reinterpret_cast<const float2*>(rwt + 16 * blk(j >> 1) + 8 * (j & 1) + 2 * tq);
#pragma unroll
        for (int m = 0; m < MT; m++) {
          o[m][j][0] *= w.x;
          o[m][j][1] *= w.y;
          o[m][j][2] *= w.x;
          o[m][j][3] *= w.y;
        }
      }
      // ---- o^T += z^T P^T
#pragma unroll
      for (int kk = 0; kk < 4; kk++) {
        uint32_t zr[MT][4];
#pragma unroll
        for (int m = 0; m < MT; m++) ldsm_t(zr[m], v2.at(tZ, 16 * blk(kk), r0 + 16 * m));
#pragma unroll
        for (int b = 1; b >= 0; b--) {
          uint32_t fb[4][4];
#pragma unroll
          for (int p = kk; p < 4; p++) ldsm(fb[p], p2 + b * PART + pair_at(p, kk));
#pragma unroll
          for (int m = 0; m < MT; m++)
#pragma unroll
            for (int p = kk; p < 4; p++) {
              mma::mma_bf16(o[m][2 * p], zr[m], fb[p][0], fb[p][1]);
              mma::mma_bf16(o[m][2 * p + 1], zr[m], fb[p][2], fb[p][3]);
            }
        }
      }
      // ---- out: transposed into tO, and from there as a tile (a chunk that is not full: row by row)
#pragma unroll
      for (int m = 0; m < MT; m++) stage_tile<DVS>(tO, r0 + 16 * m, o[m], rev);
      out_t0 = n == C ? t0 : -1;
      if (n < C) copy_rows<DVS, 16 * MT>(tO, r0, (bf16*)op.out + ((int64_t)t0 * H + h) * DVt + c0, (int64_t)H * DVt, n);
    }
    // ---- the state: S^T = e^{-an} S^T + (weighted z)^T y.  The product is summed apart from the
    // state (the tensor core truncates what an addition shifts out: into a long chain's state that
    // would be a bias), smallest parts first.
    float d[MT][NTK][4];
#pragma unroll
    for (int m = 0; m < MT; m++) mma::zero<NTK>(d[m]);
#pragma unroll
    for (int kk = 0; kk < 4; kk++) {
      uint32_t za[MT][3][4], fb[NTK / 2][4];
#pragma unroll
      for (int p = 0; p < NTK / 2; p++) ldsm_t(fb[p], k1.at(tY, 16 * blk(kk), 16 * p));
      const float2 w0 = *reinterpret_cast<const float2*>(sw + 16 * blk(kk) + 2 * tq);
      const float2 w1 = *reinterpret_cast<const float2*>(sw + 16 * blk(kk) + 2 * tq + 8);
#pragma unroll
      for (int m = 0; m < MT; m++) {
        uint32_t zr[4];
        ldsm_t(zr, v2.at(tZ, 16 * blk(kk), r0 + 16 * m));
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const float2 w = q >> 1 ? w1 : w0;
          uint32_t s[3];
          split2<3>(w.x * even(zr[q]), w.y * odd(zr[q]), s);
#pragma unroll
          for (int b = 0; b < 3; b++) za[m][b][q] = s[b];
        }
      }
#pragma unroll
      for (int b = 2; b >= 0; b--)
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int p = 0; p < NTK / 2; p++) {
            mma::mma_bf16(d[m][2 * p], za[m][b], fb[p][0], fb[p][1]);
            mma::mma_bf16(d[m][2 * p + 1], za[m][b], fb[p][2], fb[p][3]);
          }
    }
    const Decay dec(a, n);
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int j = 0; j < NTK; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) S[m][j][e] = dec(S[m][j][e]) + d[m][j][e];
    if (SH::STG == 1 && c + 1 < nch) {
      mma::fence_async_smem();
      __syncthreads();
      if (tid == 0) load(c + 1);
    }
  }
  if (!ONLY && nch > 0) {  // the last output tile, and every tile's reads before the CTA ends
    mma::fence_async_smem();
    __syncthreads();
    if (tid == 0) {
      if (good && out_t0 >= 0) {
        tma_store_2d(&maps.o, h * DVt + c0, out_t0, tO);
        mma::bulk_commit();
      }
      mma::bulk_wait_all();
    }
  }
  if (!good) {  // a wait ran out
    if (tid == 0) *P.err = KDA_ERR_DEVICE;
    return;
  }

  // ---- the unit's state
  if (ONLY) {
    float* p = op.segc + ((int64_t)u * H + h) * stN;
    each_at(0, [&](float& s, int64_t at) { p[at] = s; });
  } else if (op.fin && un.seg == (rev ? 0 : un.nseg - 1)) {
    float* p = op.fin + ((int64_t)un.doc * H + h) * stN;
    const float mul = rev ? P.scale : 1.0f;
    each_at(0, [&](float& s, int64_t at) { p[at] = mul * s; });
  }
}

template <int DK, int DVS, bool ONLY, bool rev>
__global__ void __launch_bounds__(Shape<DK, DVS, ONLY>::NTH, Shape<DK, DVS, ONLY>::CTAS)
    lin_chain_kernel(const __grid_constant__ LinMaps maps, LinP P, LinOp op, int fwd) {
  pdl_wait();
  pdl_release();
  if (!ready(P, fwd)) return;
  const int ns = op.DVt / DVS;
  chain<DK, DVS, ONLY, rev>(P, op, maps, blockIdx.x / (ns * P.H), (blockIdx.x / ns) % P.H, blockIdx.x % ns);
}

// ------------------------------------------------------------ dq and dk, bf16
// Every chunk by itself, from its entry state S and its exit state's gradient
// R (fp32): with P = scale e^{-a(i-j)} (dO_i . v_j), i >= j,
//   dq_i = sum_j P_ij k_j + scale e^{-a(i+1)} S dO_i
//   dk_j = sum_i P_ij q_i + e^{-a(n-1-j)} R v_j
// and, with DA, the decay gradient's A, B, C, D.  A CTA takes CPB chunks of a
// head and a DVS-column slice of dk; warp w forms rows 16 w .. of dq^T and dk^T
// and reads its rows of S and R from memory as operand fragments, once (128/128,
// 4 x 8192: 484 us, 3.9 TB/s, tensor pipe 52%, without DA 424 us; three chains
// instead of it took 1.9 ms for the backward where this took 1.2).
constexpr int CPB = 4;

// A warp's blocks (row r, column c <= r) of the pairs, a byte 4 r + c + 1 each,
// 0 ends.
template <int NW>
__device__ __forceinline__ uint64_t pair_list(int warp) {
  if (NW == 2) return warp == 0 ? 0x01100f0e0dull : 0x06050b0a09ull;
  return warp == 0 ? 0x0f0e0dull : warp == 1 ? 0x0a0910ull : warp == 2 ? 0x050bull : 0x0106ull;
}

template <int DV, int DVS, bool DA>
struct DShape {
  static constexpr int NW = DVS / 16, NTH = 32 * NW;
  static constexpr int OB = 128 * DV, QB = 128 * DVS;  // bytes of the dO and v, the q and k tiles
  // one chunk's tiles: a second set would hide their loads, but takes more CTAs off the SM than that is worth
  // (32/64 74 us for 69, 64/64 at 8 x 4096 tokens 105 for 94)
  static constexpr int STAGE = 2 * OB + 2 * QB;
  static constexpr int PB = 2 * PART;
  static constexpr int SMEM = 1024 + STAGE + PB + 1024 /* lut */ + 272 /* tab */ + 512 + 32;
  // parts of the states as operands: the decay gradient's fp32 sums need the third, and dq and dk keep their bits
  // whether it is wanted or not
  static constexpr int SP = 3;
  static constexpr int BY_REG = 65536 / (NTH * 168), BY_SMEM = 227 * 1024 / (SMEM + 1024);
  static constexpr int CTAS = BY_REG < BY_SMEM ? BY_REG : BY_SMEM;
};

struct DqkMaps {
  CUtensorMap q, k, v, dO, dq, dk;
};
struct DqkOp {
  void *dq, *dk;
  const float *S, *R;
  double* pda;
};

template <int DV, int DVS, bool DA>
__global__ void __launch_bounds__(DShape<DV, DVS, DA>::NTH, DShape<DV, DVS, DA>::CTAS)
    lin_dqk_kernel(const __grid_constant__ DqkMaps maps, LinP P, DqkOp op, int DKt) {
  using SH = DShape<DV, DVS, DA>;
  constexpr int NTH = SH::NTH, NW = SH::NW, SP = SH::SP;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (mma::smem_u32(smem_raw) & 1023u)) & 1023u);
  unsigned char* tP = smem + SH::STAGE;  // the pairs
  float2* lut = reinterpret_cast<float2*>(tP + SH::PB);
  float* tab = reinterpret_cast<float*>(lut + 128);
  float* rq = tab + 68;  // [64] scale e^{-a(i+1)}
  float* rk = rq + 64;   // [64] e^{-a(n-1-j)}
  uint64_t* bar = reinterpret_cast<uint64_t*>(rk + 64);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int ns = DKt / DVS, slice = blockIdx.x % ns, h = (blockIdx.x / ns) % P.H, g0 = blockIdx.x / (ns * P.H) * CPB;
  pdl_wait();
  pdl_release();
  if (!ready(P, 0)) return;
  const int nchunks = P.rows ? P.nc : P.counts[1], nch = min(CPB, nchunks - g0);
  if (nch <= 0) {
    if (DA && tid == 0) op.pda[blockIdx.x] = 0.0;
    return;
  }
  const int H = P.H, c0 = slice * DVS;
  const float a = decay_of(P.A_log, h);
  auto chunk = [&](int c) -> int2 {  // {first token, tokens}
    const int g = g0 + c;
    if (!P.rows) return P.chunks[g];
    const int cpr = (P.T + C - 1) / C, r = g / cpr, i = g % cpr;
    return make_int2(r * P.T + i * C, min(C, P.T - i * C));
  };
  // A chunk's tiles, by one thread: dO and v on barrier 0, q and k on 1, each pair as soon as its place is free.
  auto load_ov = [&](int c) {
    const int t0 = chunk(c).x;
    mma::mbar_expect_tx(bar, 2 * SH::OB);
#pragma unroll
    for (int b = 0; b < (DV + 63) / 64; b++) {
      mma::tma_load_2d(smem + 8192 * b, &maps.dO, h * DV + 64 * b, t0, bar);
      mma::tma_load_2d(smem + SH::OB + 8192 * b, &maps.v, h * DV + 64 * b, t0, bar);
    }
  };
  auto load_qk = [&](int c) {
    const int t0 = chunk(c).x;
    mma::mbar_expect_tx(bar + 1, 2 * SH::QB);
    mma::tma_load_2d(smem + 2 * SH::OB, &maps.q, h * DKt + c0, t0, bar + 1);
    mma::tma_load_2d(smem + 2 * SH::OB + SH::QB, &maps.k, h * DKt + c0, t0, bar + 1);
  };
  if (tid == 0) {
    for (int s = 0; s < 2; s++) mma::mbar_init(bar + s, 1);
    mma::mbar_init_fence();
    load_ov(0);
    load_qk(0);
  }
  // the states of a chunk on their way to L2 a chunk ahead: 78 -> 74 us at 32/64 (300M), but 484 -> 494 at
  // 128/128, whose CTAs have 64 KB of them under way anyhow
  auto warm = [&](int c) {
    if (DV == 64 && c < nch && tid < 2 * DV / 16)
      mma::bulk_prefetch_l2(
          (tid & 1 ? op.R : op.S) + (((int64_t)(g0 + c) * H + h) * DV + 16 * (tid >> 1)) * DKt + 16 * c0, 64 * DVS);
  };
  warm(0);
  for (int i = tid; i < 65; i += NTH) tab[i] = decay_pow(a, i);
  __syncthreads();
  for (int i = tid; i < 128; i += NTH) {
    const int m = i - 64;
    lut[i] = make_float2(m >= 0 ? P.scale * tab[m] : 0.f, m >= 1 ? P.scale * tab[m - 1] : 0.f);
  }
  for (int i = tid; i < C; i += NTH) rq[i] = P.scale * tab[i + 1];
  int n_w = -1;  // rows for which rk is set

  const Frag<DV, 1> o1;   // dO and v tiles
  const Frag<DV, 2> o2;
  const Frag<DVS, 1> v1;  // q and k tiles
  const Frag<DVS, 2> v2;
  const uint32_t p1 = mma::smem_u32(tP) + pair_lane<1>(), p2 = mma::smem_u32(tP) + pair_lane<2>();

  double dacc = 0.0;
  bool good = true;
  for (int c = 0; c < nch; c++) {
    const int2 ck = chunk(c);
    const int t0 = ck.x, n = ck.y;
    const uint32_t tO = mma::smem_u32(smem), tV = tO + SH::OB, tQ = tV + SH::OB, tK = tQ + SH::QB;
    warm(c + 1);
    good = mma::mbar_wait(bar, c & 1);
    good &= mma::mbar_wait(bar + 1, c & 1);
    if (n != n_w) {
      if (n_w >= 0) __syncthreads();
      for (int i = tid; i < C; i += NTH) rk[i] = i < n ? tab[n - 1 - i] : 0.f;
      n_w = n;
    }
    zero_rows<SH::STAGE, 2 * SH::OB, 128, DVS == 32 ? 64 : 128, NTH>(smem, n);
    if (__syncthreads_or(!good)) {
      good = false;
      break;
    }

    float part = 0.f;
    // ---- pairs, three blocks at a time (the same code for every warp: a copy for each, as the chain
    // has, overflows the instruction caches here, 551 -> 898 us at 128/128)
    for (uint64_t todo = pair_list<NW>(warp); todo; todo >>= 24) {
      int rr[3], cc[3];
      float p[3][2][4];
#pragma unroll
      for (int t = 0; t < 3; t++) {
        int code = (int)(todo >> (8 * t)) & 255;
        if (!code) code = (int)todo & 255;  // (the first once more, not stored)
        rr[t] = (code - 1) >> 2;
        cc[t] = (code - 1) & 3;
        mma::zero<2>(p[t]);
      }
#pragma unroll
      for (int kk = 0; kk < DV / 16; kk++) {
        uint32_t fa[3][4], fb[3][4];
#pragma unroll
        for (int t = 0; t < 3; t++) {
          ldsm(fa[t], o1.at(tO, 16 * rr[t], 16 * kk));
          ldsm(fb[t], o2.at(tV, 16 * cc[t], 16 * kk));
        }
#pragma unroll
        for (int t = 0; t < 3; t++) {
          mma::mma_bf16(p[t][0], fa[t], fb[t][0], fb[t][1]);
          mma::mma_bf16(p[t][1], fa[t], fb[t][2], fb[t][3]);
        }
      }
#pragma unroll
      for (int t = 0; t < 3; t++) {
        if (t > 0 && !((todo >> (8 * t)) & 255)) continue;
        const int d = 16 * (rr[t] - cc[t]) + gq - 2 * tq;  // row - column of the thread's first pair
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
          for (int k = 0; k < 2; k++) {
            const float2 w = lut[64 + d + 8 * k - 8 * j];
            p[t][j][2 * k] *= w.x;
            p[t][j][2 * k + 1] *= w.y;
            uint32_t s[2];
            split2<2>(p[t][j][2 * k], p[t][j][2 * k + 1], s);
            unsigned char* at = tP + pair_at(rr[t], cc[t]) + (8 * k + gq) * 32 + ((j ^ (gq >> 2)) << 4) + 4 * tq;
            *reinterpret_cast<uint32_t*>(at) = s[0];
            *reinterpret_cast<uint32_t*>(at + PART) = s[1];
          }
        if constexpr (DA) {  // A: the same pairs of q and k (this slice's columns)
          float m2[2][4];
          mma::zero<2>(m2);
#pragma unroll
          for (int kk = 0; kk < DVS / 16; kk++) {
            uint32_t fa[4], fb[4];
            ldsm(fa, v1.at(tQ, 16 * rr[t], 16 * kk));
            ldsm(fb, v2.at(tK, 16 * cc[t], 16 * kk));
            mma::mma_bf16(m2[0], fa, fb[0], fb[1]);
            mma::mma_bf16(m2[1], fa, fb[2], fb[3]);
          }
#pragma unroll
          for (int j = 0; j < 2; j++)
#pragma unroll
            for (int e = 0; e < 4; e++)
              part = fmaf((float)(d + 8 * (e >> 1) - 8 * j - (e & 1)) * p[t][j][e], m2[j][e], part);
        }
      }
    }
    // ---- the states' rows: gq^T = S dO^T, gk^T = R v^T
    float dq[8][4], dk[8][4];
    mma::zero<8>(dq);
    mma::zero<8>(dk);
    const int64_t sat = ((int64_t)(g0 + c) * H + h) * DV * DKt + 16 * (c0 + 16 * warp) + 8 * tq + gq;
    const float *pS = op.S + sat, *pR = op.R + sat;
    float dot = 0.f;
#pragma unroll (DA ? 2 : DV / 16)  // (the instruction caches again)
    for (int kk = 0; kk < DV / 16; kk++) {
      uint32_t fs[SP][4], fr[SP][4];
#pragma unroll
      for (int k = 0; k < 2; k++) {  // rows (dk) gq + 8 k: columns (dv) 16 kk + 2 tq, + 1 and those 8 further
        const float* at = pS + 16 * kk * DKt + 128 * k;
        const float* ar = pR + 16 * kk * DKt + 128 * k;
        const float sx[4] = {__ldg(at), __ldg(at + 32), __ldg(at + 64), __ldg(at + 96)};
        const float rx[4] = {__ldg(ar), __ldg(ar + 32), __ldg(ar + 64), __ldg(ar + 96)};
#pragma unroll
        for (int g = 0; g < 2; g++) {
          const int q = k + 2 * g;
          if constexpr (DA) dot = fmaf(sx[2 * g], rx[2 * g], fmaf(sx[2 * g + 1], rx[2 * g + 1], dot));
          uint32_t w[SP];
          split2<SP>(sx[2 * g], sx[2 * g + 1], w);
#pragma unroll
          for (int b = 0; b < SP; b++) fs[b][q] = w[b];
          split2<SP>(rx[2 * g], rx[2 * g + 1], w);
#pragma unroll
          for (int b = 0; b < SP; b++) fr[b][q] = w[b];
        }
      }
      uint32_t fo[4][4], fv[4][4];
#pragma unroll
      for (int p = 0; p < 4; p++) {
        ldsm(fo[p], o2.at(tO, 16 * p, 16 * kk));
        ldsm(fv[p], o2.at(tV, 16 * p, 16 * kk));
      }
#pragma unroll
      for (int b = SP - 1; b >= 0; b--)
#pragma unroll
        for (int p = 0; p < 4; p++) {
          mma::mma_bf16(dq[2 * p], fs[b], fo[p][0], fo[p][1]);
          mma::mma_bf16(dq[2 * p + 1], fs[b], fo[p][2], fo[p][3]);
          mma::mma_bf16(dk[2 * p], fr[b], fv[p][0], fv[p][1]);
          mma::mma_bf16(dk[2 * p + 1], fr[b], fv[p][2], fv[p][3]);
        }
    }
    uint32_t fq[4][4], fk[4][4];  // q^T and k^T, rows 16 warp ..
#pragma unroll
    for (int p = 0; p < 4; p++) {
      ldsm_t(fq[p], v2.at(tQ, 16 * p, 16 * warp));
      ldsm_t(fk[p], v2.at(tK, 16 * p, 16 * warp));
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int i = 8 * j + 2 * tq;
      const float2 wq = *reinterpret_cast<const float2*>(rq + i), wk = *reinterpret_cast<const float2*>(rk + i);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        dq[j][e] *= e & 1 ? wq.y : wq.x;
        dk[j][e] *= e & 1 ? wk.y : wk.x;
        if constexpr (DA) {  // B and C (the fragments' rows and tokens are the accumulators')
          const uint32_t uq = fq[j >> 1][2 * (j & 1) + (e >> 1)], uk = fk[j >> 1][2 * (j & 1) + (e >> 1)];
          part = fmaf((float)(i + (e & 1) + 1) * (e & 1 ? odd(uq) : even(uq)), dq[j][e], part);
          part = fmaf((float)(n - 1 - i - (e & 1)) * (e & 1 ? odd(uk) : even(uk)), dk[j][e], part);
        }
      }
    }
    if constexpr (DA) dacc += (double)part + (double)(dot * (float)n * tab[n]);
    mma::fence_async_smem();
    __syncthreads();  // the pairs of every warp; dO and v have been read
    if (tid == 0 && c + 1 < nch) load_ov(c + 1);
    // ---- dq^T += k^T P^T, dk^T += q^T P
#pragma unroll
    for (int kk = 0; kk < 4; kk++)
#pragma unroll
      for (int b = 1; b >= 0; b--) {
        uint32_t fp[4][4];
#pragma unroll
        for (int p = kk; p < 4; p++) ldsm(fp[p], p2 + b * PART + pair_at(p, kk));  // tokens i of block p, j of kk
#pragma unroll
        for (int p = kk; p < 4; p++) {
          mma::mma_bf16(dq[2 * p], fk[kk], fp[p][0], fp[p][1]);
          mma::mma_bf16(dq[2 * p + 1], fk[kk], fp[p][2], fp[p][3]);
        }
#pragma unroll
        for (int p = 0; p <= kk; p++)
          ldsm_t(fp[p], p1 + b * PART + pair_at(kk, p));  // tokens i of block kk, j of p
#pragma unroll
        for (int p = 0; p <= kk; p++) {
          mma::mma_bf16(dk[2 * p], fq[kk], fp[p][0], fp[p][1]);
          mma::mma_bf16(dk[2 * p + 1], fq[kk], fp[p][2], fp[p][3]);
        }
      }
    // ---- out, in the place of the q and k tiles (their last reads were before the barrier)
    unsigned char *uQ = smem + 2 * SH::OB, *uK = uQ + SH::QB;
    stage_tile<DVS>(uQ, 16 * warp, dq, false);
    stage_tile<DVS>(uK, 16 * warp, dk, false);
    if (n < C) {
      const int64_t at = ((int64_t)t0 * H + h) * DKt + c0;
      copy_rows<DVS, 16>(uQ, 16 * warp, (bf16*)op.dq + at, (int64_t)H * DKt, n);
      copy_rows<DVS, 16>(uK, 16 * warp, (bf16*)op.dk + at, (int64_t)H * DKt, n);
    }
    mma::fence_async_smem();
    __syncthreads();
    if (tid == 0) {
      if (n == C) {
        tma_store_2d(&maps.dq, h * DKt + c0, t0, uQ);
        tma_store_2d(&maps.dk, h * DKt + c0, t0, uK);
        mma::bulk_commit();
      }
      if (c + 1 < nch) {
        mma::bulk_wait_read();
        load_qk(c + 1);
      }
    }
  }
  if (tid == 0) mma::bulk_wait_all();
  if (!good) {  // a wait ran out
    if (tid == 0) *P.err = KDA_ERR_DEVICE;
    return;
  }
  if constexpr (DA) {  // the CTA's partial, summed in a fixed order
    double* red = reinterpret_cast<double*>(lut);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dacc += __shfl_xor_sync(0xffffffffu, dacc, s);
    __syncthreads();
    if (lane == 0) red[warp] = dacc;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < NW; w++) s += red[w];
      op.pda[blockIdx.x] = s;
    }
  }
}

// dA_log[h] = -a (sum of the partials), in a fixed order: per head n1 of each of
// cnt1 groups, n2 of each of cnt2.
__global__ void __launch_bounds__(256) lin_decay_kernel(LinP P, const double* p1, int64_t cnt1, int n1,
                                                        const double* p2, int64_t cnt2, int n2, float* dA) {
  __shared__ double red[256];
  const int h = blockIdx.x;
  pdl_wait();
  if (*P.wtag != P.tag || *P.err != KDA_OK) return;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < cnt1 * n1; i += 256) s += p1[((i / n1) * P.H + h) * n1 + i % n1];
  for (int64_t i = threadIdx.x; i < cnt2 * n2; i += 256) s += p2[((i / n2) * P.H + h) * n2 + i % n2];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) dA[h] = -decay_of(P.A_log, h) * (float)red[0];
}

// ------------------------------------------------------------ launches
template <int DK, int DVS, bool ONLY, bool rev>
cudaError_t launch_chain(int kid, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  using SH = Shape<DK, DVS, ONLY>;
  cudaError_t e = raise_smem<lin_chain_kernel<DK, DVS, ONLY, rev>>(SH::SMEM);
  if (e != cudaSuccess) return e;
  LinMaps m = {};
  if ((!ONLY && !encode_head_rows(&m.x, op.x, P.Ntok, P.H, DK)) || !encode_head_rows(&m.y, op.y, P.Ntok, P.H, DK) ||
      !encode_head_rows(&m.z, op.z, P.Ntok, P.H, op.DVt) ||
      (!ONLY && !encode_head_rows(&m.o, op.out, P.Ntok, P.H, op.DVt)))
    return cudaErrorInvalidValue;
  prof_begin(kid, st);
  e = launch_after(op.after, lin_chain_kernel<DK, DVS, ONLY, rev>,
                   dim3((unsigned)((int64_t)P.nu * P.H * (op.DVt / DVS))), SH::NTH, SH::SMEM, st, m, P, op, fwd);
  prof_end(kid, st);
  return e;
}

template <bool ONLY, bool rev>
cudaError_t launch_key(int kid, int key, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  if (key == 32) return launch_chain<32, 64, ONLY, rev>(kid, P, op, fwd, st);
  if (key == 64) return launch_chain<64, 64, ONLY, rev>(kid, P, op, fwd, st);
  return launch_chain<128, 64, ONLY, rev>(kid, P, op, fwd, st);
}
template <bool ONLY>
cudaError_t launch_bf16(int kid, int key, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  return op.rev ? launch_key<ONLY, true>(kid, key, P, op, fwd, st) : launch_key<ONLY, false>(kid, key, P, op, fwd, st);
}

struct LinGrads {
  const void *q, *k, *v, *dO;
  const float *h0, *dhf;
  void *dq, *dk, *dv;
  float *dA, *dh0;
};

int64_t dqk_groups(const LinP& P) { return (P.nc + CPB - 1) / CPB; }

template <int DV, int DVS, bool DA>
cudaError_t launch_dqk(const LinP& P, const LinGrads& g, const DqkOp& op, int dk, cudaStream_t st) {
  using SH = DShape<DV, DVS, DA>;
  cudaError_t e = raise_smem<lin_dqk_kernel<DV, DVS, DA>>(SH::SMEM);
  if (e != cudaSuccess) return e;
  DqkMaps m = {};
  if (!encode_head_rows(&m.q, g.q, P.Ntok, P.H, dk) || !encode_head_rows(&m.k, g.k, P.Ntok, P.H, dk) ||
      !encode_head_rows(&m.v, g.v, P.Ntok, P.H, DV) || !encode_head_rows(&m.dO, g.dO, P.Ntok, P.H, DV) ||
      !encode_head_rows(&m.dq, g.dq, P.Ntok, P.H, dk) || !encode_head_rows(&m.dk, g.dk, P.Ntok, P.H, dk))
    return cudaErrorInvalidValue;
  prof_begin(K_LIN_DQK, st);
  e = launch_after(true, lin_dqk_kernel<DV, DVS, DA>, dim3((unsigned)(dqk_groups(P) * P.H * (dk / DVS))), SH::NTH,
                   SH::SMEM, st, m, P, op, dk);
  prof_end(K_LIN_DQK, st);
  return e;
}

template <bool DA>
cudaError_t dqk(const LinP& P, const Dims& d, const LinGrads& g, const DqkOp& op, cudaStream_t st) {
  if (d.dk == 32) return launch_dqk<64, 32, DA>(P, g, op, 32, st);
  if (d.dv == 64) return launch_dqk<64, 64, DA>(P, g, op, 64, st);
  return launch_dqk<128, 64, DA>(P, g, op, d.dk, st);
}

// Value columns of a chain's CTA whose state has `key` key columns.
int value_slice(int dtype, int key, int DVt) { return DVt == 32 || (dtype == KDA_F32 && key == 128) ? 32 : 64; }

// ------------------------------------------------------------ plan, workspace
struct LinLayout {
  size_t off_counts, off_units, off_ch0, off_longs, off_chunks, off_segf, off_segr, off_S, off_R, off_p1, off_p2, total;
};

// Chain CTAs that an SM holds.
int chain_ctas(int dtype, int dk) {
  if (dtype == KDA_F32) return dk == 32 ? 2 : 1;
  return dk == 32 ? Shape<32, 64, false>::CTAS : dk == 64 ? Shape<64, 64, false>::CTAS : Shape<128, 64, false>::CTAS;
}

// Segment length in tokens (whole chunks, at least SEG_TOK): long documents are
// cut into equal pieces of at most that.  `per`: CTAs of a unit, `slots`: CTAs that
// run at once.
// Equal rows: the number of pieces that costs least, in chunk times: waves of
// CTAs x (chunks of a piece + a start of one and a half), the segments' own
// states (0.45 of that over all pieces but the last) and the fold (a fortieth per
// piece).  300M (2048 tokens, 128 chains): whole rows 114 us, 8 pieces (1024 CTAs
// on 912 slots) 43, 7 pieces 37.
// Packed documents, whose lengths only the device may know: N / L + n_docs / 2
// units fill the least number of waves that holds 2.5 units per document, so
// that the documents' last, shorter pieces do not decide (300M packed 48 us with
// pieces of 256 tokens, 51 with 320, 45 with 384, 49 with 448).
int seg_len(const Dims& d, int64_t per, int64_t slots) {
  if (d.rows) {
    int best = 1;
    double least = 1e300;
    const int most = (d.T + SEG_TOK - 1) / SEG_TOK;
    for (int ns = 1; ns <= most && ns <= 4096; ns++) {
      const double len = (double)((((int64_t)d.T + ns - 1) / ns + C - 1) / C);
      auto waves = [&](int64_t units) { return (double)((units * per + slots - 1) / slots); };
      double cost = waves((int64_t)d.B * ns) * (len + 1.5);
      if (ns > 1) cost += 0.45 * waves((int64_t)d.B * (ns - 1)) * (len + 1.5) + ns / 40.0 + 1.0;
      if (cost < least) { least = cost; best = ns; }
    }
    return ((d.T + best - 1) / best + C - 1) / C * C;
  }
  const int64_t want = 5 * (int64_t)d.n_docs / 2 + 1;
  const int64_t k = (want * per + slots - 1) / slots, units = k * slots / per - d.n_docs / 2;
  int64_t L = (d.Ntok + units - 1) / units;
  if (L < SEG_TOK) L = SEG_TOK;
  return (int)((L + C - 1) / C * C);
}
void lin_plan(const kda_problem* p, const Dims& d, LinP& P) {
  const int64_t per = (int64_t)d.H * (d.dv / value_slice(p->dtype, d.dk, d.dv));
  const int L = seg_len(d, per, (int64_t)LIN_SMS * chain_ctas(p->dtype, d.dk));
  P.Ntok = d.Ntok;
  P.H = d.H;
  P.n_docs = d.n_docs;
  P.T = d.T;
  P.rows = d.rows;
  P.L = L;
  P.nc = d.nc_max;
  P.scale = d.scale;
  P.cu = p->cu_seqlens;
  if (P.rows) {
    P.seg = d.T > L;
    P.nu = d.B * ((d.T + L - 1) / L);
    P.n_long = d.B;
  } else {
    P.nu = d.n_docs + d.Ntok / L;
    P.n_long = d.Ntok / L;
    P.seg = d.Ntok > L;
    if (p->cu_seqlens_host && P.seg) {
      P.seg = 0;
      for (int i = 0; i < d.n_docs; i++) P.seg |= p->cu_seqlens_host[i + 1] - p->cu_seqlens_host[i] > L;
    }
  }
  // the sizes' hash, and what else the layout of a saved workspace follows
  uint32_t tag = (uint32_t)d.tag ^ 0x4c696eu;
  for (const int32_t v : {P.rows, P.L}) tag = (tag ^ (uint32_t)v) * 16777619u;
  P.tag = (int32_t)(tag | 1u);
}

LinLayout lin_layout(const kda_problem* p, const Dims& d, const LinP& P, int for_bwd) {
  LinLayout L = {};
  size_t o = 256;  // error word, saved-problem tag
  auto take = [&](size_t bytes) { const size_t r = o; o = (o + bytes + 255) & ~(size_t)255; return r; };
  const size_t st = (size_t)d.H * d.dk * d.dv * 4;
  if (!P.rows) {
    L.off_counts = take(12);
    L.off_units = take(16 * (size_t)P.nu);
    L.off_ch0 = take(8 * (size_t)P.nu);
    L.off_longs = take(8 * (size_t)(P.n_long + 1));
  }
  // sized as if every long document were cut: whether any is may be known on the device alone
  const bool seg = P.rows ? P.seg : d.Ntok > P.L;
  L.off_segf = take(seg ? P.nu * st : 0);
  if (for_bwd) {
    L.off_chunks = take(!P.rows && p->dtype == KDA_BF16 ? 8 * (size_t)P.nc : 0);
    L.off_segr = take(seg ? P.nu * st : 0);
    L.off_S = take(P.nc * st);
    if (p->dtype == KDA_F32) {
      L.off_p1 = take(8 * (size_t)P.nu * d.H * (d.dk / 32));
      L.off_p2 = take(8 * (size_t)P.nu * d.H * (d.dk / 32));
    } else {
      L.off_R = take(P.nc * st);
      L.off_p1 = take(8 * (size_t)dqk_groups(P) * d.H * (d.dk / value_slice(p->dtype, d.dv, d.dk)));
    }
  }
  L.total = o;
  return L;
}

bool al(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

kda_status lin_setup(const kda_problem* p, int for_bwd, void* ws, size_t bytes, const float* A_log, Dims& d, LinP& P,
                     LinLayout& L) {
  const kda_status s = check_problem(p, &d);
  if (s != KDA_OK) return s;
  lin_plan(p, d, P);
  L = lin_layout(p, d, P, for_bwd);
  // one CTA per unit (chunk group, split document), head and slice on one grid axis
  if ((int64_t)P.nu * d.H * 4 > 2147483647LL || (int64_t)P.nc * d.H * 4 > 2147483647LL) return KDA_ERR_INVALID_ARG;
  if (!ws) return KDA_ERR_WORKSPACE;
  if (!al(ws, 256)) return KDA_ERR_ALIGNMENT;
  if (bytes < L.total) return KDA_ERR_WORKSPACE;
  char* w = (char*)ws;
  P.err = (int32_t*)w;
  P.wtag = (int32_t*)(w + 4);
  P.counts = (int32_t*)(w + L.off_counts);
  P.units = (int4*)(w + L.off_units);
  P.unit_at = (int2*)(w + L.off_ch0);
  P.longs = (int2*)(w + L.off_longs);
  P.chunks = (int2*)(w + L.off_chunks);
  P.A_log = A_log;
  P.save = for_bwd;
  return KDA_OK;
}

// The segments' start states of one direction (y, z: k, v, or in reverse q, dO).
template <typename T>
cudaError_t run_seg(const LinP& P, const Dims& d, const void* y, const void* z, const float* init, float* segc, int rev,
                    int fwd, cudaStream_t st) {
  LinOp op = {};
  op.y = y;
  op.z = z;
  op.x = y;
  op.rev = rev;
  op.DVt = d.dv;
  op.segc = segc;
  op.after = !rev && !P.rows;  // behind the table
  cudaError_t e = sizeof(T) == 4 ? launch_f32(3, K_LIN_SEG, d.dk, P, op, fwd, st)
                                 : launch_bf16<true>(K_LIN_SEG, d.dk, P, op, fwd, st);
  if (e != cudaSuccess) return e;
  const int N = d.dk * d.dv;
  prof_begin(K_LIN_FOLD, st);
  e = launch_pdl(lin_fold_kernel, dim3(FCTAS), dim3(FTH), 0, st, P, segc, init, rev, N,
                 fwd == 1 ? 2 : fwd);
  prof_end(K_LIN_FOLD, st);
  return e;
}

template <typename T>
cudaError_t lin_forward(const LinP& P, const Dims& d, const void* q, const void* k, const void* v, const float* h0,
                        void* o, float* hf, float* segf, float* S, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (!P.rows) {
    prof_begin(K_TABLE, st);
    lin_table_kernel<<<1, 1024, 0, st>>>(P);
    prof_end(K_TABLE, st);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && P.seg) e = run_seg<T>(P, d, k, v, h0, segf, 0, P.rows ? 1 : 2, st);
  if (e != cudaSuccess) return e;
  LinOp op = {};
  op.x = q;
  op.y = k;
  op.z = v;
  op.out = o;
  op.init = h0;
  op.fin = hf;
  op.DVt = d.dv;
  op.segc = P.seg ? segf : nullptr;
  op.states = P.save ? S : nullptr;
  op.after = !P.rows || P.seg;
  const int fwd = P.rows && !P.seg ? 1 : 2;
  return sizeof(T) == 4 ? launch_f32(0, K_LIN_CHAIN, d.dk, P, op, fwd, st)
                        : launch_bf16<false>(K_LIN_CHAIN, d.dk, P, op, fwd, st);
}

struct LinBwdWs {
  float *segf, *segr, *S, *R;
  double *p1, *p2;
};

template <typename T>
cudaError_t lin_backward(const LinP& P, const Dims& d, const LinGrads& g, const LinBwdWs& w, cudaStream_t st) {
  constexpr bool F = sizeof(T) == 4;
  cudaError_t e = cudaSuccess;
  if (P.seg) e = run_seg<T>(P, d, g.q, g.dO, g.dhf, w.segr, 1, 0, st);
  if (e != cudaSuccess) return e;
  LinOp op = {};
  op.x = g.k; op.y = g.q; op.z = g.dO; op.out = g.dv; op.init = g.dhf; op.fin = g.dh0; op.rev = 1; op.DVt = d.dv;
  op.segc = P.seg ? w.segr : nullptr;
  if (!F) op.states = w.R;
  op.after = P.seg;
  e = F ? launch_f32(0, K_LIN_CHAIN, d.dk, P, op, 0, st) : launch_bf16<false>(K_LIN_CHAIN, d.dk, P, op, 0, st);
  if (e != cudaSuccess) return e;
  const int ns = d.dk / value_slice(F ? KDA_F32 : KDA_BF16, d.dv, d.dk);
  if constexpr (!F) {
    const DqkOp dop{g.dq, g.dk, w.S, w.R, w.p1};
    e = g.dA ? dqk<true>(P, d, g, dop, st) : dqk<false>(P, d, g, dop, st);
  } else {
    op = LinOp{};
    op.x = g.dO; op.y = g.v; op.z = g.k; op.out = g.dq; op.init = g.h0; op.tr = 1; op.DVt = d.dk;
    op.segc = P.seg ? w.segf : nullptr; op.wx = g.q; op.pda = w.p1; op.after = 1;
    e = launch_f32(g.dA ? 1 : 0, K_LIN_CHAIN, d.dv, P, op, 0, st);
    if (e != cudaSuccess) return e;
    op = LinOp{};
    op.x = g.v; op.y = g.dO; op.z = g.q; op.out = g.dk; op.init = g.dhf; op.tr = 1; op.rev = 1; op.DVt = d.dk;
    op.segc = P.seg ? w.segr : nullptr; op.wx = g.k; op.ent = w.S; op.pda = w.p2; op.after = 1;
    e = launch_f32(g.dA ? 2 : 0, K_LIN_CHAIN, d.dv, P, op, 0, st);
  }
  if (e != cudaSuccess || !g.dA) return e;
  const int64_t cnt = F ? P.nu : dqk_groups(P);
  prof_begin(K_LIN_DECAY, st);
  e = launch_pdl(lin_decay_kernel, dim3(d.H), dim3(256), 0, st, P, (const double*)w.p1, cnt, ns, (const double*)w.p2,
                 F ? cnt : (int64_t)0, ns, g.dA);
  prof_end(K_LIN_DECAY, st);
  return e;
}

// ------------------------------------------------------------ single-token step
// One CTA per (sequence, head): the state is read and written once (fp32), so
// the step is bound by HBM (256 sequences, H 16, 128/128: 541 MB in 80.6 us, the
// measured copy bandwidth).  Thread t owns four value columns 4 (t % (DV / 4))
// of the key rows of its group, every load and store 16 bytes.
template <int DK, int DV, typename T>
__global__ void __launch_bounds__(256) lin_decode_kernel(int H, float scale, const T* __restrict__ q,
                                                         const T* __restrict__ k, const T* __restrict__ v,
                                                         const float* __restrict__ A_log, float* __restrict__ state,
                                                         T* __restrict__ o) {
  constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG;
  __shared__ float qs[DK], ks[DK];
  __shared__ __align__(16) float red[RG][DV];
  const int64_t sh = blockIdx.x;
  const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
  float4* S = reinterpret_cast<float4*>(state + sh * DK * DV) + cg;
  float4 s[RPT];
#pragma unroll
  for (int e = 0; e < RPT; e++) s[e] = S[(rg + e * RG) * CG];
  if (tid < DK) {
    qs[tid] = ldf(q + sh * DK + tid);
    ks[tid] = ldf(k + sh * DK + tid);
  }
  float vv[4];
#pragma unroll
  for (int e = 0; e < 4; e++) vv[e] = ldf(v + sh * DV + 4 * cg + e);
  const float dec = decay_pow(decay_of(A_log, (int)(sh % H)), 1);
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int e = 0; e < RPT; e++) {
    const int i = rg + e * RG;
    const float kk = ks[i], qq = qs[i];
    s[e].x = fmaf(dec, s[e].x, kk * vv[0]);
    s[e].y = fmaf(dec, s[e].y, kk * vv[1]);
    s[e].z = fmaf(dec, s[e].z, kk * vv[2]);
    s[e].w = fmaf(dec, s[e].w, kk * vv[3]);
    S[i * CG] = s[e];
    acc.x = fmaf(qq, s[e].x, acc.x);
    acc.y = fmaf(qq, s[e].y, acc.y);
    acc.z = fmaf(qq, s[e].z, acc.z);
    acc.w = fmaf(qq, s[e].w, acc.w);
  }
  *reinterpret_cast<float4*>(&red[rg][4 * cg]) = acc;
  __syncthreads();
  if (tid < DV) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < RG; g++) t += red[g][tid];
    stf(o + sh * DV + tid, scale * t);
  }
}

template <int DK, int DV>
cudaError_t launch_lin_decode(int dtype, int64_t n, int H, float scale, const void* q, const void* k, const void* v,
                              const float* A_log, float* state, void* o, cudaStream_t st) {
  prof_begin(K_LIN_DECODE, st);
  if (dtype == KDA_BF16)
    lin_decode_kernel<DK, DV, bf16><<<(unsigned)n, 256, 0, st>>>(H, scale, (const bf16*)q, (const bf16*)k,
                                                                 (const bf16*)v, A_log, state, (bf16*)o);
  else
    lin_decode_kernel<DK, DV, float><<<(unsigned)n, 256, 0, st>>>(H, scale, (const float*)q, (const float*)k,
                                                                  (const float*)v, A_log, state, (float*)o);
  prof_end(K_LIN_DECODE, st);
  return cudaGetLastError();
}

}  // namespace
}  // namespace lin
}  // namespace kda

using namespace kda;
using namespace kda::lin;

extern "C" KDA_API size_t kda_linear_workspace_size(const kda_problem* p, int for_backward) {
  Dims d;
  if (check_problem(p, &d) != KDA_OK) return 0;
  LinP P = {};
  lin_plan(p, d, P);
  return lin_layout(p, d, P, for_backward ? 1 : 0).total;
}

extern "C" KDA_API kda_status kda_linear_fwd(const kda_problem* p, const void* q, const void* k, const void* v,
                                             const float* A_log, const float* h0, void* o, float* h_final,
                                             int save_for_backward, void* workspace, size_t workspace_bytes,
                                             cudaStream_t stream) {
  Dims d;
  LinP P = {};
  LinLayout L;
  const kda_status c = check_problem(p, &d);
  if (c != KDA_OK) return c;
  if (!q || !k || !v || !A_log || !o) return KDA_ERR_INVALID_ARG;
  if (save_for_backward && h0 && h_final == h0) return KDA_ERR_INVALID_ARG;  // (the backward reads h0)
  const void* ptrs[] = {q, k, v, A_log, h0, o, h_final};
  for (const void* x : ptrs)
    if (!al(x, 16)) return KDA_ERR_ALIGNMENT;
  const kda_status s = lin_setup(p, save_for_backward ? 1 : 0, workspace, workspace_bytes, A_log, d, P, L);
  if (s != KDA_OK) return s;
  float *segf = (float*)((char*)workspace + L.off_segf), *S = (float*)((char*)workspace + L.off_S);
  const cudaError_t e = p->dtype == KDA_F32 ? lin_forward<float>(P, d, q, k, v, h0, o, h_final, segf, S, stream)
                                            : lin_forward<bf16>(P, d, q, k, v, h0, o, h_final, segf, S, stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" KDA_API kda_status kda_linear_bwd(const kda_problem* p, const void* q, const void* k, const void* v,
                                             const float* A_log, const float* h0, const void* dO,
                                             const float* dh_final, void* dq, void* dk, void* dv, float* dA_log,
                                             float* dh0, void* workspace, size_t workspace_bytes,
                                             cudaStream_t stream) {
  Dims d;
  LinP P = {};
  LinLayout L;
  const kda_status c = check_problem(p, &d);
  if (c != KDA_OK) return c;
  if (!q || !k || !v || !A_log || !dO || !dq || !dk || !dv) return KDA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, A_log, h0, dO, dh_final, dq, dk, dv, dA_log, dh0};
  for (const void* x : ptrs)
    if (!al(x, 16)) return KDA_ERR_ALIGNMENT;
  const kda_status s = lin_setup(p, 1, workspace, workspace_bytes, A_log, d, P, L);
  if (s != KDA_OK) return s;
  char* w = (char*)workspace;
  const LinGrads g{q, k, v, dO, h0, dh_final, dq, dk, dv, dA_log, dh0};
  const LinBwdWs bw{(float*)(w + L.off_segf), (float*)(w + L.off_segr), (float*)(w + L.off_S), (float*)(w + L.off_R),
                    (double*)(w + L.off_p1), (double*)(w + L.off_p2)};
  const cudaError_t e = p->dtype == KDA_F32 ? lin_backward<float>(P, d, g, bw, stream)
                                            : lin_backward<bf16>(P, d, g, bw, stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" KDA_API kda_status kda_linear_decode(int n_seq, int H, int dk, int dv, int dtype, float scale,
                                                const void* q, const void* k, const void* v, const float* A_log,
                                                float* state, void* o, cudaStream_t stream) {
  if (n_seq <= 0 || H <= 0 || H > 4096 || (int64_t)n_seq * H > ((int64_t)1 << 30)) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
  if (!q || !k || !v || !A_log || !state || !o) return KDA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, A_log, state, o};
  for (const void* x : ptrs)
    if (!al(x, 16)) return KDA_ERR_ALIGNMENT;
  const float sc = scale > 0.f ? scale : 1.0f / sqrtf((float)dk);
  const int64_t n = (int64_t)n_seq * H;
  cudaError_t e;
  if (dk == 32 && dv == 64) e = launch_lin_decode<32, 64>(dtype, n, H, sc, q, k, v, A_log, state, o, stream);
  else if (dk == 64 && dv == 64) e = launch_lin_decode<64, 64>(dtype, n, H, sc, q, k, v, A_log, state, o, stream);
  else if (dk == 64 && dv == 128) e = launch_lin_decode<64, 128>(dtype, n, H, sc, q, k, v, A_log, state, o, stream);
  else if (dk == 128 && dv == 128) e = launch_lin_decode<128, 128>(dtype, n, H, sc, q, k, v, A_log, state, o, stream);
  else return KDA_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
