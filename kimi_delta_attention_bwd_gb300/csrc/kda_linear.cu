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
// One kernel body (chain) therefore serves the forward and the three gradients.
//
// Decay gradient: with a exponent per token distance,
//   dL/da = -(A + B + D + C + E), all sums of products of one sign pattern (no
//   difference of large position sums):
//   A  pairs inside a chunk, sum_{j<i} (i-j) e^{-a(i-j)} scale (dO_i . v_j)(q_i . k_j)
//   B  entry state to row, sum_i (i+1) e^{-a(i+1)} scale q_i . S dO_i
//   D  the same with S replaced by R^ (the state weighted by the tokens that
//      passed since the end of the chunk each term came from):
//      R^' = e^{-an} (R^ + n S)
//   C  a chunk's terms to its exit state's gradient, sum_i i (k_i . dk_i^state)
//   E  <R^ at the document's end, dh_final>
// A, B, D, E ride on the dq chain, C on the dk chain.
//
// Products run on tcgen05 (M = 64).  Operands that are not inputs (the
// weighted pairs, the state, the weighted values) are split bf16 hi + lo (about 16
// bits); fp32 io splits everything in three (24 bits, six products).  The
// state stays in fp32 registers.
#include "kda_internal.cuh"
#include "kda_mma.cuh"
#include "kda_tc.cuh"
#include "../../include/kda.h"

#include <atomic>

namespace kda {

kda_status check_problem(const kda_problem* p, Dims* d);

namespace {

using bf16 = __nv_bfloat16;
constexpr int LTH = 256;        // threads of a chain CTA: warp w holds rows 16 (w % 4) .., column half w / 4
constexpr int LIN_SMS = 152;    // SMs of a GB300: the segment rule's denominator
constexpr int SEG_TOK = 256;    // shortest segment (tokens)

struct LinP {
  int Ntok, H, n_docs, T, rows;  // rows: documents are the rows of T tokens
  int nu, L, seg;                // units (an upper bound with cu_seqlens), segment length, any document split
  int save, tag;
  float scale;
  const int32_t* cu;
  const float* A_log;
  int32_t *err, *wtag, *n_units;
  int4* units;                   // {document, first token, tokens, segment}
};

// One application of the operator (see above).  z, out and the state's value
// side have DVt columns per head; the state is stored [key][DVt], or, with tr,
// [DVt][key].
struct LinOp {
  const void *x, *y, *z;
  void* out;
  const float* init;  // state at the chain's start (nullptr: 0)
  float* fin;         // state at its end (nullptr: not wanted)
  int tr, rev, DVt;
  const float* segc;  // segments' own states [nu][H][2][key * DVt] (rev: [nu][H][key * DVt])
  const void* wx;     // decay gradient: q (dq chain) or k (dk chain), laid out like z
  const float* dfin;  // decay gradient: dh_final
  double* pda;        // decay gradient: per CTA partial
};

// ------------------------------------------------------------ geometry
struct Unit {
  int doc, tok0, ntok, seg, d0, dlen;  // document start and length
};
__device__ __forceinline__ bool unit_of(const LinP& P, int u, Unit& t) {
  if (P.rows) {
    const int ns = (P.T + P.L - 1) / P.L;
    t.doc = u / ns;
    t.seg = u % ns;
    t.d0 = t.doc * P.T;
    t.dlen = P.T;
    t.tok0 = t.d0 + t.seg * P.L;
    t.ntok = min(P.L, P.T - t.seg * P.L);
    return true;
  }
  if (u >= *P.n_units) return false;
  const int4 v = P.units[u];
  t.doc = v.x;
  t.tok0 = v.y;
  t.ntok = v.z;
  t.seg = v.w;
  t.d0 = t.tok0 - t.seg * P.L;
  t.dlen = P.cu[t.doc + 1] - t.d0;
  return true;
}

// The unit table of packed documents: a document of n tokens has max(1,
// ceil(n / L)) units.  One CTA; also validates the offsets.
__global__ void __launch_bounds__(1024) lin_table_kernel(LinP P) {
  __shared__ int s_bad, s_carry, s_w[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = P.n_docs;
  if (tid == 0) {
    s_bad = P.cu[0] != 0 || P.cu[n] != P.Ntok;
    s_carry = 0;
  }
  __syncthreads();
  for (int i = tid; i < n; i += 1024)
    if (P.cu[i + 1] < P.cu[i]) s_bad = 1;
  __syncthreads();
  if (s_bad) {
    if (tid == 0) { *P.err = KDA_ERR_BAD_SEQLENS; *P.n_units = 0; *P.wtag = 0; }
    return;
  }
  for (int base = 0; base < n; base += 1024) {
    const int i = base + tid;
    const int t0 = i < n ? P.cu[i] : 0, len = i < n ? P.cu[i + 1] - t0 : 0;
    const int ns = i < n ? max(1, (len + P.L - 1) / P.L) : 0;
    int x = ns;
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
    const int u0 = s_carry + x - ns + (warp ? s_w[warp - 1] : 0);
    for (int s = 0; s < ns; s++) P.units[u0 + s] = make_int4(i, t0 + s * P.L, min(P.L, len - s * P.L), s);
    __syncthreads();
    if (tid == 0) s_carry += s_w[31];
    __syncthreads();
  }
  if (tid == 0) {
    *P.n_units = s_carry;  // <= n + Ntok / L = nu
    *P.err = KDA_OK;
    *P.wtag = P.save ? P.tag : 0;
  }
}

// Equal rows have no table: the first kernel of a forward resets the words.
__device__ __forceinline__ void rows_reset(const LinP& P) {
  if (P.rows && blockIdx.x == 0 && threadIdx.x == 0) {
    *P.err = KDA_OK;
    *P.wtag = P.save ? P.tag : 0;
  }
}

__device__ __forceinline__ float decay_of(const float* A_log, int h) { return fminf(expf(A_log[h]), 1e30f); }
__device__ __forceinline__ float decay_pow(float a, int m) { return m > 0 ? expf(-a * (float)m) : 1.0f; }

// ------------------------------------------------------------ tiles
// x = sum of N bf16 parts, each the rounding of what the parts before it leave
// (two parts: about 16 bits, three: 24).
template <int N>
__device__ __forceinline__ void split8(const float (&v)[8], bf16* dst, int stride) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; e++) r[e] = v[e];
#pragma unroll
  for (int p = 0; p < N; p++) {
    uint4 u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(r[2 * e], r[2 * e + 1]);
      const float2 f = __bfloat1622float2(h);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
      r[2 * e] -= f.x;
      r[2 * e + 1] -= f.y;
    }
    *reinterpret_cast<uint4*>(dst + p * stride) = u;
  }
}
template <int N>
__device__ __forceinline__ void split2(float x0, float x1, bf16* dst, int stride) {
#pragma unroll
  for (int p = 0; p < N; p++) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const float2 f = __bfloat1622float2(h);
    *reinterpret_cast<__nv_bfloat162*>(dst + p * stride) = h;
    x0 -= f.x;
    x1 -= f.y;
  }
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; e++) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// cp.async of 16 bytes that reads only `bytes` of them (0: fills with zeros).
__device__ __forceinline__ void cp16z(void* smem, const void* gmem, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(mma::smem_u32(smem)), "l"(gmem), "r"(bytes)
               : "memory");
}

// A chunk's rows: row i is token t0 + dir * i, i < n (later rows read as 0).
struct Rows {
  int64_t t0;
  int dir, n;
};

// Loads a 64 x W tile (columns c0 .. of a head's D) into core-matrix order.
// Element group idx (8 columns of a row) lands at element 8 idx: eight lanes
// fill one 128-byte core matrix, a warp reads 64 bytes of eight rows.
template <int W>
__device__ __forceinline__ void load_tile(bf16* dst, const bf16* g, const Rows& r, int H, int h, int D, int c0) {
  for (int idx = threadIdx.x; idx < 8 * W; idx += LTH) {
    const int row = (idx & 7) + 8 * (idx / W), cg = (idx >> 3) % (W / 8);
    const bool in = row < r.n;
    const int64_t t = in ? r.t0 + (int64_t)r.dir * row : r.t0;
    cp16z(dst + 8 * idx, g + (t * H + h) * D + c0 + 8 * cg, in ? 16 : 0);
  }
}
template <int W>
__device__ __forceinline__ void load_tile(bf16* dst, const float* g, const Rows& r, int H, int h, int D, int c0) {
  for (int idx = threadIdx.x; idx < 8 * W; idx += LTH) {
    const int row = (idx & 7) + 8 * (idx / W), cg = (idx >> 3) % (W / 8);
    float v[8];
    if (row < r.n) {
      const float4* p = reinterpret_cast<const float4*>(g + ((r.t0 + (int64_t)r.dir * row) * H + h) * D + c0 + 8 * cg);
      const float4 f0 = __ldg(p), f1 = __ldg(p + 1);
      v[0] = f0.x; v[1] = f0.y; v[2] = f0.z; v[3] = f0.w;
      v[4] = f1.x; v[5] = f1.y; v[6] = f1.z; v[7] = f1.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = 0.f;
    }
    split8<3>(v, dst + 8 * idx, 64 * W);
  }
}

// sc = the 64 x W tile `raw` (NX parts) with row i times sw[i], in NS parts; each
// thread scales the groups that it loaded itself (load_tile's mapping), so it
// needs no barrier in between.
template <int W, int NX, int NS>
__device__ __forceinline__ void scale_tile(bf16* sc, const bf16* raw, const float* sw) {
  for (int idx = threadIdx.x; idx < 8 * W; idx += LTH) {
    const float w = sw[(idx & 7) + 8 * (idx / W)];
    float v[8], u[8];
    unpack8(*reinterpret_cast<const uint4*>(raw + 8 * idx), v);
#pragma unroll
    for (int p = 1; p < NX; p++) {
      unpack8(*reinterpret_cast<const uint4*>(raw + p * 64 * W + 8 * idx), u);
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] += u[e];
    }
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] *= w;
    split8<NS>(v, sc + 8 * idx, 64 * W);
  }
}

// D = A B over ksteps x 16 with A in NA parts (sa elements apart) and B in NB:
// the products of parts i, j with i + j <= 2.  One thread issues.
template <int NA, int NB>
__device__ __forceinline__ void gemm_parts(uint32_t d, const tc::View& A, int sa, const tc::View& B, int sb, int N,
                                           int ksteps) {
  const uint32_t id = tc::idesc_bf16(64, N, A.mn, B.mn);
  const uint64_t da = tc::vstep(A), db = tc::vstep(B);
  uint32_t acc = 0;
#pragma unroll
  for (int i = 0; i < NA; i++)
#pragma unroll
    for (int j = 0; j < NB; j++) {
      if (i + j > 2) continue;
      uint64_t a = tc::vdesc(A, A.hi + i * sa, 0), b = tc::vdesc(B, B.hi + j * sb, 0);
      for (int ks = 0; ks < ksteps; ks++) {
        tc::mma_issue(d, a, b, id, acc);
        acc = 1;
        a += da;
        b += db;
      }
    }
}
__device__ __forceinline__ tc::View kview(const bf16* p, int Kc) { return tc::View{p, nullptr, Kc, 0, 0, false}; }
__device__ __forceinline__ tc::View mview(const bf16* p, int Kc) { return tc::View{p, nullptr, Kc, 0, 0, true}; }

template <int NT>
__device__ __forceinline__ void ld_tiles(uint32_t tbase, int c0, float (&v)[NT][4]) {
  if constexpr (NT <= 4) {
    tc::ld_frag<NT>(tbase, c0, v);
  } else {
#pragma unroll
    for (int b = 0; b < NT / 4; b++) {
      float t[4][4];
      tc::ld_frag<4>(tbase, c0 + 32 * b, t);
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) v[4 * b + j][e] = t[j][e];
    }
  }
}

// ------------------------------------------------------------ chain shape
// DEC: 0 plain, 1 the dq chain with the decay gradient's A, B, D, E, 2 the dk
// chain with its C, 3 state only (a segment's own state), 4 the same with R^.
template <int DK, int DVS, typename T, int DEC>
struct Shape {
  static constexpr bool F = sizeof(T) == 4;
  static constexpr int NX = F ? 3 : 1;      // parts of an input tile
  static constexpr int NS = F ? 3 : 2;      // parts of a computed operand
  static constexpr bool ONLY = DEC >= 3;    // no output rows
  static constexpr bool HASR = DEC == 1 || DEC == 4;
  static constexpr bool SCY = DK < DVS;     // the narrower of y and z carries the state weights
  static constexpr int SCW = SCY ? DK : DVS;
  // two stages of input tiles where that leaves two CTAs per SM
  static constexpr int STG = !F && (DK <= 64 || ONLY) && DEC != 1 ? 2 : 1;
  static constexpr int XE = ONLY ? 0 : NX * 64 * DK, YE = NX * 64 * DK, ZE = NX * 64 * DVS;
  static constexpr int STAGE = XE + YE + ZE;
  static constexpr int SE = ONLY ? 0 : NS * DVS * DK, SCE = NS * 64 * SCW, PE = ONLY ? 0 : NS * 64 * 64;
  static constexpr int QE = DEC == 1 ? NX * 64 * DVS : 0, RE = DEC == 1 ? NS * DVS * DK : 0;
  // 512 bytes after the tiles: an M = 64 view of a 32-column tile reads up to four cores past it
  static constexpr int ELEMS = STG * STAGE + SE + SCE + PE + QE + RE + 256;
  static constexpr int TMEM = DEC == 1 || 64 + DK > 128 ? 256 : 128;
  static constexpr int SMEM = ELEMS * 2 + 1024 /* lut */ + 512 /* tab, sw */ + 256 /* sw */ + 64;
  static constexpr int NTV = DVS / 16;      // 8-column tiles of a warp's half of the value side
  static constexpr int NTK = DK / 16;       // and of the key side
};

// Element (value j, key i) of a stored state.
__device__ __forceinline__ int64_t st_at(int tr, int j, int i, int DK, int DVt) {
  return tr ? (int64_t)j * DK + i : (int64_t)i * DVt + j;
}

template <int DK, int DVS, typename T, int DEC>
__device__ void chain(const LinP& P, const LinOp& op, int u, int h, int slice) {
  using SH = Shape<DK, DVS, T, DEC>;
  constexpr int NX = SH::NX, NS = SH::NS, NTV = SH::NTV, NTK = SH::NTK;
  constexpr bool ONLY = SH::ONLY;
  extern __shared__ __align__(1024) unsigned char smem[];
  bf16* stage0 = reinterpret_cast<bf16*>(smem);
  bf16* tS = stage0 + SH::STG * SH::STAGE;
  bf16* tSC = tS + SH::SE;
  bf16* tP = tSC + SH::SCE;
  bf16* tQ = tP + SH::PE;
  bf16* tR = tQ + SH::QE;
  float2* lut = reinterpret_cast<float2*>(smem + SH::ELEMS * 2);  // [128] (w(m), w(m - 1)), m = index - 64
  float* tab = reinterpret_cast<float*>(lut + 128);               // [65] e^{-a m}
  float* sw = tab + 96;                                           // [64] state weights of the chunk's rows
  uint64_t* bar = reinterpret_cast<uint64_t*>(sw + 64);
  uint32_t* slot = reinterpret_cast<uint32_t*>(bar + 1);
  int* s_fail = reinterpret_cast<int*>(slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int q4 = warp & 3, half = warp >> 2, r0 = 16 * q4 + gq;

  Unit un;
  if (!unit_of(P, u, un)) return;
  const int nseg = P.seg ? max(1, (un.dlen + P.L - 1) / P.L) : 1;
  if (ONLY && un.seg == (op.rev ? 0 : nseg - 1)) return;  // the last segment of its direction feeds nobody
  const int H = P.H, DVt = op.DVt, c0 = slice * DVS;
  const float a = decay_of(P.A_log, h);

  if (warp == 0) tc::tmem_alloc(slot, SH::TMEM);
  if (tid == 0) {
    mma::mbar_init(bar, 1);
    mma::mbar_init_fence();
    *s_fail = 0;
  }
  if (tid < 65) tab[tid] = decay_pow(a, tid);
  __syncthreads();
  if (tid < 128) {
    const int m = tid - 64;
    lut[tid] = make_float2(m >= 0 ? P.scale * tab[m] : 0.f, m >= 1 ? P.scale * tab[m - 1] : 0.f);
  }
  tc::fence_after();
  const uint32_t tm = *slot;

  const int nch = (un.ntok + C - 1) / C;
  auto rows_of = [&](int c) {
    const int idx = op.rev ? nch - 1 - c : c;
    const int n = min(C, un.ntok - idx * C);
    Rows r;
    r.n = n;
    r.dir = op.rev ? -1 : 1;
    r.t0 = un.tok0 + idx * C + (op.rev ? n - 1 : 0);
    return r;
  };
  auto load_x = [&](int c) {
    if constexpr (!ONLY) load_tile<DK>(stage0 + (c % SH::STG) * SH::STAGE, (const T*)op.x, rows_of(c), H, h, DK, 0);
  };
  auto load_yz = [&](int c) {
    bf16* s = stage0 + (c % SH::STG) * SH::STAGE + SH::XE;
    load_tile<DK>(s, (const T*)op.y, rows_of(c), H, h, DK, 0);
    load_tile<DVS>(s + SH::YE, (const T*)op.z, rows_of(c), H, h, DVt, c0);
    if constexpr (DEC == 1) load_tile<DVS>(tQ, (const T*)op.wx, rows_of(c), H, h, DVt, c0);
  };
  if (!SH::F && nch > 0) {
    load_x(0);
    load_yz(0);
    mma::cp_commit();
  }

  // ---- the state at the unit's start: the initial state and the earlier segments, decayed to here
  const bool st_rows = 16 * q4 < DVS;  // a warp whose rows exist (DVS = 32: warps 0, 1 of each half)
  float S[NTK][4], R[SH::HASR ? NTK : 1][4];
  mma::zero<NTK>(S);
  mma::zero<SH::HASR ? NTK : 1>(R);
  if (!ONLY && st_rows) {
    const int64_t stN = (int64_t)DK * DVt;
    auto each_st = [&](auto fn) {
#pragma unroll
      for (int j = 0; j < NTK; j++)
#pragma unroll
        for (int e = 0; e < 4; e++)
          fn(j, e, st_at(op.tr, c0 + r0 + 8 * (e >> 1), half * (DK / 2) + 8 * j + 2 * tq + (e & 1), DK, DVt));
    };
    const int age0 = op.rev ? un.dlen - un.seg * P.L - un.ntok : un.seg * P.L;
    if (op.init) {
      const float* p = op.init + ((int64_t)un.doc * H + h) * stN;
      const float w = decay_pow(a, age0) * (op.rev ? 1.0f / P.scale : 1.0f);
      each_st([&](int j, int e, int64_t at) {
        const float v = w * p[at];
        S[j][e] = v;
        if constexpr (DEC == 1) R[j][e] = (float)age0 * v;
      });
    }
    if (op.segc) {
      const int r1 = op.rev ? un.seg + 1 : 0, r2 = op.rev ? nseg : un.seg;
      for (int r = r1; r < r2; r++) {
        const int age = P.L * (op.rev ? r - un.seg - 1 : un.seg - 1 - r);
        const float w = decay_pow(a, age);
        const float* p = op.segc + ((int64_t)(u - un.seg + r) * H + h) * stN * (op.rev ? 1 : 2);
        each_st([&](int j, int e, int64_t at) {
          const float v = p[at];
          S[j][e] = fmaf(w, v, S[j][e]);
          if constexpr (DEC == 1) R[j][e] = fmaf(w, fmaf((float)age, v, p[stN + at]), R[j][e]);
        });
      }
    }
  }
  auto put_state = [&]() {
    if (st_rows) {
#pragma unroll
      for (int j = 0; j < NTK; j++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int at = mma::opix(r0 + 8 * k, half * (DK / 2) + 8 * j + 2 * tq, DK);
          split2<NS>(S[j][2 * k], S[j][2 * k + 1], tS + at, DVS * DK);
          if constexpr (DEC == 1) split2<NS>(R[j][2 * k], R[j][2 * k + 1], tR + at, DVS * DK);
        }
    }
  };
  if constexpr (!ONLY) put_state();

  double dacc = 0.0;  // this thread's part of the decay gradient's sums
  uint32_t ph = 0;
  bool good = true;
  for (int c = 0; c < nch; c++) {
    const Rows rw = rows_of(c);
    const int n = rw.n;
    bf16* tX = stage0 + (c % SH::STG) * SH::STAGE;
    bf16 *tY = tX + SH::XE, *tZ = tY + SH::YE;
    if (tid < C) sw[tid] = tid < n ? tab[n - 1 - tid + (op.rev ? 1 : 0)] : 0.f;
    if constexpr (SH::F) {
      load_x(c);
      load_yz(c);
    } else {
      mma::cp_wait_all();
    }
    [[maybe_unused]] float kx[NTV][4];
    if constexpr (DEC == 2) {  // k's rows in fragment order, used after the first products
#pragma unroll
      for (int j = 0; j < NTV; j++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int row = r0 + 8 * k;
          const T* p = (const T*)op.wx + ((rw.t0 + (int64_t)rw.dir * (row < n ? row : 0)) * H + h) * DVt + c0 +
                       half * (DVS / 2) + 8 * j + 2 * tq;
          kx[j][2 * k] = row < n ? ldf(p) : 0.f;
          kx[j][2 * k + 1] = row < n ? ldf(p + 1) : 0.f;
        }
    }
    __syncthreads();  // sw
    scale_tile<SH::SCW, NX, NS>(tSC, SH::SCY ? tY : tZ, sw);
    mma::fence_async_smem();
    tc::fence_before();
    __syncthreads();
    if (SH::STG == 2 && c + 1 < nch) {  // the other stage's last readers finished in the chunk before
      load_x(c + 1);
      load_yz(c + 1);
      mma::cp_commit();
    }
    float o[NTV][4];
    if constexpr (!ONLY) {
      if (tid == 0) {
        tc::fence_after();
        gemm_parts<NX, NX>(tm, kview(tX, DK), 64 * DK, kview(tY, DK), 64 * DK, 64, DK / 16);
        gemm_parts<NX, NS>(tm + 64, kview(tX, DK), 64 * DK, kview(tS, DK), DVS * DK, DVS, DK / 16);
        if constexpr (DEC == 1) {
          gemm_parts<NX, NX>(tm + 128, kview(tQ, DVS), 64 * DVS, kview(tZ, DVS), 64 * DVS, 64, DVS / 16);
          gemm_parts<NX, NS>(tm + 192, kview(tX, DK), 64 * DK, kview(tR, DK), DVS * DK, DVS, DK / 16);
        }
        tc::commit(bar);
      }
      __syncwarp();
      if (!mma::mbar_wait(bar, ph)) *s_fail = 1;
      ph ^= 1;
      tc::fence_after();
      if (!SH::F && SH::STG == 1 && c + 1 < nch) {  // x has been read
        load_x(c + 1);
        mma::cp_commit();
      }
      float p[4][4];
      ld_tiles<4>(tm, half * 32, p);
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int row = r0 + 8 * k, col = half * 32 + 8 * j + 2 * tq;
          const float2 w = lut[64 + row - col];
          p[j][2 * k] *= w.x;
          p[j][2 * k + 1] *= w.y;
          split2<NS>(p[j][2 * k], p[j][2 * k + 1], tP + mma::opix(row, col, 64), 64 * 64);
        }
      const float rs[2] = {P.scale * tab[r0 + (op.rev ? 0 : 1)], P.scale * tab[r0 + 8 + (op.rev ? 0 : 1)]};
      ld_tiles<NTV>(tm + 64, half * (DVS / 2), o);
      if constexpr (DEC == 1) {
        {  // A: pairs inside the chunk
          float m2[4][4];
          ld_tiles<4>(tm + 128, half * 32, m2);
#pragma unroll
          for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const int d = r0 + 8 * (e >> 1) - (half * 32 + 8 * j + 2 * tq + (e & 1));
              part = fmaf((float)d * p[j][e], m2[j][e], part);
            }
        }
        float qr[NTV][4];
        ld_tiles<NTV>(tm + 192, half * (DVS / 2), qr);
#pragma unroll
        for (int j = 0; j < NTV; j++)
#pragma unroll
          for (int e = 0; e < 4; e++) {  // B and D
            const int row = r0 + 8 * (e >> 1), at = mma::opix(row, half * (DVS / 2) + 8 * j + 2 * tq + (e & 1), DVS);
            float qv = 0.f;
#pragma unroll
            for (int b = 0; b < NX; b++) qv += __bfloat162float(tQ[b * 64 * DVS + at]);
            part = fmaf(rs[e >> 1] * qv, fmaf((float)(row + 1), o[j][e], qr[j][e]), part);
          }
      }
#pragma unroll
      for (int j = 0; j < NTV; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          o[j][e] *= rs[e >> 1];
          if constexpr (DEC == 2) part = fmaf((float)(r0 + 8 * (e >> 1)) * kx[j][e], o[j][e], part);
        }
      if constexpr (DEC == 1 || DEC == 2) dacc += (double)part;
      mma::fence_async_smem();
      tc::fence_before();
      __syncthreads();
    }
    if (tid == 0) {
      tc::fence_after();
      // S'^T += z^T (weighted) y: rows are the value columns
      if constexpr (SH::SCY)
        gemm_parts<NX, NS>(tm + 64, mview(tZ, DVS), 64 * DVS, mview(tSC, DK), 64 * DK, DK, 4);
      else
        gemm_parts<NS, NX>(tm + 64, mview(tSC, DVS), 64 * DVS, mview(tY, DK), 64 * DK, DK, 4);
      if constexpr (!ONLY) gemm_parts<NS, NX>(tm, kview(tP, 64), 64 * 64, mview(tZ, DVS), 64 * DVS, DVS, 4);
      tc::commit(bar);
    }
    __syncwarp();
    if (!mma::mbar_wait(bar, ph)) *s_fail = 1;
    ph ^= 1;
    tc::fence_after();
    if (!SH::F && SH::STG == 1 && c + 1 < nch) {
      if (ONLY) load_x(c + 1);
      load_yz(c + 1);
      mma::cp_commit();
    }
    {  // S' = e^{-an} S + ...: as S + (e^{-an} - 1) S where the decay is slow, so that its rounding is
       // relative to what a chunk loses and hundreds of chunks add up no bias; as a product where it
       // is fast, where that sum would cancel
      const bool slow = a * (float)n < 0.5f;
      const float g = slow ? expm1f(-a * (float)n) : expf(-a * (float)n);
      float d[NTK][4];
      ld_tiles<NTK>(tm + 64, half * (DK / 2), d);
#pragma unroll
      for (int j = 0; j < NTK; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          if constexpr (SH::HASR) {
            const float t = fmaf((float)n, S[j][e], R[j][e]);
            R[j][e] = fmaf(g, t, slow ? t : 0.f);
          }
          S[j][e] = fmaf(g, S[j][e], slow ? S[j][e] : 0.f) + d[j][e];
        }
    }
    if constexpr (!ONLY) {
      if (c + 1 < nch) put_state();
      float v[NTV][4];
      ld_tiles<NTV>(tm, half * (DVS / 2), v);
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int row = r0 + 8 * k;
        T* po = (T*)op.out + ((rw.t0 + (int64_t)rw.dir * row) * H + h) * DVt + c0 + half * (DVS / 2);
        if constexpr (SH::F) {
          if (row < n) {
#pragma unroll
            for (int j = 0; j < NTV; j++)
              *reinterpret_cast<float2*>(po + 8 * j + 2 * tq) =
                  make_float2(o[j][2 * k] + v[j][2 * k], o[j][2 * k + 1] + v[j][2 * k + 1]);
          }
        } else {
          uint32_t w[NTV];
#pragma unroll
          for (int j = 0; j < NTV; j++) {
            const __nv_bfloat162 b2 =
                __floats2bfloat162_rn(o[j][2 * k] + v[j][2 * k], o[j][2 * k + 1] + v[j][2 * k + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          if constexpr (NTV == 4) {  // transpose the quad: lane tq gets the 8 columns of tile tq
            uint32_t t[4];
#pragma unroll
            for (int x = 0; x < 4; x++) {
              uint32_t give = w[0];
#pragma unroll
              for (int y = 1; y < 4; y++)
                if ((tq ^ x) == y) give = w[y];
              t[x] = __shfl_xor_sync(0xffffffffu, give, x);
            }
            uint4 st;
            uint32_t* sp = reinterpret_cast<uint32_t*>(&st);
#pragma unroll
            for (int x = 0; x < 4; x++) {
              // t[x] came from lane tq ^ x: word tq ^ x of this lane's tile
#pragma unroll
              for (int y = 0; y < 4; y++)
                if ((tq ^ x) == y) sp[y] = t[x];
            }
            if (row < n) *reinterpret_cast<uint4*>(po + 8 * tq) = st;
          } else {
            if (row < n) {
#pragma unroll
              for (int j = 0; j < NTV; j++) *reinterpret_cast<uint32_t*>(po + 8 * j + 2 * tq) = w[j];
            }
          }
        }
      }
    }
    tc::fence_before();
    if (*s_fail) {  // a wait ran out: no thread starts another chunk
      good = false;
    }
    if (__syncthreads_or(!good)) {
      good = false;
      break;
    }
  }
  if (!good && tid == 0) *P.err = KDA_ERR_DEVICE;
  mma::cp_wait_all();

  // ---- the unit's state
  if (good && st_rows) {
    const int64_t stN = (int64_t)DK * DVt;
    const bool last = un.seg == (op.rev ? 0 : nseg - 1);
    float* pf = nullptr;
    float mul = 1.0f;
    if (ONLY) {
      pf = const_cast<float*>(op.segc) + ((int64_t)u * H + h) * stN * (op.rev ? 1 : 2);
    } else if (last && op.fin) {
      pf = op.fin + ((int64_t)un.doc * H + h) * stN;
      mul = op.rev ? P.scale : 1.0f;
    }
    const float* pd = DEC == 1 && last && op.dfin ? op.dfin + ((int64_t)un.doc * H + h) * stN : nullptr;
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < NTK; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int64_t at = st_at(op.tr, c0 + r0 + 8 * (e >> 1), half * (DK / 2) + 8 * j + 2 * tq + (e & 1), DK, DVt);
        if (pf) pf[at] = mul * S[j][e];
        if constexpr (DEC == 4) pf[stN + at] = R[j][e];
        if constexpr (DEC == 1) {
          if (pd) part = fmaf(R[j][e], pd[at], part);
        }
      }
    dacc += (double)part;
  }
  __syncthreads();
  if constexpr (DEC == 1 || DEC == 2) {  // the CTA's partial, summed in a fixed order
    double* red = reinterpret_cast<double*>(smem);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dacc += __shfl_xor_sync(0xffffffffu, dacc, s);
    if (lane == 0) red[warp] = dacc;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < LTH / 32; w++) s += red[w];
      op.pda[((int64_t)u * H + h) * (DVt / DVS) + slice] = s;
    }
  }
  if (warp == 0) tc::tmem_dealloc(tm, SH::TMEM);
}

template <int DK, int DVS, typename T, int DEC>
__global__ void __launch_bounds__(LTH, Shape<DK, DVS, T, DEC>::SMEM <= 113 * 1024 ? 2 : 1)
    lin_chain_kernel(LinP P, LinOp op, int fwd) {
  const int ns = op.DVt / DVS;
  const int slice = blockIdx.x % ns, h = (blockIdx.x / ns) % P.H, u = blockIdx.x / (ns * P.H);
  if (fwd == 1) {
    rows_reset(P);
  } else if (fwd == 2) {  // after this forward's first kernel
    if (*P.err != KDA_OK) return;
  } else if (*P.wtag != P.tag || *P.err != KDA_OK) {  // no forward saved this workspace, or it failed
    if (threadIdx.x == 0 && *P.wtag != P.tag) *P.err = KDA_ERR_WORKSPACE;
    return;
  }
  chain<DK, DVS, T, DEC>(P, op, u, h, slice);
}

// dA_log[h] = -a (sum of the partials), in a fixed order.
__global__ void __launch_bounds__(256) lin_decay_kernel(LinP P, const double* p1, int n1, const double* p2, int n2,
                                                        float* dA) {
  __shared__ double red[256];
  const int h = blockIdx.x;
  if (*P.wtag != P.tag || *P.err != KDA_OK) return;
  const int nu = P.rows ? P.nu : *P.n_units;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < (int64_t)nu * n1; i += 256) s += p1[((i / n1) * P.H + h) * n1 + i % n1];
  for (int64_t i = threadIdx.x; i < (int64_t)nu * n2; i += 256) s += p2[((i / n2) * P.H + h) * n2 + i % n2];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) dA[h] = -decay_of(P.A_log, h) * (float)red[0];
}

// ------------------------------------------------------------ launches
// The dynamic shared memory limit of kernel K, raised once per device.
template <auto K>
cudaError_t raise_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load() & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit);
  return e;
}

template <int DK, int DVS, typename T, int DEC>
cudaError_t launch_chain(int kid, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  constexpr int smem = Shape<DK, DVS, T, DEC>::SMEM;
  cudaError_t e = raise_smem<lin_chain_kernel<DK, DVS, T, DEC>>(smem);
  if (e != cudaSuccess) return e;
  prof_begin(kid, st);
  lin_chain_kernel<DK, DVS, T, DEC><<<(unsigned)((int64_t)P.nu * P.H * (op.DVt / DVS)), LTH, smem, st>>>(P, op, fwd);
  prof_end(kid, st);
  return cudaGetLastError();
}

template <typename T, int DEC>
cudaError_t dispatch(int kid, int key, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  if constexpr (sizeof(T) == 4) {
    if (key == 32) return launch_chain<32, 32, T, DEC>(kid, P, op, fwd, st);
    if (key == 64) return launch_chain<64, 32, T, DEC>(kid, P, op, fwd, st);
    return launch_chain<128, 32, T, DEC>(kid, P, op, fwd, st);
  } else {
    if (key == 32) return launch_chain<32, 64, T, DEC>(kid, P, op, fwd, st);
    if (key == 64 && op.DVt == 32) return launch_chain<64, 32, T, DEC>(kid, P, op, fwd, st);
    if (key == 64) return launch_chain<64, 64, T, DEC>(kid, P, op, fwd, st);
    return launch_chain<128, 64, T, DEC>(kid, P, op, fwd, st);
  }
}

int value_slice(int dtype, int DVt) { return dtype == KDA_F32 || DVt == 32 ? 32 : 64; }

// ------------------------------------------------------------ plan, workspace
struct LinLayout {
  size_t off_nu, off_units, off_segf, off_segr, off_p1, off_p2, total;
};

// Segment length: long documents are cut so that about two chain CTAs per SM
// exist, in whole chunks and at least SEG_TOK tokens.
void lin_plan(const kda_problem* p, const Dims& d, LinP& P) {
  const int64_t per = (int64_t)d.H * (d.dv / value_slice(p->dtype, d.dv));
  int64_t L = ((int64_t)d.Ntok * per + 2 * LIN_SMS - 1) / (2 * LIN_SMS);
  L = (L + C - 1) / C * C;
  if (L < SEG_TOK) L = SEG_TOK;
  P.Ntok = d.Ntok;
  P.H = d.H;
  P.n_docs = d.n_docs;
  P.T = d.T;
  P.rows = d.rows;
  P.L = (int)L;
  P.scale = d.scale;
  P.cu = p->cu_seqlens;
  if (P.rows) {
    P.seg = d.T > L;
    P.nu = d.B * (int)((d.T + L - 1) / L);
  } else {
    P.nu = d.n_docs + (int)(d.Ntok / L);
    P.seg = d.Ntok > L;
    if (p->cu_seqlens_host && P.seg) {
      P.seg = 0;
      for (int i = 0; i < d.n_docs; i++) P.seg |= p->cu_seqlens_host[i + 1] - p->cu_seqlens_host[i] > L;
    }
  }
  P.tag = d.tag ^ 0x4c696e;
}

LinLayout lin_layout(const Dims& d, const LinP& P, int for_bwd) {
  LinLayout L = {};
  size_t o = 256;  // error word, saved-problem tag
  auto take = [&](size_t bytes) { const size_t r = o; o = (o + bytes + 255) & ~(size_t)255; return r; };
  const size_t st = (size_t)P.nu * d.H * d.dk * d.dv * 4;
  L.off_nu = take(4);
  L.off_units = take(P.rows ? 0 : 16 * (size_t)P.nu);
  // sized as if every long document were cut: whether any is may be known on the device alone
  const bool seg = P.rows ? P.seg : d.Ntok > P.L;
  L.off_segf = take(seg ? 2 * st : 0);
  if (for_bwd) {
    L.off_segr = take(seg ? st : 0);
    L.off_p1 = take(8 * (size_t)P.nu * d.H * (d.dk / 32));
    L.off_p2 = take(8 * (size_t)P.nu * d.H * (d.dk / 32));
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
  L = lin_layout(d, P, for_bwd);
  if ((int64_t)P.nu * d.H * 4 > 2147483647LL) return KDA_ERR_INVALID_ARG;  // one CTA per unit, head and slice
  if (!ws) return KDA_ERR_WORKSPACE;
  if (!al(ws, 256)) return KDA_ERR_ALIGNMENT;
  if (bytes < L.total) return KDA_ERR_WORKSPACE;
  char* w = (char*)ws;
  P.err = (int32_t*)w;
  P.wtag = (int32_t*)(w + 4);
  P.n_units = (int32_t*)(w + L.off_nu);
  P.units = (int4*)(w + L.off_units);
  P.A_log = A_log;
  P.save = for_bwd;
  return KDA_OK;
}

// The segments' own states of one direction.
template <typename T>
cudaError_t run_seg(const LinP& P, const Dims& d, const void* y, const void* z, float* segc, int rev, int want_r,
                    int fwd, cudaStream_t st) {
  LinOp op = {};
  op.x = y;
  op.y = y;
  op.z = z;
  op.rev = rev;
  op.DVt = d.dv;
  op.segc = segc;
  return want_r ? dispatch<T, 4>(K_LIN_SEG, d.dk, P, op, fwd, st) : dispatch<T, 3>(K_LIN_SEG, d.dk, P, op, fwd, st);
}

template <typename T>
cudaError_t lin_forward(const LinP& P, const Dims& d, const void* q, const void* k, const void* v, const float* h0,
                        void* o, float* hf, float* segf, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (!P.rows) {
    prof_begin(K_TABLE, st);
    lin_table_kernel<<<1, 1024, 0, st>>>(P);
    prof_end(K_TABLE, st);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && P.seg) e = run_seg<T>(P, d, k, v, segf, 0, P.save, P.rows ? 1 : 2, st);
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
  return dispatch<T, 0>(K_LIN_CHAIN, d.dk, P, op, P.rows && !P.seg ? 1 : 2, st);
}

struct LinGrads {
  const void *q, *k, *v, *dO;
  const float *h0, *dhf;
  void *dq, *dk, *dv;
  float *dA, *dh0;
};

template <typename T>
cudaError_t lin_backward(const LinP& P, const Dims& d, const LinGrads& g, float* segf, float* segr, double* p1,
                         double* p2, int dtype, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (P.seg) e = run_seg<T>(P, d, g.q, g.dO, segr, 1, 0, 0, st);
  if (e != cudaSuccess) return e;
  LinOp op = {};
  op.x = g.dO; op.y = g.v; op.z = g.k; op.out = g.dq; op.init = g.h0; op.tr = 1; op.DVt = d.dk;
  op.segc = P.seg ? segf : nullptr; op.wx = g.q; op.dfin = g.dhf; op.pda = p1;
  e = g.dA ? dispatch<T, 1>(K_LIN_CHAIN, d.dv, P, op, 0, st) : dispatch<T, 0>(K_LIN_CHAIN, d.dv, P, op, 0, st);
  if (e != cudaSuccess) return e;
  op = LinOp{};
  op.x = g.v; op.y = g.dO; op.z = g.q; op.out = g.dk; op.init = g.dhf; op.tr = 1; op.rev = 1; op.DVt = d.dk;
  op.segc = P.seg ? segr : nullptr; op.wx = g.k; op.pda = p2;
  e = g.dA ? dispatch<T, 2>(K_LIN_CHAIN, d.dv, P, op, 0, st) : dispatch<T, 0>(K_LIN_CHAIN, d.dv, P, op, 0, st);
  if (e != cudaSuccess) return e;
  op = LinOp{};
  op.x = g.k; op.y = g.q; op.z = g.dO; op.out = g.dv; op.init = g.dhf; op.fin = g.dh0; op.rev = 1; op.DVt = d.dv;
  op.segc = P.seg ? segr : nullptr;
  e = dispatch<T, 0>(K_LIN_CHAIN, d.dk, P, op, 0, st);
  if (e != cudaSuccess || !g.dA) return e;
  const int ns = d.dk / value_slice(dtype, d.dk);
  prof_begin(K_LIN_DECAY, st);
  lin_decay_kernel<<<d.H, 256, 0, st>>>(P, p1, ns, p2, ns, g.dA);
  prof_end(K_LIN_DECAY, st);
  return cudaGetLastError();
}

// ------------------------------------------------------------ single-token step
// One CTA per (sequence, head): the state is read and written once (fp32), so
// the step is bound by HBM.  Thread t owns four value columns 4 (t % (DV / 4))
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
}  // namespace kda

using namespace kda;

extern "C" KDA_API size_t kda_linear_workspace_size(const kda_problem* p, int for_backward) {
  Dims d;
  if (check_problem(p, &d) != KDA_OK) return 0;
  LinP P = {};
  lin_plan(p, d, P);
  return lin_layout(d, P, for_backward ? 1 : 0).total;
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
  const void* ptrs[] = {q, k, v, A_log, h0, o, h_final};
  for (const void* x : ptrs)
    if (!al(x, 16)) return KDA_ERR_ALIGNMENT;
  const kda_status s = lin_setup(p, save_for_backward ? 1 : 0, workspace, workspace_bytes, A_log, d, P, L);
  if (s != KDA_OK) return s;
  float* segf = (float*)((char*)workspace + L.off_segf);
  const cudaError_t e = p->dtype == KDA_F32 ? lin_forward<float>(P, d, q, k, v, h0, o, h_final, segf, stream)
                                            : lin_forward<bf16>(P, d, q, k, v, h0, o, h_final, segf, stream);
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
  float *segf = (float*)(w + L.off_segf), *segr = (float*)(w + L.off_segr);
  double *p1 = (double*)(w + L.off_p1), *p2 = (double*)(w + L.off_p2);
  const cudaError_t e = p->dtype == KDA_F32
                            ? lin_backward<float>(P, d, g, segf, segr, p1, p2, p->dtype, stream)
                            : lin_backward<bf16>(P, d, g, segf, segr, p1, p2, p->dtype, stream);
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
