// Linear attention with one decay per head: declarations shared by its two
// chain kernels (bf16: kda_linear.cu, fp32: kda_linear_f32.cu).
#pragma once
#include "kda_internal.cuh"
#include "kda_mma.cuh"
#include "../../include/kda.h"

#include <atomic>

namespace kda {
namespace lin {

using bf16 = __nv_bfloat16;

struct LinP {
  int Ntok, H, n_docs, T, rows;  // rows: documents are the rows of T tokens
  int nu, L, seg;                // units (an upper bound with cu_seqlens), segment length, any document split
  int nc, n_long;                // upper bounds: chunks, split documents
  int save, tag;
  float scale;
  const int32_t* cu;
  const float* A_log;
  int32_t *err, *wtag, *counts;  // counts: units, chunks, split documents (cu_seqlens)
  int4* units;                   // {document, first token, tokens, segment}
  int2* unit_at;                 // {first chunk, segments of the document}
  int2* longs;                   // split documents: {first unit, segments}
  int2* chunks;                  // {first token, tokens} by packed documents' chunk, from the saving bf16 forward
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
  int after;          // launched behind another kernel of the same call (programmatic dependent launch)
  float* segc;        // per unit [nu][H][key * DVt]: a segment's own state, then (lin_fold) its start state
  float* states;      // per chunk [nc][H][dv dk]: the state where the chain enters it (fp32 io: [dv][dk];
                      // bf16: tiles, see chain); nullptr: not kept
  const void* wx;     // fp32 decay gradient: q (dq chain) or k (dk chain), laid out like z
  const float* ent;   // fp32 decay gradient, dk chain: the forward's states
  double* pda;        // fp32 decay gradient: per CTA partial
};

// Tokens of the equal pieces (whole chunks) of a document of len tokens, at most
// L (a multiple of C).
__host__ __device__ inline int seg_tokens(int L, int len) {
  const int ns = (len + L - 1) / L;
  return ns <= 1 ? L : ((len + ns - 1) / ns + C - 1) / C * C;
}

struct Unit {
  int doc, tok0, ntok, seg, nseg, ch0;
};
__device__ __forceinline__ bool unit_of(const LinP& P, int u, Unit& t) {
  if (P.rows) {
    const int ns = (P.T + P.L - 1) / P.L;
    t.doc = u / ns;
    t.seg = u % ns;
    t.nseg = ns;
    t.tok0 = t.doc * P.T + t.seg * P.L;
    t.ntok = min(P.L, P.T - t.seg * P.L);
    t.ch0 = t.doc * ((P.T + C - 1) / C) + t.seg * (P.L / C);
    return true;
  }
  if (u >= P.counts[0]) return false;
  const int4 v = P.units[u];
  t.doc = v.x;
  t.tok0 = v.y;
  t.ntok = v.z;
  t.seg = v.w;
  const int2 at = P.unit_at[u];
  t.ch0 = at.x;
  t.nseg = at.y;
  return true;
}

// Equal rows have no table: the first kernel of a forward resets the words.
__device__ __forceinline__ void rows_reset(const LinP& P) {
  if (P.rows && blockIdx.x == 0 && threadIdx.x == 0) {
    *P.err = KDA_OK;
    *P.wtag = P.save ? P.tag : 0;
  }
}

// a = exp(A_log), finite (0 tokens of an infinite decay would be NaN); a NaN stays one.
__device__ __forceinline__ float decay_of(const float* A_log, int h) {
  const float a = expf(A_log[h]);
  return a > 1e30f ? 1e30f : a;
}
__device__ __forceinline__ float decay_pow(float a, int m) { return m > 0 ? expf(-a * (float)m) : 1.0f; }

// Launches k, behind another kernel of the same call as its programmatic
// dependent (every kernel here waits for the grid before it, first thing).
template <typename... KA, typename... A>
inline cudaError_t launch_after(bool after, void (*k)(KA...), dim3 grid, int block, size_t smem, cudaStream_t st,
                                A... args) {
  if (after) return launch_pdl(k, grid, dim3(block), smem, st, args...);
  k<<<grid, block, smem, st>>>(args...);
  return cudaGetLastError();
}

// Whether a chain CTA has work: fwd 1 is a forward's first kernel (it resets
// the words of equal rows), 2 a later one, 0 a backward, which needs the
// workspace that a saving forward of the same problem filled.
__device__ __forceinline__ bool ready(const LinP& P, int fwd) {
  if (fwd == 1) {
    rows_reset(P);
    return true;
  }
  if (fwd == 2) return *P.err == KDA_OK;
  // (a forward that cut documents, and a backward whose host offsets hold none to cut)
  if (*P.wtag != P.tag || (!P.rows && !P.seg && P.counts[2] > 0)) {
    if (threadIdx.x == 0) *P.err = KDA_ERR_WORKSPACE;
    return false;
  }
  return *P.err == KDA_OK;
}

// Element (value j, key i) of a stored state.
__device__ __forceinline__ int64_t st_at(int tr, int j, int i, int DK, int DVt) {
  return tr ? (int64_t)j * DK + i : (int64_t)i * DVt + j;
}

// A chunk's rows: row i is token t0 + dir * i, i < n (later rows read as 0).
struct Rows {
  int64_t t0;
  int dir, n;
};
// The c-th chunk of a unit in the chain's direction.
__device__ __forceinline__ Rows rows_of(const Unit& un, int rev, int c) {
  const int nch = (un.ntok + C - 1) / C, idx = rev ? nch - 1 - c : c;
  Rows r;
  r.n = min(C, un.ntok - idx * C);
  r.dir = rev ? -1 : 1;
  r.t0 = un.tok0 + idx * C + (rev ? r.n - 1 : 0);
  return r;
}

// The state at a unit's start (of a document in pieces always from segc: its
// last piece may already have written an h_final that is h0).  each(fn) calls fn(s, at) for every state
// element a thread holds.
template <class EACH>
__device__ __forceinline__ void start_state(const LinP& P, const LinOp& op, const Unit& un, int u, int h, int64_t stN,
                                            EACH each) {
  const float *p = nullptr;
  float w = 1.0f;
  if (op.segc && un.nseg > 1) {
    p = op.segc + ((int64_t)u * P.H + h) * stN;
  } else if (op.init) {
    p = op.init + ((int64_t)un.doc * P.H + h) * stN;
    if (op.rev) w = 1.0f / P.scale;
  }
  if (p) each([&](float& s, int64_t at) { s = w * p[at]; });
}

// The state after n tokens of decay, S' = e^{-an} S: as S + (e^{-an} - 1) S where
// the decay is slow, so that its rounding is relative to what a chunk loses
// and hundreds of chunks add up no bias; as a product where it is fast, where
// that sum would cancel.
struct Decay {
  float g;
  bool slow;
  __device__ __forceinline__ Decay(float a, int n) : slow(a * (float)n < 0.5f) {
    g = slow ? expm1f(-a * (float)n) : expf(-a * (float)n);
  }
  __device__ __forceinline__ float operator()(float s) const { return fmaf(g, s, slow ? s : 0.f); }
};

// Two values as N bf16 parts, each the rounding of what the parts before it
// leave (two parts: about 16 bits, three: 24).
template <int N>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t (&w)[N]) {
#pragma unroll
  for (int p = 0; p < N; p++) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    w[p] = *reinterpret_cast<const uint32_t*>(&h);
    x0 -= __uint_as_float(w[p] << 16);
    x1 -= __uint_as_float(w[p] & 0xffff0000u);
  }
}

// The fp32 chain (kda_linear_f32.cu): `dec` as in kda_linear.cu.
cudaError_t launch_f32(int dec, int kid, int key, const LinP& P, const LinOp& op, int fwd, cudaStream_t st);

}  // namespace lin
}  // namespace kda
