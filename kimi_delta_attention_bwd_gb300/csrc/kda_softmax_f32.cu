// Softmax attention, the backward of fp32 io at D = 128, on the fp32 pipe (the other
// fp32 passes run on the tensor cores in three bf16 parts; here both own blocks in three
// parts would fill shared memory).  Per document, query head h and its key head h / G:
//   p_ij = exp(scale q_i k_j - lse_i),  dv_j = sum_i p_ij dO_i
//   ds_ij = p_ij (dO_i v_j - delta_i),  delta_i = o_i dO_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
// Tiles of 16 R own rows by 64 of the other side, 256 threads with R x 4 pairs each;
// operands of the pair products lie transposed in shared memory ([d][row]) so that a
// thread's rows are one 16-byte load; the next block's values are on their way to
// registers meanwhile.  dk and dv of a key tile are summed by one CTA over the queries
// of its whole head group, dq by one CTA over the keys: no atomics, a fixed order.
#include "kda_softmax.cuh"

namespace kda {
namespace smx {
namespace {

constexpr int TM = 64, NT = 256;  // rows of the other side's blocks; threads

__device__ __forceinline__ void ld4(const float* p, float* v) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
__device__ __forceinline__ void st4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// A block of ROWS rows of x (ld elements apart) on its way to shared memory: rows from n on are zeros, so that a
// neighbour's values never enter a product.
template <int D, int ROWS>
struct Block {
  static constexpr int N = ROWS * D / 4 / NT;
  float4 v[N];
  __device__ __forceinline__ void load(const float* x, size_t ld, int n) {
#pragma unroll
    for (int k = 0; k < N; k++) {
      const int i = threadIdx.x + k * NT, r = i % ROWS, d = i / ROWS * 4;
      v[k] = r < n ? *reinterpret_cast<const float4*>(x + r * ld + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  // to tr[d][row], and to pl[row][d], where not null
  __device__ __forceinline__ void store(float* tr, float* pl) const {
#pragma unroll
    for (int k = 0; k < N; k++) {
      const int i = threadIdx.x + k * NT, r = i % ROWS, d = i / ROWS * 4;
      if (tr) {
        tr[d * ROWS + r] = v[k].x;
        tr[(d + 1) * ROWS + r] = v[k].y;
        tr[(d + 2) * ROWS + r] = v[k].z;
        tr[(d + 3) * ROWS + r] = v[k].w;
      }
      if (pl) *reinterpret_cast<float4*>(pl + r * D + d) = v[k];
    }
  }
};

// c[i][j] = sum_d a[d][r0 + i] b[d][c0 + j]: a has 16 R rows, b TM
template <int D, int R>
__device__ __forceinline__ void pairs(const float* a, const float* b, int r0, int c0, float (&c)[R][4]) {
#pragma unroll
  for (int i = 0; i < R; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) c[i][j] = 0.f;
#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += 32) {  // (sums of 32, then their sum: a third of one long sum's rounding)
    float u[R][4] = {};
#pragma unroll 8
    for (int d = d0; d < d0 + 32; d++) {
      float x[R], y[4];
#pragma unroll
      for (int i = 0; i < R; i += 4) ld4(a + d * 16 * R + r0 + i, x + i);
      ld4(b + d * TM + c0, y);
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) u[i][j] = fmaf(x[i], y[j], u[i][j]);
    }
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) c[i][j] += u[i][j];
  }
}
// c[i][64 m + 4 tx + e] += sum_n w[n][r0 + i] x[n][64 m + 4 tx + e]: w's rows are PP apart
template <int R>
constexpr int PP = 16 * R + 4;
template <int D, int R>
__device__ __forceinline__ void apply(const float* w, const float* x, int r0, int tx, float (&c)[R][D / 16]) {
#pragma unroll 4
  for (int n = 0; n < TM; n++) {
    float a[R];
#pragma unroll
    for (int i = 0; i < R; i += 4) ld4(w + n * PP<R> + r0 + i, a + i);
#pragma unroll
    for (int m = 0; m < D / 64; m++) {
      float y[4];
      ld4(x + n * D + 64 * m + 4 * tx, y);
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) c[i][4 * m + e] = fmaf(a[i], y[e], c[i][4 * m + e]);
    }
  }
}
template <int R>
__device__ __forceinline__ void put_column(float* dst, const float (&v)[R]) {
#pragma unroll
  for (int i = 0; i < R; i += 4) st4(dst + i, v + i);
}

// dk and dv of 16 R keys of one key head.  Threads: keys R ty .., queries 4 tx ..
template <int D, int R>
__global__ void __launch_bounds__(NT) smx_dkv_kernel(SmxP P, const float* __restrict__ q, const float* __restrict__ k,
                                                    const float* __restrict__ v, const float* __restrict__ dO,
                                                    float* __restrict__ dk, float* __restrict__ dv) {
  constexpr int OWN = 16 * R;
  extern __shared__ __align__(16) float sm[];
  float *tK = sm, *tV = tK + D * OWN, *tQ = tV + D * OWN, *tG = tQ + D * TM, *sQ = tG + D * TM, *sG = sQ + D * TM;
  float *sP = sG + D * TM, *sl = sP + TM * PP<R>, *sd = sl + TM;  // (the weights, then their gradients)
  pdl_wait();
  pdl_release();  // dq's CTAs may follow this grid's last ones: they wait for it at their end only
  if (!saved(P)) return;
  const int hk = blockIdx.x % P.Hkv, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  Tile t;
  if (!tile_of(P, 2, blockIdx.x / P.Hkv, true, t)) return;
  const int j0 = t.t * OWN, nk = min(OWN, t.Lk - j0);
  {
    const size_t at = ((size_t)(t.k0 + j0) * P.Hkv + hk) * D;
    Block<D, OWN> b;
    b.load(k + at, (size_t)P.Hkv * D, nk);
    b.store(tK, nullptr);
    b.load(v + at, (size_t)P.Hkv * D, nk);
    b.store(tV, nullptr);
  }
  float ak[R][D / 16] = {}, av[R][D / 16] = {};
  const int first = first_query(P.causal, j0, t.Lq, t.Lk) / TM, per = max(0, (t.Lq + TM - 1) / TM - first);
  const size_t ld = (size_t)P.Hq * D;
  Block<D, TM> bq, bg;
  float nl = 0.f, nd = 0.f;
  auto load = [&](int x) {  // block x of the group's heads' queries
    const int y = t.j0 + x, h = hk * P.G + y / per, i0 = (first + y % per) * TM;
    const size_t at = ((size_t)(t.q0 + i0) * P.Hq + h) * D;
    bq.load(q + at, ld, t.Lq - i0);
    bg.load(dO + at, ld, t.Lq - i0);
    if (threadIdx.x < TM) {
      const bool in = i0 + (int)threadIdx.x < t.Lq;
      const size_t r = (size_t)h * P.Nq + t.q0 + i0 + threadIdx.x;
      nl = in ? P.lse2[r] : 0.f;
      nd = in ? P.delta[r] : 0.f;
    }
  };
  const int n = min(per * P.G, t.j1) - t.j0;
  if (n > 0) load(0);
  for (int x = 0; x < n; x++) {
    const int i0 = (first + (t.j0 + x) % per) * TM;
    __syncthreads();
    bq.store(tQ, sQ);
    bg.store(tG, sG);
    if (threadIdx.x < TM) {
      sl[threadIdx.x] = nl;
      sd[threadIdx.x] = nd;
    }
    __syncthreads();
    if (x + 1 < n) load(x + 1);
    float s[R][4], dp[R][4];
    pairs<D, R>(tK, tQ, R * ty, 4 * tx, s);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int i = i0 + 4 * tx + j, lim = i < t.Lq ? keys_of(P.causal, i, t.Lq, t.Lk) : 0;
      float p[R];
#pragma unroll
      for (int e = 0; e < R; e++) {
        p[e] = j0 + R * ty + e < lim ? ex2(fmaf(s[e][j], P.scale2, -sl[4 * tx + j])) : 0.f;
        s[e][j] = p[e];
      }
      put_column<R>(sP + (4 * tx + j) * PP<R> + R * ty, p);
    }
    __syncwarp();
    apply<D, R>(sP, sG, R * ty, tx, av);
    pairs<D, R>(tV, tG, R * ty, 4 * tx, dp);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float d[R];
#pragma unroll
      for (int e = 0; e < R; e++) d[e] = s[e][j] == 0.f ? 0.f : s[e][j] * (dp[e][j] - sd[4 * tx + j]);
      put_column<R>(sP + (4 * tx + j) * PP<R> + R * ty, d);
    }
    __syncwarp();
    apply<D, R>(sP, sQ, R * ty, tx, ak);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < R; i++) {
    const int r = R * ty + i;
    if (r >= nk) continue;
    const bool whole = t.piece < 0;
    const size_t row = ((size_t)(t.k0 + j0 + r) * P.Hkv + hk) * D, pa = (((size_t)t.piece * P.Hkv + hk) * OWN + r) * D;
    float* ok = whole ? dk + row : P.po[2] + pa;
    float* ov = whole ? dv + row : P.po[2] + (size_t)P.pieces[2] * P.Hkv * OWN * D + pa;
    const float f = whole ? P.scale : 1.0f;
#pragma unroll
    for (int c = 0; c < D / 64; c++) {
      const float x[4] = {ak[i][4 * c] * f, ak[i][4 * c + 1] * f, ak[i][4 * c + 2] * f, ak[i][4 * c + 3] * f};
      const float y[4] = {av[i][4 * c], av[i][4 * c + 1], av[i][4 * c + 2], av[i][4 * c + 3]};
      st4(ok + 64 * c + 4 * tx, x);
      st4(ov + 64 * c + 4 * tx, y);
    }
  }
}

// dq of 16 R queries of one head.  Threads: queries R ty .., keys 4 tx ..
template <int D, int R>
__global__ void __launch_bounds__(NT) smx_dq_kernel(SmxP P, const float* __restrict__ q, const float* __restrict__ k,
                                                   const float* __restrict__ v, const float* __restrict__ dO,
                                                   float* __restrict__ dq) {
  constexpr int OWN = 16 * R;
  extern __shared__ __align__(16) float sm[];
  float *tQ = sm, *tG = tQ + D * OWN, *tK = tG + D * OWN, *tV = tK + D * TM, *sK = tV + D * TM, *sD = sK + D * TM;
  struct Last {  // what follows this grid follows dk and dv too
    __device__ ~Last() { pdl_wait(); }
  } last;
  if (!saved(P)) return;
  const int h = blockIdx.x % P.Hq, hk = h / P.G, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  Tile t;
  if (!tile_of(P, 1, blockIdx.x / P.Hq, false, t)) return;
  const int i0 = t.t * OWN, nq = min(OWN, t.Lq - i0);
  const size_t qa = ((size_t)(t.q0 + i0) * P.Hq + h) * D;
  {
    Block<D, OWN> b;
    b.load(q + qa, (size_t)P.Hq * D, nq);
    b.store(tQ, nullptr);
    b.load(dO + qa, (size_t)P.Hq * D, nq);
    b.store(tG, nullptr);
  }
  float acc[R][D / 16] = {}, l2[R], del[R];
  int lim[R];
#pragma unroll
  for (int i = 0; i < R; i++) {
    const int r = R * ty + i;
    const size_t at = (size_t)h * P.Nq + t.q0 + i0 + r;
    l2[i] = r < nq ? P.lse2[at] : 0.f;
    del[i] = r < nq ? P.delta[at] : 0.f;
    lim[i] = r < nq ? keys_of(P.causal, i0 + r, t.Lq, t.Lk) : 0;
  }
  const int nk = (int)min((int64_t)keys_of(P.causal, i0 + nq - 1, t.Lq, t.Lk), (int64_t)t.j1 * TM);
  const size_t ld = (size_t)P.Hkv * D, at = ((size_t)t.k0 * P.Hkv + hk) * D;
  Block<D, TM> bk, bv;
  const int first = t.j0 * TM;
  if (first < nk) {
    bk.load(k + at + first * ld, ld, t.Lk - first);
    bv.load(v + at + first * ld, ld, t.Lk - first);
  }
  for (int j0 = first; j0 < nk; j0 += TM) {
    __syncthreads();
    bk.store(tK, sK);
    bv.store(tV, nullptr);
    __syncthreads();
    if (j0 + TM < nk) {
      bk.load(k + at + (j0 + TM) * ld, ld, t.Lk - j0 - TM);
      bv.load(v + at + (j0 + TM) * ld, ld, t.Lk - j0 - TM);
    }
    float s[R][4], dp[R][4];
    pairs<D, R>(tQ, tK, R * ty, 4 * tx, s);
    pairs<D, R>(tG, tV, R * ty, 4 * tx, dp);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float d[R];
#pragma unroll
      for (int i = 0; i < R; i++)
        d[i] = j0 + 4 * tx + j < lim[i] ? ex2(fmaf(s[i][j], P.scale2, -l2[i])) * (dp[i][j] - del[i]) : 0.f;
      put_column<R>(sD + (4 * tx + j) * PP<R> + R * ty, d);
    }
    __syncwarp();
    apply<D, R>(sD, sK, R * ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < R; i++) {
    const int r = R * ty + i;
    if (r >= nq) continue;
    const bool whole = t.piece < 0;
    float* out = whole ? dq + qa + (size_t)r * P.Hq * D : P.po[1] + (((size_t)t.piece * P.Hq + h) * OWN + r) * D;
    const float f = whole ? P.scale : 1.0f;
#pragma unroll
    for (int c = 0; c < D / 64; c++) {
      const float x[4] = {acc[i][4 * c] * f, acc[i][4 * c + 1] * f, acc[i][4 * c + 2] * f, acc[i][4 * c + 3] * f};
      st4(out + 64 * c + 4 * tx, x);
    }
  }
}

}  // namespace

cudaError_t launch_f32_bwd(const SmxP& P, const float* q, const float* k, const float* v, const float* dO, float* dq,
                           float* dk, float* dv, cudaStream_t st) {
  constexpr int D = 128, R = F32_TILE / 16;
  const size_t s1 = (2 * D * 16 * R + 4 * D * TM + TM * PP<R> + 2 * TM) * sizeof(float);
  const size_t s2 = (2 * D * 16 * R + 3 * D * TM + TM * PP<R>) * sizeof(float);
  const int64_t gk = (int64_t)max_tiles(P, 2) * P.Hkv, gq = (int64_t)max_tiles(P, 1) * P.Hq;
  cudaError_t e = raise_smem<smx_dkv_kernel<D, R>>((int)s1);
  if (e == cudaSuccess) e = raise_smem<smx_dq_kernel<D, R>>((int)s2);
  if (e != cudaSuccess) return e;
  prof_begin(K_SMX_DKV, st);
  e = launch_pdl(smx_dkv_kernel<D, R>, dim3((unsigned)gk), dim3(NT), s1, st, P, q, k, v, dO, dk, dv);
  prof_end(K_SMX_DKV, st);
  if (e != cudaSuccess) return e;
  prof_begin(K_SMX_DQ, st);
  e = launch_pdl(smx_dq_kernel<D, R>, dim3((unsigned)gq), dim3(NT), s2, st, P, q, k, v, dO, dq);
  prof_end(K_SMX_DQ, st);
  return e;
}

}  // namespace smx
}  // namespace kda
