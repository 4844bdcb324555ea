// Softmax attention on the fp32 pipe: the fp32 io path (and any io type).
// Per document, query head h and its key head h / G:
//   s_ij = scale q_i k_j,  p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   dv_j = sum_i p_ij dO_i,  ds_ij = p_ij (dO_i v_j - delta_i),  delta_i = o_i dO_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
// 64 x 64 tiles of pairs, 256 threads with 4 x 4 pairs each; operands of the pair
// products lie transposed in shared memory ([d][row]) so that a thread's four rows
// are one 16-byte load.  The forward keeps a running maximum and sum per row.  dk
// and dv of a key tile are summed by one CTA over the queries of its whole head
// group, dq by one CTA over the keys: no atomics, a fixed order.
#include "kda_softmax.cuh"

namespace kda {
namespace smx {
namespace {

constexpr int TM = 64, NT = 256, PP = TM + 4;

__device__ __forceinline__ void ld4(const float* p, float (&v)[4]) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
__device__ __forceinline__ void ld4(const bf16* p, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void st4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st4(bf16* p, const float (&v)[4]) {
  uint2 u;
  *reinterpret_cast<__nv_bfloat162*>(&u.x) = __floats2bfloat162_rn(v[0], v[1]);
  *reinterpret_cast<__nv_bfloat162*>(&u.y) = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = u;
}

// Rows 0 .. n - 1 (of TM; the rest zero, so that a neighbour's values never enter a
// product) of x, whose rows are ld elements apart: tr[d][row], and pl[row][d] where wanted.
template <int D, typename T>
__device__ __forceinline__ void load_tile(const T* x, size_t ld, int n, float* tr, float* pl) {
  for (int i = threadIdx.x; i < TM * D / 4; i += NT) {
    const int r = i % TM, d = i / TM * 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < n) ld4(x + r * ld + d, v);
    if (tr)
#pragma unroll
      for (int e = 0; e < 4; e++) tr[(d + e) * TM + r] = v[e];
    if (pl) st4(pl + r * D + d, v);
  }
}

// c[i][j] = sum_d a[d][r0 + i] b[d][c0 + j]
template <int D>
__device__ __forceinline__ void pairs(const float* a, const float* b, int r0, int c0, float (&c)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) c[i][j] = 0.f;
#pragma unroll 8
  for (int d = 0; d < D; d++) {
    float x[4], y[4];
    ld4(a + d * TM + r0, x);
    ld4(b + d * TM + c0, y);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) c[i][j] = fmaf(x[i], y[j], c[i][j]);
  }
}
// c[i][64 m + 4 tx + e] += sum_n w[n][r0 + i] x[n][64 m + 4 tx + e]
template <int D>
__device__ __forceinline__ void apply(const float* w, const float* x, int r0, int tx, float (&c)[4][D / 16]) {
#pragma unroll 4
  for (int n = 0; n < TM; n++) {
    float a[4];
    ld4(w + n * PP + r0, a);
#pragma unroll
    for (int m = 0; m < D / 64; m++) {
      float y[4];
      ld4(x + n * D + 64 * m + 4 * tx, y);
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int e = 0; e < 4; e++) c[i][4 * m + e] = fmaf(a[i], y[e], c[i][4 * m + e]);
    }
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(NT) smx_fwd_kernel(SmxP P, const T* __restrict__ q, const T* __restrict__ k,
                                                    const T* __restrict__ v, T* __restrict__ o,
                                                    float* __restrict__ lse) {
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm, *sK = sQ + D * TM, *sV = sK + D * TM, *sP = sV + D * TM;
  pdl_wait();
  if (P.rows && blockIdx.x == 0 && threadIdx.x == 0) {
    *P.err = KDA_OK;
    *P.wtag = P.save ? P.tag : 0;
  }
  const int h = blockIdx.x % P.Hq, hk = h / P.G, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  Tile t;
  if (!tile_of(P, 0, blockIdx.x / P.Hq, false, t)) return;
  const int i0 = t.t * TM, nq = min(TM, t.Lq - i0);
  load_tile<D>(q + ((size_t)(t.q0 + i0) * P.Hq + h) * D, (size_t)P.Hq * D, nq, sQ, (float*)nullptr);
  float acc[4][D / 16] = {}, m[4], l[4];
  int lim[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    lim[i] = keys_of(P.causal, i0 + 4 * ty + i, t.Lq, t.Lk);
  }
  const int nk = keys_of(P.causal, i0 + nq - 1, t.Lq, t.Lk);
  for (int j0 = 0; j0 < nk; j0 += TM) {
    __syncthreads();
    const size_t at = ((size_t)(t.k0 + j0) * P.Hkv + hk) * D;
    load_tile<D>(k + at, (size_t)P.Hkv * D, t.Lk - j0, sK, (float*)nullptr);
    load_tile<D>(v + at, (size_t)P.Hkv * D, t.Lk - j0, (float*)nullptr, sV);
    __syncthreads();
    float s[4][4];
    pairs<D>(sQ, sK, 4 * ty, 4 * tx, s);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        s[i][j] = j0 + 4 * tx + j < lim[i] ? s[i][j] * P.scale2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[i], mx), mu = mn == -INFINITY ? 0.f : mn, c = ex2(m[i] - mu);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        s[i][j] = ex2(s[i][j] - mu);
        sum += s[i][j];
      }
      l[i] = l[i] * c + sum;
      m[i] = mn;
#pragma unroll
      for (int e = 0; e < D / 16; e++) acc[i][e] *= c;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float col[4] = {s[0][j], s[1][j], s[2][j], s[3][j]};
      st4(sP + (4 * tx + j) * PP + 4 * ty, col);
    }
    __syncwarp();  // a row's pairs are formed and used by one half warp
    apply<D>(sP, sV, 4 * ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    const int r = 4 * ty + i;
    if (r >= nq) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i], l2 = m[i] + log2f(l[i]);
    const size_t row = (size_t)(t.q0 + i0 + r) * P.Hq + h;
#pragma unroll
    for (int c = 0; c < D / 64; c++) {
      const float y[4] = {acc[i][4 * c] * inv, acc[i][4 * c + 1] * inv, acc[i][4 * c + 2] * inv,
                          acc[i][4 * c + 3] * inv};
      st4(o + row * D + 64 * c + 4 * tx, y);
      if (P.save && sizeof(T) == 2) {
        float z[4];
        ld4(o + row * D + 64 * c + 4 * tx, z);
#pragma unroll
        for (int e = 0; e < 4; e++) z[e] = y[e] - z[e];
        st4(P.res + row * D + 64 * c + 4 * tx, z);
      }
    }
    if (tx == 0) {
      lse[row] = l2 * LN2;
      if (P.save) P.lse2[(size_t)h * P.Nq + t.q0 + i0 + r] = l2;
    }
  }
}

// dk and dv of 64 keys of one key head.  Threads: keys 4 ty .., queries 4 tx ..
template <int D, typename T>
__global__ void __launch_bounds__(NT) smx_dkv_kernel(SmxP P, const T* __restrict__ q, const T* __restrict__ k,
                                                    const T* __restrict__ v, const T* __restrict__ dO,
                                                    T* __restrict__ dk, T* __restrict__ dv) {
  extern __shared__ __align__(16) float sm[];
  float *tK = sm, *tV = tK + D * TM, *tQ = tV + D * TM, *tG = tQ + D * TM, *sQ = tG + D * TM, *sG = sQ + D * TM;
  float *sP = sG + D * TM, *sD = sP + TM * PP, *sl = sD + TM * PP, *sd = sl + TM;
  pdl_wait();
  if (!saved(P)) return;
  const int hk = blockIdx.x % P.Hkv, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  Tile t;
  if (!tile_of(P, 2, blockIdx.x / P.Hkv, true, t)) return;
  const int j0 = t.t * TM, nk = min(TM, t.Lk - j0);
  const size_t at = ((size_t)(t.k0 + j0) * P.Hkv + hk) * D;
  load_tile<D>(k + at, (size_t)P.Hkv * D, nk, tK, (float*)nullptr);
  load_tile<D>(v + at, (size_t)P.Hkv * D, nk, tV, (float*)nullptr);
  float ak[4][D / 16] = {}, av[4][D / 16] = {};
  const int first = first_query(P.causal, j0, t.Lq, t.Lk) / TM * TM;
  for (int g = 0; g < P.G; g++) {
    const int h = hk * P.G + g;
    for (int i0 = first; i0 < t.Lq; i0 += TM) {
      __syncthreads();
      const size_t qa = ((size_t)(t.q0 + i0) * P.Hq + h) * D;
      load_tile<D>(q + qa, (size_t)P.Hq * D, t.Lq - i0, tQ, sQ);
      load_tile<D>(dO + qa, (size_t)P.Hq * D, t.Lq - i0, tG, sG);
      if (threadIdx.x < TM) {
        const bool in = i0 + (int)threadIdx.x < t.Lq;
        const size_t r = (size_t)h * P.Nq + t.q0 + i0 + threadIdx.x;
        sl[threadIdx.x] = in ? P.lse2[r] : 0.f;
        sd[threadIdx.x] = in ? P.delta[r] : 0.f;
      }
      __syncthreads();
      float s[4][4], dp[4][4];
      pairs<D>(tK, tQ, 4 * ty, 4 * tx, s);
      pairs<D>(tV, tG, 4 * ty, 4 * tx, dp);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int i = i0 + 4 * tx + j, lim = i < t.Lq ? keys_of(P.causal, i, t.Lq, t.Lk) : 0;
        float p[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const bool seen = j0 + 4 * ty + e < lim;
          p[e] = seen ? ex2(fmaf(s[e][j], P.scale2, -sl[4 * tx + j])) : 0.f;
          d[e] = seen ? p[e] * (dp[e][j] - sd[4 * tx + j]) : 0.f;
        }
        st4(sP + (4 * tx + j) * PP + 4 * ty, p);
        st4(sD + (4 * tx + j) * PP + 4 * ty, d);
      }
      __syncwarp();
      apply<D>(sP, sG, 4 * ty, tx, av);
      apply<D>(sD, sQ, 4 * ty, tx, ak);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * ty + i;
    if (r >= nk) continue;
    const size_t row = ((size_t)(t.k0 + j0 + r) * P.Hkv + hk) * D;
#pragma unroll
    for (int c = 0; c < D / 64; c++) {
      const float x[4] = {ak[i][4 * c] * P.scale, ak[i][4 * c + 1] * P.scale, ak[i][4 * c + 2] * P.scale,
                          ak[i][4 * c + 3] * P.scale};
      const float y[4] = {av[i][4 * c], av[i][4 * c + 1], av[i][4 * c + 2], av[i][4 * c + 3]};
      st4(dk + row + 64 * c + 4 * tx, x);
      st4(dv + row + 64 * c + 4 * tx, y);
    }
  }
}

// dq of 64 queries of one head.  Threads: queries 4 ty .., keys 4 tx ..
template <int D, typename T>
__global__ void __launch_bounds__(NT) smx_dq_kernel(SmxP P, const T* __restrict__ q, const T* __restrict__ k,
                                                   const T* __restrict__ v, const T* __restrict__ dO,
                                                   T* __restrict__ dq) {
  extern __shared__ __align__(16) float sm[];
  float *tQ = sm, *tG = tQ + D * TM, *tK = tG + D * TM, *tV = tK + D * TM, *sK = tV + D * TM, *sD = sK + D * TM;
  pdl_wait();
  if (!saved(P)) return;
  const int h = blockIdx.x % P.Hq, hk = h / P.G, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  Tile t;
  if (!tile_of(P, 1, blockIdx.x / P.Hq, false, t)) return;
  const int i0 = t.t * TM, nq = min(TM, t.Lq - i0);
  const size_t qa = ((size_t)(t.q0 + i0) * P.Hq + h) * D;
  load_tile<D>(q + qa, (size_t)P.Hq * D, nq, tQ, (float*)nullptr);
  load_tile<D>(dO + qa, (size_t)P.Hq * D, nq, tG, (float*)nullptr);
  float acc[4][D / 16] = {}, l2[4], del[4];
  int lim[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * ty + i;
    const size_t at = (size_t)h * P.Nq + t.q0 + i0 + r;
    l2[i] = r < nq ? P.lse2[at] : 0.f;
    del[i] = r < nq ? P.delta[at] : 0.f;
    lim[i] = r < nq ? keys_of(P.causal, i0 + r, t.Lq, t.Lk) : 0;
  }
  const int nk = keys_of(P.causal, i0 + nq - 1, t.Lq, t.Lk);
  for (int j0 = 0; j0 < nk; j0 += TM) {
    __syncthreads();
    const size_t at = ((size_t)(t.k0 + j0) * P.Hkv + hk) * D;
    load_tile<D>(k + at, (size_t)P.Hkv * D, t.Lk - j0, tK, sK);
    load_tile<D>(v + at, (size_t)P.Hkv * D, t.Lk - j0, tV, (float*)nullptr);
    __syncthreads();
    float s[4][4], dp[4][4];
    pairs<D>(tQ, tK, 4 * ty, 4 * tx, s);
    pairs<D>(tG, tV, 4 * ty, 4 * tx, dp);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float d[4];
#pragma unroll
      for (int i = 0; i < 4; i++)
        d[i] = j0 + 4 * tx + j < lim[i] ? ex2(fmaf(s[i][j], P.scale2, -l2[i])) * (dp[i][j] - del[i]) : 0.f;
      st4(sD + (4 * tx + j) * PP + 4 * ty, d);
    }
    __syncwarp();
    apply<D>(sD, sK, 4 * ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * ty + i;
    if (r >= nq) continue;
#pragma unroll
    for (int c = 0; c < D / 64; c++) {
      const float x[4] = {acc[i][4 * c] * P.scale, acc[i][4 * c + 1] * P.scale, acc[i][4 * c + 2] * P.scale,
                          acc[i][4 * c + 3] * P.scale};
      st4(dq + qa + (size_t)r * P.Hq * D + 64 * c + 4 * tx, x);
    }
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch(int kid, void (*kern)(KArgs...), int64_t grid, size_t smem, cudaStream_t st, Args... args) {
  if (grid <= 0 || grid > 2147483647) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  prof_begin(kid, st);
  e = launch_pdl(kern, dim3((unsigned)grid), dim3(NT), smem, st, args...);
  prof_end(kid, st);
  return e;
}

template <int D, typename T>
cudaError_t fwd(const SmxP& P, const void* q, const void* k, const void* v, void* o, float* lse, cudaStream_t st) {
  const size_t smem = (3 * D * TM + TM * PP) * sizeof(float);
  return launch(K_SMX_FWD, smx_fwd_kernel<D, T>, (int64_t)max_tiles(P, 0) * P.Hq, smem, st, P, (const T*)q,
                (const T*)k, (const T*)v, (T*)o, lse);
}
template <int D, typename T>
cudaError_t bwd(const SmxP& P, const void* q, const void* k, const void* v, const void* dO, void* dq, void* dk,
                void* dv, cudaStream_t st) {
  const size_t s1 = (6 * D * TM + 2 * TM * PP + 2 * TM) * sizeof(float), s2 = (5 * D * TM + TM * PP) * sizeof(float);
  cudaError_t e = launch(K_SMX_DKV, smx_dkv_kernel<D, T>, (int64_t)max_tiles(P, 2) * P.Hkv, s1, st, P, (const T*)q,
                         (const T*)k, (const T*)v, (const T*)dO, (T*)dk, (T*)dv);
  if (e != cudaSuccess) return e;
  return launch(K_SMX_DQ, smx_dq_kernel<D, T>, (int64_t)max_tiles(P, 1) * P.Hq, s2, st, P, (const T*)q, (const T*)k,
                (const T*)v, (const T*)dO, (T*)dq);
}

}  // namespace

cudaError_t launch_f32_fwd(const SmxP& P, int D, int dtype, const void* q, const void* k, const void* v, void* o,
                           float* lse, cudaStream_t st) {
  if (dtype == KDA_F32)
    return D == 64 ? fwd<64, float>(P, q, k, v, o, lse, st) : fwd<128, float>(P, q, k, v, o, lse, st);
  return D == 64 ? fwd<64, bf16>(P, q, k, v, o, lse, st) : fwd<128, bf16>(P, q, k, v, o, lse, st);
}
cudaError_t launch_f32_bwd(const SmxP& P, int D, int dtype, const void* q, const void* k, const void* v,
                           const void* dO, void* dq, void* dk, void* dv, cudaStream_t st) {
  if (dtype == KDA_F32)
    return D == 64 ? bwd<64, float>(P, q, k, v, dO, dq, dk, dv, st) : bwd<128, float>(P, q, k, v, dO, dq, dk, dv, st);
  return D == 64 ? bwd<64, bf16>(P, q, k, v, dO, dq, dk, dv, st) : bwd<128, bf16>(P, q, k, v, dO, dq, dk, dv, st);
}

}  // namespace smx
}  // namespace kda
