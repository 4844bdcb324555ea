// Layer norm over the last axis of n rows of D values:
//   mu = mean_j x_j,  r = 1 / sqrt(mean_j (x_j - mu)^2 + eps),  xh_j = (x_j - mu) r,
//   y_j = xh_j w_j + b_j,
// and its backward
//   g_j = dy_j w_j,  dx_j = r (g_j - mean(g) - xh_j mean(g xh)),
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
// Bound by HBM: the forward reads x and writes y once, the backward reads x
// and dy and writes dx once.  A row sits in the registers of G threads (at
// most 16 values each) from its load to its store, so the variance is the
// second moment of the centred values (no E[x^2] - mu^2 cancellation) at no
// further read.  G <= 32: several rows per warp, sums by shuffles; above,
// one row per CTA of G threads.  The backward's CTAs are persistent over rows and keep their
// columns' dw / db sums in registers (a thread owns the same columns of every
// row); the per-CTA partials are then added in a fixed order (deterministic).
// Loads are 16 bytes where D allows it, else 4 or a single value: D = 5003 in
// bf16 has no wider aligned load in most rows.
#include "kda_internal.cuh"
#include "../../include/kda.h"

namespace kda {
namespace {

constexpr int LN_NTHR = 256;         // threads per CTA where a row takes at most a warp
constexpr int LN_PER = 16;           // values of a row per thread
constexpr int LN_REG_D = 16384;      // widest row held in registers (1024 threads)
constexpr int LN_SMS = 152;          // the backward's grid: a few persistent CTAs per SM
constexpr int LN_MAX_D = 1 << 24;

template <typename T, int VEC> struct Vec;
template <> struct Vec<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void ld(const __nv_bfloat16* p, float* v) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; e++) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void st(__nv_bfloat16* p, const float* v) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int e = 0; e < 4; e++) h[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    *reinterpret_cast<uint4*>(p) = u;
  }
};
template <> struct Vec<__nv_bfloat16, 2> {
  static __device__ __forceinline__ void ld(const __nv_bfloat16* p, float* v) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ void st(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
  }
};
template <typename T> struct Vec<T, 1> {
  static __device__ __forceinline__ void ld(const T* p, float* v) { v[0] = ldf(p); }
  static __device__ __forceinline__ void st(T* p, const float* v) { stf(p, v[0]); }
};
template <> struct Vec<float, 4> {
  static __device__ __forceinline__ void ld(const float* p, float* v) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  }
  static __device__ __forceinline__ void st(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// Sum of x over the G threads of a row: the whole CTA (BLK; red: 32 floats,
// reused only after another barrier), or an aligned group of G lanes.
template <bool BLK>
__device__ __forceinline__ float group_sum(float x, int G, float* red) {
  if (!BLK) {
    for (int o = G >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  }
  x = warp_sum(x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = x;
  __syncthreads();
  float s = lane < nw ? red[lane] : 0.f;
  return warp_sum(s);
}

template <typename T, int VEC, int NCH, bool BLK>
__global__ void __launch_bounds__(BLK ? 1024 : LN_NTHR) ln_fwd_kernel(int64_t n, int D, int G, float eps,
                                                                      const T* __restrict__ x,
                                                                      const float* __restrict__ w,
                                                                      const float* __restrict__ b, T* __restrict__ y,
                                                                      float* __restrict__ mean,
                                                                      float* __restrict__ rstd) {
  __shared__ float red[2][32];
  const int gid = BLK ? 0 : threadIdx.x / G, lane = BLK ? threadIdx.x : threadIdx.x % G;
  const int rpc = BLK ? 1 : LN_NTHR / G;
  const float inv = 1.0f / (float)D;
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < n; base += (int64_t)gridDim.x * rpc) {
    const int64_t row = base + gid;
    const bool ok = row < n;  // a group's lanes agree; shuffles stay warp-wide
    const T* xr = x + row * D;
    float v[NCH * VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int c = (i * G + lane) * VEC;
      if (ok && c < D) {
        Vec<T, VEC>::ld(xr + c, v + i * VEC);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e++) v[i * VEC + e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < VEC; e++) s += v[i * VEC + e];
    }
    const float mu = group_sum<BLK>(s, G, red[0]) * inv;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const bool in = (i * G + lane) * VEC < D;
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        v[i * VEC + e] -= mu;
        if (in) q += v[i * VEC + e] * v[i * VEC + e];
      }
    }
    const float r = 1.0f / sqrtf(group_sum<BLK>(q, G, red[1]) * inv + eps);
    if (ok && mean && lane == 0) {
      mean[row] = mu;
      rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int c = (i * G + lane) * VEC;
      if (ok && c < D) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e++) o[e] = v[i * VEC + e] * r * __ldg(w + c + e) + (b ? __ldg(b + c + e) : 0.f);
        Vec<T, VEC>::st(y + row * D + c, o);
      }
    }
    if (BLK) __syncthreads();  // red is free again
  }
}

// MODE 0: rows within warps; 1: a row per CTA, dw / db sums in registers; 2: a
// row per CTA of up to 1024 threads, the sums in shared memory (a thread's own
// slots; 64 registers per thread would not hold them).
template <typename T, int VEC, int NCH, int MODE>
__global__ void __launch_bounds__(MODE == 0 ? LN_NTHR : MODE == 1 ? 512 : 1024)
    ln_bwd_kernel(int64_t n, int D, int G, const T* __restrict__ x, const float* __restrict__ w,
                  const T* __restrict__ dy, const float* __restrict__ mean, const float* __restrict__ rstd,
                  T* __restrict__ dx, float* __restrict__ part) {
  constexpr bool BLK = MODE != 0;
  constexpr int E = NCH * VEC;
  __shared__ float red[4][32];
  extern __shared__ float acc[];  // MODE 0: [256 / G][D]; MODE 2: [2][E][blockDim.x]
  pdl_release();
  const int gid = BLK ? 0 : threadIdx.x / G, lane = BLK ? threadIdx.x : threadIdx.x % G;
  const int rpc = BLK ? 1 : LN_NTHR / G;
  const float inv = 1.0f / (float)D;
  float aw[MODE == 2 ? 1 : E], ab[MODE == 2 ? 1 : E];
  if (MODE == 2) {
#pragma unroll
    for (int e = 0; e < E; e++) acc[e * blockDim.x + threadIdx.x] = acc[(E + e) * blockDim.x + threadIdx.x] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < (MODE == 2 ? 1 : E); e++) aw[e] = ab[e] = 0.f;
  }
  int flip = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpc; base < n; base += (int64_t)gridDim.x * rpc) {
    const int64_t row = base + gid;
    const bool ok = row < n;
    float xh[E], g[E];
    const float mu = ok ? __ldg(mean + row) : 0.f, r = ok ? __ldg(rstd + row) : 0.f;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int c = (i * G + lane) * VEC;
      if (ok && c < D) {
        Vec<T, VEC>::ld(x + row * D + c, xh + i * VEC);
        Vec<T, VEC>::ld(dy + row * D + c, g + i * VEC);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; e++) { xh[i * VEC + e] = mu; g[i * VEC + e] = 0.f; }
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int c = (i * G + lane) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        const int j = i * VEC + e;
        const float h = (xh[j] - mu) * r, d = g[j];
        xh[j] = h;
        if (MODE == 2) {
          acc[j * blockDim.x + threadIdx.x] += d * h;
          acc[(E + j) * blockDim.x + threadIdx.x] += d;
        } else {
          aw[MODE == 2 ? 0 : j] += d * h;
          ab[MODE == 2 ? 0 : j] += d;
        }
        const float gw = c < D ? d * __ldg(w + c + e) : 0.f;
        g[j] = gw;
        s1 += gw;
        s2 += gw * h;
      }
    }
    float m1, m2;
    if (BLK) {  // both sums across one barrier; the buffers alternate between rows
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      const int ln = threadIdx.x & 31, wp = threadIdx.x >> 5, nw = blockDim.x >> 5;
      if (ln == 0) { red[flip][wp] = s1; red[flip + 1][wp] = s2; }
      __syncthreads();
      m1 = warp_sum(ln < nw ? red[flip][ln] : 0.f) * inv;
      m2 = warp_sum(ln < nw ? red[flip + 1][ln] : 0.f) * inv;
      flip ^= 2;
    } else {
      m1 = group_sum<false>(s1, G, nullptr) * inv;
      m2 = group_sum<false>(s2, G, nullptr) * inv;
    }
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      const int c = (i * G + lane) * VEC;
      if (ok && c < D) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; e++) o[e] = r * (g[i * VEC + e] - m1 - xh[i * VEC + e] * m2);
        Vec<T, VEC>::st(dx + row * D + c, o);
      }
    }
  }
  float* pw = part + (int64_t)blockIdx.x * 2 * D;
  if (MODE == 0) {  // the CTA's row groups in order, dw then db
#pragma unroll
    for (int k = 0; k < 2; k++) {
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        const int c = (i * G + lane) * VEC;
        if (c < D) {
#pragma unroll
          for (int e = 0; e < VEC; e++) {
            const int j = MODE == 2 ? 0 : i * VEC + e;
            acc[gid * D + c + e] = k ? ab[j] : aw[j];
          }
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += LN_NTHR) {
        float s = 0.f;
        for (int q = 0; q < LN_NTHR / G; q++) s += acc[q * D + c];
        pw[k * D + c] = s;
      }
      __syncthreads();
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int c = (i * G + lane) * VEC;
    if (c < D) {
#pragma unroll
      for (int e = 0; e < VEC; e++) {
        const int j = i * VEC + e;
        pw[c + e] = MODE == 2 ? acc[j * blockDim.x + threadIdx.x] : aw[MODE == 2 ? 0 : j];
        pw[D + c + e] = MODE == 2 ? acc[(E + j) * blockDim.x + threadIdx.x] : ab[MODE == 2 ? 0 : j];
      }
    }
  }
}

// Rows wider than LN_REG_D: a CTA per row, the row read once per pass (its
// later passes hit L2), the backward's column sums in its partial row.
template <typename T>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(int64_t n, int D, float eps, const T* __restrict__ x,
                                                           const float* __restrict__ w, const float* __restrict__ b,
                                                           T* __restrict__ y, float* __restrict__ mean,
                                                           float* __restrict__ rstd) {
  __shared__ float red[2][32];
  const float inv = 1.0f / (float)D;
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const T* xr = x + row * D;
    float s = 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) s += ldf(xr + c);
    const float mu = group_sum<true>(s, 0, red[0]) * inv;
    float q = 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      const float d = ldf(xr + c) - mu;
      q += d * d;
    }
    const float r = 1.0f / sqrtf(group_sum<true>(q, 0, red[1]) * inv + eps);
    if (mean && threadIdx.x == 0) {
      mean[row] = mu;
      rstd[row] = r;
    }
    for (int c = threadIdx.x; c < D; c += blockDim.x)
      stf(y + row * D + c, (ldf(xr + c) - mu) * r * w[c] + (b ? b[c] : 0.f));
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) ln_bwd_wide_kernel(int64_t n, int D, const T* __restrict__ x,
                                                           const float* __restrict__ w, const T* __restrict__ dy,
                                                           const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, T* __restrict__ dx,
                                                           float* __restrict__ part) {
  __shared__ float red[2][32];
  const float inv = 1.0f / (float)D;
  float* pw = part + (int64_t)blockIdx.x * 2 * D;
  pdl_release();
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const float mu = mean[row], r = rstd[row];
    const bool first = row == blockIdx.x;
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      const float h = (ldf(x + row * D + c) - mu) * r, d = ldf(dy + row * D + c), g = d * w[c];
      pw[c] = (first ? 0.f : pw[c]) + d * h;
      pw[D + c] = (first ? 0.f : pw[D + c]) + d;
      s1 += g;
      s2 += g * h;
    }
    const float m1 = group_sum<true>(s1, 0, red[0]) * inv, m2 = group_sum<true>(s2, 0, red[1]) * inv;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      const float h = (ldf(x + row * D + c) - mu) * r;
      stf(dx + row * D + c, r * (ldf(dy + row * D + c) * w[c] - m1 - h * m2));
    }
    __syncthreads();
  }
}

// dw | db [2 D] = the sums over the nblk partial rows, in a fixed order: a CTA
// owns 32 columns, each of its 32 warps every 32nd row, then the warps in order.
__global__ void __launch_bounds__(1024) ln_reduce_kernel(const float* __restrict__ part, int nblk, int D,
                                                         float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float red[32][33];
  const int cx = threadIdx.x & 31, gy = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
  const int64_t nc = 2 * (int64_t)D;
  pdl_wait();
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < nc) {
    int r = gy;
    for (; r + 96 < nblk; r += 128) {
#pragma unroll
      for (int u = 0; u < 4; u++) s[u] += part[(int64_t)(r + 32 * u) * nc + c];
    }
    for (; r < nblk; r += 32) s[0] += part[(int64_t)r * nc + c];
  }
  red[gy][cx] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (gy == 0 && c < nc) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < 32; g++) t += red[g][cx];
    if (c < D) dw[c] = t;
    else if (db) db[c - D] = t;
  }
}

// How a row of D values is laid over threads: vectors of vec values (16 bytes,
// or 4 or one value as D's divisors allow), G threads a row.
struct LnShape {
  int vec, G;
  bool blk;
};
LnShape ln_shape(int D, int dtype) {
  LnShape s;
  if (dtype == KDA_BF16) s.vec = D % 8 == 0 ? 8 : D % 2 == 0 ? 2 : 1;
  else s.vec = D % 4 == 0 ? 4 : 1;
  int G = 1;
  while (G < 32 && G * LN_PER < D) G *= 2;
  if (G * LN_PER < D) G = ((D + LN_PER - 1) / LN_PER + 31) / 32 * 32;  // whole warps, no power of two needed
  s.G = G;
  s.blk = G > 32;
  return s;
}

// Persistent CTAs of the backward: at least one row group each, and no more
// than what the SMs hold at once.
int ln_bwd_blocks(int64_t n, int D, int dtype) {
  if (D > LN_REG_D) return (int)(n < LN_SMS ? n : LN_SMS);
  const LnShape s = ln_shape(D, dtype);
  const int thr = s.blk ? s.G : LN_NTHR, rpc = s.blk ? 1 : LN_NTHR / s.G;
  int per = 1024 / thr;
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  const int64_t need = (n + rpc - 1) / rpc;
  return (int)(need < (int64_t)LN_SMS * per ? need : (int64_t)LN_SMS * per);
}

struct LnArgs {
  int64_t n;
  int D;
  float eps;
  const void *x, *dy;
  const float *w, *b;
  void *y, *dx;
  float *mean, *rstd, *part;
  cudaStream_t st;
};

template <typename T, int VEC>
cudaError_t ln_fwd_launch(const LnShape& s, const LnArgs& a) {
  constexpr int NCH = LN_PER / VEC;
  const int rpc = s.blk ? 1 : LN_NTHR / s.G;
  const int64_t need = (a.n + rpc - 1) / rpc;
  const unsigned grid = (unsigned)(need < (1 << 30) ? need : (1 << 30));
  if (s.blk)
    ln_fwd_kernel<T, VEC, NCH, true><<<grid, s.G, 0, a.st>>>(a.n, a.D, s.G, a.eps, (const T*)a.x, a.w, a.b, (T*)a.y,
                                                             a.mean, a.rstd);
  else
    ln_fwd_kernel<T, VEC, NCH, false><<<grid, LN_NTHR, 0, a.st>>>(a.n, a.D, s.G, a.eps, (const T*)a.x, a.w, a.b,
                                                                  (T*)a.y, a.mean, a.rstd);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t ln_bwd_launch(const LnShape& s, const LnArgs& a, int nblk) {
  constexpr int NCH = LN_PER / VEC;
  if (!s.blk) {
    const size_t smem = (size_t)(LN_NTHR / s.G) * a.D * sizeof(float);  // at most 256 * 16 floats
    ln_bwd_kernel<T, VEC, NCH, 0><<<nblk, LN_NTHR, smem, a.st>>>(a.n, a.D, s.G, (const T*)a.x, a.w, (const T*)a.dy,
                                                                 a.mean, a.rstd, (T*)a.dx, a.part);
  } else if (s.G <= 512) {
    ln_bwd_kernel<T, VEC, NCH, 1><<<nblk, s.G, 0, a.st>>>(a.n, a.D, s.G, (const T*)a.x, a.w, (const T*)a.dy, a.mean,
                                                          a.rstd, (T*)a.dx, a.part);
  } else {
    const int smem = 2 * LN_PER * s.G * (int)sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(ln_bwd_kernel<T, VEC, NCH, 2>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ln_bwd_kernel<T, VEC, NCH, 2><<<nblk, s.G, smem, a.st>>>(a.n, a.D, s.G, (const T*)a.x, a.w, (const T*)a.dy,
                                                             a.mean, a.rstd, (T*)a.dx, a.part);
  }
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

kda_status ln_check(int64_t n, int D, int dtype) {
  if (n <= 0 || D <= 0 || n > ((int64_t)1 << 34)) return KDA_ERR_INVALID_ARG;
  if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
  if (D > LN_MAX_D) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" KDA_API size_t kda_layer_norm_workspace_size(int64_t n_rows, int D, int dtype) {
  if (ln_check(n_rows, D, dtype) != KDA_OK) return 0;
  return (size_t)ln_bwd_blocks(n_rows, D, dtype) * 2 * (size_t)D * sizeof(float);
}

extern "C" KDA_API kda_status kda_layer_norm_fwd(int64_t n_rows, int D, int dtype, float eps, const void* x,
                                                 const float* w, const float* bias, void* y, float* mean,
                                                 float* rstd, cudaStream_t st) {
  const kda_status c = ln_check(n_rows, D, dtype);
  if (c != KDA_OK) return c;
  if (!x || !w || !y || !mean != !rstd) return KDA_ERR_INVALID_ARG;
  const void* ptrs[] = {x, w, bias, y, mean, rstd};
  for (const void* p : ptrs)
    if (!aligned16(p)) return KDA_ERR_ALIGNMENT;
  const LnShape s = ln_shape(D, dtype);
  LnArgs a = {};
  a.n = n_rows; a.D = D; a.eps = eps > 0.f ? eps : 1e-6f;
  a.x = x; a.w = w; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd; a.st = st;
  typedef __nv_bfloat16 B;
  cudaError_t e;
  prof_begin(K_LN_FWD, st);
  if (D > LN_REG_D) {
    const unsigned grid = (unsigned)(n_rows < (1 << 30) ? n_rows : (1 << 30));
    if (dtype == KDA_BF16)
      ln_fwd_wide_kernel<B><<<grid, 1024, 0, st>>>(n_rows, D, a.eps, (const B*)x, w, bias, (B*)y, mean, rstd);
    else
      ln_fwd_wide_kernel<float><<<grid, 1024, 0, st>>>(n_rows, D, a.eps, (const float*)x, w, bias, (float*)y, mean,
                                                       rstd);
    e = cudaGetLastError();
  } else if (dtype == KDA_BF16) {
    e = s.vec == 8 ? ln_fwd_launch<B, 8>(s, a) : s.vec == 2 ? ln_fwd_launch<B, 2>(s, a) : ln_fwd_launch<B, 1>(s, a);
  } else {
    e = s.vec == 4 ? ln_fwd_launch<float, 4>(s, a) : ln_fwd_launch<float, 1>(s, a);
  }
  prof_end(K_LN_FWD, st);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" KDA_API kda_status kda_layer_norm_bwd(int64_t n_rows, int D, int dtype, const void* x, const float* w,
                                                 const void* dy, const float* mean, const float* rstd, void* dx,
                                                 float* dw, float* dbias, void* workspace, size_t workspace_bytes,
                                                 cudaStream_t st) {
  const kda_status c = ln_check(n_rows, D, dtype);
  if (c != KDA_OK) return c;
  if (!x || !w || !dy || !mean || !rstd || !dx || !dw) return KDA_ERR_INVALID_ARG;
  const void* ptrs[] = {x, w, dy, mean, rstd, dx, dw, dbias};
  for (const void* p : ptrs)
    if (!aligned16(p)) return KDA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kda_layer_norm_workspace_size(n_rows, D, dtype)) return KDA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return KDA_ERR_ALIGNMENT;
  const LnShape s = ln_shape(D, dtype);
  const int nblk = ln_bwd_blocks(n_rows, D, dtype);
  LnArgs a = {};
  a.n = n_rows; a.D = D;
  a.x = x; a.w = w; a.dy = dy; a.dx = dx; a.mean = (float*)mean; a.rstd = (float*)rstd; a.part = (float*)workspace;
  a.st = st;
  typedef __nv_bfloat16 B;
  cudaError_t e;
  prof_begin(K_LN_BWD, st);
  if (D > LN_REG_D) {
    if (dtype == KDA_BF16)
      ln_bwd_wide_kernel<B><<<nblk, 1024, 0, st>>>(n_rows, D, (const B*)x, w, (const B*)dy, mean, rstd, (B*)dx, a.part);
    else
      ln_bwd_wide_kernel<float><<<nblk, 1024, 0, st>>>(n_rows, D, (const float*)x, w, (const float*)dy, mean, rstd,
                                                       (float*)dx, a.part);
    e = cudaGetLastError();
  } else if (dtype == KDA_BF16) {
    e = s.vec == 8 ? ln_bwd_launch<B, 8>(s, a, nblk)
                   : s.vec == 2 ? ln_bwd_launch<B, 2>(s, a, nblk) : ln_bwd_launch<B, 1>(s, a, nblk);
  } else {
    e = s.vec == 4 ? ln_bwd_launch<float, 4>(s, a, nblk) : ln_bwd_launch<float, 1>(s, a, nblk);
  }
  prof_end(K_LN_BWD, st);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  prof_begin(K_LN_RED, st);
  e = launch_pdl(ln_reduce_kernel, dim3((unsigned)((2 * (int64_t)D + 31) / 32)), dim3(1024), 0, st,
                 (const float*)a.part, nblk, D, dw, dbias);
  prof_end(K_LN_RED, st);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
