// Layer norm over the last axis of n rows of D values:
//   mu = mean_j x_j,  r = 1 / sqrt(mean_j (x_j - mu)^2 + eps),  xh_j = (x_j - mu) r,
//   y_j = xh_j w_j + b_j,
// and its backward
//   g_j = dy_j w_j,  dx_j = r (g_j - mean(g) - xh_j mean(g xh)),
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
// Bound by HBM: the forward reads x and writes y once, the backward reads x
// and dy and writes dx once.  A row sits in the registers of G threads from
// its load to its store, so the variance is the second moment of the centred
// values (no E[x^2] - mu^2 cancellation) at no further read.  G <= 32: rows
// within warps, sums by shuffles; above, one row per CTA of G threads.
//
// Every access is an aligned 16-byte vector whatever D is.  Row r starts r D
// values into the tensor, s = r D mod V values past a vector's start (V values
// a vector); the CTAs are persistent and their row step is a multiple of V, so
// a thread meets the same s, hence the same columns, in all its rows: it keeps
// their w and b, and the backward their dw and db sums, in registers.  The two
// vectors that a row shares with its neighbours are read and written value by
// value.  Eight columns a thread, so that 1024 threads fit an SM; two rows at a
// time share the sums' barriers, and the next rows are under way to the
// thread's own slots of shared memory (cp.async, no barrier) meanwhile.  The
// backward's per-CTA partials are added in a fixed order (deterministic).
#include "kda_internal.cuh"
#include "../../include/kda.h"

namespace kda {
namespace {

constexpr int LN_NTHR = 256;     // threads per CTA where a row takes at most a warp
constexpr int LN_CTAS = 3;       // and resident CTAs per SM of those
constexpr int LN_PER = 8;        // values of a row per thread (16 in rows past LN_WIDE)
constexpr int LN_WIDE = 8184;    // widest row of 1024 threads at eight values each (and a vector of offset)
constexpr int LN_REG_D = 16368;  // and at sixteen; wider rows are read once per pass
constexpr int LN_SMS = 152;      // the grids: what the SMs hold at once
constexpr int LN_MAX_D = 1 << 24;

// 16 bytes as loaded (half the registers for bf16) until they are used.
template <typename T>
struct Pack {
  static constexpr int V = 16 / (int)sizeof(T);
  uint4 u;
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (sizeof(T) == 4) {
      u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    } else {
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int e = 0; e < 4; e++) h[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    }
  }
};

// A thread's vector: columns c .. c + V - 1 of its rows, of which those in
// [0, D) exist.
template <typename T>
struct Cols {
  static constexpr int V = Pack<T>::V;
  int c, D;
  __device__ __forceinline__ Cols(int first, int D_) : c(first), D(D_) {}
  __device__ __forceinline__ bool full() const { return c >= 0 && c + V <= D; }
  __device__ __forceinline__ bool any() const { return c < D && c + V > 0; }
  __device__ __forceinline__ bool in(int e) const { return (unsigned)(c + e) < (unsigned)D; }
  __device__ __forceinline__ Pack<T> load(const T* row) const {  // missing columns read as 0
    Pack<T> p;
    if (full()) {
      p.u = __ldg(reinterpret_cast<const uint4*>(row + c));
    } else {
      float v[V];
#pragma unroll
      for (int e = 0; e < V; e++) v[e] = in(e) ? ldf(row + c + e) : 0.f;
      p.set(v);
    }
    return p;
  }
  // The whole aligned vector to shared memory, its neighbours' columns included, but nothing at or
  // past `end` (the tensor's).
  __device__ __forceinline__ void copy(uint4* slot, const T* row, const T* end) const {
    const int64_t left = (const char*)end - (const char*)(row + c);
    const int bytes = left < 16 ? (int)left : 16;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(slot)),
                 "l"(row + c), "r"(bytes)
                 : "memory");
  }
  __device__ __forceinline__ void clear(float* v) const {  // the columns that are not this row's
    if (!full()) {
#pragma unroll
      for (int e = 0; e < V; e++)
        if (!in(e)) v[e] = 0.f;
    }
  }
  __device__ __forceinline__ void store(T* row, const float* v) const {
    if (full()) {
      Pack<T> p;
      p.set(v);
      *reinterpret_cast<uint4*>(row + c) = p.u;
    } else {
#pragma unroll
      for (int e = 0; e < V; e++)
        if (in(e)) stf(row + c + e, v[e]);
    }
  }
  __device__ __forceinline__ void param(const float* w, float* v) const {
#pragma unroll
    for (int e = 0; e < V; e++) v[e] = w && in(e) ? __ldg(w + c + e) : 0.f;
  }
};

// Sums of NS values over the G threads of a row at once: the whole CTA (BLK;
// red: NS x 32 floats, free again after the CTA's next barrier but one), or an
// aligned group of G lanes.
template <bool BLK, int NS>
__device__ __forceinline__ void row_sums(float (&x)[NS], int G, float (*red)[32]) {
  if constexpr (!BLK) {
    for (int o = G >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < NS; k++) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
  } else {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int k = 0; k < NS; k++) x[k] = warp_sum(x[k]);
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < NS; k++) red[k][warp] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NS; k++) x[k] = warp_sum(lane < nw ? red[k][lane] : 0.f);
  }
}

// The input vectors of a persistent CTA's rows, NT tensors, NR rows at a time,
// NCH vectors a row and thread: one group ahead in the thread's own slots of
// shared memory.
template <typename T, int NT, int NR, int NCH>
struct Ahead {
  static constexpr int SLOTS = NT * NR * NCH;  // 16-byte slots per thread of a group; two groups
  uint4* base;
  __device__ __forceinline__ uint4* slot(int g, int t, int k, int i) const {
    return base + (((g & 1) * SLOTS + (t * NR + k) * NCH + i) * blockDim.x) + threadIdx.x;
  }
  __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
  // all but the newest group are here
  __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group 1;\n" ::: "memory"); }
};

// KEEP: w and b in registers and NR rows at a time (eight columns a thread);
// else (sixteen columns) neither.
template <typename T, int NCH, bool BLK, bool KEEP, int NR>
__global__ void __launch_bounds__(BLK ? 1024 : LN_NTHR, BLK ? 1 : LN_CTAS)
    ln_fwd_kernel(int64_t n, int D, int G, float eps, const T* __restrict__ x, const float* __restrict__ w,
                  const float* __restrict__ b, T* __restrict__ y, float* __restrict__ mean,
                  float* __restrict__ rstd) {
  constexpr int V = Pack<T>::V, E = NCH * V;
  __shared__ float red[4][NR][32];
  extern __shared__ __align__(16) unsigned char smem[];
  const Ahead<T, 1, NR, NCH> q = {reinterpret_cast<uint4*>(smem)};
  const int gid = BLK ? 0 : threadIdx.x / G, lane = BLK ? threadIdx.x : threadIdx.x % G, rpc = BLK ? 1 : LN_NTHR / G;
  const int64_t row0 = (int64_t)blockIdx.x * rpc + gid, step = (int64_t)gridDim.x * rpc;
  const int s = (int)((row0 % V) * (D % V) % V);
  const float inv = 1.0f / (float)D;
  const T* end = x + n * D;
  auto cols = [&](int i) { return Cols<T>((i * G + lane) * V - s, D); };
  auto fetch = [&](int g) {
#pragma unroll
    for (int k = 0; k < NR; k++) {
      const int64_t row = row0 + ((int64_t)g * NR + k) * step;
#pragma unroll
      for (int i = 0; i < NCH; i++)
        if (row < n && cols(i).any()) cols(i).copy(q.slot(g, 0, k, i), x + row * D, end);
    }
    q.commit();
  };
  if constexpr (KEEP) fetch(0);
  float wv[KEEP ? E : 1], bv[KEEP ? E : 1];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      cols(i).param(w, wv + i * V);
      cols(i).param(b, bv + i * V);
    }
  }
  int flip = 0;
  // (the trip count is the CTA's: a group past the last row takes part in the shuffles)
  for (int g = 0; row0 - gid + (int64_t)g * NR * step < n; g++) {
    const int64_t row = row0 + (int64_t)g * NR * step;
    float v[NR][E], m[NR], var[NR];
    if constexpr (KEEP) {
      fetch(g + 1);
      q.wait();
    }
#pragma unroll
    for (int k = 0; k < NR; k++) {
      m[k] = var[k] = 0.f;
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        Pack<T> p;
        p.u = make_uint4(0, 0, 0, 0);
        if (row + k * step < n && cols(i).any()) {
          if constexpr (KEEP) p.u = *q.slot(g, 0, k, i);
          else p = cols(i).load(x + (row + k * step) * D);
        }
        p.get(v[k] + i * V);
        if constexpr (KEEP) cols(i).clear(v[k] + i * V);
#pragma unroll
        for (int e = 0; e < V; e++) m[k] += v[k][i * V + e];
      }
    }
    row_sums<BLK, NR>(m, G, red[flip]);
#pragma unroll
    for (int k = 0; k < NR; k++) {
      m[k] *= inv;
#pragma unroll
      for (int i = 0; i < NCH; i++) {
#pragma unroll
        for (int e = 0; e < V; e++) v[k][i * V + e] -= m[k];
        cols(i).clear(v[k] + i * V);
#pragma unroll
        for (int e = 0; e < V; e++) var[k] += v[k][i * V + e] * v[k][i * V + e];
      }
    }
    row_sums<BLK, NR>(var, G, red[flip + 1]);
    flip ^= 2;
#pragma unroll
    for (int k = 0; k < NR; k++) {
      const int64_t rk = row + k * step;
      const float r = 1.0f / sqrtf(var[k] * inv + eps);
      if (rk >= n) continue;
      if (mean && lane == 0) {
        mean[rk] = m[k];
        rstd[rk] = r;
      }
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        if (!cols(i).any()) continue;
        float o[V], pw[V], pb[V];
        if constexpr (!KEEP) {
          cols(i).param(w, pw);
          cols(i).param(b, pb);
        }
#pragma unroll
        for (int e = 0; e < V; e++)
          o[e] = KEEP ? v[k][i * V + e] * r * wv[KEEP ? i * V + e : 0] + bv[KEEP ? i * V + e : 0]
                      : v[k][i * V + e] * r * pw[e] + pb[e];
        cols(i).store(y + rk * D, o);
      }
    }
  }
}

// KEEP: the dw / db sums and w in registers; else (sixteen columns a thread)
// the sums in shared memory, in slots of the thread's own.
template <typename T, int NCH, bool BLK, bool KEEP, int NR>
__global__ void __launch_bounds__(BLK ? 1024 : LN_NTHR, BLK ? 1 : LN_CTAS)
    ln_bwd_kernel(int64_t n, int D, int G, const T* __restrict__ x, const float* __restrict__ w,
                  const T* __restrict__ dy, const float* __restrict__ mean, const float* __restrict__ rstd,
                  T* __restrict__ dx, float* __restrict__ part) {
  constexpr int V = Pack<T>::V, E = NCH * V;
  __shared__ float red[2][2 * NR][32];
  extern __shared__ __align__(16) unsigned char smem[];
  const Ahead<T, 2, NR, NCH> q = {reinterpret_cast<uint4*>(smem)};
  float* acc = reinterpret_cast<float*>(smem);  // !KEEP: [2][E][blockDim.x]; !BLK, at the end: [256 / G][D]
  pdl_release();
  const int gid = BLK ? 0 : threadIdx.x / G, lane = BLK ? threadIdx.x : threadIdx.x % G;
  const int rpc = BLK ? 1 : LN_NTHR / G;
  const int64_t row0 = (int64_t)blockIdx.x * rpc + gid, step = (int64_t)gridDim.x * rpc;
  const int s = (int)((row0 % V) * (D % V) % V);
  const float inv = 1.0f / (float)D;
  const T *xend = x + n * D, *dend = dy + n * D;
  auto cols = [&](int i) { return Cols<T>((i * G + lane) * V - s, D); };
  auto fetch = [&](int g) {
#pragma unroll
    for (int k = 0; k < NR; k++) {
      const int64_t row = row0 + ((int64_t)g * NR + k) * step;
#pragma unroll
      for (int i = 0; i < NCH; i++)
        if (row < n && cols(i).any()) {
          cols(i).copy(q.slot(g, 0, k, i), x + row * D, xend);
          cols(i).copy(q.slot(g, 1, k, i), dy + row * D, dend);
        }
    }
    q.commit();
  };
  float aw[KEEP ? E : 1], ab[KEEP ? E : 1], wv[KEEP ? E : 1];
  if constexpr (KEEP) {
    fetch(0);
#pragma unroll
    for (int i = 0; i < NCH; i++) cols(i).param(w, wv + i * V);
#pragma unroll
    for (int e = 0; e < E; e++) aw[e] = ab[e] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 2 * E; e++) acc[e * blockDim.x + threadIdx.x] = 0.f;
  }
  int flip = 0;
  for (int g = 0; row0 - gid + (int64_t)g * NR * step < n; g++) {
    const int64_t row = row0 + (int64_t)g * NR * step;
    float xh[NR][E], dd[NR][E], m[2 * NR], r[NR];
    if constexpr (KEEP) fetch(g + 1);
#pragma unroll
    for (int k = 0; k < NR; k++) {
      const int64_t rk = row + k * step;
      m[k] = rk < n ? __ldg(mean + rk) : 0.f;
      r[k] = rk < n ? __ldg(rstd + rk) : 0.f;
    }
    if constexpr (KEEP) q.wait();
#pragma unroll
    for (int k = 0; k < NR; k++) {
      const int64_t rk = row + k * step;
      const float mu = m[k];
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        Pack<T> px, pd;
        px.u = pd.u = make_uint4(0, 0, 0, 0);
        if (rk < n && cols(i).any()) {
          if constexpr (KEEP) {
            px.u = *q.slot(g, 0, k, i);
            pd.u = *q.slot(g, 1, k, i);
          } else {
            px = cols(i).load(x + rk * D);
            pd = cols(i).load(dy + rk * D);
          }
        }
        px.get(xh[k] + i * V);
        pd.get(dd[k] + i * V);
        if constexpr (KEEP) {  // (a missing column then has dy = 0, and h finite: nothing enters a sum)
          cols(i).clear(xh[k] + i * V);
          cols(i).clear(dd[k] + i * V);
        }
        float wl[V];
        if constexpr (!KEEP) cols(i).param(w, wl);
#pragma unroll
        for (int e = 0; e < V; e++) {
          const int j = i * V + e;
          const float h = (xh[k][j] - mu) * r[k], d = dd[k][j];
          xh[k][j] = h;
          if constexpr (KEEP) {
            aw[j] += d * h;
            ab[j] += d;
            dd[k][j] = d * wv[j];
          } else {
            acc[j * blockDim.x + threadIdx.x] += d * h;
            acc[(E + j) * blockDim.x + threadIdx.x] += d;
            dd[k][j] = d * wl[e];
          }
          s1 += dd[k][j];
          s2 += dd[k][j] * h;
        }
      }
      m[k] = s1;
      m[NR + k] = s2;
    }
    row_sums<BLK, 2 * NR>(m, G, red[flip]);
    flip ^= 1;
#pragma unroll
    for (int k = 0; k < NR; k++) {
      const int64_t rk = row + k * step;
      if (rk >= n) continue;
      const float m1 = m[k] * inv, m2 = m[NR + k] * inv;
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        if (!cols(i).any()) continue;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = r[k] * (dd[k][i * V + e] - m1 - xh[k][i * V + e] * m2);
        cols(i).store(dx + rk * D, o);
      }
    }
  }
  if constexpr (KEEP && !BLK) {
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();  // the slots are free: acc takes their place
  }
  float* pw = part + (int64_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int k = 0; k < 2; k++) {  // dw, then db
#pragma unroll
    for (int i = 0; i < NCH; i++)
#pragma unroll
      for (int e = 0; e < V; e++) {
        const int j = i * V + e, c = cols(i).c + e;
        if (!cols(i).in(e)) continue;
        if constexpr (!KEEP) pw[(int64_t)k * D + c] = acc[(k * E + j) * blockDim.x + threadIdx.x];
        else if constexpr (BLK) pw[(int64_t)k * D + c] = k ? ab[j] : aw[j];
        else acc[gid * D + c] = k ? ab[j] : aw[j];
      }
    if constexpr (!BLK) {  // the CTA's row groups in order
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += LN_NTHR) {
        float t = 0.f;
        for (int o = 0; o < LN_NTHR / G; o++) t += acc[o * D + c];
        pw[(int64_t)k * D + c] = t;
      }
      __syncthreads();
    }
  }
}

// Rows wider than LN_REG_D: a CTA per row, the row read once per pass (its
// later passes hit L2), the backward's column sums in its partial row.
__device__ __forceinline__ float one_sum(float x, float (*red)[32]) {
  float v[1] = {x};
  row_sums<true>(v, 0, red);
  return v[0];
}

template <typename T>
__global__ void __launch_bounds__(1024) ln_fwd_wide_kernel(int64_t n, int D, float eps, const T* __restrict__ x,
                                                           const float* __restrict__ w, const float* __restrict__ b,
                                                           T* __restrict__ y, float* __restrict__ mean,
                                                           float* __restrict__ rstd) {
  __shared__ float red[2][1][32];
  const float inv = 1.0f / (float)D;
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const T* xr = x + row * D;
    float s = 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) s += ldf(xr + c);
    const float mu = one_sum(s, red[0]) * inv;
    float q = 0.f;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      const float d = ldf(xr + c) - mu;
      q += d * d;
    }
    const float r = 1.0f / sqrtf(one_sum(q, red[1]) * inv + eps);
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
  __shared__ float red[2][1][32];
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
    const float m1 = one_sum(s1, red[0]) * inv, m2 = one_sum(s2, red[1]) * inv;
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

// How a row is laid over threads: G threads of `per` values each, blk: a CTA a row.
struct LnShape {
  int G, per;
  bool blk;
};
LnShape ln_shape(int D, int dtype) {
  const int V = dtype == KDA_BF16 ? 8 : 4, span = D % V ? D + V - 1 : D;  // with the offset of a row's start
  LnShape s = {1, LN_PER, false};
  while (s.G < 32 && s.G * s.per < span) s.G *= 2;
  if (s.G * s.per < span) {
    s.blk = true;
    if (D > LN_WIDE) s.per = 2 * LN_PER;
    s.G = ((span + s.per - 1) / s.per + 31) / 32 * 32;
  }
  return s;
}

// Persistent CTAs: no more than the rows need or than the SMs hold at once (a
// thread of the one-row CTAs has 64 registers), in a number that makes the row
// step a multiple of a vector's values.
int ln_blocks(int64_t n, int D, int dtype) {
  if (D > LN_REG_D) return (int)(n < LN_SMS ? n : LN_SMS);
  const LnShape s = ln_shape(D, dtype);
  const int rpc = s.blk ? 1 : LN_NTHR / s.G, per = s.blk ? 1024 / s.G : LN_CTAS;
  const int64_t need = (n + rpc - 1) / rpc;
  const int64_t most = (int64_t)LN_SMS * per;  // a multiple of 8
  return (int)(need < most ? (need + 7) / 8 * 8 : most);
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

// Launches K with smem dynamic bytes, its limit raised where they pass 48 KB.
template <typename... KA, typename... A>
cudaError_t ln_run(void (*k)(KA...), int nblk, int thr, size_t smem, cudaStream_t st, A... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  k<<<nblk, thr, smem, st>>>(args...);
  return cudaGetLastError();
}

template <typename T>
cudaError_t ln_fwd_launch(const LnShape& s, const LnArgs& a, int nblk) {
  constexpr int NCH = LN_PER * (int)sizeof(T) / 16, NR = 2;
  auto run = [&](auto* kernel, int thr, size_t slots) {
    return ln_run(kernel, nblk, thr, slots * 32 * thr, a.st, a.n, a.D, s.G, a.eps, (const T*)a.x, a.w, a.b, (T*)a.y,
                  a.mean, a.rstd);
  };
  if (!s.blk) return run(ln_fwd_kernel<T, NCH, false, true, NR>, LN_NTHR, NR * NCH);
  if (s.per == LN_PER) return run(ln_fwd_kernel<T, NCH, true, true, NR>, s.G, NR * NCH);
  return run(ln_fwd_kernel<T, 2 * NCH, true, false, 1>, s.G, 0);
}

template <typename T>
cudaError_t ln_bwd_launch(const LnShape& s, const LnArgs& a, int nblk) {
  // (two fp32 rows at a time would take 256 KB of slots)
  constexpr int NCH = LN_PER * (int)sizeof(T) / 16, NR = sizeof(T) == 4 ? 1 : 2;
  auto run = [&](auto* kernel, int thr, size_t smem) {
    return ln_run(kernel, nblk, thr, smem, a.st, a.n, a.D, s.G, (const T*)a.x, a.w, (const T*)a.dy,
                  (const float*)a.mean, (const float*)a.rstd, (T*)a.dx, a.part);
  };
  const size_t slots = 2 * NR * NCH * 32;  // bytes a thread
  if (!s.blk) {  // at most 256 x 8 floats at the end
    const size_t acc = (size_t)(LN_NTHR / s.G) * a.D * sizeof(float);
    return run(ln_bwd_kernel<T, NCH, false, true, NR>, LN_NTHR, acc > slots * LN_NTHR ? acc : slots * LN_NTHR);
  }
  if (s.per == LN_PER) return run(ln_bwd_kernel<T, NCH, true, true, NR>, s.G, slots * s.G);
  return run(ln_bwd_kernel<T, 2 * NCH, true, false, 1>, s.G, 4 * LN_PER * (size_t)s.G * sizeof(float));
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
  return (size_t)ln_blocks(n_rows, D, dtype) * 2 * (size_t)D * sizeof(float);
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
  const int nblk = ln_blocks(n_rows, D, dtype);
  LnArgs a = {};
  a.n = n_rows; a.D = D; a.eps = eps > 0.f ? eps : 1e-6f;
  a.x = x; a.w = w; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd; a.st = st;
  typedef __nv_bfloat16 B;
  cudaError_t e;
  prof_begin(K_LN_FWD, st);
  if (D > LN_REG_D) {
    if (dtype == KDA_BF16)
      ln_fwd_wide_kernel<B><<<nblk, 1024, 0, st>>>(n_rows, D, a.eps, (const B*)x, w, bias, (B*)y, mean, rstd);
    else
      ln_fwd_wide_kernel<float><<<nblk, 1024, 0, st>>>(n_rows, D, a.eps, (const float*)x, w, bias, (float*)y, mean,
                                                       rstd);
    e = cudaGetLastError();
  } else {
    e = dtype == KDA_BF16 ? ln_fwd_launch<B>(s, a, nblk) : ln_fwd_launch<float>(s, a, nblk);
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
  const int nblk = ln_blocks(n_rows, D, dtype);
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
  } else {
    e = dtype == KDA_BF16 ? ln_bwd_launch<B>(s, a, nblk) : ln_bwd_launch<float>(s, a, nblk);
  }
  prof_end(K_LN_BWD, st);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  prof_begin(K_LN_RED, st);
  e = launch_pdl(ln_reduce_kernel, dim3((unsigned)((2 * (int64_t)D + 31) / 32)), dim3(1024), 0, st,
                 (const float*)a.part, nblk, D, dw, dbias);
  prof_end(K_LN_RED, st);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
