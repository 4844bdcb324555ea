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
// value.  Sixteen columns a thread: with eight, the shuffles of the row sums and
// the bookkeeping took the larger part of the issue slots (bf16 32768 x 2048
// forward: 68 us at 76% of them, 44 now, 68% of them; backward 68).  The next
// rows are under way to the thread's own slots of shared memory (cp.async, no
// barrier) while a row is summed.  The backward's per-CTA partials are added in
// a fixed order (deterministic).
#include "kda_internal.cuh"
#include "../../include/kda.h"

namespace kda {
namespace {

constexpr int LN_NTHR = 256;     // threads per CTA where a row takes at most a warp
constexpr int LN_CTHR = 512;     // most threads of a one-row CTA (128 registers each)
constexpr int LN_PER = 16;       // values of a row per thread, twice that in rows that LN_CTHR threads do not hold
constexpr int LN_SMS = 152;      // the grids: what the SMs hold at once
constexpr int LN_FWD_THR = 512, LN_BWD_THR = 512;  // resident threads per SM (their registers)
// A forward's CTAs of 257 to LN_PAIR threads leave an SM of LN_FWD_THR half empty: in bf16 two of them there, at
// 102 registers a thread (128 MB: 5003 columns 84 us with one, 68 with two, 5120 columns 59 and 49).  fp32 has
// twice the bytes under way and gains nothing (5003 columns 65 and 69).
constexpr int LN_PAIR = 320;
constexpr int LN_MAX_D = 1 << 24;
constexpr size_t LN_SMEM = 225 * 1024;  // dynamic shared memory of a CTA at most

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
// [0, D) exist.  EDGE: rows may share vectors with their neighbours (else a
// vector is a row's or nobody's).
template <typename T, bool EDGE>
struct Cols {
  static constexpr int V = Pack<T>::V;
  int c, D;
  __device__ __forceinline__ bool full() const { return EDGE ? c >= 0 && c + V <= D : c < D; }
  __device__ __forceinline__ bool any() const { return EDGE ? c < D && c + V > 0 : c < D; }
  __device__ __forceinline__ bool in(int e) const { return EDGE ? (unsigned)(c + e) < (unsigned)D : c < D; }
  // The whole aligned vector to shared memory, its neighbours' columns included, but nothing at or
  // past `end` (the tensor's).
  __device__ __forceinline__ void copy(uint4* slot, const T* row, const T* end) const {
    int bytes = 16;
    if constexpr (EDGE) {
      const int64_t left = (const char*)end - (const char*)(row + c);
      if (left < 16) bytes = (int)left;
    }
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"((uint32_t)__cvta_generic_to_shared(slot)),
                 "l"(row + c), "r"(bytes)
                 : "memory");
  }
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
    } else if (EDGE) {
#pragma unroll
      for (int e = 0; e < V; e++)
        if (in(e)) stf(row + c + e, v[e]);
    }
  }
  __device__ __forceinline__ void param(const float* w, float* v) const {
    if (!EDGE && w && full()) {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(w + c + e));
        v[e] = f.x; v[e + 1] = f.y; v[e + 2] = f.z; v[e + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; e++) v[e] = w && in(e) ? __ldg(w + c + e) : 0.f;
    }
  }
};

// Sums of NS values over the G threads of a row at once: the whole CTA (BLK; up
// to 16 warps; red: NS x 32 floats, free again after the CTA's next barrier but
// one), or an aligned group of G lanes.
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
    for (int k = 0; k < NS; k++) {
      x[k] = (lane & 15) < nw ? red[k][lane & 15] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
    }
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
  // all but the newest N groups are here
  template <int N>
  __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }
};

// KEEP: w and b in registers and the next rows under way; else (32 columns a
// thread) w and b in the thread's own words of shared memory, and the next row
// under way from when this one is in registers (bf16, 128 MB: 8200 columns
// 124 us with w, b and the rows read as they were needed, 79 so; 10001 columns
// 257 and 81).
template <typename T, bool BLK, bool EDGE, bool KEEP, int NR, bool PAIR = false>
__global__ void __launch_bounds__(BLK ? (PAIR ? LN_PAIR : LN_CTHR) : LN_NTHR,
                                  BLK ? (PAIR ? 2 : 1) : LN_FWD_THR / LN_NTHR)
    ln_fwd_kernel(int64_t n, int D, int G, float eps, const T* __restrict__ x, const float* __restrict__ w,
                  const float* __restrict__ b, T* __restrict__ y, float* __restrict__ mean,
                  float* __restrict__ rstd) {
  constexpr int V = Pack<T>::V, E = KEEP ? LN_PER : 2 * LN_PER, NCH = E / V;
  __shared__ float red[4][NR][32];
  extern __shared__ __align__(16) unsigned char smem[];
  const Ahead<T, 1, NR, NCH> q = {reinterpret_cast<uint4*>(smem)};
  const int gid = BLK ? 0 : threadIdx.x / G, lane = BLK ? threadIdx.x : threadIdx.x % G, rpc = BLK ? 1 : LN_NTHR / G;
  const int64_t row0 = (int64_t)blockIdx.x * rpc + gid, step = (int64_t)gridDim.x * rpc, stepD = step * D;
  const int s = EDGE ? (int)((row0 % V) * (D % V) % V) : 0;
  const float inv = 1.0f / (float)D;
  const T* end = x + n * D;
  auto cols = [&](int i) { return Cols<T, EDGE>{(i * G + lane) * V - s, D}; };
  auto fetch = [&](int g, int64_t row, const T* p) {
#pragma unroll
    for (int k = 0; k < NR; k++) {
      if (row + k * step < n) {
#pragma unroll
        for (int i = 0; i < NCH; i++)
          if (cols(i).any()) cols(i).copy(q.slot(g, 0, k, i), p + k * stepD, end);
      }
    }
    q.commit();
  };
  const T* px = x + row0 * D;
  T* py = y + row0 * D;
  float wv[KEEP ? E : V], bv[KEEP ? E : V];
  // !KEEP: word e of vector i of w, E * blockDim.x further on of b
  float* own = reinterpret_cast<float*>(smem) + (KEEP ? 0 : NCH * 4 * blockDim.x) + threadIdx.x;
  fetch(0, row0, px);
#pragma unroll
  for (int i = 0; i < NCH; i++) {
    const int at = KEEP ? i * V : 0;
    cols(i).param(w, wv + at);
    cols(i).param(b, bv + at);
    if constexpr (!KEEP) {
#pragma unroll
      for (int e = 0; e < V; e++) {
        own[(i * V + e) * blockDim.x] = wv[e];
        own[(E + i * V + e) * blockDim.x] = bv[e];
      }
    }
  }
  int flip = 0;
  // (the trip count is the CTA's: a group past the last row takes part in the shuffles)
  int64_t row = row0;
  for (int g = 0; row - gid < n; g++) {
    float v[NR][E], m[NR], var[NR];
    px += NR * stepD;
    if constexpr (KEEP) {
      fetch(g + 1, row + NR * step, px);
      q.template wait<1>();
    } else {
      q.template wait<0>();
    }
#pragma unroll
    for (int k = 0; k < NR; k++) {
      m[k] = var[k] = 0.f;
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        Pack<T> p;
        p.u = make_uint4(0, 0, 0, 0);
        // (a row past the last: whatever the slot held, not stored)
        if (cols(i).any()) p.u = *q.slot(KEEP ? g : 0, 0, k, i);
        p.get(v[k] + i * V);
        if constexpr (EDGE) cols(i).clear(v[k] + i * V);
#pragma unroll
        for (int e = 0; e < V; e++) m[k] += v[k][i * V + e];
      }
    }
    row_sums<BLK, NR>(m, G, red[flip]);
    if constexpr (!KEEP) fetch(0, row + NR * step, px);
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
      const float r = 1.0f / sqrtf(var[k] * inv + eps);
      if (row + k * step >= n) continue;
      if (mean && lane == 0) {
        mean[row + k * step] = m[k];
        rstd[row + k * step] = r;
      }
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        if (!cols(i).any()) continue;
        const int at = KEEP ? i * V : 0;
        if constexpr (!KEEP) {
#pragma unroll
          for (int e = 0; e < V; e++) {
            wv[e] = own[(i * V + e) * blockDim.x];
            bv[e] = own[(E + i * V + e) * blockDim.x];
          }
        }
        float o[V];
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = v[k][i * V + e] * r * wv[at + e] + bv[at + e];
        cols(i).store(py + k * stepD, o);
      }
    }
    row += NR * step;
    py += NR * stepD;
  }
}

// KEEP as in the forward; without it the dw / db sums are in shared memory, in
// words of the thread's own and, where shared memory has room, the next row under
// way as in the forward (MORE >= 1) and w too (MORE = 2) (bf16, 128 MB: 8200
// columns 242 us without, 166 with; 10001 columns 269 and 213).
template <typename T, bool BLK, bool EDGE, bool KEEP, int MORE>
__global__ void __launch_bounds__(BLK ? LN_CTHR : LN_NTHR, BLK ? 1 : LN_BWD_THR / LN_NTHR)
    ln_bwd_kernel(int64_t n, int D, int G, const T* __restrict__ x, const float* __restrict__ w,
                  const T* __restrict__ dy, const float* __restrict__ mean, const float* __restrict__ rstd,
                  T* __restrict__ dx, float* __restrict__ part) {
  constexpr int V = Pack<T>::V, E = KEEP ? LN_PER : 2 * LN_PER, NCH = E / V;
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) unsigned char smem[];
  float* acc = reinterpret_cast<float*>(smem);  // !KEEP: [2][E][blockDim.x]; !BLK, at the end: [256 / G][D]
  const Ahead<T, 2, 1, NCH> q = {reinterpret_cast<uint4*>(acc + (KEEP ? 0 : 2 * E * blockDim.x))};
  float* own = reinterpret_cast<float*>(q.base + 2 * NCH * blockDim.x) + threadIdx.x;  // MORE = 2: w
  pdl_release();
  const int gid = BLK ? 0 : threadIdx.x / G, lane = BLK ? threadIdx.x : threadIdx.x % G;
  const int rpc = BLK ? 1 : LN_NTHR / G;
  const int64_t row0 = (int64_t)blockIdx.x * rpc + gid, step = (int64_t)gridDim.x * rpc, stepD = step * D;
  int s = EDGE ? (int)((row0 % V) * (D % V) % V) : 0;
  const float inv = 1.0f / (float)D;
  const T *xend = x + n * D, *dend = dy + n * D;
  auto cols = [&](int i) { return Cols<T, EDGE>{(i * G + lane) * V - s, D}; };
  float nmu = 0.f, nr = 0.f;
  auto fetch = [&](int g, int64_t row, int64_t at) {
    if (row < n) {
      nmu = __ldg(mean + row);
      nr = __ldg(rstd + row);
#pragma unroll
      for (int i = 0; i < NCH; i++)
        if (cols(i).any()) {
          cols(i).copy(q.slot(g, 0, 0, i), x + at, xend);
          cols(i).copy(q.slot(g, 1, 0, i), dy + at, dend);
        }
    }
    q.commit();
  };
  int64_t at = row0 * D, row = row0;
  float aw[KEEP ? E : 1], ab[KEEP ? E : 1], wv[KEEP ? E : V];
  if constexpr (MORE > 0) fetch(0, row, at);
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NCH; i++) cols(i).param(w, wv + i * V);
#pragma unroll
    for (int e = 0; e < E; e++) aw[e] = ab[e] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 2 * E; e++) acc[e * blockDim.x + threadIdx.x] = 0.f;
    if constexpr (MORE == 2) {
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        cols(i).param(w, wv);
#pragma unroll
        for (int e = 0; e < V; e++) own[(i * V + e) * blockDim.x] = wv[e];
      }
    }
  }
  int flip = 0;
  for (int g = 0; row - gid < n; g++) {
    const bool ok = row < n;
    if (MORE == 0 && ok) {
      nmu = mean[row];
      nr = rstd[row];
    }
    // (a row's columns are found anew: kept over the rows, as the compiler would, they spill)
    if constexpr (EDGE && !KEEP) asm volatile("" : "+r"(s));
    const float mu = nmu, r = nr;
    if constexpr (KEEP) {
      fetch(g + 1, row + step, at + stepD);
      q.template wait<1>();
    } else {
      q.template wait<0>();
    }
    float xh[E], dd[E], m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NCH; i++) {
      Pack<T> px, pd;
      px.u = pd.u = make_uint4(0, 0, 0, 0);
      if (ok && cols(i).any()) {
        if constexpr (MORE > 0) {
          px.u = *q.slot(KEEP ? g : 0, 0, 0, i);
          pd.u = *q.slot(KEEP ? g : 0, 1, 0, i);
        } else {
          px = cols(i).load(x + at);
          pd = cols(i).load(dy + at);
        }
      }
      px.get(xh + i * V);
      pd.get(dd + i * V);
      if constexpr (!KEEP) {
        if constexpr (MORE == 2) {
#pragma unroll
          for (int e = 0; e < V; e++) wv[e] = own[(i * V + e) * blockDim.x];
        } else {
          cols(i).param(w, wv);
        }
      }
      if constexpr (EDGE) {
        cols(i).clear(xh + i * V);
        cols(i).clear(dd + i * V);
      }
#pragma unroll
      for (int e = 0; e < V; e++) {  // (a missing column or row has dy = 0, and h finite: nothing enters a sum)
        const int j = i * V + e;
        const float h = (xh[j] - mu) * r, d = dd[j];
        xh[j] = h;
        if constexpr (KEEP) {
          aw[j] += d * h;
          ab[j] += d;
        } else {
          acc[j * blockDim.x + threadIdx.x] += d * h;
          acc[(E + j) * blockDim.x + threadIdx.x] += d;
        }
        dd[j] = d * wv[KEEP ? j : e];
        m[0] += dd[j];
        m[1] += dd[j] * h;
      }
      if constexpr (!KEEP) asm volatile("" ::: "memory");  // (the next vector's loads not before: registers)
    }
    row_sums<BLK, 2>(m, G, red[flip]);
    flip ^= 1;
    if constexpr (!KEEP && MORE > 0) fetch(0, row + step, at + stepD);
    if (ok) {
      m[0] *= inv;
      m[1] *= inv;
#pragma unroll
      for (int i = 0; i < NCH; i++) {
        if (!cols(i).any()) continue;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; e++) o[e] = r * (dd[i * V + e] - m[0] - xh[i * V + e] * m[1]);
        cols(i).store(dx + at, o);
      }
    }
    row += step;
    at += stepD;
  }
  float* pw = part + (int64_t)blockIdx.x * 2 * D;
  if constexpr (!BLK) {  // acc takes the slots' place
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();
  }
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

// Rows wider than 32 columns for each of LN_CTHR threads: a CTA per row, the row read once per pass (its
// later passes hit L2), the backward's column sums in its partial row.  A thread's sums, of up to 2^15 values
// here, are compensated (Kahan 1965; 128 MB of bf16, 16386 columns: forward 538 us, 521 without, backward 856 and
// 852).  Bound by the latency of single values: 0.5 TB/s in bf16, 0.8 in fp32.
struct LongSum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float y = x - c, t = s + y;
    c = (t - s) - y;
    s = t;
  }
};

template <typename T>
__global__ void __launch_bounds__(LN_CTHR) ln_fwd_wide_kernel(int64_t n, int D, float eps, const T* __restrict__ x,
                                                           const float* __restrict__ w, const float* __restrict__ b,
                                                           T* __restrict__ y, float* __restrict__ mean,
                                                           float* __restrict__ rstd) {
  __shared__ float red[2][2][32];
  const float inv = 1.0f / (float)D;
  for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
    const T* xr = x + row * D;
    LongSum s;
    for (int c = threadIdx.x; c < D; c += blockDim.x) s.add(ldf(xr + c));
    float m[1] = {s.s};
    row_sums<true>(m, 0, red[0]);
    float mu = m[0] * inv;
    // the centred values' own mean is what rounding left in mu: against a spread near sqrt(eps) it would show
    LongSum q, t;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      const float d = ldf(xr + c) - mu;
      q.add(d * d);
      t.add(d);
    }
    float v[2] = {q.s, t.s};
    row_sums<true>(v, 0, red[1]);
    const float off = v[1] * inv, var = v[0] * inv - off * off;
    mu += off;
    const float r = 1.0f / sqrtf((var < 0.f ? 0.f : var) + eps);
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
__global__ void __launch_bounds__(LN_CTHR) ln_bwd_wide_kernel(int64_t n, int D, const T* __restrict__ x,
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
    LongSum s1, s2;
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      const float h = (ldf(x + row * D + c) - mu) * r, d = ldf(dy + row * D + c), g = d * w[c];
      pw[c] = (first ? 0.f : pw[c]) + d * h;
      pw[D + c] = (first ? 0.f : pw[D + c]) + d;
      s1.add(g);
      s2.add(g * h);
    }
    float m[2] = {s1.s, s2.s};
    row_sums<true>(m, 0, red);
    const float m1 = m[0] * inv, m2 = m[1] * inv;
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

// How a row is laid over threads: G threads of LN_PER values each (twice that
// without keep), blk: a CTA a row.  wide: not held in registers.
struct LnShape {
  int G;
  bool blk, edge, keep, wide;
};
LnShape ln_shape(int D, int dtype) {
  const int V = dtype == KDA_BF16 ? 8 : 4, span = D % V ? D + V - 1 : D;  // with the offset of a row's start
  LnShape s = {1, false, D % V != 0, span <= LN_CTHR * LN_PER, span > 2 * LN_CTHR * LN_PER};
  while (s.G < 32 && s.G * LN_PER < span) s.G *= 2;
  if (s.G * LN_PER < span) {
    const int per = s.keep ? LN_PER : 2 * LN_PER;
    s.blk = true;
    s.G = ((span + per - 1) / per + 31) / 32 * 32;
  }
  return s;
}

bool ln_pair(const LnShape& s, int dtype) {
  return dtype == KDA_BF16 && s.blk && s.keep && s.G > LN_FWD_THR / 2 && s.G <= LN_PAIR;
}

// Persistent CTAs: no more than the rows need or than the SMs hold at once, in
// a number that makes the row step a multiple of a vector's values.
int ln_blocks(int64_t n, int D, int dtype, bool bwd) {
  const LnShape s = ln_shape(D, dtype);
  if (s.wide) return (int)(n < LN_SMS ? n : LN_SMS);
  const int rpc = s.blk ? 1 : LN_NTHR / s.G;
  const int per = !bwd && ln_pair(s, dtype) ? 2 : (bwd ? LN_BWD_THR : LN_FWD_THR) / (s.blk ? s.G : LN_NTHR);
  const int64_t need = (n + rpc - 1) / rpc;
  const int64_t most = (int64_t)LN_SMS * (per < 1 ? 1 : per);  // a multiple of 8
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

// Launches K with smem dynamic bytes, its limit raised where they and the static kilobyte pass 48 KB.
template <typename... KA, typename... A>
cudaError_t ln_run(void (*k)(KA...), int nblk, int thr, size_t smem, cudaStream_t st, A... args) {
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  k<<<nblk, thr, smem, st>>>(args...);
  return cudaGetLastError();
}

template <typename T>
cudaError_t ln_fwd_launch(const LnShape& s, const LnArgs& a, int nblk) {
  constexpr int NR = 2;
  const int thr = s.blk ? s.G : LN_NTHR;
  auto run = [&](auto* kernel) {
    return ln_run(kernel, nblk, thr, (s.keep ? 2 * NR * LN_PER * sizeof(T) : 2 * LN_PER * (sizeof(T) + 8)) * thr, a.st,
                  a.n, a.D, s.G, a.eps, (const T*)a.x, a.w, a.b, (T*)a.y, a.mean, a.rstd);
  };
  if (!s.keep)
    return s.edge ? run(ln_fwd_kernel<T, true, true, false, 1>) : run(ln_fwd_kernel<T, true, false, false, 1>);
  if constexpr (sizeof(T) == 2) {
    if (ln_pair(s, KDA_BF16))
      return s.edge ? run(ln_fwd_kernel<T, true, true, true, NR, true>)
                    : run(ln_fwd_kernel<T, true, false, true, NR, true>);
  }
  if (s.blk) return s.edge ? run(ln_fwd_kernel<T, true, true, true, NR>) : run(ln_fwd_kernel<T, true, false, true, NR>);
  return s.edge ? run(ln_fwd_kernel<T, false, true, true, NR>) : run(ln_fwd_kernel<T, false, false, true, NR>);
}

template <typename T>
cudaError_t ln_bwd_launch(const LnShape& s, const LnArgs& a, int nblk) {
  const int thr = s.blk ? s.G : LN_NTHR;
  const size_t slots = 2 * 2 * LN_PER * sizeof(T) * thr;
  const size_t acc = !s.keep ? 4 * LN_PER * sizeof(float) * thr : s.blk ? 0 : (size_t)(LN_NTHR / s.G) * a.D * 4;
  // (without keep: the sums, then what has room of the next row and of w)
  const size_t wb = 2 * LN_PER * 4 * thr;
  const int more = acc + slots + wb <= LN_SMEM ? 2 : acc + slots <= LN_SMEM ? 1 : 0;
  const size_t smem = s.keep ? (acc > slots ? acc : slots) : acc + (more > 0 ? slots : 0) + (more > 1 ? wb : 0);
  auto run = [&](auto* kernel) {
    return ln_run(kernel, nblk, thr, smem, a.st, a.n, a.D, s.G, (const T*)a.x, a.w,
                  (const T*)a.dy, (const float*)a.mean, (const float*)a.rstd, (T*)a.dx, a.part);
  };
  if (!s.keep && more == 2)
    return s.edge ? run(ln_bwd_kernel<T, true, true, false, 2>) : run(ln_bwd_kernel<T, true, false, false, 2>);
  if (!s.keep && (more == 1 || sizeof(T) == 2))  // (bf16 rows always fit)
    return s.edge ? run(ln_bwd_kernel<T, true, true, false, 1>) : run(ln_bwd_kernel<T, true, false, false, 1>);
  if constexpr (sizeof(T) == 4) {
    if (!s.keep)
      return s.edge ? run(ln_bwd_kernel<T, true, true, false, 0>) : run(ln_bwd_kernel<T, true, false, false, 0>);
  }
  if (s.blk)
    return s.edge ? run(ln_bwd_kernel<T, true, true, true, 1>) : run(ln_bwd_kernel<T, true, false, true, 1>);
  return s.edge ? run(ln_bwd_kernel<T, false, true, true, 1>) : run(ln_bwd_kernel<T, false, false, true, 1>);
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
  return (size_t)ln_blocks(n_rows, D, dtype, true) * 2 * (size_t)D * sizeof(float);
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
  const int nblk = ln_blocks(n_rows, D, dtype, false);
  LnArgs a = {};
  a.n = n_rows; a.D = D; a.eps = eps > 0.f ? eps : 1e-6f;
  a.x = x; a.w = w; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd; a.st = st;
  typedef __nv_bfloat16 B;
  cudaError_t e;
  prof_begin(K_LN_FWD, st);
  if (s.wide) {
    if (dtype == KDA_BF16)
      ln_fwd_wide_kernel<B><<<nblk, LN_CTHR, 0, st>>>(n_rows, D, a.eps, (const B*)x, w, bias, (B*)y, mean, rstd);
    else
      ln_fwd_wide_kernel<float><<<nblk, LN_CTHR, 0, st>>>(n_rows, D, a.eps, (const float*)x, w, bias, (float*)y, mean,
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
  const int nblk = ln_blocks(n_rows, D, dtype, true);
  LnArgs a = {};
  a.n = n_rows; a.D = D;
  a.x = x; a.w = w; a.dy = dy; a.dx = dx; a.mean = (float*)mean; a.rstd = (float*)rstd; a.part = (float*)workspace;
  a.st = st;
  typedef __nv_bfloat16 B;
  cudaError_t e;
  prof_begin(K_LN_BWD, st);
  if (s.wide) {
    if (dtype == KDA_BF16)
      ln_bwd_wide_kernel<B><<<nblk, LN_CTHR, 0, st>>>(n_rows, D, (const B*)x, w, (const B*)dy, mean, rstd, (B*)dx,
                                                      a.part);
    else
      ln_bwd_wide_kernel<float><<<nblk, LN_CTHR, 0, st>>>(n_rows, D, (const float*)x, w, (const float*)dy, mean, rstd,
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
