// Rotary positions of queries and keys, per token, head and pair i < rot / 2:
//   (a, b) -> s (a cos w - b sin w, b cos w + a sin w),   w = position * inv_freq_i
// (the inverse turns by -w: with the same s it is the transpose, the gradient's map).
// A pair is (x_i, x_{i + rot/2}) (half) or (x_{2i}, x_{2i+1}) (interleaved); values from rot on pass.
//
// w is needed modulo a turn, and far positions leave fp32 no fraction: inv_freq / 2 pi
// becomes a 64-bit fraction of a turn once per thread, position times it wraps modulo
// 2^64 by itself, and the upper 32 bits are the angle to 2^-32 of a turn at any int32
// position (what the conversion leaves is 2^-53 of the total turns).  A CTA forms
// its tokens' cosines and sines once, in shared memory, and turns all heads' vectors with
// them: one pass, 16-byte accesses, bound by HBM.
#include "kda_internal.cuh"
#include "../../include/kda.h"

namespace kda {
namespace {

using bf16 = __nv_bfloat16;
constexpr int RT = 256;

struct RotP {
  int64_t n_tok, T;
  int Hq, Hkv, D, rot, interleaved, inverse, n_docs, per;  // per: tokens a CTA
  float scale;
  const float* freq;
  const int32_t *pos, *cu;
};

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  float v[N];
  __device__ __forceinline__ void ld(const T* p);
  __device__ __forceinline__ void st(T* p) const;
};
template <>
__device__ __forceinline__ void Vec<float>::ld(const float* p) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
template <>
__device__ __forceinline__ void Vec<float>::st(float* p) const {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void Vec<bf16>::ld(const bf16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const float2 f = __bfloat1622float2(h[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void Vec<bf16>::st(bf16* p) const {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int e = 0; e < 4; e++) h[e] = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
  *reinterpret_cast<uint4*>(p) = u;
}

__device__ __forceinline__ int64_t position_of(const RotP& P, int64_t tok) {
  if (P.pos) return P.pos[tok];
  if (!P.cu) return tok % P.T;
  int lo = 0, hi = P.n_docs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.cu[mid] <= tok) lo = mid;
    else hi = mid - 1;
  }
  return tok - P.cu[lo];
}

// Whether this CTA sees offsets that are no documents of the tokens: the first looks at both ends, and 256 offsets at a time
// are shared out, so that wrong ones show in some tokens at least and most CTAs have none to look at.  (All CTAs with the ends
// to look at: 16384 tokens of 8 and 8 heads of 64 17.7 -> 18.8 us.)
__device__ __forceinline__ bool bad_offsets(const RotP& P) {
  int bad = blockIdx.x == 0 && (P.cu[0] != 0 || P.cu[P.n_docs] != P.n_tok);
  for (int64_t i = (int64_t)blockIdx.x * RT + threadIdx.x; i < P.n_docs; i += (int64_t)gridDim.x * RT)
    bad |= P.cu[i + 1] < P.cu[i];
  return __syncthreads_or(bad);
}

// VEC: 16-byte vectors divide the rows and (half) the turned halves or (interleaved) the turned part.
template <typename T, bool VEC>
__global__ void __launch_bounds__(RT) rotary_kernel(RotP P, const T* q, const T* k, T* oq, T* ok) {
  extern __shared__ float2 cs[];  // [per][rot / 2]
  constexpr int N = VEC ? Vec<T>::N : 1;
  const int half = P.rot / 2, H = P.Hq + P.Hkv;
  const int64_t t0 = (int64_t)blockIdx.x * P.per;
  const int nt = (int)(P.n_tok - t0 < P.per ? P.n_tok - t0 : P.per);
  const bool bad = P.cu && (int64_t)blockIdx.x * RT < P.n_docs && bad_offsets(P);
  for (int i = threadIdx.x; i < nt * half; i += RT) {
    const int t = i / half, f = i - t * half;
    const float w = P.freq[f];
    double x = (double)w * 0.15915494309189535;  // turns a position
    x -= floor(x);
    const uint64_t turn = (uint64_t)position_of(P, t0 + t) * __double2ull_rn(x * 18446744073709551616.0);
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // in half turns: 2^-31
    if (!isfinite(w) || bad) s = c = __int_as_float(0x7fffffff);
    cs[i] = make_float2(c * P.scale, (P.inverse ? -s : s) * P.scale);
  }
  __syncthreads();
  // a head's work: its turned pairs in pieces of N (a piece of `half` has two vectors), then the vectors that pass
  const int turned = P.interleaved ? (VEC ? P.rot / N : half) : half / N;
  const int passed = (q == oq) ? 0 : (P.D - P.rot) / N;  // (both are in place, or neither)
  const int per_head = turned + passed, all = nt * H * per_head;
  for (int i = threadIdx.x; i < all; i += RT) {
    const int hv = i / per_head, u = i - hv * per_head, t = hv / H, h = hv - t * H;
    const T* x = h < P.Hq ? q + ((t0 + t) * P.Hq + h) * P.D : k + ((t0 + t) * P.Hkv + (h - P.Hq)) * P.D;
    T* y = h < P.Hq ? oq + ((t0 + t) * P.Hq + h) * P.D : ok + ((t0 + t) * P.Hkv + (h - P.Hq)) * P.D;
    const float2* w = cs + t * half;
    if (u >= turned) {
      const int at = P.rot + (u - turned) * N;
      if constexpr (VEC) *reinterpret_cast<uint4*>(y + at) = *reinterpret_cast<const uint4*>(x + at);
      else y[at] = x[at];
    } else if constexpr (VEC) {
      if (P.interleaved) {
        Vec<T> a;
        a.ld(x + u * N);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 r = w[(u * N + e) / 2];
          const float p = a.v[e], o = a.v[e + 1];
          a.v[e] = p * r.x - o * r.y;
          a.v[e + 1] = o * r.x + p * r.y;
        }
        a.st(y + u * N);
      } else {
        Vec<T> a, b;
        a.ld(x + u * N);
        b.ld(x + half + u * N);
#pragma unroll
        for (int e = 0; e < N; e++) {
          const float2 r = w[u * N + e];
          const float p = a.v[e], o = b.v[e];
          a.v[e] = p * r.x - o * r.y;
          b.v[e] = o * r.x + p * r.y;
        }
        a.st(y + u * N);
        b.st(y + half + u * N);
      }
    } else {
      const int ia = P.interleaved ? 2 * u : u, ib = P.interleaved ? 2 * u + 1 : u + half;
      const float p = ldf(x + ia), o = ldf(x + ib);
      const float2 r = w[u];
      stf(y + ia, p * r.x - o * r.y);
      stf(y + ib, o * r.x + p * r.y);
    }
  }
}

template <typename T>
cudaError_t launch(const RotP& P, const void* q, const void* k, void* oq, void* ok, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const bool vec = P.D % N == 0 && (P.interleaved ? P.rot % N == 0 : (P.rot / 2) % N == 0 && P.rot % N == 0);
  const int64_t grid = (P.n_tok + P.per - 1) / P.per;
  const size_t smem = (size_t)P.per * (P.rot / 2) * sizeof(float2);
  prof_begin(K_ROTARY, st);
  if (vec)
    rotary_kernel<T, true><<<(unsigned)grid, RT, smem, st>>>(P, (const T*)q, (const T*)k, (T*)oq, (T*)ok);
  else
    rotary_kernel<T, false><<<(unsigned)grid, RT, smem, st>>>(P, (const T*)q, (const T*)k, (T*)oq, (T*)ok);
  prof_end(K_ROTARY, st);
  return cudaGetLastError();
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" KDA_API kda_status kda_rotary(int64_t n_tok, int64_t T, int Hq, int Hkv, int D, int rot, int dtype,
                                         int interleaved, int inverse, float scale, const float* inv_freq,
                                         const int32_t* positions, const int32_t* cu_seqlens, int n_docs,
                                         const void* q, const void* k, void* q_out, void* k_out, cudaStream_t st) {
  if (n_tok <= 0 || n_tok > ((int64_t)1 << 31) - 1 || Hq <= 0 || Hkv < 0 || Hq > 4096 || Hkv > 4096)
    return KDA_ERR_INVALID_ARG;
  if (D <= 0 || D > 1024 || rot <= 0 || rot > D || rot % 2 != 0) return KDA_ERR_INVALID_ARG;
  if ((dtype != KDA_BF16 && dtype != KDA_F32) || !isfinite(scale)) return KDA_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return KDA_ERR_INVALID_ARG;
  if (!inv_freq || !q || !q_out || (Hkv > 0 && (!k || !k_out))) return KDA_ERR_INVALID_ARG;
  if (positions && cu_seqlens) return KDA_ERR_INVALID_ARG;
  if (cu_seqlens && n_docs <= 0) return KDA_ERR_INVALID_ARG;
  if (!positions && !cu_seqlens && T <= 0) return KDA_ERR_INVALID_ARG;
  if (Hkv > 0 && (q == q_out) != (k == k_out)) return KDA_ERR_INVALID_ARG;
  for (const void* x : {q, k, (const void*)q_out, (const void*)k_out})
    if ((uintptr_t)x % 16 != 0) return KDA_ERR_ALIGNMENT;
  for (const void* x : {(const void*)inv_freq, (const void*)positions, (const void*)cu_seqlens})
    if ((uintptr_t)x % 4 != 0) return KDA_ERR_ALIGNMENT;
  RotP P;
  P.n_tok = n_tok;
  P.T = T;
  P.Hq = Hq;
  P.Hkv = Hkv;
  P.D = D;
  P.rot = rot;
  P.interleaved = interleaved;
  P.inverse = inverse;
  P.n_docs = n_docs;
  P.scale = scale > 0.f ? scale : 1.f;
  P.freq = inv_freq;
  P.pos = positions;
  P.cu = cu_seqlens;
  P.per = n_tok >= 8 * SMS ? 4 : 1;
  const cudaError_t e = dtype == KDA_BF16 ? launch<bf16>(P, q, k, q_out, k_out, st)
                                          : launch<float>(P, q, k, q_out, k_out, st);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
