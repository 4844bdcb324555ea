// Softmax attention, single-token step: every sequence's new key and value are
// appended to its cache and its new query reads the cache,
//   o_h = sum_j p_j v_j,   p_j = exp(scale q_h k_j) / sum,   j = 0 .. length (the new token last).
// The cache is read once: a CTA takes all query heads of a key head (up to 16) over one
// piece of a sequence, so the bytes are the cache's and the step is bound by HBM
// bandwidth.  Where sequences and heads do not fill the GPU the length is cut into equal
// pieces, whose (maximum, sum, o) are joined by a second kernel in a fixed order.
//
// bf16: a warp takes 16 keys at a time straight from global memory into mma.sync
// fragments; which d (of a key) or which column (of a value) a lane's 16-byte load
// stands for is free as long as both operands agree, so no shared memory and no
// transposing loads are needed.  The weights enter the value product as two bf16 parts
// (off by 2^-16): the tensor pipe has room, and the output is rounded once.
#include "kda_internal.cuh"
#include "kda_mma.cuh"
#include "../../include/kda.h"

namespace kda {
namespace smx {
namespace {

using bf16 = __nv_bfloat16;
constexpr int WARPS = 4, MH = 16;  // warps a CTA; query heads a CTA

struct DecP {
  int n, cap, Hq, Hkv, G, HG, ns;  // HG: groups of MH query heads of a key head; ns: pieces of a sequence
  float scale2;
  const int32_t* len;
  int32_t* err;
  float* part;  // per (sequence, key head, head group, piece): MH maxima, MH sums, MH x D outputs
};

// The CTA's place; false for a sequence that takes no step (its outputs are zeros).
struct Place {
  int seq, hk, h0, nh, L;   // first query head and how many; the new token's index
  int lo, hi;               // keys of this piece
  size_t unit;              // (sequence, key head, head group)
};
__device__ __forceinline__ bool place_of(const DecP& P, Place& c) {
  const int piece = blockIdx.x % P.ns;
  c.unit = blockIdx.x / P.ns;
  const int hg = (int)(c.unit % P.HG);
  const size_t sh = c.unit / P.HG;
  c.hk = (int)(sh % P.Hkv);
  c.seq = (int)(sh / P.Hkv);
  c.h0 = c.hk * P.G + hg * MH;
  c.nh = min(MH, P.G - hg * MH);
  c.L = P.len[c.seq];
  c.lo = c.hi = 0;
  if (c.L < 0 || c.L >= P.cap) return false;
  const int64_t total = (int64_t)c.L + 1, step = ((total + P.ns - 1) / P.ns + 63) / 64 * 64;
  const int64_t lo = step * piece;
  c.lo = (int)(lo < total ? lo : total);
  c.hi = (int)(lo + step < total ? lo + step : total);
  return true;
}

__device__ __forceinline__ void dec_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void dec_out(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// Joins the warps' rows in shared memory (sm: m[WARPS][MH], l[WARPS][MH], o[WARPS][MH][D]) and writes the
// output, or the piece's part.
template <int D, typename T>
__device__ __forceinline__ void finish(const DecP& P, const Place& c, const float* sm, T* o) {
  const float *m = sm, *l = sm + WARPS * MH, *a = l + WARPS * MH;
  float* part = P.part + (size_t)blockIdx.x * (MH * (D + 2));
  for (int i = threadIdx.x; i < c.nh * D; i += WARPS * 32) {
    const int r = i / D, d = i % D;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; w++) mx = fmaxf(mx, m[w * MH + r]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
      const float e = ex2(m[w * MH + r] - mu);
      sum += e * l[w * MH + r];
      x += e * a[((size_t)w * MH + r) * D + d];
    }
    if (P.ns == 1) {
      dec_out(o + ((size_t)c.seq * P.Hq + c.h0 + r) * D + d, x / sum);
    } else {
      part[2 * MH + r * D + d] = x;
      if (d == 0) {
        part[r] = mx;
        part[MH + r] = sum;
      }
    }
  }
}

// Outputs of a sequence that takes no step: zeros.
template <int D, typename T>
__device__ __forceinline__ void no_step(const DecP& P, const Place& c, T* o) {
  if (P.ns == 1)
    for (int i = threadIdx.x; i < c.nh * D; i += WARPS * 32) dec_out(o + ((size_t)c.seq * P.Hq + c.h0) * D + i, 0.f);
}

// The error word: a length without room in its cache (block 0 looks at all).
__device__ __forceinline__ void check_lengths(const DecP& P) {
  if (blockIdx.x != 0) return;
  int bad = 0;
  for (int i = threadIdx.x; i < P.n; i += WARPS * 32) bad |= P.len[i] >= P.cap;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *P.err = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
}

__device__ __forceinline__ uint4 ldg16(const bf16* p, bool in) {
  return in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }
// two probabilities as a bf16 pair and what that left
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

// Lane (g, t) = (lane / 4, lane % 4).  q k: step 2 j + s of the contraction holds d = 32 j + 8 t + 4 s .. + 3 of
// lane t's 16-byte load j.  p v: column g of tile (c, e) is d = 64 c + 8 g + e, so a lane's load c of a key
// gives it one column of eight tiles, and it ends with d = 64 c + 16 t .. + 15 of rows g and g + 8.
template <int D>
__global__ void __launch_bounds__(WARPS * 32) smx_decode_kernel(DecP P, const bf16* __restrict__ q,
                                                              const bf16* __restrict__ kn,
                                                              const bf16* __restrict__ vn, bf16* kc, bf16* vc,
                                                              bf16* __restrict__ o) {
  constexpr int NJ = D / 32, NC = D / 64;
  extern __shared__ __align__(16) float sm[];
  pdl_wait();
  pdl_release();
  check_lengths(P);
  Place c;
  if (!place_of(P, c)) return no_step<D>(P, c, o);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const size_t row = (size_t)P.Hkv * D, cache = ((size_t)c.seq * P.cap * P.Hkv + c.hk) * D;
  const bf16 *kb = kc + cache, *vb = vc + cache, *k1 = kn + ((size_t)c.seq * P.Hkv + c.hk) * D,
             *v1 = vn + ((size_t)c.seq * P.Hkv + c.hk) * D;
  if (c.h0 == c.hk * P.G && blockIdx.x % P.ns == 0 && warp == 0 && lane < D / 8) {  // (no reader takes it from the cache)
    *reinterpret_cast<uint4*>(kc + cache + (size_t)c.L * row + 8 * lane) = ldg16(k1 + 8 * lane, true);
    *reinterpret_cast<uint4*>(vc + cache + (size_t)c.L * row + 8 * lane) = ldg16(v1 + 8 * lane, true);
  }
  uint4 qa[NJ], qb[NJ];
#pragma unroll
  for (int j = 0; j < NJ; j++) {
    const bf16* p = q + ((size_t)c.seq * P.Hq + c.h0) * D + 32 * j + 8 * t;
    qa[j] = ldg16(p + g * D, g < c.nh);
    qb[j] = ldg16(p + (g + 8) * D, g + 8 < c.nh);
  }
  float acc[NC * 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll 1
  for (int j0 = c.lo + 16 * warp; j0 < c.hi; j0 += 16 * WARPS) {
    uint4 kr[2][NJ], vr[4][NC];
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const int j = j0 + 8 * x + g;
      const bf16* p = (j == c.L ? k1 : kb + (size_t)j * row) + 8 * t;
#pragma unroll
      for (int y = 0; y < NJ; y++) kr[x][y] = j < c.hi ? *reinterpret_cast<const uint4*>(p + 32 * y) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int x = 0; x < 4; x++) {
      const int j = j0 + 2 * t + (x & 1) + 8 * (x >> 1);
      const bf16* p = (j == c.L ? v1 : vb + (size_t)j * row) + 8 * g;
#pragma unroll
      for (int y = 0; y < NC; y++) vr[x][y] = j < c.hi ? *reinterpret_cast<const uint4*>(p + 64 * y) : make_uint4(0, 0, 0, 0);
    }
    float s[2][4] = {};
#pragma unroll
    for (int y = 0; y < NJ; y++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const uint32_t a[4] = {word(qa[y], 2 * h), word(qb[y], 2 * h), word(qa[y], 2 * h + 1), word(qb[y], 2 * h + 1)};
#pragma unroll
        for (int x = 0; x < 2; x++) mma::mma_bf16(s[x], a, word(kr[x][y], 2 * h), word(kr[x][y], 2 * h + 1));
      }
    uint32_t ph[4], pl[4];
    bool grew = false;
    float corr[2];
#pragma unroll
    for (int r = 0; r < 2; r++) {
      float mx = m[r];
#pragma unroll
      for (int x = 0; x < 2; x++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float& z = s[x][2 * r + e];
          z = j0 + 8 * x + 2 * t + e < c.hi ? z * P.scale2 : -INFINITY;
          mx = fmaxf(mx, z);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mu = mx == -INFINITY ? 0.f : mx;
      corr[r] = ex2(m[r] - mu);
      grew |= mx != m[r];
      m[r] = mx;
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < 2; x++) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
          s[x][2 * r + e] = ex2(s[x][2 * r + e] - mu);
          sum += s[x][2 * r + e];
        }
        split2(s[x][2 * r], s[x][2 * r + 1], ph[2 * x + r], pl[2 * x + r]);
      }
      l[r] = l[r] * corr[r] + sum;
    }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int i = 0; i < NC * 8; i++) {
        acc[i][0] *= corr[0];
        acc[i][1] *= corr[0];
        acc[i][2] *= corr[1];
        acc[i][3] *= corr[1];
      }
    }
#pragma unroll
    for (int y = 0; y < NC; y++)
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
        const uint32_t b0 = __byte_perm(word(vr[0][y], e / 2), word(vr[1][y], e / 2), sel);
        const uint32_t b1 = __byte_perm(word(vr[2][y], e / 2), word(vr[3][y], e / 2), sel);
        mma::mma_bf16(acc[8 * y + e], ph, b0, b1);
        mma::mma_bf16(acc[8 * y + e], pl, b0, b1);
      }
  }
  float *sM = sm, *sL = sm + WARPS * MH, *sO = sL + WARPS * MH;
#pragma unroll
  for (int r = 0; r < 2; r++) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int i = warp * MH + g + 8 * r;
    if (t == 0) {
      sM[i] = m[r];
      sL[i] = l[r];
    }
#pragma unroll
    for (int y = 0; y < NC; y++)
#pragma unroll
      for (int e = 0; e < 2; e++)
#pragma unroll
        for (int z = 0; z < 8; z++) sO[(size_t)i * D + 64 * y + 16 * t + 8 * e + z] = acc[8 * y + z][2 * r + e];
  }
  __syncthreads();
  finish<D>(P, c, sm, o);
}

// fp32: lanes (g, t) form the pairs of key g (t a quarter of d), then every lane sums its D / 32 columns.
template <int D>
__global__ void __launch_bounds__(WARPS * 32) smx_decode_f32_kernel(DecP P, const float* __restrict__ q,
                                                                  const float* __restrict__ kn,
                                                                  const float* __restrict__ vn, float* kc, float* vc,
                                                                  float* __restrict__ o) {
  constexpr int NJ = D / 16, NV = D / 32;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm + WARPS * MH * (D + 2);
  pdl_wait();
  pdl_release();
  check_lengths(P);
  Place c;
  if (!place_of(P, c)) return no_step<D>(P, c, o);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const size_t row = (size_t)P.Hkv * D, cache = ((size_t)c.seq * P.cap * P.Hkv + c.hk) * D;
  const float *kb = kc + cache, *vb = vc + cache, *k1 = kn + ((size_t)c.seq * P.Hkv + c.hk) * D,
              *v1 = vn + ((size_t)c.seq * P.Hkv + c.hk) * D;
  if (c.h0 == c.hk * P.G && blockIdx.x % P.ns == 0 && warp == 0)
    for (int d = lane; d < D; d += 32) {
      kc[cache + (size_t)c.L * row + d] = k1[d];
      vc[cache + (size_t)c.L * row + d] = v1[d];
    }
  for (int i = threadIdx.x; i < c.nh * D; i += WARPS * 32) sq[i] = q[((size_t)c.seq * P.Hq + c.h0) * D + i];
  __syncthreads();
  float acc[MH][NV] = {}, m[MH], l[MH] = {};
#pragma unroll
  for (int h = 0; h < MH; h++) m[h] = -INFINITY;
#pragma unroll 1
  for (int j0 = c.lo + 8 * warp; j0 < c.hi; j0 += 8 * WARPS) {
    float4 kr[NJ];
    float vr[8][NV];
    const int j = j0 + g;
    const float* p = (j == c.L ? k1 : kb + (size_t)j * row) + 4 * t;
#pragma unroll
    for (int y = 0; y < NJ; y++) kr[y] = j < c.hi ? *reinterpret_cast<const float4*>(p + 16 * y) : make_float4(0, 0, 0, 0);
#pragma unroll
    for (int x = 0; x < 8; x++) {
      const float* z = (j0 + x == c.L ? v1 : vb + (size_t)(j0 + x) * row) + lane * NV;
#pragma unroll
      for (int e = 0; e < NV; e++) vr[x][e] = j0 + x < c.hi ? z[e] : 0.f;
    }
#pragma unroll
    for (int h = 0; h < MH; h++) {
      if (h >= c.nh) break;
      float s = 0.f;
#pragma unroll
      for (int y = 0; y < NJ; y++) {
        const float4 a = *reinterpret_cast<const float4*>(sq + h * D + 16 * y + 4 * t);
        s = fmaf(a.x, kr[y].x, s);
        s = fmaf(a.y, kr[y].y, s);
        s = fmaf(a.z, kr[y].z, s);
        s = fmaf(a.w, kr[y].w, s);
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      s = j < c.hi ? s * P.scale2 : -INFINITY;
      float mx = s;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      mx = fmaxf(mx, m[h]);
      const float mu = mx == -INFINITY ? 0.f : mx, corr = ex2(m[h] - mu), w = ex2(s - mu);
      m[h] = mx;
      l[h] = l[h] * corr + w;  // (this lane's key; the lanes t of a key hold the same)
#pragma unroll
      for (int e = 0; e < NV; e++) acc[h][e] *= corr;
#pragma unroll
      for (int x = 0; x < 8; x++) {
        const float wx = __shfl_sync(0xffffffffu, w, 4 * x);
#pragma unroll
        for (int e = 0; e < NV; e++) acc[h][e] = fmaf(wx, vr[x][e], acc[h][e]);
      }
    }
  }
  float *sM = sm, *sL = sm + WARPS * MH, *sO = sL + WARPS * MH;
#pragma unroll
  for (int h = 0; h < MH; h++) {
    if (h >= c.nh) break;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
    if (lane == 0) {
      sM[warp * MH + h] = m[h];
      sL[warp * MH + h] = l[h];
    }
#pragma unroll
    for (int e = 0; e < NV; e++) sO[(size_t)(warp * MH + h) * D + lane * NV + e] = acc[h][e];
  }
  __syncthreads();
  finish<D>(P, c, sm, o);
}

// Joins the pieces of one (sequence, query head): their weights first, then warp w sums pieces w, w + JW, .. whose loads
// do not wait for one another (with a running maximum along them 114 pieces took 12.7 us, so 5).
constexpr int JW = 16;
template <int D, typename T>
__global__ void __launch_bounds__(JW * 32) smx_join_kernel(DecP P, T* __restrict__ o) {
  constexpr int NV = D / 32;
  extern __shared__ float sw[];  // [ns]
  __shared__ float red[JW], so[JW][D];
  const int seq = blockIdx.x / P.Hq, h = blockIdx.x % P.Hq, hk = h / P.G, r = h % P.G;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, rr = r % MH;
  pdl_wait();
  const int L = P.len[seq];
  T* out = o + ((size_t)seq * P.Hq + h) * D;
  if (L < 0 || L >= P.cap) {
    if (threadIdx.x < D) dec_out(out + threadIdx.x, 0.f);
    return;
  }
  constexpr size_t ST = MH * (D + 2);
  const float* part = P.part + (((size_t)seq * P.Hkv + hk) * P.HG + r / MH) * P.ns * ST;
  float m = -INFINITY;
  for (int s = threadIdx.x; s < P.ns; s += JW * 32) {
    sw[s] = part[s * ST + rr];
    m = fmaxf(m, sw[s]);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  if (lane == 0) red[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < JW; w++) m = fmaxf(m, red[w]);
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int s = threadIdx.x; s < P.ns; s += JW * 32) {
    sw[s] = ex2(sw[s] - mu);
    l += sw[s] * part[s * ST + MH + rr];
  }
  l = warp_sum(l);
  __syncthreads();  // (red is read, the weights are there)
  if (lane == 0) red[warp] = l;
  float acc[NV] = {};
  const float* p = part + 2 * MH + rr * D + lane * NV;
#pragma unroll 8
  for (int s = warp; s < P.ns; s += JW) {
    const float w = sw[s];
#pragma unroll
    for (int e = 0; e < NV; e++) acc[e] = fmaf(w, p[s * ST + e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < NV; e++) so[warp][lane * NV + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < JW; w++) {
      sum += red[w];
      x += so[w][threadIdx.x];
    }
    dec_out(out + threadIdx.x, x / sum);
  }
}

// Pieces of a sequence, none of fewer than 128 keys of a full cache: for one sequence as many as the CTAs that 152
// SMs hold (three each), so that its equal pieces are one wave; several sequences differ in length, and smaller pieces
// even that out.
int pieces(int n, int64_t units, int cap) {
  const int64_t want = ((n == 1 ? 3 : 8) * 152 + units - 1) / units, most = ((int64_t)cap + 127) / 128;
  const int64_t ns = want < most ? want : most;
  return (int)(ns < 1 ? 1 : ns);
}

bool sizes_ok(int n, int cap, int Hq, int Hkv, int dtype) {
  return n > 0 && cap > 0 && Hq > 0 && Hkv > 0 && Hq <= 4096 && Hq % Hkv == 0 && (int64_t)n * Hq <= ((int64_t)1 << 28) &&
         (int64_t)n * cap <= ((int64_t)1 << 40) && (dtype == KDA_BF16 || dtype == KDA_F32);
}

template <int D>
cudaError_t launch(const DecP& P, int dtype, const void* q, const void* k, const void* v, void* kc, void* vc, void* o,
                   cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)P.n * P.Hkv * P.HG * P.ns);
  const size_t smem = WARPS * MH * (D + 2) * sizeof(float), s32 = smem + MH * D * sizeof(float);
  cudaError_t e;
  prof_begin(K_SMX_DECODE, st);
  if (dtype == KDA_BF16) {
    e = launch_pdl(smx_decode_kernel<D>, dim3(grid), dim3(WARPS * 32), smem, st, P, (const bf16*)q, (const bf16*)k,
                   (const bf16*)v, (bf16*)kc, (bf16*)vc, (bf16*)o);
  } else {
    e = launch_pdl(smx_decode_f32_kernel<D>, dim3(grid), dim3(WARPS * 32), s32, st, P, (const float*)q,
                   (const float*)k, (const float*)v, (float*)kc, (float*)vc, (float*)o);
  }
  prof_end(K_SMX_DECODE, st);
  if (e != cudaSuccess || P.ns == 1) return e;
  prof_begin(K_SMX_JOIN, st);
  if (dtype == KDA_BF16)
    e = launch_pdl(smx_join_kernel<D, bf16>, dim3(P.n * P.Hq), dim3(JW * 32), P.ns * sizeof(float), st, P, (bf16*)o);
  else
    e = launch_pdl(smx_join_kernel<D, float>, dim3(P.n * P.Hq), dim3(JW * 32), P.ns * sizeof(float), st, P, (float*)o);
  prof_end(K_SMX_JOIN, st);
  return e;
}

}  // namespace
}  // namespace smx
}  // namespace kda

using namespace kda;
using namespace kda::smx;

extern "C" KDA_API size_t kda_softmax_decode_workspace_size(int n_seq, int cap, int Hq, int Hkv, int D) {
  if (!sizes_ok(n_seq, cap, Hq, Hkv, KDA_BF16) || (D != 64 && D != 128)) return 0;
  const int64_t units = (int64_t)n_seq * Hkv * ((Hq / Hkv + MH - 1) / MH);
  const int ns = pieces(n_seq, units, cap);
  return 256 + (ns == 1 ? 0 : (size_t)units * ns * MH * (D + 2) * sizeof(float));
}

extern "C" KDA_API kda_status kda_softmax_decode(int n_seq, int cap, int Hq, int Hkv, int D, int dtype, float scale,
                                                 const void* q, const void* k, const void* v, void* k_cache,
                                                 void* v_cache, const int32_t* lengths, void* o, void* workspace,
                                                 size_t workspace_bytes, cudaStream_t st) {
  if (!sizes_ok(n_seq, cap, Hq, Hkv, dtype)) return KDA_ERR_INVALID_ARG;
  if (!q || !k || !v || !k_cache || !v_cache || !lengths || !o) return KDA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return KDA_ERR_UNSUPPORTED;
  for (const void* x : {q, k, v, (const void*)k_cache, (const void*)v_cache, (const void*)o})
    if ((uintptr_t)x % 16 != 0) return KDA_ERR_ALIGNMENT;
  if ((uintptr_t)lengths % 4 != 0) return KDA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kda_softmax_decode_workspace_size(n_seq, cap, Hq, Hkv, D)) return KDA_ERR_WORKSPACE;
  if ((uintptr_t)workspace % 256 != 0) return KDA_ERR_ALIGNMENT;
  DecP P;
  P.n = n_seq;
  P.cap = cap;
  P.Hq = Hq;
  P.Hkv = Hkv;
  P.G = Hq / Hkv;
  P.HG = (P.G + MH - 1) / MH;
  P.ns = pieces(n_seq, (int64_t)n_seq * Hkv * P.HG, cap);
  P.scale2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  P.len = lengths;
  P.err = (int32_t*)workspace;
  P.part = (float*)((unsigned char*)workspace + 256);
  const cudaError_t e = D == 64 ? launch<64>(P, dtype, q, k, v, k_cache, v_cache, o, st)
                                : launch<128>(P, dtype, q, k, v, k_cache, v_cache, o, st);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
