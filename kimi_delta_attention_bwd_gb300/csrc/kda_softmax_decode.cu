// Softmax attention, single-token step: every sequence's new key and value are
// appended to its cache and its new query reads the cache,
//   o_h = sum_j p_j v_j,   p_j = exp(scale q_h k_j) / sum,   j = 0 .. length (the new token last).
// The cache is read once: a CTA takes all query heads of a key head (up to 16) over one
// piece of a sequence, so the bytes are the cache's and the step is bound by HBM
// bandwidth.  Where sequences and heads do not fill the GPU the length is cut into equal
// pieces, whose (maximum, sum, o) are joined by a second kernel in a fixed order.
//
// bf16: one warp loads blocks of 64 keys and values (TMA, a ring of 96 KB a CTA, two CTAs per SM: what keeps HBM busy is
// bytes in flight; with 16 keys a warp loaded to registers 64 caches of up to 8192 places took 155 us, so 126),
// four warps take 16 keys each of a block into mma.sync.  The weights enter the value product as two bf16 parts
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
  for (int i = threadIdx.x; i < c.nh * D; i += blockDim.x) {
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
    for (int i = threadIdx.x; i < c.nh * D; i += blockDim.x) dec_out(o + ((size_t)c.seq * P.Hq + c.h0) * D + i, 0.f);
}

// The error word: a length without room in its cache (block 0 looks at all).
__device__ __forceinline__ void check_lengths(const DecP& P) {
  if (blockIdx.x != 0) return;
  int bad = 0;
  for (int i = threadIdx.x; i < P.n; i += blockDim.x) bad |= P.len[i] >= P.cap;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *P.err = bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
}

// two probabilities as a bf16 pair and what that left
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

// ------------------------------------------------------------ bf16
constexpr int KB = 64;  // keys of a block
template <int D>
struct Ring {
  static constexpr int HALF = KB * 128, BLOCK = KB * D * 2;  // 64 columns; a block of keys or of values
  static constexpr int STAGES = D == 64 ? 6 : 3;
  static constexpr int SMEM = STAGES * 2 * BLOCK + 1024;
};
// 16 bytes (columns 8 c ..) of row r of a block: halves of 64 columns, 128-byte swizzle
template <int D>
__device__ __forceinline__ unsigned char* at_chunk(unsigned char* block, int r, int c) {
  return block + (c >> 3) * Ring<D>::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          mma::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(mma::smem_u32(bar))
      : "memory");
}

// Maps: the caches as [sequence][place][Hkv D].  Lane (g, t) = (lane / 4, lane % 4) holds rows (query heads) g and g + 8.
template <int D>
__global__ void __launch_bounds__(WARPS * 32 + 32) smx_decode_kernel(DecP P, const __grid_constant__ CUtensorMap mk,
                                                                   const __grid_constant__ CUtensorMap mv,
                                                                   const bf16* __restrict__ q,
                                                                   const bf16* __restrict__ kn,
                                                                   const bf16* __restrict__ vn, bf16* kc, bf16* vc,
                                                                   bf16* __restrict__ o) {
  using R = Ring<D>;
  constexpr int NS = D / 16, NT = D / 8;  // steps of q k; tiles of p v
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[R::STAGES], empty[R::STAGES];
  __shared__ int dead;
  unsigned char* ring = raw + ((1024 - (mma::smem_u32(raw) & 1023)) & 1023);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::STAGES; i++) {
      mma::mbar_init(&full[i], 1);
      mma::mbar_init(&empty[i], WARPS);
    }
    dead = 0;
    mma::mbar_init_fence();
  }
  pdl_wait();
  pdl_release();
  check_lengths(P);
  Place c;
  const bool live = place_of(P, c);
  __syncthreads();
  if (!live) return no_step<D>(P, c, o);
  const int n = (c.hi - c.lo + KB - 1) / KB;
  const size_t row = (size_t)P.Hkv * D, cache = ((size_t)c.seq * P.cap * P.Hkv + c.hk) * D;
  const bf16 *k1 = kn + ((size_t)c.seq * P.Hkv + c.hk) * D, *v1 = vn + ((size_t)c.seq * P.Hkv + c.hk) * D;
  auto wait = [&](uint64_t* bar, int phase) -> bool {
    bool ok = mma::mbar_try(bar, phase & 1);
    for (int it = 0; !ok && it < mma::WAIT_POLLS; it++) {
      ok = mma::mbar_try(bar, phase & 1);
      if (!ok && *(volatile int*)&dead) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *(volatile int*)&dead = 1;
    return ok;
  };
  float acc[NT][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  if (warp == WARPS) {  // loads (a wait gives up after a second: by then every copy under way has landed)
    for (int x = 0; x < n; x++) {
      const int s = x % R::STAGES;
      if (x >= R::STAGES && !wait(&empty[s], x / R::STAGES - 1)) break;
      if (lane == 0) {
        unsigned char* dst = ring + s * 2 * R::BLOCK;
        mma::mbar_expect_tx(&full[s], 2 * R::BLOCK);
#pragma unroll
        for (int y = 0; y < D / 64; y++) {
          tma_load_3d(dst + y * R::HALF, &mk, c.hk * D + 64 * y, c.lo + x * KB, c.seq, &full[s]);
          tma_load_3d(dst + R::BLOCK + y * R::HALF, &mv, c.hk * D + 64 * y, c.lo + x * KB, c.seq, &full[s]);
        }
      }
      __syncwarp();
    }
  } else {
    if (c.h0 == c.hk * P.G && blockIdx.x % P.ns == 0 && warp == 0 && lane < D / 8) {  // (no reader takes it from the cache)
      *reinterpret_cast<uint4*>(kc + cache + (size_t)c.L * row + 8 * lane) = *reinterpret_cast<const uint4*>(k1 + 8 * lane);
      *reinterpret_cast<uint4*>(vc + cache + (size_t)c.L * row + 8 * lane) = *reinterpret_cast<const uint4*>(v1 + 8 * lane);
    }
    uint32_t qa[NS][4];
    const bf16* qb = q + ((size_t)c.seq * P.Hq + c.h0) * D + 2 * t;
#pragma unroll
    for (int s = 0; s < NS; s++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int r = g + 8 * (e & 1);
        qa[s][e] = r < c.nh ? *reinterpret_cast<const uint32_t*>(qb + (size_t)r * D + 16 * s + 8 * (e >> 1)) : 0u;
      }
#pragma unroll 1
    for (int x = 0; x < n; x++) {
      const int s = x % R::STAGES, r0 = 16 * warp, j0 = c.lo + x * KB + r0;  // the warp's rows of the block, its first key
      if (!wait(&full[s], x / R::STAGES)) break;
      unsigned char *bk = ring + s * 2 * R::BLOCK, *bv = bk + R::BLOCK;
      if (j0 < c.hi) {
        if (j0 + 16 >= c.hi) {  // the last keys: the new token's row, and zeros for places behind it, which hold anything
          for (int i = lane; i < 16 * (D / 8); i += 32) {
            const int r = i / (D / 8), y = i % (D / 8);
            const uint4 zero = make_uint4(0, 0, 0, 0);
            if (j0 + r == c.L) {
              *reinterpret_cast<uint4*>(at_chunk<D>(bk, r0 + r, y)) = *reinterpret_cast<const uint4*>(k1 + 8 * y);
              *reinterpret_cast<uint4*>(at_chunk<D>(bv, r0 + r, y)) = *reinterpret_cast<const uint4*>(v1 + 8 * y);
            } else if (j0 + r >= c.hi) {
              *reinterpret_cast<uint4*>(at_chunk<D>(bv, r0 + r, y)) = zero;
            }
          }
          __syncwarp();
        }
        float sc[2][4] = {};
#pragma unroll
        for (int y = 0; y < NS / 2; y++)
#pragma unroll
          for (int z = 0; z < 2; z++) {
            uint32_t b[4];
            mma::ldsm4(b, at_chunk<D>(bk, r0 + 8 * z + (lane & 7), 4 * y + (lane >> 3)));
            mma::mma_bf16(sc[z], qa[2 * y], b[0], b[1]);
            mma::mma_bf16(sc[z], qa[2 * y + 1], b[2], b[3]);
          }
        uint32_t ph[4], pl[4];
        bool grew = false;
        float corr[2];
#pragma unroll
        for (int r = 0; r < 2; r++) {
          float mx = m[r];
#pragma unroll
          for (int z = 0; z < 2; z++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              float& v = sc[z][2 * r + e];
              v = j0 + 8 * z + 2 * t + e < c.hi ? v * P.scale2 : -INFINITY;
              mx = fmaxf(mx, v);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mu = mx == -INFINITY ? 0.f : mx;
          corr[r] = ex2(m[r] - mu);
          grew |= mx != m[r];
          m[r] = mx;
          float sum = 0.f;
#pragma unroll
          for (int z = 0; z < 2; z++) {
#pragma unroll
            for (int e = 0; e < 2; e++) {
              sc[z][2 * r + e] = ex2(sc[z][2 * r + e] - mu);
              sum += sc[z][2 * r + e];
            }
            split2(sc[z][2 * r], sc[z][2 * r + 1], ph[2 * z + r], pl[2 * z + r]);
          }
          l[r] = l[r] * corr[r] + sum;
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int i = 0; i < NT; i++) {
            acc[i][0] *= corr[0];
            acc[i][1] *= corr[0];
            acc[i][2] *= corr[1];
            acc[i][3] *= corr[1];
          }
        }
#pragma unroll
        for (int y = 0; y < NT / 2; y++) {
          uint32_t b[4];
          mma::ldsm4t(b, at_chunk<D>(bv, r0 + 8 * ((lane >> 3) & 1) + (lane & 7), 2 * y + (lane >> 4)));
          mma::mma_bf16(acc[2 * y], ph, b[0], b[1]);
          mma::mma_bf16(acc[2 * y + 1], ph, b[2], b[3]);
          mma::mma_bf16(acc[2 * y], pl, b[0], b[1]);
          mma::mma_bf16(acc[2 * y + 1], pl, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mma::mbar_arrive(&empty[s]);  // (a block that was written to is the last: no copy follows)
    }
  }
  __syncthreads();
  if (dead) {  // (uniform: written before the barrier)
    if (threadIdx.x == 0) *P.err = KDA_ERR_DEVICE;
    return;
  }
  float* sm = reinterpret_cast<float*>(ring);  // (no copy is under way, no block is read)
  float *sM = sm, *sL = sm + WARPS * MH, *sO = sL + WARPS * MH;
  if (warp < WARPS)
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
      for (int y = 0; y < NT; y++)
        *reinterpret_cast<float2*>(sO + (size_t)i * D + 8 * y + 2 * t) = make_float2(acc[y][2 * r], acc[y][2 * r + 1]);
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
  for (int i = threadIdx.x; i < c.nh * D; i += blockDim.x) sq[i] = q[((size_t)c.seq * P.Hq + c.h0) * D + i];
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

// Joins the pieces of one (sequence, query head): their weights first, then warp w sums pieces w, w + nw, .. whose loads
// do not wait for one another (with a running maximum along them 114 pieces took 12.7 us, so 5).
constexpr int JW = 32;  // warps at most
template <int D, typename T>
__global__ void __launch_bounds__(JW * 32) smx_join_kernel(DecP P, T* __restrict__ o) {
  constexpr int NV = D / 32;
  extern __shared__ float sw[];  // [ns]
  __shared__ float red[JW], so[JW][D];
  const int seq = blockIdx.x / P.Hq, h = blockIdx.x % P.Hq, hk = h / P.G, r = h % P.G;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, rr = r % MH, nw = blockDim.x / 32;
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
  for (int s = threadIdx.x; s < P.ns; s += blockDim.x) {
    sw[s] = part[s * ST + rr];
    m = fmaxf(m, sw[s]);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  for (int w = 0; w < nw; w++) m = fmaxf(m, red[w]);
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int s = threadIdx.x; s < P.ns; s += blockDim.x) {
    sw[s] = ex2(sw[s] - mu);
    l += sw[s] * part[s * ST + MH + rr];
  }
  l = warp_sum(l);
  __syncthreads();  // (red is read, the weights are there)
  if (lane == 0) red[warp] = l;
  float acc[NV] = {};
  const float* p = part + 2 * MH + rr * D + lane * NV;
#pragma unroll 8
  for (int s = warp; s < P.ns; s += nw) {
    const float w = sw[s];
#pragma unroll
    for (int e = 0; e < NV; e++) acc[e] = fmaf(w, p[s * ST + e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < NV; e++) so[warp][lane * NV + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f, x = 0.f;
    for (int w = 0; w < nw; w++) {
      sum += red[w];
      x += so[w][threadIdx.x];
    }
    dec_out(out + threadIdx.x, x / sum);
  }
}

// Pieces of a sequence, none of fewer than 128 keys of a full cache: for one sequence a CTA for each of 152 SMs, for several
// four, since they differ in length and smaller pieces even that out.  Both sides, 16 heads on 4 of 128, one CTA an SM and four
// (as graphs): one of 131072 places 51.7 and 60.3 us, a quarter full 22.4 and 28.6; two of 65536, full, 51.3 and 58.1, of
// uneven lengths 47.7 and 46.1; four of 32768 54.6 and 57.8, uneven 48.4 and 40.2; 16 of 16384 89.5 and 101, uneven 73.9 and
// 56.7; 64 of up to 8192 109 and 100.  Equal lengths lose up to 13% by the rule, uneven ones up to 30% by the other; lengths
// are known on the device alone.
int pieces(int n, int64_t units, int cap) {
  const int64_t want = ((n == 1 ? 1 : 4) * SMS + units - 1) / units, most = ((int64_t)cap + 127) / 128;
  const int64_t ns = want < most ? want : most;
  return (int)(ns < 1 ? 1 : ns);
}

bool sizes_ok(int n, int cap, int Hq, int Hkv, int dtype) {
  return n > 0 && cap > 0 && Hq > 0 && Hkv > 0 && Hq <= 4096 && Hq % Hkv == 0 && (int64_t)n * Hq <= ((int64_t)1 << 28) &&
         (int64_t)n * cap <= ((int64_t)1 << 40) && (dtype == KDA_BF16 || dtype == KDA_F32);
}

// A cache [n][cap][Hkv D] with boxes of 64 columns by KB places of one sequence, in the 128-byte swizzle.
bool encode_cache(CUtensorMap* m, const void* base, int n, int cap, int width) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)cap, (cuuint64_t)n};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)width * 2 * (cuuint64_t)cap};
  const cuuint32_t box[3] = {64, KB, 1}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const DecP& P, int dtype, const void* q, const void* k, const void* v, void* kc, void* vc, void* o,
                   cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)P.n * P.Hkv * P.HG * P.ns);
  const size_t s32 = (WARPS * MH * (D + 2) + MH * D) * sizeof(float);
  cudaError_t e = cudaSuccess;
  CUtensorMap mk, mv;
  if (dtype == KDA_BF16) {
    e = raise_smem<smx_decode_kernel<D>>(Ring<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (!encode_cache(&mk, kc, P.n, P.cap, P.Hkv * D) || !encode_cache(&mv, vc, P.n, P.cap, P.Hkv * D))
      return cudaErrorInvalidValue;
  }
  prof_begin(K_SMX_DECODE, st);
  if (dtype == KDA_BF16) {
    e = launch_pdl(smx_decode_kernel<D>, dim3(grid), dim3(WARPS * 32 + 32), Ring<D>::SMEM, st, P, mk, mv, (const bf16*)q,
                   (const bf16*)k, (const bf16*)v, (bf16*)kc, (bf16*)vc, (bf16*)o);
  } else {
    e = launch_pdl(smx_decode_f32_kernel<D>, dim3(grid), dim3(WARPS * 32), s32, st, P, (const float*)q,
                   (const float*)k, (const float*)v, (float*)kc, (float*)vc, (float*)o);
  }
  prof_end(K_SMX_DECODE, st);
  if (e != cudaSuccess || P.ns == 1) return e;
  const int jw = P.ns >= 4 * JW ? JW : P.ns <= 16 ? 4 : (P.ns + 3) / 4;  // about four pieces a warp; D threads at least
  prof_begin(K_SMX_JOIN, st);
  if (dtype == KDA_BF16)
    e = launch_pdl(smx_join_kernel<D, bf16>, dim3(P.n * P.Hq), dim3(jw * 32), P.ns * sizeof(float), st, P, (bf16*)o);
  else
    e = launch_pdl(smx_join_kernel<D, float>, dim3(P.n * P.Hq), dim3(jw * 32), P.ns * sizeof(float), st, P, (float*)o);
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
  if (!sizes_ok(n_seq, cap, Hq, Hkv, dtype) || !isfinite(scale)) return KDA_ERR_INVALID_ARG;
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
