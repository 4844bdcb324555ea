// Softmax attention on the 5th-generation tensor cores (tcgen05, accumulators in tensor memory): bf16 io, and fp32 io as
// three bf16 parts of every value (kda_softmax_tc.cuh) but for its backward at D = 128 (kda_softmax_f32.cu).
//
// Forward, per CTA: 256 queries of one head as two tiles of 128 over the keys in blocks of 128.  One warp loads
// (TMA, a ring of key and value blocks), one issues the products, and per tile four warps, a thread a row,
// turn the block of logits S = q k^T into weights P = 2^(scale2 S - m): row maximum, exponentials, row sum.  P goes
// back to tensor memory over S, as bf16, and is the product P v's operand there.  While one tile's weights are formed
// the other's products run.  The maximum m that the exponents are taken against is raised (and o and the sum scaled
// down) only where a row's maximum has grown by 2^8: weights stay below 2^8, which bf16 and fp32 hold with the same
// relative precision as those below 1.
// Weights are rounded to bf16 (2^-8, the operand's type; o's error with that is that of one rounding of o times
// sqrt(2)), but in a first block that a mask cuts they enter as two parts (2^-16): rows with few keys have theirs there,
// and the backward's delta = o dO cancels against dO v in just those rows.  Documents
// of few rows, or against few of the other side (FEW_ROWS, FEW), take two parts throughout, in the backward too: a handful
// of roundings does not average out (up to 1.8 times the error of weights that are multiplied in fp32 and a result rounded
// once; with two parts 1.5).  The rule looks at the document alone, whatever batch it stands in, and that costs batches of
// short ones up to 12% (training steps of 64 rows of 256, 8 heads of 64: 101 us with one part, 113 with two; 100 documents
// of 164, 16 heads on 4 of 128: 428 and 474; 256 documents of 64, 8 heads of 64: 156 and 159).
#include "kda_softmax_tc.cuh"

#include <type_traits>

namespace kda {
namespace smx {
namespace {

constexpr int FEW_ROWS = 64, FEW = 256;  // a document's rows on a kernel's own side, and on the other, for two parts
constexpr float GROW = 8.0f;   // log2 of what a weight may exceed 1 by

// f with `twice` as a constant (a branch inside its loop cost dk and dv 8% and dq 5% at D = 128)
template <int PARTS, class F>
__device__ __forceinline__ bool with_parts(bool twice, F f) {
  if constexpr (PARTS == 1)
    if (twice) return f(std::true_type{});
  return f(std::false_type{});
}
template <int PARTS>
struct Io {
  using T = bf16;
};
template <>
struct Io<3> {
  using T = float;
};

// ------------------------------------------------------------ forward
// A CTA has two tiles that share every block of keys and values.  At D = 128 the products bound it, with one CTA per SM
// and blocks of 128 keys.  At D = 64 they are half of that, and the exponentials and the waits between the steps count:
// blocks of 64 keys let two CTAs share an SM (256 columns of tensor memory, 80 registers a thread), so that four tiles'
// steps hide each other (300M batch: 88 us; with tiles and blocks as at D = 128 116 us, two CTAs of one tile 104).
// fp32 io (three parts a value): blocks of 64 keys, one CTA per SM, at D = 128 of one tile.
template <int D, int PARTS>
struct Fwd {
  static constexpr int NT = D == 128 && PARTS == 3 ? 1 : 2, XB = D == 64 || PARTS == 3 ? 64 : 128;
  static constexpr int OWN = BLK * D * 2 * PARTS, BYTES = XB * D * 2 * PARTS;  // a tile of queries, a block of keys or values
  static constexpr int STAGES = PARTS == 3 ? (D == 64 ? 5 : 2) : D == 64 ? 8 : 5;  // blocks in their ring
  static constexpr int SMEM = NT * OWN + STAGES * BYTES + 1024;
  static constexpr int COLS = D == 64 && PARTS == 1 ? 256 : 512, PER_SM = COLS == 256 ? 2 : 1;
  // tensor memory columns: S of the tiles, o of the tiles, third parts of the weights
  static constexpr uint32_t S0 = 0, O0 = NT * XB, X0 = O0 + NT * D;
  // Weights lie over the logits they come from: those of 16 keys at part(s), their second parts SECOND further.
  static constexpr int SECOND = XB == 64 ? 8 : 16;
  static __device__ constexpr int part(int s) { return XB == 64 ? 16 * s : 32 * (s >> 1) + 8 * (s & 1); }
  static constexpr int THREADS = NT * BLK + 64;
};

struct FwdBars {
  uint64_t q[2], full[8], empty[8], s[2], p[2], o[2], drain;
  uint32_t tmem;
  int dead;
};

template <int D, int PARTS>
__global__ void __launch_bounds__(Fwd<D, PARTS>::THREADS, Fwd<D, PARTS>::PER_SM)
smx_tc_fwd_kernel(SmxP P, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, typename Io<PARTS>::T* __restrict__ o,
                  float* __restrict__ lse) {
  using F = Fwd<D, PARTS>;
  constexpr int NT = F::NT, XB = F::XB, W_MMA = 4 * NT, W_LOAD = W_MMA + 1;
  extern __shared__ unsigned char raw[];
  __shared__ FwdBars B;
  unsigned char* sm = raw + ((1024 - (mma::smem_u32(raw) & 1023)) & 1023);
  unsigned char* ring = sm + NT * F::OWN;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == W_MMA) tc::tmem_alloc(&B.tmem, F::COLS);
  if (threadIdx.x == 32 * W_LOAD) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; i++) {
      mma::mbar_init(&B.q[i], 1);
      mma::mbar_init(&B.s[i], 1);
      mma::mbar_init(&B.p[i], 4);
      mma::mbar_init(&B.o[i], 1);
    }
    for (int i = 0; i < F::STAGES; i++) {
      mma::mbar_init(&B.full[i], 1);
      mma::mbar_init(&B.empty[i], 1);
    }
    mma::mbar_init(&B.drain, 1);
    B.dead = 0;
    mma::mbar_init_fence();
  }
  pdl_wait();
  if (P.rows && blockIdx.x == 0 && threadIdx.x == 0) {
    *P.err = KDA_OK;
    *P.wtag = P.save ? P.tag : 0;
  }
  Tile t;
  const int h = blockIdx.x % P.Hq, hk = h / P.G;
  const bool live = tile_of(P, 0, blockIdx.x / P.Hq, false, t);
  int i0 = 0, nq = 0, nb[2] = {0, 0}, clean[2] = {0, 0};  // blocks of each tile; those that no mask cuts
  bool twice = false;                                     // every weight in two parts
  if (live) {
    i0 = t.t * (NT * BLK);
    nq = min(NT * BLK, t.Lq - i0);
    twice = PARTS == 1 && (t.Lq <= FEW_ROWS || t.Lk <= FEW);
#pragma unroll
    for (int i = 0; i < NT; i++)
      if (i * BLK < nq) {
        nb[i] = (keys_of(P.causal, i0 + min(nq, (i + 1) * BLK) - 1, t.Lq, t.Lk) + XB - 1) / XB;
        nb[i] = max(0, min(nb[i], t.j1) - t.j0);
        clean[i] = keys_of(P.causal, i0 + i * BLK, t.Lq, t.Lk) / XB;
      }
  }
  const int n = max(nb[0], nb[1]);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = tm_base<F::COLS>(B.tmem);

  if (warp == W_LOAD) {  // loads
    if (lane == 0 && n > 0) {
      for (int i = 0; i < NT; i++)
        if (nb[i]) {
          mma::mbar_expect_tx(&B.q[i], F::OWN);
          load_block<D, BLK, PARTS>(sm + i * F::OWN, &mq, h, t.q0 + i0 + i * BLK, P.Nq, &B.q[i]);
        }
    }
    __syncwarp();
    int x = 0;
    for (; x < 2 * n; x++) {
      const int s = x % F::STAGES, r = x / F::STAGES;
      if (r > 0 && !wait(&B.empty[s], (r - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.full[s], F::BYTES);
        load_block<D, XB, PARTS>(ring + s * F::BYTES, x & 1 ? &mv : &mk, hk, t.k0 + (t.j0 + x / 2) * XB, P.Nk, &B.full[s]);
      }
      __syncwarp();
    }
    if (*(volatile int*)&B.dead) {  // every copy lands before the shared memory is released
      for (int y = max(0, x - F::STAGES); y < x; y++)
        for (int it = 0; it < mma::WAIT_POLLS && !mma::mbar_try(&B.full[y % F::STAGES], (y / F::STAGES) & 1); it++) {}
      for (int i = 0; i < NT; i++)
        if (nb[i])
          for (int it = 0; it < mma::WAIT_POLLS && !mma::mbar_try(&B.q[i], 0); it++) {}
    }
  } else if (warp == W_MMA) {  // products
    const uint32_t q0 = mma::smem_u32(sm), r0 = mma::smem_u32(ring);
    constexpr uint32_t id_s = idesc(BLK, XB, false), id_o = idesc(BLK, D, true);
    const uint32_t me = elect();
    auto logits = [&](int i, int j) {  // S of tile i and key block j
      prod_ss<D, PARTS, BLK, XB>(tm + F::S0 + i * XB, q0 + i * F::OWN, r0 + 2 * j % F::STAGES * F::BYTES, id_s, me);
      commit(&B.s[i], me);
    };
    auto run = [&]() -> bool {
      if (!wait(&B.full[0], 0, &B.dead)) return false;
#pragma unroll
      for (int i = 0; i < NT; i++)
        if (nb[i]) {
          if (!wait(&B.q[i], 0, &B.dead)) return false;
          logits(i, 0);
        }
      commit(&B.empty[0], me);
      for (int j = 0; j < n; j++) {
        const int xv = 2 * j + 1, xk = 2 * j + 2, sv = xv % F::STAGES, sk = xk % F::STAGES;
        if (!wait(&B.full[sv], (xv / F::STAGES) & 1, &B.dead)) return false;
        const int left = t.Lk - (t.j0 + j) * XB;
        if (left < XB) zero_rows<D, XB, PARTS>(ring + sv * F::BYTES, left);
        if (j + 1 < n && !wait(&B.full[sk], (xk / F::STAGES) & 1, &B.dead)) return false;
        const uint32_t vb = r0 + sv * F::BYTES;
#pragma unroll
        for (int i = 0; i < NT; i++) {
          if (j >= nb[i]) continue;
          if (!wait(&B.p[i], j & 1, &B.dead)) return false;
          tc::fence_after();
          const uint32_t a = tm + F::S0 + i * XB, d = tm + F::O0 + i * D, c = tm + F::X0 + i * (XB / 2);
          using Q = Prod<PARTS>;
#pragma unroll
          for (int y = 0; y < Q::N; y++)
#pragma unroll
            for (int s = 0; s < XB / 16; s++)
              mma_ts(d, Q::a(y) == 2 ? c + 8 * s : a + F::part(s) + Q::a(y) * F::SECOND,
                     desc_mn<XB>(vb + Q::b(y) * (XB * D * 2), s), id_o, (PARTS == 1 && j > 0) || y > 0 || s > 0, me);
          if (PARTS == 1 && (twice || (t.j0 + j == 0 && clean[i] == 0)))
#pragma unroll
            for (int s = 0; s < XB / 16; s++)
              mma_ts(d, a + F::part(s) + F::SECOND, desc_mn<XB>(vb, s), id_o, true, me);
          commit(&B.o[i], me);
          if (i == NT - 1 || j >= nb[1]) commit(&B.empty[sv], me);
          if (j + 1 < nb[i]) logits(i, j + 1);
          if (j + 1 < n && (i == NT - 1 || j + 1 >= nb[1])) commit(&B.empty[sk], me);
        }
      }
      return true;
    };
    if (n > 0 && !run()) {  // (its products end before the tensor memory is released)
      commit(&B.drain, me);
      for (int it = 0; it < mma::WAIT_POLLS && !mma::mbar_try(&B.drain, 0); it++) {}
    }
  } else if (warp < W_MMA && live) {  // weights: a thread a row
    const int i = warp / 4, r = i * BLK + (threadIdx.x & 127), nbi = i ? nb[1] : nb[0], cleani = i ? clean[1] : clean[0];
    const bool in = r < nq;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tm + F::S0 + i * XB + lanes, to = tm + F::O0 + i * D + lanes;
    const int lim = keys_of(P.causal, i0 + r, t.Lq, t.Lk);  // (grows with the row)
    const uint64_t sc = two(P.scale2, P.scale2);
    float m = -INFINITY, l = 0.f;
    float sums[PARTS == 3 ? D : 1] = {};  // (three parts) o
    auto take_block = [&]() {  // the product of the block before is done: its S was issued earlier than this one's
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        float v[16];
        tm_ld16(to + c, v);
        tm_wait_ld(v);
#pragma unroll
        for (int e = 0; e < 16; e++) sums[c + e] += v[e];
      }
    };
    // A new reference, the block's maximum `top`, in rows where it has grown by 2^GROW (or that ask for it): o and l are
    // scaled down to it.  False: a wait gave up.
    auto raise = [&](int j, float top, bool ask) -> bool {
      const bool grew = top > m && (ask || !((top - m) * P.scale2 <= GROW));
      if (!__any_sync(0xffffffffu, grew)) return true;
      const float up = grew ? ex2((m - top) * P.scale2) : 1.0f;
      if (grew) m = top;
      l *= up;
      if (j == 0) return true;
      if constexpr (PARTS == 3) {
#pragma unroll
        for (int c = 0; c < D; c++) sums[c] *= up;
        return true;
      }
      if (!wait(&B.o[i], (j - 1) & 1, &B.dead)) return false;
      tc::fence_after();
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float v[16];
        tm_ld16(to + c, v);
        tm_wait_ld(v);
#pragma unroll
        for (int e = 0; e < 16; e++) v[e] *= up;
        tm_st16(to + c, reinterpret_cast<const uint32_t*>(v));
      }
      return true;
    };
    auto reference = [&]() { return m == -INFINITY ? 0.f : -m * P.scale2; };
    bool ok = true;
    for (int j = 0; j < nbi; j++) {
      ok = wait(&B.s[i], j & 1, &B.dead);
      if (!ok) break;
      tc::fence_after();
      if constexpr (PARTS == 3)
        if (j > 0) take_block();
      const bool cut = t.j0 + j >= cleani, few = twice || (cut && t.j0 + j == 0);  // a mask cuts the block; two parts
      const int left = lim - (t.j0 + j) * XB, least = cut ? __shfl_sync(0xffffffffu, left, 0) : XB;  // (the warp's first row's)
      uint64_t sum[2] = {0, 0};
      float s0, s1;
      if constexpr (XB == 128) {
        float s[4][32], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; c++) tm_ld32(ts + 32 * c, s[c]);
#pragma unroll
        for (int c = 0; c < 4; c++) tm_wait_ld(s[c]);
        if (cut)
#pragma unroll
          for (int c = 0; c < 4; c++) mask(s[c], left - 32 * c);
#pragma unroll
        for (int c = 0; c < 4; c++) row_max(s[c], mx);
        ok = raise(j, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), false);
        if (!ok) break;
        const float neg = reference();
        const uint64_t ng = two(neg, neg);
#pragma unroll
        for (int c = 0; c < 4; c++) {
          uint32_t w[16];
          weights(s[c], sc, ng, sum, w);
          tm_st16(ts + 32 * c, w);
          if (few) {
            second_parts(s[c], w);
            tm_st16(ts + 32 * c + 16, w);
          }
        }
      } else {
        // The weights against the reference as it is: a row's sum of at most 2^GROW says that none is above it, and the
        // maximum need not be known.  Else, and in the first block, the maximum first (a NaN row: every time).
        float a[16], b[16];
        bool ask = false, again = j == 0 || few || PARTS == 3;
        if (PARTS == 1 && !again) {
          const float neg = reference();
          const uint64_t ng = two(neg, neg);
          uint32_t w[32];
          tm_ld16(ts, a);
          tm_wait_ld(a);
          tm_ld16(ts + 16, b);
          if (least < 16) mask(a, left);
          weights(a, sc, ng, sum, w);
          tm_wait_ld(b);
          tm_ld16(ts + 32, a);
          if (least < 32) mask(b, left - 16);
          weights(b, sc, ng, sum, w + 8);
          tm_wait_ld(a);
          tm_ld16(ts + 48, b);
          if (least < 48) mask(a, left - 32);
          weights(a, sc, ng, sum, w + 16);
          tm_wait_ld(b);
          if (least < 64) mask(b, left - 48);
          weights(b, sc, ng, sum, w + 24);
          one(add2(sum[0], sum[1]), s0, s1);
          ask = !(s0 + s1 <= 256.0f) || m == -INFINITY;
          again = __any_sync(0xffffffffu, ask);
          if (!again)
#pragma unroll
            for (int c = 0; c < 4; c++) tm_st8(ts + 16 * c, w + 8 * c);
        }
        if (again) {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < 4; c++) {
            tm_ld16(ts + 16 * c, a);
            tm_wait_ld(a);
            if (least < 16 * (c + 1)) mask(a, left - 16 * c);
            row_max(a, mx);
          }
          ok = raise(j, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), ask);
          if (!ok) break;
          const float neg = reference();
          const uint64_t ng = two(neg, neg);
          sum[0] = sum[1] = 0;
#pragma unroll 1
          for (int c = 0; c < 4; c++) {
            uint32_t w[8];
            tm_ld16(ts + 16 * c, a);
            tm_wait_ld(a);
            if (least < 16 * (c + 1)) mask(a, left - 16 * c);
            weights(a, sc, ng, sum, w);
            if (PARTS == 3) {
              next_part(a, w);
              tm_st8(ts + 16 * c, w);
              next_part(a, w);
              tm_st8(ts + 16 * c + 8, w);
              next_part(a, w);
              tm_st8(tm + F::X0 + i * (XB / 2) + lanes + 8 * c, w);
            } else {
              tm_st8(ts + 16 * c, w);
              if (few) {
                second_parts(a, w);
                tm_st8(ts + 16 * c + 8, w);
              }
            }
          }
        }
      }
      one(add2(sum[0], sum[1]), s0, s1);
      l += s0 + s1;
      tm_wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mma::mbar_arrive(&B.p[i]);
    }
    if (ok && nbi > 0) {
      ok = wait(&B.o[i], (nbi - 1) & 1, &B.dead);
      tc::fence_after();
      if constexpr (PARTS == 3)
        if (ok) take_block();
    }
    if (ok) {
      const float inv = l == 0.f ? 0.f : 1.0f / l, l2 = m * P.scale2 + log2f(l);
      const int w0 = r & ~31, rows = nq - w0;  // the warp's first row, rows from there on
      const size_t row = (size_t)(t.q0 + i0 + r) * P.Hq + h, row0 = (size_t)(t.q0 + i0 + w0) * P.Hq + h;
      unsigned char* buf = sm + i * F::OWN + (w0 & 127) * 128;  // (the tile's queries are no longer read)
      // a piece's o, or o of fp32 io
      const size_t at = ((size_t)t.piece * P.Hq + h) * (NT * BLK);
      if (PARTS == 3 || t.piece >= 0) {
        float* dst = t.piece >= 0 ? P.po[0] + (at + w0) * D : (float*)o + row0 * D;
        const size_t ld = t.piece >= 0 ? D : (size_t)P.Hq * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float v[32];
          if constexpr (PARTS == 3) {
#pragma unroll
            for (int e = 0; e < 32; e++) v[e] = sums[c + e];
          } else if (nbi > 0) {
            tm_ld32(to + c, v);
            tm_wait_ld(v);
          }
          uint32_t u[32];
#pragma unroll
          for (int e = 0; e < 32; e++) u[e] = __float_as_uint(l == 0.f ? 0.f : v[e] * inv);
          store_rows(buf, u, dst + c, ld, rows);
        }
      } else if constexpr (PARTS == 1) {
#pragma unroll
        for (int c = 0; c < D; c += 64) {
          uint32_t u[32], w[32];  // o, and what its rounding leaves
#pragma unroll
          for (int y = 0; y < 2; y++) {
            float v[32];
            if (nbi > 0) {
              tm_ld32(to + c + 32 * y, v);
              tm_wait_ld(v);
            }
#pragma unroll
            for (int e = 0; e < 32; e++) v[e] = l == 0.f ? 0.f : v[e] * inv;
            next_part(v, u + 16 * y);
            next_part(v, w + 16 * y);
          }
          store_rows(buf, u, o + row0 * D + c, (size_t)P.Hq * D, rows);
          if (P.save) store_rows(buf, w, P.res + row0 * D + c, (size_t)P.Hq * D, rows);
        }
      }
      if (in && t.piece >= 0) {
        P.pl[at + r] = l2;
      } else if (in) {
        lse[row] = l2 * LN2;
        if (P.save) P.lse2[(size_t)h * P.Nq + t.q0 + i0 + r] = l2;
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && B.dead) *P.err = KDA_ERR_DEVICE;
  if (warp == W_MMA) {
    tc::fence_after();
    tc::tmem_dealloc(tm, F::COLS);
  }
}

template <int D, int PARTS>
cudaError_t fwd(const SmxP& P, const void* q, const void* k, const void* v, void* o, float* lse, cudaStream_t st) {
  using F = Fwd<D, PARTS>;
  cudaError_t e = raise_smem<smx_tc_fwd_kernel<D, PARTS>>(F::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!encode_head_rows(&mq, q, PARTS * P.Nq, P.Hq, D, BLK) || !encode_head_rows(&mk, k, PARTS * P.Nk, P.Hkv, D, F::XB) ||
      !encode_head_rows(&mv, v, PARTS * P.Nk, P.Hkv, D, F::XB))
    return cudaErrorInvalidValue;
  const int64_t grid = (int64_t)max_tiles(P, 0) * P.Hq;
  prof_begin(K_SMX_FWD, st);
  e = launch_pdl(smx_tc_fwd_kernel<D, PARTS>, dim3((unsigned)grid), dim3(F::THREADS), F::SMEM, st, P, mq, mk, mv,
                 (typename Io<PARTS>::T*)o, lse);
  prof_end(K_SMX_FWD, st);
  return e;
}

// ------------------------------------------------------------ backward
// 32 H pairs of a row as operands: bf16 at `to`, second parts (three parts, or TWICE) 16 H columns further,
// third at `x3`.
template <int PARTS, bool TWICE, int H>
__device__ __forceinline__ void put_parts(float (&v)[H][32], uint32_t to, uint32_t x3) {
#pragma unroll
  for (int y = 0; y < (TWICE ? 2 : PARTS); y++) {
#pragma unroll
    for (int c = 0; c < H; c++) {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; e++) w[e] = rest(v[c][2 * e], v[c][2 * e + 1], y);
      tm_st16((y == 2 ? x3 : to + 16 * H * y) + 16 * c, w);
    }
  }
}
// The same in dq, whose three parts lie XB / 2 columns apart, or second of two at `over`.
template <int PARTS, bool TWICE, int XB, int H>
__device__ __forceinline__ void put_dq(float (&v)[H][32], uint32_t to, uint32_t over) {
#pragma unroll
  for (int y = 0; y < (TWICE ? 2 : PARTS); y++) {
#pragma unroll
    for (int c = 0; c < H; c++) {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; e++) w[e] = rest(v[c][2 * e], v[c][2 * e + 1], y);
      tm_st16((TWICE && y == 1 ? over : to + XB / 2 * y) + 16 * c, w);
    }
  }
}
// dk and dv, per CTA: 128 keys of one key head, over the blocks of 128 queries of its group's heads.  The pairs lie
// transposed, a key a lane: S' = k q^T, P' = 2^(scale2 S' - lse2), dP' = v dO^T, dS' = P' (dP' - delta), and P' and
// dS' (bf16, over S' and dP' in tensor memory) are the operands of dv += P' dO and dk += dS' q.  Eight warps form
// them, each half of the queries' columns; the row sums of the queries come through shared memory.  The products are
// issued as dv, next S', dk, next dP': while two run, the other two's operand is formed.
//
// Both kernels keep two blocks of their own (dq with bf16 io one) and two rings: A, of the blocks that a first product and then the last one
// reads (q for dk and dv, k for dq), and B, of those that are free earlier (dO, v).
// The other side's blocks have XB rows: 128, and eight warps for the pairs, at D = 128; at D = 64 half of both (dk and dv
// keep the eight), and two CTAs per SM.
template <int D, int PARTS>
struct Bwd {
  static_assert(PARTS == 1 || D == 64, "at D = 128 three parts of both own blocks leave no room: kda_softmax_f32.cu");
  static constexpr int XB = D == 64 ? 64 : 128;
  static constexpr int OWN = BLK * D * 2 * PARTS, BYTES = XB * D * 2 * PARTS;  // a block of either side
  static constexpr int NA = D == 64 && PARTS == 1 ? 5 : 3, NB = D == 64 && PARTS == 1 ? 4 : 2;
  static constexpr int BLOCKS = 2 * OWN + (NA + NB) * BYTES;
  // warps of the pairs: 64 of a row's pairs a thread, at D = 64 in dk and dv 32 (300M packed step: 93 us, 97 with 64); with
  // three parts there also 32 columns of both sums.  (16 warps at D = 128: dk and dv the same, dq 6% slower.)
  static constexpr int EW = XB / 16, EWK = 8;
  static constexpr int COLS = D == 64 && PARTS == 1 ? 256 : 512, PER_SM = COLS == 256 ? 2 : 1;
  // dq with bf16 io: q is an operand in tensor memory, and its place in shared memory has further blocks of ring A
  static constexpr int QOWN = PARTS == 1 ? OWN : 2 * OWN, QA = NA + (2 * OWN - QOWN) / BYTES;
};

template <int XB>
struct BwdRest {  // (shared memory is full at D = 128: behind the blocks, whose swizzle wants 1024-byte alignment)
  float stat[2][2][XB];  // minus lse2 and minus delta of two blocks' queries
  uint64_t own, fullA[5], emptyA[5], fullB[5], emptyB[5], fullS[2], s, dp, p, ds, done, drain;
  uint32_t tmem;
  int dead;
};
template <int D, int PARTS>
constexpr int DKV_SMEM = Bwd<D, PARTS>::BLOCKS + (int)sizeof(BwdRest<Bwd<D, PARTS>::XB>);
static_assert(Bwd<64, 1>::QA <= 7 && Bwd<128, 1>::QA <= 7 && 2 * (DKV_SMEM<64, 1> + 1024) <= 233472 && DKV_SMEM<128, 1> <= 232448 && DKV_SMEM<64, 3> <= 232448,
              "shared memory of an SM, of a CTA");

template <int D, int PARTS>
__global__ void __launch_bounds__(Bwd<D, PARTS>::EWK * 32 + 96, Bwd<D, PARTS>::PER_SM)
smx_tc_dkv_kernel(SmxP P, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                  typename Io<PARTS>::T* __restrict__ dk, typename Io<PARTS>::T* __restrict__ dv) {
  using F = Bwd<D, PARTS>;
  constexpr int XB = F::XB, EW = F::EWK, H = XB / 8 / EW;
  constexpr uint32_t cS = 0, cDP = XB, cDV = 2 * XB, cDK = 2 * XB + D, cX = 2 * XB + 2 * D;  // (X: third parts)
  extern __shared__ __align__(1024) unsigned char sm[];
  BwdRest<XB>& B = *reinterpret_cast<BwdRest<XB>*>(sm + F::BLOCKS);
  if (mma::smem_u32(sm) & 1023) {  // (dynamic shared memory alone starts on such a boundary)
    if (blockIdx.x == 0 && threadIdx.x == 0) *P.err = KDA_ERR_DEVICE;
    return;
  }
  unsigned char *ringA = sm + 2 * F::OWN, *ringB = ringA + F::NA * F::BYTES;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == EW) tc::tmem_alloc(&B.tmem, F::COLS);
  if (threadIdx.x == 32 * (EW + 1)) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
    prefetch_map(&mg);
  }
  if (threadIdx.x == 0) {
    mma::mbar_init(&B.own, 1);
    for (int i = 0; i < F::NA; i++) {
      mma::mbar_init(&B.fullA[i], 1);
      mma::mbar_init(&B.emptyA[i], 1);
    }
    for (int i = 0; i < F::NB; i++) {
      mma::mbar_init(&B.fullB[i], 1);
      mma::mbar_init(&B.emptyB[i], 1);
    }
    mma::mbar_init(&B.fullS[0], 1);
    mma::mbar_init(&B.fullS[1], 1);
    mma::mbar_init(&B.s, 1);
    mma::mbar_init(&B.dp, 1);
    mma::mbar_init(&B.p, EW);
    mma::mbar_init(&B.ds, EW);
    mma::mbar_init(&B.done, 1);
    mma::mbar_init(&B.drain, 1);
    B.dead = 0;
    mma::mbar_init_fence();
  }
  pdl_wait();
  pdl_release();  // dq's CTAs may follow this grid's last ones: they wait for it at their end only
  Tile t;
  const int hk = blockIdx.x % P.Hkv;
  const bool live = tile_of(P, 2, blockIdx.x / P.Hkv, true, t);
  int j0 = 0, nk = 0, first = 0, per = 0;  // first query block, blocks a head
  if (live) {
    j0 = t.t * BLK;
    nk = min(BLK, t.Lk - j0);
    first = first_query(P.causal, j0, t.Lq, t.Lk) / XB;
    per = max(0, (t.Lq + XB - 1) / XB - first);
  }
  const bool twice = PARTS == 1 && live && (t.Lk <= FEW_ROWS || t.Lq <= FEW);
  const int n = live ? min(per * P.G, t.j1) - t.j0 : 0;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = tm_base<F::COLS>(B.tmem);

  if (warp == EW + 1) {  // copies
    if (lane == 0 && n > 0) {
      mma::mbar_expect_tx(&B.own, 2 * F::OWN);
      load_block<D, BLK, PARTS>(sm, &mk, hk, t.k0 + j0, P.Nk, &B.own);
      load_block<D, BLK, PARTS>(sm + F::OWN, &mv, hk, t.k0 + j0, P.Nk, &B.own);
    }
    __syncwarp();
    for (int x = 0; x < n; x++) {
      const int sa = x % F::NA, sb = x % F::NB, y = t.j0 + x, h = hk * P.G + y / per, row = t.q0 + (first + y % per) * XB;
      if (x >= F::NA && !wait(&B.emptyA[sa], (x / F::NA - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullA[sa], F::BYTES);
        load_block<D, XB, PARTS>(ringA + sa * F::BYTES, &mq, h, row, P.Nq, &B.fullA[sa]);
      }
      __syncwarp();
      if (x >= F::NB && !wait(&B.emptyB[sb], (x / F::NB - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullB[sb], F::BYTES);
        load_block<D, XB, PARTS>(ringB + sb * F::BYTES, &mg, h, row, P.Nq, &B.fullB[sb]);
      }
      __syncwarp();
    }
    // (a wait gives up after a second: by then every copy under way has landed)
  } else if (warp == EW + 2) {  // row sums
    for (int x = 0; x < n; x++) {
      const int s = x & 1;  // (free once block x - 2 has left ring A)
      if (x >= 2 && !wait(&B.emptyA[(x - 2) % F::NA], ((x - 2) / F::NA) & 1, &B.dead)) break;
      const int y = t.j0 + x, h = hk * P.G + y / per, i0 = (first + y % per) * XB;
      const size_t at = (size_t)h * P.Nq + t.q0 + i0;
#pragma unroll
      for (int c = lane; c < XB; c += 32) {
        const bool in = i0 + c < t.Lq;
        B.stat[s][0][c] = in ? -P.lse2[at + c] : 0.f;
        B.stat[s][1][c] = in ? -P.delta[at + c] : 0.f;
      }
      __syncwarp();
      if (lane == 0) mma::mbar_arrive(&B.fullS[s]);
    }
  } else if (warp == EW) {  // products
    const uint32_t k0 = mma::smem_u32(sm), v0 = k0 + F::OWN, a0 = mma::smem_u32(ringA), b0 = mma::smem_u32(ringB);
    constexpr uint32_t id_s = idesc(BLK, XB, false), id_o = idesc(BLK, D, true);
    const uint32_t me = elect();
    auto pairs = [&](uint32_t d, uint32_t a, uint32_t b, uint64_t* bar) {
      prod_ss<D, PARTS, BLK, XB>(tm + d, a, b, id_s, me);
      commit(bar, me);
    };
    // (a thread's pairs, 32 H columns, are 16 H of bf16, second parts 16 H further, third at x3)
    auto apply = [&](auto tw, uint32_t d, uint32_t a, uint32_t x3, uint32_t b, bool acc) {
      using Q = Prod<PARTS>;
#pragma unroll
      for (int y = 0; y < Q::N; y++)
#pragma unroll
        for (int s = 0; s < XB / 16; s++)
          mma_ts(tm + d, tm + (Q::a(y) == 2 ? x3 + 8 * s : a + 32 * H * (s / (2 * H)) + 8 * (s % (2 * H)) + 16 * H * Q::a(y)),
                 desc_mn<XB>(b + Q::b(y) * (XB * D * 2), s), id_o, (PARTS == 1 && acc) || y > 0 || s > 0, me);
      if constexpr (decltype(tw)::value)
#pragma unroll
        for (int s = 0; s < XB / 16; s++)
          mma_ts(tm + d, tm + a + 32 * H * (s / (2 * H)) + 8 * (s % (2 * H)) + 16 * H, desc_mn<XB>(b, s), id_o, true, me);
    };
    // block x of queries (of their dO) has landed; rows behind its document's last are zeros
    auto ready = [&](int x, unsigned char* block, uint64_t* full, int phase) -> bool {
      const int left = t.Lq - (first + (t.j0 + x) % per) * XB;
      if (!wait(full, phase & 1, &B.dead)) return false;
      if (left < XB) zero_rows<D, XB, PARTS>(block, left);
      return true;
    };
    auto readyA = [&](int x) { return ready(x, ringA + x % F::NA * F::BYTES, &B.fullA[x % F::NA], x / F::NA); };
    auto readyB = [&](int x) { return ready(x, ringB + x % F::NB * F::BYTES, &B.fullB[x % F::NB], x / F::NB); };
    auto run = [&](auto tw) -> bool {
      if (!wait(&B.own, 0, &B.dead) || !readyA(0)) return false;
      pairs(cS, k0, a0, &B.s);
      if (!readyB(0)) return false;
      pairs(cDP, v0, b0, &B.dp);
      for (int x = 0; x < n; x++) {
        const uint32_t qb = a0 + x % F::NA * F::BYTES, qn = a0 + (x + 1) % F::NA * F::BYTES;
        const uint32_t gb = b0 + x % F::NB * F::BYTES, gn = b0 + (x + 1) % F::NB * F::BYTES;
        const bool more = x + 1 < n;
        if (!wait(&B.p, x & 1, &B.dead)) return false;
        tc::fence_after();
        apply(tw, cDV, cS, cX, gb, x > 0);
        commit(&B.emptyB[x % F::NB], me);
        if (more) {
          if (!readyA(x + 1)) return false;
          pairs(cS, k0, qn, &B.s);
        }
        if (!wait(&B.ds, x & 1, &B.dead)) return false;
        tc::fence_after();
        apply(tw, cDK, cDP, cX + XB / 2, qb, x > 0);
        commit(&B.emptyA[x % F::NA], me);
        if (more) {
          if (!readyB(x + 1)) return false;
          pairs(cDP, v0, gn, &B.dp);
        } else {
          commit(&B.done, me);
        }
      }
      return true;
    };
    if (n > 0 && !with_parts<PARTS>(twice, run)) {
      commit(&B.drain, me);
      for (int it = 0; it < mma::WAIT_POLLS && !mma::mbar_try(&B.drain, 0); it++) {}
    }
  } else if (warp < EW && live) {  // weights and their gradients: a thread a key, 32 H of a block's queries
    const int half = warp / 4, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    constexpr int W = 32 * H;  // a thread's columns of a block's pairs
    const uint32_t ts = tm + cS + W * half + lanes, td = tm + cDP + W * half + lanes;
    const uint32_t x3 = tm + cX + W / 2 * half + lanes;
    const int fq = first_query(P.causal, j0 + r, t.Lq, t.Lk), fq_last = first_query(P.causal, j0 + nk - 1, t.Lq, t.Lk);
    const uint64_t sc = two(P.scale2, P.scale2);
    float sv[PARTS == 3 ? 32 : 1] = {}, sk[PARTS == 3 ? 32 : 1] = {};  // (three parts) dv and dk, columns 32 half ..
    auto pairs = [&](auto tw) -> bool {
      for (int x = 0; x < n; x++) {
        const int s = x & 1, i0 = (first + (t.j0 + x) % per) * XB;
        const float *l2 = B.stat[s][0] + W * half, *dl = B.stat[s][1] + W * half;
        const bool cut = i0 < fq_last || i0 + XB > t.Lq;
        const int lo = fq - i0 - W * half, hi = t.Lq - i0 - W * half;
        float a[H][32];
        if (!wait(&B.fullS[s], (x >> 1) & 1, &B.dead) || !wait(&B.s, x & 1, &B.dead)) return false;
        tc::fence_after();
#pragma unroll
        for (int c = 0; c < H; c++) tm_ld32(ts + 32 * c, a[c]);
#pragma unroll
        for (int c = 0; c < H; c++) tm_wait_ld(a[c]);
#pragma unroll
        for (int c = 0; c < H; c++) bwd_weights(a[c], l2 + 32 * c, sc, cut, lo - 32 * c, hi - 32 * c);
        // (over logits of its own: the other half's warp may still read its)
        put_parts<PARTS, decltype(tw)::value, H>(a, ts, x3);
        if constexpr (PARTS == 3)
          if (x > 0) add_columns(sv, tm + cDV + 32 * half + lanes);  // (the block before's: issued before this S')
        tm_wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mma::mbar_arrive(&B.p);
        if (!wait(&B.dp, x & 1, &B.dead)) return false;
        tc::fence_after();
#pragma unroll
        for (int c = 0; c < H; c++) {
          float g[32];
          tm_ld32(td + 32 * c, g);
          tm_wait_ld(g);
          bwd_grads(a[c], g, dl + 32 * c, cut, lo - 32 * c, hi - 32 * c);
        }
        put_parts<PARTS, decltype(tw)::value, H>(a, td, x3 + XB / 2);
        if constexpr (PARTS == 3)
          if (x > 0) add_columns(sk, tm + cDK + 32 * half + lanes);
        tm_wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mma::mbar_arrive(&B.ds);
      }
      return true;
    };
    const bool keep = saved(P);
    bool ok = with_parts<PARTS>(twice, pairs);
    if (ok && n > 0) {
      ok = wait(&B.done, 0, &B.dead);
      tc::fence_after();
    }
    if (ok && keep) {
      const int w0 = r & ~31, c = PARTS == 3 ? 32 * half : 0;  // (the CTA's own blocks are no longer read)
      const size_t at = ((size_t)(t.k0 + j0 + w0) * P.Hkv + hk) * D + c, ld = (size_t)P.Hkv * D;
      unsigned char* buf = sm + half * HALF + w0 * 128;
      const size_t pa = (((size_t)t.piece * P.Hkv + hk) * BLK + w0) * D + c;  // (a piece's place)
      const size_t more = (size_t)P.pieces[2] * P.Hkv * BLK * D;
      if constexpr (PARTS == 3) {
        if (n > 0) {
          add_columns(sv, tm + cDV + c + lanes);
          add_columns(sk, tm + cDK + c + lanes);
        }
        const bool whole = t.piece < 0;
        store_sums(buf, sv, 1.0f, whole ? dv + at : P.po[2] + more + pa, whole ? ld : D, nk - w0);
        store_sums(buf, sk, whole ? P.scale : 1.0f, whole ? dk + at : P.po[2] + pa, whole ? ld : D, nk - w0);
      } else {
        for (int y = half; y < 2 * (D / 64); y += EW / 4) {  // 64 columns: dv's, then dk's
          const bool is_k = y >= D / 64;
          const int cy = 64 * (is_k ? y - D / 64 : y);
          const uint32_t from = tm + (is_k ? cDK : cDV) + cy + lanes;
          if (t.piece >= 0)
            store_acc_f32(buf, from, n > 0, P.po[2] + (is_k ? 0 : more) + pa + cy, D, nk - w0);
          else
            store_acc(buf, from, n > 0, is_k ? P.scale : 1.0f, (is_k ? dk : dv) + at + cy, ld, nk - w0);
        }
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && B.dead) *P.err = KDA_ERR_DEVICE;
  if (warp == EW) {
    tc::fence_after();
    tc::tmem_dealloc(tm, F::COLS);
  }
}

// dq, per CTA (its grid starts behind dk and dv's last CTAs and needs nothing of theirs): 128 queries of one head over
// the blocks of keys: S = q k^T, dP = dO v^T, dS = P (dP - delta), dq += dS k.
// S and dP are each taken to registers at once and formed anew for the next block meanwhile (one barrier for both left the
// tensor pipe idle until both were taken: large heads 1085 us, so 1027).  (bf16) q is an operand in tensor memory: with both
// of S's from shared memory the copies and products of a block of 128 keep that busy for 1792 cycles, the tensor pipe for
// 1536 (300M packed step 65.5 us, 67.5 without; at D = 128 the same).
struct DqBars {
  uint64_t own, loaded, fullA[7], emptyA[7], fullB[4], emptyB[4], s, dp, takenS, takenP, ds, used[2], drain;
  uint32_t tmem;
  int dead;
};

template <int D, int PARTS>
__global__ void __launch_bounds__(Bwd<D, PARTS>::EW * 32 + 64, Bwd<D, PARTS>::PER_SM)
smx_tc_dq_kernel(SmxP P, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mg,
                 const bf16* __restrict__ q, typename Io<PARTS>::T* __restrict__ dq) {
  using F = Bwd<D, PARTS>;
  constexpr int XB = F::XB, EW = F::EW, W = 4 * XB / EW, H = W / 32;  // (W: columns of a block's pairs a thread)
  constexpr uint32_t cS = 0, cDP = XB, cDQ = 2 * XB, nDQ = PARTS == 3 ? D : 0;         // (nDQ: columns to the other dq)
  constexpr uint32_t cDS = 2 * XB + D + nDQ, nDS = PARTS == 3 ? XB / 2 * PARTS : 0;    // (nDS: to the other dS)
  constexpr uint32_t cQ = cDS + XB / 2;                                                 // (PARTS = 1)
  extern __shared__ unsigned char raw[];
  __shared__ DqBars B;
  unsigned char* sm = raw + ((1024 - (mma::smem_u32(raw) & 1023)) & 1023);
  unsigned char *ringA = sm + F::QOWN, *ringB = ringA + F::QA * F::BYTES;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == EW) tc::tmem_alloc(&B.tmem, F::COLS);
  if (threadIdx.x == 32 * (EW + 1)) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
    prefetch_map(&mg);
  }
  if (threadIdx.x == 0) {
    mma::mbar_init(&B.own, 1);
    mma::mbar_init(&B.loaded, EW);
    for (int i = 0; i < F::QA; i++) {
      mma::mbar_init(&B.fullA[i], 1);
      mma::mbar_init(&B.emptyA[i], 1);
    }
    for (int i = 0; i < F::NB; i++) {
      mma::mbar_init(&B.fullB[i], 1);
      mma::mbar_init(&B.emptyB[i], 1);
    }
    mma::mbar_init(&B.s, 1);
    mma::mbar_init(&B.dp, 1);
    mma::mbar_init(&B.takenS, EW);
    mma::mbar_init(&B.takenP, EW);
    mma::mbar_init(&B.ds, EW);
    mma::mbar_init(&B.used[0], 1);
    mma::mbar_init(&B.used[1], 1);
    mma::mbar_init(&B.drain, 1);
    B.dead = 0;
    mma::mbar_init_fence();
  }
  Tile t;
  const int h = blockIdx.x % P.Hq, hk = h / P.G;
  const bool live = tile_of(P, 1, blockIdx.x / P.Hq, false, t);
  int i0 = 0, nq = 0, n = 0, clean = 0;
  bool twice = false;  // dS in two parts, the second ones over S
  if (live) {
    i0 = t.t * BLK;
    nq = min(BLK, t.Lq - i0);
    twice = PARTS == 1 && (t.Lq <= FEW_ROWS || t.Lk <= FEW);
    n = min((keys_of(P.causal, i0 + nq - 1, t.Lq, t.Lk) + XB - 1) / XB, t.j1) - t.j0;
    clean = keys_of(P.causal, i0, t.Lq, t.Lk) / XB;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = tm_base<F::COLS>(B.tmem);
  auto place = [](int x) { return PARTS == 3 ? x & 1 : 0; };  // of block x's dS

  if (warp == EW + 1) {  // copies
    if (lane == 0 && n > 0) {
      mma::mbar_expect_tx(&B.own, F::QOWN);
      load_block<D, BLK, PARTS>(sm, &mg, h, t.q0 + i0, P.Nq, &B.own);
      if (PARTS == 3) load_block<D, BLK, PARTS>(sm + F::OWN, &mq, h, t.q0 + i0, P.Nq, &B.own);
    }
    __syncwarp();
    for (int x = 0; x < n; x++) {
      const int sa = x % F::QA, sb = x % F::NB;
      if (x >= F::QA && !wait(&B.emptyA[sa], (x / F::QA - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullA[sa], F::BYTES);
        load_block<D, XB, PARTS>(ringA + sa * F::BYTES, &mk, hk, t.k0 + (t.j0 + x) * XB, P.Nk, &B.fullA[sa]);
      }
      __syncwarp();
      if (x >= F::NB && !wait(&B.emptyB[sb], (x / F::NB - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullB[sb], F::BYTES);
        load_block<D, XB, PARTS>(ringB + sb * F::BYTES, &mv, hk, t.k0 + (t.j0 + x) * XB, P.Nk, &B.fullB[sb]);
      }
      __syncwarp();
    }
  } else if (warp == EW) {  // products
    const uint32_t g0 = mma::smem_u32(sm), a0 = mma::smem_u32(ringA), b0 = mma::smem_u32(ringB);
    constexpr uint32_t id_s = idesc(BLK, XB, false), id_o = idesc(BLK, D, true);
    const uint32_t me = elect();
    auto logits = [&](int x) -> bool {
      const int left = t.Lk - (t.j0 + x) * XB;
      const uint32_t kb = a0 + x % F::QA * F::BYTES;
      if (!wait(&B.fullA[x % F::QA], (x / F::QA) & 1, &B.dead)) return false;
      if (left < XB) zero_rows<D, XB, PARTS>(ringA + x % F::QA * F::BYTES, left);
      if (x > 0 && !wait(&B.takenS, (x - 1) & 1, &B.dead)) return false;
      tc::fence_after();
      if constexpr (PARTS == 3) {
        prod_ss<D, PARTS, BLK, XB>(tm + cS, g0 + F::OWN, kb, id_s, me);
      } else {
#pragma unroll
        for (int s = 0; s < D / 16; s++) mma_ts(tm + cS, tm + cQ + 8 * s, desc_k<XB>(kb, s), id_s, s > 0, me);
      }
      commit(&B.s, me);
      return true;
    };
    auto grads = [&](int x) -> bool {
      if (!wait(&B.fullB[x % F::NB], (x / F::NB) & 1, &B.dead)) return false;
      if (x > 0 && !wait(&B.takenP, (x - 1) & 1, &B.dead)) return false;
      tc::fence_after();
      prod_ss<D, PARTS, BLK, XB>(tm + cDP, g0, b0 + x % F::NB * F::BYTES, id_s, me);
      commit(&B.dp, me);
      commit(&B.emptyB[x % F::NB], me);
      return true;
    };
    auto run = [&](auto tw) -> bool {
      if (!wait(&B.own, 0, &B.dead) || (PARTS == 1 && !wait(&B.loaded, 0, &B.dead))) return false;
      if (!logits(0) || !grads(0)) return false;
      for (int x = 0; x < n; x++) {
        auto next = [&]() { return x + 1 == n || (logits(x + 1) && grads(x + 1)); };
        if (!decltype(tw)::value && !next()) return false;
        if (!wait(&B.ds, x & 1, &B.dead)) return false;
        tc::fence_after();
        const uint32_t kb = a0 + x % F::QA * F::BYTES;
        using Q = Prod<PARTS>;
#pragma unroll
        for (int y = 0; y < Q::N; y++)
#pragma unroll
          for (int s = 0; s < XB / 16; s++)
            mma_ts(tm + cDQ + nDQ * (x & 1), tm + cDS + nDS * place(x) + XB / 2 * Q::a(y) + 8 * s,
                   desc_mn<XB>(kb + Q::b(y) * (XB * D * 2), s), id_o, (PARTS == 1 && x > 0) || y > 0 || s > 0, me);
        if constexpr (decltype(tw)::value)
#pragma unroll
          for (int s = 0; s < XB / 16; s++)
            mma_ts(tm + cDQ, tm + cS + W * (s / (W / 16)) + 8 * (s % (W / 16)), desc_mn<XB>(kb, s), id_o, true, me);
        commit(&B.used[place(x)], me);
        commit(&B.emptyA[x % F::QA], me);
        if (decltype(tw)::value && !next()) return false;
      }
      return true;
    };
    if (n > 0 && !with_parts<PARTS>(twice, run)) {
      commit(&B.drain, me);
      for (int it = 0; it < mma::WAIT_POLLS && !mma::mbar_try(&B.drain, 0); it++) {}
    }
  } else if (warp < EW && live) {  // a thread a query, 64 of a block's keys
    const int half = warp / 4, r = threadIdx.x & 127;
    const bool in = r < nq;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tm + cS + W * half + lanes, td = tm + cDP + W * half + lanes;
    const int lim = in ? keys_of(P.causal, i0 + r, t.Lq, t.Lk) : 0;
    const size_t at = (size_t)h * P.Nq + t.q0 + i0 + r;
    const float nl = in ? -P.lse2[at] : 0.f, nd = in ? -P.delta[at] : 0.f;
    const uint64_t sc = two(P.scale2, P.scale2), l2 = two(nl, nl), dl = two(nd, nd);
    float sum[PARTS == 3 ? 64 : 1] = {};  // (three parts) dq
    if constexpr (PARTS == 1) {  // the row's q, W of its values a thread (zeros behind the document's end)
      const bf16* row = q + ((size_t)(t.q0 + i0 + r) * P.Hq + h) * D + W * half;
#pragma unroll
      for (int c = 0; c < H; c++) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const uint4 u = in ? *reinterpret_cast<const uint4*>(row + 32 * c + 8 * e) : make_uint4(0, 0, 0, 0);
          w[4 * e] = u.x, w[4 * e + 1] = u.y, w[4 * e + 2] = u.z, w[4 * e + 3] = u.w;
        }
        tm_st16(tm + cQ + W / 2 * half + 16 * c + lanes, w);
      }
      tm_wait_st();
      arrive(&B.loaded);
    }
    auto pairs = [&](auto tw) -> bool {
      constexpr bool TW = decltype(tw)::value;
      for (int x = 0; x < n; x++) {
        if (!wait(&B.s, x & 1, &B.dead)) return false;
        tc::fence_after();
        float a[H][32], g[H][32];
#pragma unroll
        for (int c = 0; c < H; c++) tm_ld32(ts + 32 * c, a[c]);
#pragma unroll
        for (int c = 0; c < H; c++) tm_wait_ld(a[c]);
        arrive(&B.takenS);
#pragma unroll
        for (int c = 0; c < H; c++) dq_weights(a[c], sc, l2);
        if (!wait(&B.dp, x & 1, &B.dead)) return false;
        tc::fence_after();
#pragma unroll
        for (int c = 0; c < H; c++) tm_ld32(td + 32 * c, g[c]);
#pragma unroll
        for (int c = 0; c < H; c++) tm_wait_ld(g[c]);
        arrive(&B.takenP);
        const int left = lim - (t.j0 + x) * XB - W * half;
        const bool cut = t.j0 + x >= clean;
#pragma unroll
        for (int c = 0; c < H; c++) dq_grads(a[c], g[c], dl, cut, left - 32 * c);
        if (x >= (PARTS == 3 ? 2 : 1)) {
          if (!wait(&B.used[place(x)], ((PARTS == 3 ? x / 2 : x) - 1) & 1, &B.dead)) return false;
          tc::fence_after();
          if constexpr (PARTS == 3) add_columns(sum, tm + cDQ + nDQ * (x & 1) + lanes);  // (block x - 2's)
        }
        const uint32_t to = tm + cDS + nDS * place(x) + W / 2 * half + lanes;
        put_dq<PARTS, TW, XB, H>(a, to, ts);
        tm_wait_st();
        arrive(&B.ds);
      }
      if (n > 0 && !wait(&B.used[place(n - 1)], (PARTS == 3 ? (n - 1) / 2 : n - 1) & 1, &B.dead)) return false;
      tc::fence_after();
      return true;
    };
    const bool keep = saved(P);
    const bool ok = with_parts<PARTS>(twice, pairs);
    if (ok && keep && half < D / 64) {
      const int w0 = r & ~31, c = 64 * half;
      unsigned char* buf = sm + half * HALF + w0 * 128;
      const size_t to = ((size_t)(t.q0 + i0 + w0) * P.Hq + h) * D + c, ld = (size_t)P.Hq * D;
      const size_t pa = (((size_t)t.piece * P.Hq + h) * BLK + w0) * D + c;  // (a piece's place)
      if constexpr (PARTS == 3) {
        for (int x = max(0, n - 2); x < n; x++) add_columns(sum, tm + cDQ + nDQ * (x & 1) + lanes);
        const bool whole = t.piece < 0;
        store_sums(buf, sum, whole ? P.scale : 1.0f, whole ? dq + to : P.po[1] + pa, whole ? ld : D, nq - w0);
      } else if (t.piece >= 0) {
        store_acc_f32(buf, tm + cDQ + c + lanes, n > 0, P.po[1] + pa, D, nq - w0);
      } else {
        store_acc(buf, tm + cDQ + c + lanes, n > 0, P.scale, dq + to, ld, nq - w0);
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && B.dead) *P.err = KDA_ERR_DEVICE;
  if (warp == EW) {
    tc::fence_after();
    tc::tmem_dealloc(tm, F::COLS);
  }
  pdl_wait();  // (what follows this grid follows dk and dv too)
}

template <int D, int PARTS>
cudaError_t bwd(const SmxP& P, const void* q, const void* k, const void* v, const void* dO, void* dq, void* dk,
                void* dv, cudaStream_t st) {
  using F = Bwd<D, PARTS>;
  using T = typename Io<PARTS>::T;
  cudaError_t e = raise_smem<smx_tc_dkv_kernel<D, PARTS>>(DKV_SMEM<D, PARTS>);
  if (e == cudaSuccess) e = raise_smem<smx_tc_dq_kernel<D, PARTS>>(F::BLOCKS + 1024);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv, mg, xq, xk, xv, xg;  // blocks of 128 rows, and of the other side's XB
  const int nq = PARTS * P.Nq, nk = PARTS * P.Nk;
  if (!encode_head_rows(&mq, q, nq, P.Hq, D, BLK) || !encode_head_rows(&mk, k, nk, P.Hkv, D, BLK) ||
      !encode_head_rows(&mv, v, nk, P.Hkv, D, BLK) || !encode_head_rows(&mg, dO, nq, P.Hq, D, BLK))
    return cudaErrorInvalidValue;
  xq = mq, xk = mk, xv = mv, xg = mg;
  if (F::XB != BLK && (!encode_head_rows(&xq, q, nq, P.Hq, D, F::XB) || !encode_head_rows(&xk, k, nk, P.Hkv, D, F::XB) ||
                       !encode_head_rows(&xv, v, nk, P.Hkv, D, F::XB) || !encode_head_rows(&xg, dO, nq, P.Hq, D, F::XB)))
    return cudaErrorInvalidValue;
  const int64_t gk = (int64_t)max_tiles(P, 2) * P.Hkv, gq = (int64_t)max_tiles(P, 1) * P.Hq;
  prof_begin(K_SMX_DKV, st);
  e = launch_pdl(smx_tc_dkv_kernel<D, PARTS>, dim3((unsigned)gk), dim3(F::EWK * 32 + 96), DKV_SMEM<D, PARTS>, st, P, xq, mk, mv, xg, (T*)dk,
                 (T*)dv);
  prof_end(K_SMX_DKV, st);
  if (e != cudaSuccess) return e;
  prof_begin(K_SMX_DQ, st);
  e = launch_pdl(smx_tc_dq_kernel<D, PARTS>, dim3((unsigned)gq), dim3(F::EW * 32 + 64), F::BLOCKS + 1024, st, P, mq, xk,
                 xv, mg, (const bf16*)q, (T*)dq);
  prof_end(K_SMX_DQ, st);
  return e;
}

// ------------------------------------------------------------ fp32 io: the parts
// Array y of up to three: its 8 n_y values as three bf16 arrays one behind the other.
struct Split {
  const float* x[3];
  bf16* parts[3];
  int64_t n[3];
};
__global__ void __launch_bounds__(256) smx_split_kernel(Split s) {
  pdl_wait();
  pdl_release();
  const int y = blockIdx.y;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < s.n[y]; i += (int64_t)gridDim.x * 256) {
    float v[8];
#pragma unroll
    for (int c = 0; c < 2; c++) {
      const float4 f = *reinterpret_cast<const float4*>(s.x[y] + 8 * i + 4 * c);
      v[4 * c] = f.x; v[4 * c + 1] = f.y; v[4 * c + 2] = f.z; v[4 * c + 3] = f.w;
    }
#pragma unroll
    for (int p = 0; p < 3; p++) {
      uint32_t w[4];
      next_part(v, w);
      *reinterpret_cast<uint4*>(s.parts[y] + 8 * (p * s.n[y] + i)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace

cudaError_t launch_tc_fwd(const SmxP& P, int D, int parts, const void* q, const void* k, const void* v, void* o,
                          float* lse, cudaStream_t st) {
  if (parts == 3) return D == 64 ? fwd<64, 3>(P, q, k, v, o, lse, st) : fwd<128, 3>(P, q, k, v, o, lse, st);
  return D == 64 ? fwd<64, 1>(P, q, k, v, o, lse, st) : fwd<128, 1>(P, q, k, v, o, lse, st);
}
cudaError_t launch_tc_bwd(const SmxP& P, int D, int parts, const void* q, const void* k, const void* v, const void* dO,
                          void* dq, void* dk, void* dv, cudaStream_t st) {
  if (parts == 3) return bwd<64, 3>(P, q, k, v, dO, dq, dk, dv, st);
  return D == 64 ? bwd<64, 1>(P, q, k, v, dO, dq, dk, dv, st) : bwd<128, 1>(P, q, k, v, dO, dq, dk, dv, st);
}
cudaError_t launch_split(int n, const float* const* x, bf16* const* parts, const int64_t* values, cudaStream_t st) {
  Split s = {};
  int64_t most = 0;
  for (int y = 0; y < n; y++) {
    s.x[y] = x[y];
    s.parts[y] = parts[y];
    s.n[y] = values[y] / 8;
    if (s.n[y] > most) most = s.n[y];
  }
  const int64_t grid = (most + 255) / 256;
  prof_begin(K_SMX_SPLIT, st);
  const cudaError_t e = launch_pdl(smx_split_kernel, dim3((unsigned)(grid < 16384 ? grid : 16384), n), dim3(256), 0, st, s);
  prof_end(K_SMX_SPLIT, st);
  return e;
}

}  // namespace smx
}  // namespace kda
