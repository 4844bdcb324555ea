// Softmax attention, the backward of fp32 io at D = 128 on the 5th-generation tensor cores, every operand as three bf16
// parts (the other passes: kda_softmax_tc.cu).  Per document, query head h and its key head h / G:
//   p_ij = exp(scale q_i k_j - lse_i),  dv_j = sum_i p_ij dO_i
//   ds_ij = p_ij (dO_i v_j - delta_i),  delta_i = o_i dO_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
// Both own blocks of 128 rows would fill shared memory (96 KB each): one lies there, the other in tensor memory (192 of
// its 512 columns), where a product can take its first operand from too.  That leaves room for a ring of blocks of 32
// rows of the other side, and 128 columns for one result: dv and dk of a block take turns in it, and their sums over the
// blocks are in registers, where they are rounded (the tensor pipe cuts its sums off).
// Eight warps, a thread a row and half of a block's pairs, of a result's columns, and of an own row to tensor memory.
// Bound by the tensor pipe: six products a product, and the first operand's reads (128 x 16 values for 32 columns: 32
// cycles, so 16 of arithmetic).  4 x 1001 rows of 8 heads, every pair seen: 559 us with the forward; on the fp32
// pipe, 64 x 64 pairs a CTA, 2105.  (16 warps would halve a thread's 128 sums of dk and dv and have too few registers for
// them; eight spill 220 bytes, a few loads a block.)
#include "kda_softmax_tc.cuh"

namespace kda {
namespace smx {
namespace {

constexpr int D = 128, XB = 32, EW = 8;                         // rows of the other side's blocks; warps of the pairs
constexpr int OWN = BLK * D * 2 * 3, BYTES = XB * D * 2 * 3;    // a block of three parts, of either side
constexpr int NA = 3, NB = 2, BLOCKS = OWN + NA * BYTES + NB * BYTES;
constexpr int PART = XB / 2;                                    // columns of one part of a block's pairs as an operand
constexpr uint32_t ID_S = idesc(BLK, XB, false), ID_O = idesc(BLK, D, true);

struct Bars {
  float stat[NA][2][XB];  // minus lse2 and minus delta of ring A's queries
  uint64_t own, loaded, fullA[NA], emptyA[NA], fullB[NB], emptyB[NB], fullS[NA], s, dp, p, ds, taken, first, second, drain;
  uint32_t tmem;
  int dead;
};
constexpr int SMEM = BLOCKS + (int)sizeof(Bars);
static_assert(SMEM <= 232448, "shared memory of a CTA");

// An own row's half (64 values, three parts `stride` values apart) to tensor memory; zeros behind the document's end.
__device__ __forceinline__ void load_own(uint32_t to, const bf16* row, size_t stride, bool in) {
#pragma unroll
  for (int y = 0; y < 3; y++)
#pragma unroll
    for (int c = 0; c < 2; c++) {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const uint4 u = in ? *reinterpret_cast<const uint4*>(row + y * stride + 32 * c + 8 * e) : make_uint4(0, 0, 0, 0);
        w[4 * e] = u.x, w[4 * e + 1] = u.y, w[4 * e + 2] = u.z, w[4 * e + 3] = u.w;
      }
      tm_st16(to + D / 2 * y + 16 * c, w);
    }
  tm_wait_st();
}
// 16 pairs of a row as an operand's three parts
__device__ __forceinline__ void put(float (&v)[16], uint32_t to) {
#pragma unroll
  for (int y = 0; y < 3; y++) {
    uint32_t w[8];
    next_part(v, w);
    tm_st8(to + PART * y, w);
  }
  tm_wait_st();
}
// d = A B^T, A's three parts in tensor memory, B a block, K-major
__device__ __forceinline__ void prod_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t me) {
  using Q = Prod<3>;
#pragma unroll
  for (int i = 0; i < Q::N; i++)
#pragma unroll
    for (int s = 0; s < D / 16; s++)
      mma_ts(d, a + D / 2 * Q::a(i) + 8 * s, desc_k<XB>(b + Q::b(i) * (XB * D * 2), s), ID_S, i > 0 || s > 0, me);
}
// d = pairs B over a block's rows
__device__ __forceinline__ void apply(uint32_t d, uint32_t a, uint32_t b, uint32_t me) {
  using Q = Prod<3>;
#pragma unroll
  for (int i = 0; i < Q::N; i++)
#pragma unroll
    for (int s = 0; s < XB / 16; s++)
      mma_ts(d, a + PART * Q::a(i) + 8 * s, desc_mn<XB>(b + Q::b(i) * (XB * D * 2), s), ID_O, i > 0 || s > 0, me);
}
__device__ __forceinline__ void init(Bars& B) {
  mma::mbar_init(&B.own, 1);
  mma::mbar_init(&B.loaded, EW);
  for (int i = 0; i < NA; i++) {
    mma::mbar_init(&B.fullA[i], 1);
    mma::mbar_init(&B.emptyA[i], 1);
    mma::mbar_init(&B.fullS[i], 1);
  }
  for (int i = 0; i < NB; i++) {
    mma::mbar_init(&B.fullB[i], 1);
    mma::mbar_init(&B.emptyB[i], 1);
  }
  mma::mbar_init(&B.s, 1);
  mma::mbar_init(&B.dp, 1);
  mma::mbar_init(&B.p, EW);
  mma::mbar_init(&B.ds, EW);
  mma::mbar_init(&B.taken, EW);
  mma::mbar_init(&B.first, 1);
  mma::mbar_init(&B.second, 1);
  mma::mbar_init(&B.drain, 1);
  B.dead = 0;
  mma::mbar_init_fence();
}
// (16 columns at a time: 128 sums a thread of dk and dv leave few registers)
__device__ __forceinline__ void add(float (&sum)[64], uint32_t tm) {
#pragma unroll
  for (int c = 0; c < 64; c += 16) {
    float v[16];
    tm_ld16(tm + c, v);
    tm_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 16; e++) sum[c + e] += v[e];
  }
}
// dk and dv of 128 keys of one key head, over the blocks of its group's queries; the pairs transposed, a key a lane.
// Products in the order S'(x + 1), dv(x), dP'(x + 1), dk(x): while two run, the weights and gradients of the others form.
__global__ void __launch_bounds__(EW * 32 + 64, 1)
smx_f32_dkv_kernel(SmxP P, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mg, float* __restrict__ dk, float* __restrict__ dv) {
  constexpr uint32_t cS = 0, cDP = XB, cP = 2 * XB, cDS = cP + 3 * PART, cO = cDS + 3 * PART, cV = cO + D;
  static_assert(cV + 3 * (D / 2) <= 512, "tensor memory");
  extern __shared__ __align__(1024) unsigned char sm[];
  Bars& B = *reinterpret_cast<Bars*>(sm + BLOCKS);
  if (mma::smem_u32(sm) & 1023) {  // (dynamic shared memory alone starts on such a boundary)
    if (blockIdx.x == 0 && threadIdx.x == 0) *P.err = KDA_ERR_DEVICE;
    return;
  }
  unsigned char *ringA = sm + OWN, *ringB = ringA + NA * BYTES;  // q, dO
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == EW) tc::tmem_alloc(&B.tmem, 512);
  if (threadIdx.x == 32 * (EW + 1)) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mg);
  }
  if (threadIdx.x == 0) init(B);
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
  const int n = live ? min(per * P.G, t.j1) - t.j0 : 0;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = tm_base<512>(B.tmem);

  if (warp == EW + 1) {  // copies, and the queries' row sums
    if (lane == 0 && n > 0) {
      mma::mbar_expect_tx(&B.own, OWN);
      load_block<D, BLK, 3>(sm, &mk, hk, t.k0 + j0, P.Nk, &B.own);
    }
    __syncwarp();
    for (int x = 0; x < n; x++) {
      const int sa = x % NA, sb = x % NB, y = t.j0 + x, h = hk * P.G + y / per, i0 = (first + y % per) * XB, row = t.q0 + i0;
      if (x >= NA && !wait(&B.emptyA[sa], (x / NA - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullA[sa], BYTES);
        load_block<D, XB, 3>(ringA + sa * BYTES, &mq, h, row, P.Nq, &B.fullA[sa]);
      }
      const bool in = i0 + lane < t.Lq;
      const size_t at = (size_t)h * P.Nq + row + lane;
      B.stat[sa][0][lane] = in ? -P.lse2[at] : 0.f;
      B.stat[sa][1][lane] = in ? -P.delta[at] : 0.f;
      __syncwarp();
      if (lane == 0) mma::mbar_arrive(&B.fullS[sa]);
      if (x >= NB && !wait(&B.emptyB[sb], (x / NB - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullB[sb], BYTES);
        load_block<D, XB, 3>(ringB + sb * BYTES, &mg, h, row, P.Nq, &B.fullB[sb]);
      }
      __syncwarp();
    }
    // (a wait gives up after a second: by then every copy under way has landed)
  } else if (warp == EW) {  // products
    const uint32_t k0 = mma::smem_u32(sm), a0 = mma::smem_u32(ringA), b0 = mma::smem_u32(ringB);
    const uint32_t me = elect();
    // block x of queries (of their dO) has landed; rows behind its document's last are zeros
    auto ready = [&](int x, unsigned char* block, uint64_t* full, int phase) -> bool {
      const int left = t.Lq - (first + (t.j0 + x) % per) * XB;
      if (!wait(full, phase & 1, &B.dead)) return false;
      if (left < XB) zero_rows<D, XB, 3>(block, left);
      return true;
    };
    auto readyA = [&](int x) { return ready(x, ringA + x % NA * BYTES, &B.fullA[x % NA], x / NA); };
    auto readyB = [&](int x) { return ready(x, ringB + x % NB * BYTES, &B.fullB[x % NB], x / NB); };
    auto logits = [&](int x) {
      prod_ss<D, 3, BLK, XB>(tm + cS, k0, a0 + x % NA * BYTES, ID_S, me);
      commit(&B.s, me);
    };
    auto grads = [&](int x) {
      prod_ts(tm + cDP, tm + cV, b0 + x % NB * BYTES, me);
      commit(&B.dp, me);
    };
    auto run = [&]() -> bool {
      if (!wait(&B.own, 0, &B.dead) || !readyA(0)) return false;
      logits(0);
      if (!readyB(0) || !wait(&B.loaded, 0, &B.dead)) return false;
      tc::fence_after();
      grads(0);
      for (int x = 0; x < n; x++) {
        const bool more = x + 1 < n;
        if (!wait(&B.p, x & 1, &B.dead)) return false;
        tc::fence_after();
        if (more) {
          if (!readyA(x + 1)) return false;
          logits(x + 1);
        }
        if (!wait(&B.ds, x & 1, &B.dead)) return false;  // (and dk of block x - 1 is taken)
        tc::fence_after();
        apply(tm + cO, tm + cP, b0 + x % NB * BYTES, me);
        commit(&B.first, me);
        commit(&B.emptyB[x % NB], me);
        if (more) {
          if (!readyB(x + 1)) return false;
          grads(x + 1);
        }
        if (!wait(&B.taken, x & 1, &B.dead)) return false;
        tc::fence_after();
        apply(tm + cO, tm + cDS, a0 + x % NA * BYTES, me);
        commit(&B.second, me);
        commit(&B.emptyA[x % NA], me);
      }
      return true;
    };
    if (n > 0 && !run()) {
      commit(&B.drain, me);
      for (int it = 0; it < mma::WAIT_POLLS && !mma::mbar_try(&B.drain, 0); it++) {}
    }
  } else if (warp < EW && live) {
    const int half = warp / 4, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t out = tm + cO + 64 * half + lanes;
    const int fq = first_query(P.causal, j0 + r, t.Lq, t.Lk), fq_last = first_query(P.causal, j0 + nk - 1, t.Lq, t.Lk);
    const uint64_t sc = two(P.scale2, P.scale2);
    float sv[64] = {}, sk[64] = {};  // dv and dk, columns 64 half ..
    load_own(tm + cV + 32 * half + lanes, P.pv + ((size_t)(t.k0 + j0 + r) * P.Hkv + hk) * D + 64 * half,
             (size_t)P.Nk * P.Hkv * D, r < nk);
    arrive(&B.loaded);
    const bool keep = saved(P);
    bool ok = true;
    for (int x = 0; x < n; x++) {
      const int s = x % NA, i0 = (first + (t.j0 + x) % per) * XB;
      const float *l2 = B.stat[s][0] + 16 * half, *dl = B.stat[s][1] + 16 * half;
      const bool cut = i0 < fq_last || i0 + XB > t.Lq;
      const int lo = fq - i0 - 16 * half, hi = t.Lq - i0 - 16 * half;
      float a[16], g[16];
      ok = wait(&B.fullS[s], (x / NA) & 1, &B.dead) && wait(&B.s, x & 1, &B.dead);
      if (!ok) break;
      tc::fence_after();
      tm_ld16(tm + cS + 16 * half + lanes, a);
      tm_wait_ld(a);
      bwd_weights(a, l2, sc, cut, lo, hi);
#pragma unroll
      for (int e = 0; e < 16; e++) g[e] = a[e];
      put(g, tm + cP + 8 * half + lanes);
      arrive(&B.p);
      ok = wait(&B.dp, x & 1, &B.dead);
      if (!ok) break;
      tc::fence_after();
      tm_ld16(tm + cDP + 16 * half + lanes, g);
      tm_wait_ld(g);
      bwd_grads(a, g, dl, cut, lo, hi);
      if (x > 0) {
        ok = wait(&B.second, (x - 1) & 1, &B.dead);
        if (!ok) break;
        tc::fence_after();
        add(sk, out);
      }
      put(a, tm + cDS + 8 * half + lanes);
      arrive(&B.ds);
      ok = wait(&B.first, x & 1, &B.dead);
      if (!ok) break;
      tc::fence_after();
      add(sv, out);
      arrive(&B.taken);
    }
    if (ok && n > 0) {
      ok = wait(&B.second, (n - 1) & 1, &B.dead);
      tc::fence_after();
      if (ok) add(sk, out);
    }
    if (ok && keep) {
      const int w0 = r & ~31, c = 64 * half;  // (the CTA's own block is no longer read)
      const bool whole = t.piece < 0;
      const size_t at = ((size_t)(t.k0 + j0 + w0) * P.Hkv + hk) * D + c, ld = whole ? (size_t)P.Hkv * D : D;
      const size_t pa = (((size_t)t.piece * P.Hkv + hk) * BLK + w0) * D + c;  // (a piece's place)
      const size_t more = (size_t)P.pieces[2] * P.Hkv * BLK * D;
      unsigned char* buf = sm + half * HALF + w0 * 128;
      store_sums(buf, sv, 1.0f, whole ? dv + at : P.po[2] + more + pa, ld, nk - w0);
      store_sums(buf, sk, whole ? P.scale : 1.0f, whole ? dk + at : P.po[2] + pa, ld, nk - w0);
    }
    tc::fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && B.dead) *P.err = KDA_ERR_DEVICE;
  if (warp == EW) {
    tc::fence_after();
    tc::tmem_dealloc(tm, 512);
  }
}

// dq of 128 queries of one head, over the blocks of keys.  S and dP are taken to registers at once, so that the next
// block's products run while dS is formed and the block before's dq is added.
__global__ void __launch_bounds__(EW * 32 + 64, 1)
smx_f32_dq_kernel(SmxP P, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, float* __restrict__ dq) {
  constexpr uint32_t cS = 0, cDP = XB, cDS = 2 * XB, cDQ = cDS + 3 * PART, cG = cDQ + D;
  static_assert(cG + 3 * (D / 2) <= 512, "tensor memory");
  extern __shared__ __align__(1024) unsigned char sm[];
  Bars& B = *reinterpret_cast<Bars*>(sm + BLOCKS);
  struct Last {  // what follows this grid follows dk and dv too
    __device__ ~Last() { pdl_wait(); }
  } last;
  if (mma::smem_u32(sm) & 1023) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *P.err = KDA_ERR_DEVICE;
    return;
  }
  unsigned char *ringA = sm + OWN, *ringB = ringA + NA * BYTES;  // k, v
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == EW) tc::tmem_alloc(&B.tmem, 512);
  if (threadIdx.x == 32 * (EW + 1)) {
    prefetch_map(&mq);
    prefetch_map(&mk);
    prefetch_map(&mv);
  }
  if (threadIdx.x == 0) init(B);
  Tile t;
  const int h = blockIdx.x % P.Hq, hk = h / P.G;
  const bool live = tile_of(P, 1, blockIdx.x / P.Hq, false, t);
  int i0 = 0, nq = 0, n = 0, clean = 0;
  if (live) {
    i0 = t.t * BLK;
    nq = min(BLK, t.Lq - i0);
    n = min((keys_of(P.causal, i0 + nq - 1, t.Lq, t.Lk) + XB - 1) / XB, t.j1) - t.j0;
    clean = keys_of(P.causal, i0, t.Lq, t.Lk) / XB;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = tm_base<512>(B.tmem);

  if (warp == EW + 1) {  // copies
    if (lane == 0 && n > 0) {
      mma::mbar_expect_tx(&B.own, OWN);
      load_block<D, BLK, 3>(sm, &mq, h, t.q0 + i0, P.Nq, &B.own);
    }
    __syncwarp();
    for (int x = 0; x < n; x++) {
      const int sa = x % NA, sb = x % NB, row = t.k0 + (t.j0 + x) * XB;
      if (x >= NA && !wait(&B.emptyA[sa], (x / NA - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullA[sa], BYTES);
        load_block<D, XB, 3>(ringA + sa * BYTES, &mk, hk, row, P.Nk, &B.fullA[sa]);
      }
      __syncwarp();
      if (x >= NB && !wait(&B.emptyB[sb], (x / NB - 1) & 1, &B.dead)) break;
      if (lane == 0) {
        mma::mbar_expect_tx(&B.fullB[sb], BYTES);
        load_block<D, XB, 3>(ringB + sb * BYTES, &mv, hk, row, P.Nk, &B.fullB[sb]);
      }
      __syncwarp();
    }
  } else if (warp == EW) {  // products
    const uint32_t q0 = mma::smem_u32(sm), a0 = mma::smem_u32(ringA), b0 = mma::smem_u32(ringB);
    const uint32_t me = elect();
    auto pairs = [&](int x) {
      prod_ss<D, 3, BLK, XB>(tm + cS, q0, a0 + x % NA * BYTES, ID_S, me);
      prod_ts(tm + cDP, tm + cG, b0 + x % NB * BYTES, me);
      commit(&B.s, me);
      commit(&B.emptyB[x % NB], me);
    };
    auto ready = [&](int x) -> bool {
      const int left = t.Lk - (t.j0 + x) * XB;
      if (!wait(&B.fullA[x % NA], (x / NA) & 1, &B.dead)) return false;
      if (left < XB) zero_rows<D, XB, 3>(ringA + x % NA * BYTES, left);
      return wait(&B.fullB[x % NB], (x / NB) & 1, &B.dead);
    };
    auto run = [&]() -> bool {
      if (!wait(&B.own, 0, &B.dead) || !ready(0) || !wait(&B.loaded, 0, &B.dead)) return false;
      tc::fence_after();
      pairs(0);
      for (int x = 0; x < n; x++) {
        if (x + 1 < n) {
          if (!ready(x + 1) || !wait(&B.taken, x & 1, &B.dead)) return false;
          tc::fence_after();
          pairs(x + 1);
        }
        if (!wait(&B.ds, x & 1, &B.dead)) return false;
        tc::fence_after();
        apply(tm + cDQ, tm + cDS, a0 + x % NA * BYTES, me);
        commit(&B.first, me);
        commit(&B.emptyA[x % NA], me);
      }
      return true;
    };
    if (n > 0 && !run()) {
      commit(&B.drain, me);
      for (int it = 0; it < mma::WAIT_POLLS && !mma::mbar_try(&B.drain, 0); it++) {}
    }
  } else if (warp < EW && live) {
    const int half = warp / 4, r = threadIdx.x & 127;
    const bool in = r < nq;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t out = tm + cDQ + 64 * half + lanes;
    const int lim = in ? keys_of(P.causal, i0 + r, t.Lq, t.Lk) : 0;
    const size_t at = (size_t)h * P.Nq + t.q0 + i0 + r;
    const float nl = in ? -P.lse2[at] : 0.f, nd = in ? -P.delta[at] : 0.f;
    const uint64_t sc = two(P.scale2, P.scale2), l2 = two(nl, nl), dl = two(nd, nd);
    float sum[64] = {};
    load_own(tm + cG + 32 * half + lanes, P.pg + ((size_t)(t.q0 + i0 + r) * P.Hq + h) * D + 64 * half,
             (size_t)P.Nq * P.Hq * D, in);
    arrive(&B.loaded);
    const bool keep = saved(P);
    bool ok = true;
    for (int x = 0; x < n; x++) {
      ok = wait(&B.s, x & 1, &B.dead);
      if (!ok) break;
      tc::fence_after();
      float a[16], g[16];
      tm_ld16(tm + cS + 16 * half + lanes, a);
      tm_ld16(tm + cDP + 16 * half + lanes, g);
      tm_wait_ld(a);
      tm_wait_ld(g);
      arrive(&B.taken);
      dq_weights(a, sc, l2);
      dq_grads(a, g, dl, t.j0 + x >= clean, lim - (t.j0 + x) * XB - 16 * half);
      if (x > 0) {
        ok = wait(&B.first, (x - 1) & 1, &B.dead);
        if (!ok) break;
        tc::fence_after();
        add(sum, out);
      }
      put(a, tm + cDS + 8 * half + lanes);
      arrive(&B.ds);
    }
    if (ok && n > 0) {
      ok = wait(&B.first, (n - 1) & 1, &B.dead);
      tc::fence_after();
      if (ok) add(sum, out);
    }
    if (ok && keep) {
      const int w0 = r & ~31, c = 64 * half;
      const bool whole = t.piece < 0;
      const size_t to = ((size_t)(t.q0 + i0 + w0) * P.Hq + h) * D + c;
      const size_t pa = (((size_t)t.piece * P.Hq + h) * BLK + w0) * D + c;  // (a piece's place)
      store_sums(sm + half * HALF + w0 * 128, sum, whole ? P.scale : 1.0f, whole ? dq + to : P.po[1] + pa,
                 whole ? (size_t)P.Hq * D : D, nq - w0);
    }
    tc::fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && B.dead) *P.err = KDA_ERR_DEVICE;
  if (warp == EW) {
    tc::fence_after();
    tc::tmem_dealloc(tm, 512);
  }
}

}  // namespace

cudaError_t launch_f32_bwd(const SmxP& P, float* dq, float* dk, float* dv, cudaStream_t st) {
  cudaError_t e = raise_smem<smx_f32_dkv_kernel>(SMEM);
  if (e == cudaSuccess) e = raise_smem<smx_f32_dq_kernel>(SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, xq, xg, xk, xv;  // own blocks of 128 rows, the other side's of 32
  const int nq = 3 * P.Nq, nk = 3 * P.Nk;
  if (!encode_head_rows(&mq, P.pq, nq, P.Hq, D, BLK) || !encode_head_rows(&mk, P.pk, nk, P.Hkv, D, BLK) ||
      !encode_head_rows(&xq, P.pq, nq, P.Hq, D, XB) || !encode_head_rows(&xg, P.pg, nq, P.Hq, D, XB) ||
      !encode_head_rows(&xk, P.pk, nk, P.Hkv, D, XB) || !encode_head_rows(&xv, P.pv, nk, P.Hkv, D, XB))
    return cudaErrorInvalidValue;
  const int64_t gk = (int64_t)max_tiles(P, 2) * P.Hkv, gq = (int64_t)max_tiles(P, 1) * P.Hq;
  prof_begin(K_SMX_DKV, st);
  e = launch_pdl(smx_f32_dkv_kernel, dim3((unsigned)gk), dim3(EW * 32 + 64), SMEM, st, P, xq, mk, xg, dk, dv);
  prof_end(K_SMX_DKV, st);
  if (e != cudaSuccess) return e;
  prof_begin(K_SMX_DQ, st);
  e = launch_pdl(smx_f32_dq_kernel, dim3((unsigned)gq), dim3(EW * 32 + 64), SMEM, st, P, mq, xk, xv, dq);
  prof_end(K_SMX_DQ, st);
  return e;
}

}  // namespace smx
}  // namespace kda
