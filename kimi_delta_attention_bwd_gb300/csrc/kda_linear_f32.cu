// The fp32 chain of linear attention (kda_linear.cu has the mathematics).
// Every operand is three bf16 parts (24 bits) and every product the six part
// products of order 2^-16 and above, on tcgen05 (M = 64, operands in shared
// memory, accumulators in TMEM): three parts of everything would not fit the
// registers of the bf16 chain.  A CTA carries one chain of a value slice of 64
// columns (32 where shared memory or the head has no more): its state in fp32
// registers, warp w with rows (value columns) 16 (w % 4) .. and the key columns
// of half w / 4.  Small part products are accumulated first: the tensor core
// truncates what an addition shifts out.
// Bound by the chunk's chain of dependent steps (loads and splits, pairs, their
// product), at one CTA per SM in most shapes: so the entry state's rows and the
// state's product run while the pairs are weighted, and the next chunk's tiles
// are under way to registers meanwhile (4 x 1001 tokens, H 8, 64/64, forward and
// backward: 196 us with every product waited for and tiles loaded between, 153 to
// 158 so; a prompt of 16 x 2048, H 8, 32/64: 158 us).
#include "kda_linear.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace lin {
namespace {

constexpr int LTH = 256;  // threads of a chain CTA
constexpr int NP = 3;     // bf16 parts of an operand

// Eight values as three parts, stored `stride` elements apart.
__device__ __forceinline__ void split8(const float (&v)[8], bf16* dst, int stride) {
  uint32_t w[4][NP];
#pragma unroll
  for (int e = 0; e < 4; e++) split2<NP>(v[2 * e], v[2 * e + 1], w[e]);
#pragma unroll
  for (int p = 0; p < NP; p++)
    *reinterpret_cast<uint4*>(dst + p * stride) = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
}
__device__ __forceinline__ void put2(float x0, float x1, bf16* dst, int stride) {
  uint32_t w[NP];
  split2<NP>(x0, x1, w);
#pragma unroll
  for (int p = 0; p < NP; p++) *reinterpret_cast<uint32_t*>(dst + p * stride) = w[p];
}
// A 64 x W tile (columns c0 .. of a head's D) on its way: loaded into registers
// at once, later put as three parts in core-matrix order: the group of eight
// columns idx lands at element 8 idx, so eight lanes fill one 128-byte core
// matrix.
template <int W>
struct Tile {
  static constexpr int IT = 8 * W / LTH;
  float v[IT][8];
  static __device__ __forceinline__ int row(int t) {
    const int idx = threadIdx.x + t * LTH;
    return (idx & 7) + 8 * (idx / W);
  }
  __device__ __forceinline__ void load(const float* g, const Rows& r, int H, int h, int D, int c0) {
#pragma unroll
    for (int t = 0; t < IT; t++) {
      const int cg = ((threadIdx.x + t * LTH) >> 3) % (W / 8);
      const bool in = row(t) < r.n;
      const float4* p =
          reinterpret_cast<const float4*>(g + ((r.t0 + (int64_t)r.dir * (in ? row(t) : 0)) * H + h) * D + c0 + 8 * cg);
      const float4 f0 = __ldg(p), f1 = __ldg(p + 1);
      v[t][0] = in ? f0.x : 0.f; v[t][1] = in ? f0.y : 0.f; v[t][2] = in ? f0.z : 0.f; v[t][3] = in ? f0.w : 0.f;
      v[t][4] = in ? f1.x : 0.f; v[t][5] = in ? f1.y : 0.f; v[t][6] = in ? f1.z : 0.f; v[t][7] = in ? f1.w : 0.f;
    }
  }
  __device__ __forceinline__ void put(bf16* dst) const {
#pragma unroll
    for (int t = 0; t < IT; t++) split8(v[t], dst + 8 * (threadIdx.x + t * LTH), 64 * W);
  }
  template <class F>
  __device__ __forceinline__ void put_weighted(bf16* dst, int n, F w) const {  // row i times w(i)
#pragma unroll
    for (int t = 0; t < IT; t++) {
      const float m = row(t) < n ? w(row(t)) : 0.f;
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; e++) u[e] = m * v[t][e];
      split8(u, dst + 8 * (threadIdx.x + t * LTH), 64 * W);
    }
  }
};

// D = A B over ksteps x 16, A's and B's parts sa and sb elements apart: the
// products of parts i, j with i + j <= 2, the smallest first.  One thread issues.
__device__ __forceinline__ void gemm_parts(uint32_t d, const tc::View& A, int sa, const tc::View& B, int sb, int N,
                                           int ksteps) {
  const uint32_t id = tc::idesc_bf16(64, N, A.mn, B.mn);
  const uint64_t da = tc::vstep(A), db = tc::vstep(B);
  uint32_t acc = 0;
#pragma unroll
  for (int o = NP - 1; o >= 0; o--)
#pragma unroll
    for (int i = 0; i <= o; i++) {
      uint64_t a = tc::vdesc(A, A.hi + i * sa, 0), b = tc::vdesc(B, B.hi + (o - i) * sb, 0);
      for (int ks = 0; ks < ksteps; ks++) {
        tc::mma_issue(d, a, b, id, acc);
        acc = 1;
        a += da;
        b += db;
      }
    }
}
__device__ __forceinline__ tc::View kview(const bf16* p, int Kc) { return tc::View{p, nullptr, Kc, 0, 0, false}; }
__device__ __forceinline__ tc::View mview(const bf16* p, int Kc) { return tc::View{p, nullptr, Kc, 0, 0, true}; }

template <int NT>
__device__ __forceinline__ void ld_tiles(uint32_t tbase, int c0, float (&v)[NT][4]) {
  if constexpr (NT <= 4) {
    tc::ld_frag<NT>(tbase, c0, v);
  } else {
#pragma unroll
    for (int b = 0; b < NT / 4; b++) {
      float t[4][4];
      tc::ld_frag<4>(tbase, c0 + 32 * b, t);
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) v[4 * b + j][e] = t[j][e];
    }
  }
}

template <int DK, int DVS, int DEC>
struct Shape {
  static constexpr bool ONLY = DEC >= 3;  // a segment's own state: no output rows
  static constexpr int XE = ONLY ? 0 : NP * 64 * DK, YE = NP * 64 * DK, ZE = ONLY ? 0 : NP * 64 * DVS;
  static constexpr int SE = ONLY ? 0 : NP * DVS * DK, SCE = NP * 64 * DVS, PE = ONLY ? 0 : NP * 64 * 64;
  static constexpr int QE = DEC == 1 ? ZE : 0;
  // 512 bytes after the tiles: an M = 64 view of a 32-column tile reads up to four cores past it
  static constexpr int ELEMS = XE + YE + ZE + SE + SCE + PE + QE + 256;
  // accumulator columns: pairs and o 64, the entry state's rows DVS, the state's product DK, pairs of q and k 64
  static constexpr int C_X = ONLY ? 0 : 64, C_S = C_X + (ONLY ? 0 : DVS), C_A = C_S + DK;
  static constexpr int COLS = C_A + (DEC == 1 ? 64 : 0);
  static constexpr int TMEM = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int SMEM = ELEMS * 2 + 1024 /* lut */ + 384 /* tab */ + 64;
  static constexpr int NTV = DVS / 16;  // 8-column tiles of a warp's half of the value side
  static constexpr int NTK = DK / 16;   // and of the key side
};

template <int DK, int DVS, int DEC>
__device__ void chain(const LinP& P, const LinOp& op, int u, int h, int slice) {
  using SH = Shape<DK, DVS, DEC>;
  constexpr int NTV = SH::NTV, NTK = SH::NTK;
  constexpr bool ONLY = SH::ONLY;
  extern __shared__ __align__(1024) unsigned char smem[];
  bf16* tX = reinterpret_cast<bf16*>(smem);
  bf16* tY = tX + SH::XE;
  bf16* tZ = tY + SH::YE;
  bf16* tS = tZ + SH::ZE;
  bf16* tSC = tS + SH::SE;
  bf16* tP = tSC + SH::SCE;
  bf16* tQ = tP + SH::PE;
  float2* lut = reinterpret_cast<float2*>(smem + SH::ELEMS * 2);  // [128] (w(m), w(m - 1)), m = index - 64
  float* tab = reinterpret_cast<float*>(lut + 128);               // [65] e^{-a m}
  uint64_t* bar = reinterpret_cast<uint64_t*>(tab + 96);          // pairs; entry state's rows and state; o
  uint32_t* slot = reinterpret_cast<uint32_t*>(bar + 3);
  int* s_fail = reinterpret_cast<int*>(slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int q4 = warp & 3, half = warp >> 2, r0 = 16 * q4 + gq;

  Unit un;
  if (!unit_of(P, u, un)) {
    if ((DEC == 1 || DEC == 2) && tid == 0) op.pda[((int64_t)u * P.H + h) * (op.DVt / DVS) + slice] = 0.0;
    return;
  }
  if (ONLY && un.seg == (op.rev ? 0 : un.nseg - 1)) return;  // the last segment of its direction feeds nobody
  const int H = P.H, DVt = op.DVt, c0 = slice * DVS;
  const int64_t stN = (int64_t)DK * DVt;
  const float a = decay_of(P.A_log, h);

  if (warp == 0) tc::tmem_alloc(slot, SH::TMEM);
  if (tid == 0) {
    for (int i = 0; i < 3; i++) mma::mbar_init(bar + i, 1);
    mma::mbar_init_fence();
    *s_fail = 0;
  }
  if (tid < 65) tab[tid] = decay_pow(a, tid);
  __syncthreads();
  if (tid < 128) {
    const int m = tid - 64;
    lut[tid] = make_float2(m >= 0 ? P.scale * tab[m] : 0.f, m >= 1 ? P.scale * tab[m - 1] : 0.f);
  }
  tc::fence_after();
  const uint32_t tm = *slot;

  const bool st_rows = 16 * q4 < DVS;  // a warp whose state rows exist (warps 0, 1 of each half)
  float S[NTK][4];
  mma::zero<NTK>(S);
  auto each_at = [&](int tr, auto fn) {
#pragma unroll
    for (int j = 0; j < NTK; j++)
#pragma unroll
      for (int e = 0; e < 4; e++)
        fn(S[j][e],
           st_at(tr, c0 + r0 + 8 * (e >> 1), half * (DK / 2) + 8 * j + 2 * tq + (e & 1), DK, DVt));
  };
  auto each_st = [&](auto fn) { each_at(op.tr, fn); };
  if (!ONLY && st_rows) start_state(P, op, un, u, h, stN, each_st);
  auto put_state = [&]() {
    if (st_rows) {
#pragma unroll
      for (int j = 0; j < NTK; j++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int at = mma::opix(r0 + 8 * k, half * (DK / 2) + 8 * j + 2 * tq, DK);
          put2(S[j][2 * k], S[j][2 * k + 1], tS + at, DVS * DK);
        }
    }
  };
  if constexpr (!ONLY) put_state();

  double dacc = 0.0;  // this thread's part of the decay gradient's sums
  uint32_t ph = 0;
  bool good = true;
  const int nch = (un.ntok + C - 1) / C;
  auto rows = [&](int c) { return rows_of(un, op.rev, c); };
  Tile<DK> x, y;
  Tile<DVS> z, wq;
  auto load_xy = [&](const Rows& r) {
    if constexpr (!ONLY) x.load((const float*)op.x, r, H, h, DK, 0);
    y.load((const float*)op.y, r, H, h, DK, 0);
  };
  auto put_xy = [&]() {
    if constexpr (!ONLY) x.put(tX);
    y.put(tY);
  };
  auto load_z = [&](const Rows& r) {
    z.load((const float*)op.z, r, H, h, DVt, c0);
    if constexpr (DEC == 1) wq.load((const float*)op.wx, r, H, h, DVt, c0);
  };
  auto put_z = [&](int n) {  // the state's operand with the weights of row to exit state
    if constexpr (!ONLY) z.put(tZ);
    z.put_weighted(tSC, n, [&](int row) { return tab[n - 1 - row + (op.rev ? 1 : 0)]; });
    if constexpr (DEC == 1) wq.put(tQ);
  };
  auto wait = [&](int b) {
    __syncwarp();
    if (!mma::mbar_wait(bar + b, ph)) *s_fail = 1;
    tc::fence_after();
  };
  if (nch > 0) {
    load_xy(rows(0));
    load_z(rows(0));
    put_xy();
    put_z(rows(0).n);
  }
  for (int c = 0; c < nch; c++) {
    const Rows rw = rows(c);
    const int n = rw.n, idx = op.rev ? nch - 1 - c : c;
    mma::fence_async_smem();
    tc::fence_before();
    // the chunk's tiles and state of every warp; the last chunk's accumulators have been read
    if (__syncthreads_or(!good)) {
      good = false;
      break;
    }
    if (tid == 0) {
      tc::fence_after();
      if constexpr (!ONLY) {
        gemm_parts(tm, kview(tX, DK), 64 * DK, kview(tY, DK), 64 * DK, 64, DK / 16);
        if constexpr (DEC == 1)
          gemm_parts(tm + SH::C_A, kview(tQ, DVS), 64 * DVS, kview(tZ, DVS), 64 * DVS, 64, DVS / 16);
        tc::commit(bar);
        gemm_parts(tm + SH::C_X, kview(tX, DK), 64 * DK, kview(tS, DK), DVS * DK, DVS, DK / 16);
      }
      // S'^T += (weighted z)^T y: rows are the value columns
      gemm_parts(tm + SH::C_S, mview(tSC, DVS), 64 * DVS, mview(tY, DK), 64 * DK, DK, 4);
      tc::commit(bar + 1);
    }
    if (!ONLY && st_rows) {
      const int64_t at0 = ((int64_t)(un.ch0 + idx) * H + h) * stN;
      if (op.states) each_at(1, [&](float& s, int64_t at) { op.states[at0 + at] = s; });  // saving forward: [dv][dk]
      if constexpr (DEC == 2) {  // D: n e^{-an} <the chunk's exit gradient, its entry state>
        float part = 0.f;
        each_at(0, [&](float& s, int64_t at) { part = fmaf(s, op.ent[at0 + at], part); });
        dacc += (double)(part * P.scale * (float)n * tab[n]);
      }
    }
    [[maybe_unused]] float kx[NTV][4];
    if constexpr (DEC == 2) {  // k's rows in fragment order
#pragma unroll
      for (int j = 0; j < NTV; j++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int row = r0 + 8 * k;
          float2 f = make_float2(0.f, 0.f);
          if (row < n)
            f = *reinterpret_cast<const float2*>((const float*)op.wx +
                                                 ((rw.t0 + (int64_t)rw.dir * row) * H + h) * DVt + c0 +
                                                 half * (DVS / 2) + 8 * j + 2 * tq);
          kx[j][2 * k] = f.x;
          kx[j][2 * k + 1] = f.y;
        }
    }
    float o[NTV][4];
    float part = 0.f;
    if constexpr (!ONLY) {
      wait(0);
      float p[4][4];
      ld_tiles<4>(tm, half * 32, p);
#pragma unroll
      for (int j = 0; j < 4; j++)
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int row = r0 + 8 * k, col = half * 32 + 8 * j + 2 * tq;
          const float2 w = lut[64 + row - col];
          p[j][2 * k] *= w.x;
          p[j][2 * k + 1] *= w.y;
          put2(p[j][2 * k], p[j][2 * k + 1], tP + mma::opix(row, col, 64), 64 * 64);
        }
      if constexpr (DEC == 1) {  // A: pairs inside the chunk
        float m2[4][4];
        ld_tiles<4>(tm + SH::C_A, half * 32, m2);
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int d = r0 + 8 * (e >> 1) - (half * 32 + 8 * j + 2 * tq + (e & 1));
            part = fmaf((float)d * p[j][e], m2[j][e], part);
          }
      }
      mma::fence_async_smem();
      tc::fence_before();
      __syncthreads();  // the pairs of every warp
      if (tid == 0) {
        tc::fence_after();
        gemm_parts(tm, kview(tP, 64), 64 * 64, mview(tZ, DVS), 64 * DVS, DVS, 4);
        tc::commit(bar + 2);
      }
    }
    // ---- the entry state's rows and the state, while the tensor core forms o
    if (c + 1 < nch) load_xy(rows(c + 1));
    wait(1);
    if constexpr (!ONLY) {
      const float rs[2] = {P.scale * tab[r0 + (op.rev ? 0 : 1)], P.scale * tab[r0 + 8 + (op.rev ? 0 : 1)]};
      ld_tiles<NTV>(tm + SH::C_X, half * (DVS / 2), o);
#pragma unroll
      for (int j = 0; j < NTV; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int row = r0 + 8 * (e >> 1);
          if constexpr (DEC == 1) {  // B
            const int at = mma::opix(row, half * (DVS / 2) + 8 * j + 2 * tq + (e & 1), DVS);
            float qv = 0.f;
#pragma unroll
            for (int b = 0; b < NP; b++) qv += __bfloat162float(tQ[b * 64 * DVS + at]);
            part = fmaf(rs[e >> 1] * qv * (float)(row + 1), o[j][e], part);
          }
          o[j][e] *= rs[e >> 1];
          if constexpr (DEC == 2) part = fmaf((float)row * kx[j][e], o[j][e], part);  // C
        }
      if constexpr (DEC == 1 || DEC == 2) dacc += (double)part;
    }
    {
      const Decay dec(a, n);
      float d[NTK][4];
      ld_tiles<NTK>(tm + SH::C_S, half * (DK / 2), d);
#pragma unroll
      for (int j = 0; j < NTK; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) S[j][e] = dec(S[j][e]) + d[j][e];
    }
    // the next chunk's x, y and state: every product that reads these tiles has completed
    if (c + 1 < nch) {
      if constexpr (!ONLY) put_state();
      put_xy();
      load_z(rows(c + 1));
    }
    if constexpr (!ONLY) {
      wait(2);
      float v[NTV][4];
      ld_tiles<NTV>(tm, half * (DVS / 2), v);
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const int row = r0 + 8 * k;
        if (row < n) {
          float* po = (float*)op.out + ((rw.t0 + (int64_t)rw.dir * row) * H + h) * DVt + c0 + half * (DVS / 2);
#pragma unroll
          for (int j = 0; j < NTV; j++)
            *reinterpret_cast<float2*>(po + 8 * j + 2 * tq) =
                make_float2(o[j][2 * k] + v[j][2 * k], o[j][2 * k + 1] + v[j][2 * k + 1]);
        }
      }
    }
    ph ^= 1;
    if (DEC == 1) __syncthreads();  // q's rows (B) have been read
    if (c + 1 < nch) put_z(rows(c + 1).n);
    if (*(volatile int*)s_fail) good = false;  // a wait ran out: no thread starts another chunk
  }
  tc::fence_before();
  __syncthreads();
  if (*s_fail) good = false;
  if (!good && tid == 0) *P.err = KDA_ERR_DEVICE;

  if (good && st_rows) {  // the unit's state
    const bool last = un.seg == (op.rev ? 0 : un.nseg - 1);
    float* pf = nullptr;
    float mul = 1.0f;
    if (ONLY) {
      pf = op.segc + ((int64_t)u * H + h) * stN;
    } else if (last && op.fin) {
      pf = op.fin + ((int64_t)un.doc * H + h) * stN;
      mul = op.rev ? P.scale : 1.0f;
    }
    if (pf) each_st([&](float& s, int64_t at) { pf[at] = mul * s; });
  }
  __syncthreads();
  if constexpr (DEC == 1 || DEC == 2) {  // the CTA's partial, summed in a fixed order
    double* red = reinterpret_cast<double*>(smem);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dacc += __shfl_xor_sync(0xffffffffu, dacc, s);
    if (lane == 0) red[warp] = dacc;
    __syncthreads();
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < LTH / 32; w++) s += red[w];
      op.pda[((int64_t)u * H + h) * (DVt / DVS) + slice] = s;
    }
  }
  if (warp == 0) tc::tmem_dealloc(tm, SH::TMEM);
}

template <int DK, int DVS, int DEC>
__global__ void __launch_bounds__(LTH, Shape<DK, DVS, DEC>::SMEM <= 113 * 1024 ? 2 : 1)
    lin_f32_kernel(LinP P, LinOp op, int fwd) {
  pdl_wait();
  pdl_release();
  if (!ready(P, fwd)) return;
  const int ns = op.DVt / DVS;
  chain<DK, DVS, DEC>(P, op, blockIdx.x / (ns * P.H), (blockIdx.x / ns) % P.H, blockIdx.x % ns);
}

template <int DK, int DVS, int DEC>
cudaError_t launch(int kid, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  constexpr int smem = Shape<DK, DVS, DEC>::SMEM;
  cudaError_t e = raise_smem<lin_f32_kernel<DK, DVS, DEC>>(smem);
  if (e != cudaSuccess) return e;
  prof_begin(kid, st);
  e = launch_after(op.after, lin_f32_kernel<DK, DVS, DEC>, dim3((unsigned)((int64_t)P.nu * P.H * (op.DVt / DVS))), LTH,
                   smem, st, P, op, fwd);
  prof_end(kid, st);
  return e;
}

template <int DEC>
cudaError_t by_key(int kid, int key, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  // (the gradients' chains have dv as their key side, the others dk)
  if constexpr (DEC != 1 && DEC != 2) {
    if (key == 32) return launch<32, 64, DEC>(kid, P, op, fwd, st);
  }
  if constexpr (DEC != 3) {
    if (key == 64 && op.DVt == 32) return launch<64, 32, DEC>(kid, P, op, fwd, st);
  }
  if (key == 64) return launch<64, 64, DEC>(kid, P, op, fwd, st);
  return launch<128, 32, DEC>(kid, P, op, fwd, st);
}

}  // namespace

cudaError_t launch_f32(int dec, int kid, int key, const LinP& P, const LinOp& op, int fwd, cudaStream_t st) {
  switch (dec) {
    case 0: return by_key<0>(kid, key, P, op, fwd, st);
    case 1: return by_key<1>(kid, key, P, op, fwd, st);
    case 2: return by_key<2>(kid, key, P, op, fwd, st);
    default: return by_key<3>(kid, key, P, op, fwd, st);
  }
}

}  // namespace lin
}  // namespace kda
