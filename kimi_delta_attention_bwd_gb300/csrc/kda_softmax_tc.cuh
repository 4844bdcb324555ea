// What the tensor-core kernels of softmax attention share: products (tcgen05, operands in 128-byte swizzled shared memory
// or in tensor memory), accumulator loads and stores, bounded waits, blocks of rows, the backward's elementwise steps.
#pragma once
#include "kda_softmax.cuh"
#include "kda_mma.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace smx {

constexpr int BLK = 128;       // rows of a block of keys (or queries)
constexpr int HALF = 16384;    // bytes of 128 rows by 64 columns, one swizzled half of a block

// The tensor memory's address, the same for the whole warp: with all 512 columns its first one.
template <int COLS>
__device__ __forceinline__ uint32_t tm_base(uint32_t slot) {
  return COLS == 512 ? 0u : __shfl_sync(0xffffffffu, slot, 0);
}

// ------------------------------------------------------------ helpers
// Descriptors of a block of rows in 128-byte swizzled halves of 64 columns (TMA's layout): 8-row groups 1024 bytes apart.
// K-major (rows are M or N): 16 columns of the contraction are 32 bytes of the swizzled row.  MN-major (rows are the
// contraction): 16 rows are 2048 bytes, and the next 64 columns are a half away.
//
// A warp issues products as a whole, one elected lane's predicate on the instruction: descriptors and addresses then
// stay in uniform registers.  Issued inside a branch of one lane, from registers of that lane, a product took 70 to 180
// cycles to issue, and 64 (128 x 128 x 16) to run.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) | (lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61);
}
template <int ROWS>
__device__ __forceinline__ uint64_t desc_k(uint32_t block, int step) {  // columns 16 step ..
  return sdesc(block + (step >> 2) * (ROWS * 128) + (step & 3) * 32, 16);
}
template <int ROWS>
__device__ __forceinline__ uint64_t desc_mn(uint32_t block, int step) {  // rows 16 step ..
  return sdesc(block + step * 2048, ROWS * 128);
}
constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)b_mn << 16 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p;
}
// (whole warp; me: the elected lane)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc, uint32_t me) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc), "r"(me)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc, uint32_t me) {  // A in tensor memory
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc), "r"(me)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t me) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(mma::smem_u32(bar)),
      "r"(me)
      : "memory");
}

// 32 columns of this warp's lanes, a lane a row.
__device__ __forceinline__ void tm_ld32(uint32_t a, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(a));
}
__device__ __forceinline__ void tm_ld16(uint32_t a, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(a));
}
__device__ __forceinline__ void tm_st8(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};\n" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(a)
               : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
      : "memory");
}
// Waits for the loads in flight; the values they bring depend on it, so that no use moves before it.
__device__ __forceinline__ void tm_wait_ld(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
                 "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]),
                 "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                 "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tm_wait_ld(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
                 "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// The second (y = 1) or third bf16 parts of two floats.
__device__ __forceinline__ uint32_t rest(float a, float b, int y) {
  for (int i = 0; i < y; i++) {
    const uint32_t u = pack(a, b);
    a -= low(u);
    b -= high(u);
  }
  return pack(a, b);
}

// Whole-warp wait on a barrier's phase; gives up (and lets every other wait of the CTA give up) after mma::WAIT_POLLS.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* dead) {
  bool ok = mma::mbar_try(bar, parity);
  for (int it = 0; !ok && it < mma::WAIT_POLLS; it++) {
    ok = mma::mbar_try(bar, parity);
    if (!ok && *(volatile int*)dead) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) *(volatile int*)dead = 1;
  return ok;
}

// This warp's part of a step is in tensor memory, or taken from it.
__device__ __forceinline__ void arrive(uint64_t* bar) {
  tc::fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mma::mbar_arrive(bar);
}

// Logits of a row: those from `left` on are not seen.
template <int N>
__device__ __forceinline__ void mask(float (&v)[N], int left) {
#pragma unroll
  for (int e = 0; e < N; e++) v[e] = e < left ? v[e] : -INFINITY;
}
template <int N>
__device__ __forceinline__ void row_max(const float (&v)[N], float (&mx)[4]) {
#pragma unroll
  for (int e = 0; e < N; e += 8)
#pragma unroll
    for (int y = 0; y < 4; y++)
      asm("max.f32 %0, %1, %2, %3;" : "=f"(mx[y]) : "f"(mx[y]), "f"(v[e + 2 * y]), "f"(v[e + 2 * y + 1]));
}
// Pairs of floats in one register pair, for the two-wide fp32 instructions.
__device__ __forceinline__ uint64_t two(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void one(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Logits into weights 2^(sc v + ng), their sum, and as bf16 pairs; what that rounding leaves.
template <int N>
__device__ __forceinline__ void weights(float (&v)[N], uint64_t sc, uint64_t ng, uint64_t (&sum)[2], uint32_t* w) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    one(fma2(two(v[e], v[e + 1]), sc, ng), v[e], v[e + 1]);
    v[e] = ex2(v[e]);
    v[e + 1] = ex2(v[e + 1]);
    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], two(v[e], v[e + 1]));
    w[e / 2] = pack(v[e], v[e + 1]);
  }
}
template <int N>
__device__ __forceinline__ void second_parts(const float (&v)[N], uint32_t* w) {
#pragma unroll
  for (int e = 0; e < N / 2; e++) {
    const uint32_t h = pack(v[2 * e], v[2 * e + 1]);
    w[e] = pack(v[2 * e] - low(h), v[2 * e + 1] - high(h));
  }
}

// 128 bytes (u: 64 bf16 or 32 fp32 values of this lane's row) of each of a warp's 32 rows to global memory, through 4 KB
// of shared memory of its own (16-byte pieces swizzled): a lane's row alone would make every store 32 half sectors.
// The first n rows are stored; dst is the warp's first row, ld elements a row.
template <typename T>
__device__ __forceinline__ void store_rows(unsigned char* buf, const uint32_t (&u)[32], T* dst, size_t ld, int n) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < 8; c++)
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int r = 4 * i + lane / 8, c = lane & 7;
    const uint4 x = *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
    if (r < n) *reinterpret_cast<uint4*>(dst + r * ld + 16 / sizeof(T) * c) = x;
  }
  __syncwarp();
}
// 64 columns of an accumulator, times f, as bf16 (zeros where nothing was accumulated).
__device__ __forceinline__ void store_acc(unsigned char* buf, uint32_t tm, bool any, float f, bf16* dst, size_t ld,
                                          int n) {
  uint32_t u[32];
#pragma unroll
  for (int c = 0; c < 2; c++) {
    float v[32];
    if (any) {
      tm_ld32(tm + 32 * c, v);
      tm_wait_ld(v);
    }
#pragma unroll
    for (int e = 0; e < 16; e++) u[16 * c + e] = any ? pack(v[2 * e] * f, v[2 * e + 1] * f) : 0u;
  }
  store_rows(buf, u, dst, ld, n);
}
__device__ __forceinline__ void store_acc_f32(unsigned char* buf, uint32_t tm, bool any, float* dst, size_t ld, int n) {
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    float v[32];
    uint32_t u[32];
    if (any) {
      tm_ld32(tm + c, v);
      tm_wait_ld(v);
    }
#pragma unroll
    for (int e = 0; e < 32; e++) u[e] = any ? __float_as_uint(v[e]) : 0u;
    store_rows(buf, u, dst + c, ld, n);
  }
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
}

// A block in shared memory: PARTS arrays (below) of ROWS rows by D columns, each in halves of 64 columns.
// Its rows from n on (other documents' tokens) become zeros, by one warp, before products read them.
template <int D, int ROWS, int PARTS>
__device__ __forceinline__ void zero_rows(unsigned char* block, int n) {
  for (int i = threadIdx.x & 31; i < (ROWS - n) * 8; i += 32)
#pragma unroll
    for (int c = 0; c < D / 64 * PARTS; c++)
      *reinterpret_cast<uint4*>(block + (c * ROWS + n) * 128 + i * 16) = make_uint4(0, 0, 0, 0);
  mma::fence_async_smem();
  __syncwarp();
}
// Its load; the parts lie `stride` rows apart in the map.
template <int D, int ROWS, int PARTS>
__device__ __forceinline__ void load_block(unsigned char* dst, const CUtensorMap* map, int head, int row, int stride,
                                           uint64_t* bar) {
#pragma unroll
  for (int p = 0; p < PARTS; p++)
#pragma unroll
    for (int c = 0; c < D / 64; c++)
      mma::tma_load_2d(dst + (p * (D / 64) + c) * (ROWS * 128), map, head * D + 64 * c, row + p * stride, bar);
}

// fp32 io comes as three bf16 parts of every value (x = x0 + x1 + x2 to 2^-24), and a product is the six products of
// parts above that, smallest first: bytes and time of six, and the fp32 pipe's precision.  The tensor pipe truncates its
// sums, so a sum over many blocks would be off by 2^-24 for every 16 of its terms (o after 1001 keys by 6e-6): each
// block's product starts from zero and is added to the row's sum in registers (3e-7).
template <int PARTS>
struct Prod {
  static constexpr int N = 1;
  static __device__ constexpr int a(int) { return 0; }
  static __device__ constexpr int b(int) { return 0; }
};
template <>
struct Prod<3> {
  static constexpr int N = 6;
  static __device__ constexpr int a(int i) { return i == 0 ? 0 : i == 1 ? 2 : i == 2 ? 1 : i == 3 ? 0 : i == 4 ? 1 : 0; }
  static __device__ constexpr int b(int i) { return i == 0 ? 2 : i == 1 ? 0 : i == 2 ? 1 : i == 3 ? 1 : 0; }
};
// d = A B^T over D columns, both K-major blocks
template <int D, int PARTS, int RA, int RB>
__device__ __forceinline__ void prod_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t me) {
  using Q = Prod<PARTS>;
#pragma unroll
  for (int i = 0; i < Q::N; i++)
#pragma unroll
    for (int s = 0; s < D / 16; s++)
      mma_ss(d, desc_k<RA>(a + Q::a(i) * (RA * D * 2), s), desc_k<RB>(b + Q::b(i) * (RB * D * 2), s), id, i > 0 || s > 0,
             me);
}
// Three parts of 2 n floats as bf16 pairs, taken off v one by one.
template <int N>
__device__ __forceinline__ void next_part(float (&v)[N], uint32_t* w) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const uint32_t u = pack(v[e], v[e + 1]);
    w[e / 2] = u;
    v[e] -= low(u);
    v[e + 1] -= high(u);
  }
}

// ------------------------------------------------------------ the backward
// The backward's weights of N logits of a key: queries lo .. hi - 1 of them see it; l2: the queries' log2 sums,
// negated.
template <int N>
__device__ __forceinline__ void bwd_weights(float (&v)[N], const float* l2, uint64_t sc, bool cut, int lo, int hi) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(l2 + e);
    one(fma2(two(v[e], v[e + 1]), sc, l.x), v[e], v[e + 1]);
    one(fma2(two(v[e + 2], v[e + 3]), sc, l.y), v[e + 2], v[e + 3]);
#pragma unroll
    for (int y = 0; y < 4; y++) v[e + y] = ex2(v[e + y]);
  }
  if (cut)
#pragma unroll
    for (int e = 0; e < N; e++) v[e] = e >= lo && e < hi ? v[e] : 0.f;
}
// N gradients p <- p (dp - delta) (an unseen pair's is zero whatever dp holds); dl: -delta.
template <int N>
__device__ __forceinline__ void bwd_grads(float (&p)[N], const float (&dp)[N], const float* dl, bool cut, int lo, int hi) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(dl + e);
    one(mul2(two(p[e], p[e + 1]), add2(two(dp[e], dp[e + 1]), l.x)), p[e], p[e + 1]);
    one(mul2(two(p[e + 2], p[e + 3]), add2(two(dp[e + 2], dp[e + 3]), l.y)), p[e + 2], p[e + 3]);
  }
  if (cut)
#pragma unroll
    for (int e = 0; e < N; e++) p[e] = e >= lo && e < hi ? p[e] : 0.f;
}
// The same of a query's row: its (negated) sums are scalars, its keys end at `left`.
template <int N>
__device__ __forceinline__ void dq_weights(float (&v)[N], uint64_t sc, uint64_t l2) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    one(fma2(two(v[e], v[e + 1]), sc, l2), v[e], v[e + 1]);
    v[e] = ex2(v[e]);
    v[e + 1] = ex2(v[e + 1]);
  }
}
template <int N>
__device__ __forceinline__ void dq_grads(float (&p)[N], const float (&dp)[N], uint64_t dl, bool cut, int left) {
#pragma unroll
  for (int e = 0; e < N; e += 2)
    one(mul2(two(p[e], p[e + 1]), add2(two(dp[e], dp[e + 1]), dl)), p[e], p[e + 1]);
  if (cut)
#pragma unroll
    for (int e = 0; e < N; e++) p[e] = e < left ? p[e] : 0.f;
}
template <int N>
__device__ __forceinline__ void add_columns(float (&sum)[N], uint32_t tm) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    float v[32];
    tm_ld32(tm + c, v);
    tm_wait_ld(v);
#pragma unroll
    for (int e = 0; e < 32; e++) sum[c + e] += v[e];
  }
}
template <int N>
__device__ __forceinline__ void store_sums(unsigned char* buf, const float (&sum)[N], float f, float* dst, size_t ld, int n) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    uint32_t u[32];
#pragma unroll
    for (int e = 0; e < 32; e++) u[e] = __float_as_uint(sum[c + e] * f);
    store_rows(buf, u, dst + c, ld, n);
  }
}

}  // namespace smx
}  // namespace kda
