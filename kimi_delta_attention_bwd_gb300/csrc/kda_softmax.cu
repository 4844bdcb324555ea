// Softmax attention with grouped heads: tile tables of packed documents, the
// backward's row sums, argument checks, workspace and the C entries.
#include "kda_softmax.cuh"

#include <string.h>

namespace kda {
namespace smx {
namespace {

// ------------------------------------------------------------ tile tables
// Block l builds list l: every document's tiles of queries (keys for list
// 2), by decreasing pairs, so that the longest tiles start first and the grid's
// end is short ones (a counting sort; tiles of equal weight in any order, which no
// result depends on).  The offsets are checked before any of them is used.  A saving
// forward builds the backward's lists too, so that a step has one launch of this kernel and
// the backward reads no offsets: they may be gone or others by then.
// Tiles with more than 1.5 times the load that `target` CTAs would have on average are
// cut along the other side into pieces of about that load, which a further kernel joins:
// a few queries against long prefixes, or few heads, would else leave most SMs idle
// behind the longest (11 pieces of prompts, 4096 queries on 30011 keys: 127 us whole, 97
// cut; 128 queries of 16 heads on 16384 keys: 176 and 51; a training step of 8192 tokens,
// four heads on one key head at 64: 627 and 303).
constexpr int TT = 1024, NB = 1024;

__device__ int incl_scan(int x, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_warp[lane] = y;
  }
  __syncthreads();
  const int r = x + (warp ? s_warp[warp - 1] : 0);
  *total = s_warp[31];
  __syncthreads();
  return r;
}

__global__ void __launch_bounds__(TT) smx_table_kernel(SmxP P) {
  constexpr int NS = 1024;  // documents whose offsets shared memory holds
  __shared__ int s_bad, s_piece, s_join, s_warp[32], s_cnt[NB], s_off[3][NS + 1];
  __shared__ unsigned long long s_blocks;
  const int l = blockIdx.x, tid = threadIdx.x, n = P.n_docs, tile = P.tile[l];
  const bool by_key = l == 2, near = n <= NS;
  pdl_wait();
  pdl_release();
  if (!P.list[l]) return;
  const int32_t *cu = P.cu, *cuk = P.cuk;
  int32_t* pre = P.pre[l];
  if (near) {
    for (int i = tid; i <= n; i += TT) {
      s_off[0][i] = P.rows ? i * P.T : cu[i];
      s_off[1][i] = P.rows ? i * P.Tk : cuk[i];
    }
    cu = s_off[0];
    cuk = s_off[1];
    pre = s_off[2];
  }
  const int32_t* own = by_key ? cuk : cu;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  if (tid == 0 && (cu[0] != 0 || cu[n] != P.Nq || cuk[0] != 0 || cuk[n] != P.Nk)) s_bad = 1;
  for (int i = tid; i < n; i += TT)
    if (cu[i + 1] < cu[i] || cuk[i + 1] < cuk[i]) s_bad = 1;
  __syncthreads();
  if (tid == 0 && l == 0) {
    *P.err = s_bad ? KDA_ERR_BAD_SEQLENS : KDA_OK;
    *P.wtag = P.save && !s_bad ? P.tag : 0;
  }
  if (s_bad) {
    if (tid == 0) P.counts[l] = 0;
    return;
  }
  int carry = 0;
  for (int base = 0; base < n; base += TT) {
    const int i = base + tid, nt = i < n ? (own[i + 1] - own[i] + tile - 1) / tile : 0;
    int total;
    const int r = carry + incl_scan(nt, s_warp, &total) - nt;
    if (i < n) pre[i] = r;
    carry += total;
  }
  for (int b = tid; b < NB; b += TT) s_cnt[b] = 0;
  if (tid == 0) s_piece = s_join = 0, s_blocks = 0;
  __syncthreads();
  const int xb = P.xb[l], H = by_key ? P.Hkv : P.Hq;
  const Tiles tiles{cu, cuk, pre, n, tile, xb, P.G, P.causal, by_key};
  const bool may_cut = P.target[l] > 0;
  int64_t per = 0;  // blocks a piece
  if (may_cut) {
    int64_t blocks = tiles.blocks(tid, carry, TT);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
    if (tid % 32 == 0) atomicAdd(&s_blocks, (unsigned long long)blocks);
    __syncthreads();
    per = piece_blocks((int64_t)s_blocks, H, P.target[l], xb);
  }
  auto pieces_of = [&](const Tiles::Found& f) { return may_cut ? pieces_in(f.nb, per) : 1; };
  auto bucket = [&](const Tiles::Found& f, int np) { return NB - 1 - min(NB - 1, f.nb / np); };
  for (int x = tid; x < carry; x += TT) {
    const Tiles::Found f = tiles.find(x);
    const int np = pieces_of(f);
    atomicAdd(&s_cnt[bucket(f, np)], np);
  }
  __syncthreads();
  int entries;
  {
    static_assert(NB == TT, "a bucket a thread");
    const int c = s_cnt[tid], r = incl_scan(c, s_warp, &entries) - c;
    s_cnt[tid] = r;
  }
  __syncthreads();
  for (int x = tid; x < carry; x += TT) {
    const Tiles::Found f = tiles.find(x);
    const int np = pieces_of(f), at = atomicAdd(&s_cnt[bucket(f, np)], np);
    int first = -1;
    if (np > 1) {  // (there is room: piece_room)
      first = atomicAdd(&s_piece, np);
      const int j = atomicAdd(&s_join, 1), i0 = f.t * tile;
      P.joins[l][j] = by_key ? make_int4(f.doc.z + i0, min(tile, f.doc.w - i0), first, np)
                             : make_int4(f.doc.x + i0, min(tile, f.doc.y - i0), first, np);
    }
    const int len = (f.nb + np - 1) / np;
    for (int y = 0; y < np; y++) {
      P.list[l][2 * (size_t)(at + y)] = f.doc;
      P.list[l][2 * (size_t)(at + y) + 1] =
          np > 1 ? make_int4(f.t, y * len, (y + 1) * len, first + y) : make_int4(f.t, 0, INT_MAX, -1);
    }
  }
  __syncthreads();
  if (tid == 0) {
    P.counts[l] = entries;
    P.counts[3 + l] = s_join;
  }
}

// Joins the pieces of the cut tiles, a warp a row: o = sum_p 2^(l_p - l) o_p, 2^l = sum_p 2^l_p.
template <int D, typename T>
__global__ void __launch_bounds__(256) smx_join_rows_kernel(SmxP P, T* __restrict__ o, float* __restrict__ lse) {
  constexpr int NV = D / 32;
  pdl_wait();
  const int tile = P.tile[0], lane = threadIdx.x % 32;
  const size_t step = (size_t)P.Hq * tile;
  const int rows = P.counts[0] == 0 ? 0 : P.counts[3] * tile * P.Hq;  // (at most pieces / 2 tiles of them)
  for (int x = blockIdx.x * 8 + threadIdx.x / 32; x < rows; x += gridDim.x * 8) {
    const int h = x % P.Hq, r = x / P.Hq % tile;
    const int4 e = P.joins[0][x / (P.Hq * tile)];
    if (r >= e.y) continue;
    const size_t at = ((size_t)e.z * P.Hq + h) * tile + r;
    float m = -INFINITY;
    for (int p = 0; p < e.w; p++) m = fmaxf(m, P.pl[at + p * step]);
    const float mu = m == -INFINITY ? 0.f : m;
    float sum = 0.f, acc[NV] = {};
#pragma unroll 4
    for (int p = 0; p < e.w; p++) {
      const float l = P.pl[at + p * step], w = l == -INFINITY ? 0.f : ex2(l - mu);  // (NaN stays)
      sum += w;
#pragma unroll
      for (int y = 0; y < NV; y++) acc[y] = fmaf(w, P.po[0][(at + p * step) * D + lane * NV + y], acc[y]);
    }
    const size_t row = (size_t)(e.x + r) * P.Hq + h;
    const float inv = sum == 0.f ? 0.f : 1.0f / sum, l2 = sum != sum ? sum : m + log2f(sum);
#pragma unroll
    for (int y = 0; y < NV; y++) {
      const float z = acc[y] * inv;
      stf(o + row * D + lane * NV + y, z);
      if constexpr (sizeof(T) == 2)
        if (P.save) stf(P.res + row * D + lane * NV + y, z - __bfloat162float(__float2bfloat16_rn(z)));
    }
    if (lane == 0) {
      lse[row] = l2 * LN2;
      if (P.save) P.lse2[(size_t)h * P.Nq + e.x + r] = l2;
    }
  }
}

// The same of the backward, sums of pieces: blockIdx.y 0: dq, 1: dk, 2: dv.
template <int D, typename T>
__global__ void __launch_bounds__(256) smx_join_grads_kernel(SmxP P, T* __restrict__ dq, T* __restrict__ dk,
                                                            T* __restrict__ dv) {
  constexpr int NV = D / 32;
  pdl_wait();
  const int l = blockIdx.y == 0 ? 1 : 2, H = l == 1 ? P.Hq : P.Hkv, tile = P.tile[l], lane = threadIdx.x % 32;
  if (!P.list[l] || !P.target[l] || *P.err != KDA_OK) return;
  const size_t step = (size_t)H * tile;
  const float* part = P.po[l] + (blockIdx.y == 2 ? (size_t)P.pieces[l] * step * D : 0);
  const float f = blockIdx.y == 2 ? 1.0f : P.scale;
  T* out = blockIdx.y == 0 ? dq : blockIdx.y == 1 ? dk : dv;
  const int rows = P.counts[l] == 0 ? 0 : P.counts[3 + l] * tile * H;
  for (int x = blockIdx.x * 8 + threadIdx.x / 32; x < rows; x += gridDim.x * 8) {
    const int h = x % H, r = x / H % tile;
    const int4 e = P.joins[l][x / (H * tile)];
    if (r >= e.y) continue;
    const size_t at = ((size_t)e.z * H + h) * tile + r;
    float acc[NV] = {};
#pragma unroll 4
    for (int p = 0; p < e.w; p++)
#pragma unroll
      for (int y = 0; y < NV; y++) acc[y] += part[(at + p * step) * D + lane * NV + y];
#pragma unroll
    for (int y = 0; y < NV; y++) stf(out + ((size_t)(e.x + r) * H + h) * D + lane * NV + y, acc[y] * f);
  }
}

// ------------------------------------------------------------ delta
// delta_i = sum_d o_i dO_i per row (token, head), D / 8 threads a row.  With bf16
// io o is the stored output plus what its rounding left: delta is subtracted from
// dO v, and a rounded o would put a further rounding's error into every gradient.
// A backward that is refused (its workspace holds no forward of this problem) gets NaN gradients here: nothing after this
// kernel writes any.
template <typename T>
__device__ void fill_nan(T* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    stf(p + i, __int_as_float(0x7fffffff));
}
template <int D, typename T>
__global__ void __launch_bounds__(256) smx_delta_kernel(SmxP P, const T* __restrict__ o, const T* __restrict__ dO,
                                                       T* __restrict__ dq, T* __restrict__ dk, T* __restrict__ dv) {
  constexpr int TR = D / 8;
  pdl_wait();
  pdl_release();
  if (!saved(P)) {
    fill_nan(dq, (int64_t)P.Nq * P.Hq * D);
    fill_nan(dk, (int64_t)P.Nk * P.Hkv * D);
    fill_nan(dv, (int64_t)P.Nk * P.Hkv * D);
    return;
  }
  const int64_t row = (int64_t)blockIdx.x * (256 / TR) + threadIdx.x / TR;
  const bool in = row < (int64_t)P.Nq * P.Hq;
  float s = 0.f;
  if (in) {
    const size_t at = (size_t)row * D + threadIdx.x % TR * 8;
    if constexpr (sizeof(T) == 2) {
      const uint4 a = *reinterpret_cast<const uint4*>(o + at), b = *reinterpret_cast<const uint4*>(dO + at),
                  r = *reinterpret_cast<const uint4*>(P.res + at);
      const __nv_bfloat162 *pa = reinterpret_cast<const __nv_bfloat162*>(&a),
                           *pb = reinterpret_cast<const __nv_bfloat162*>(&b),
                           *pr = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float2 x = __bfloat1622float2(pa[e]), y = __bfloat1622float2(pb[e]), z = __bfloat1622float2(pr[e]);
        s = fmaf(x.x + z.x, y.x, s);
        s = fmaf(x.y + z.y, y.y, s);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 2; c++) {
        const float4 a = *reinterpret_cast<const float4*>(o + at + 4 * c),
                     b = *reinterpret_cast<const float4*>(dO + at + 4 * c);
        s = fmaf(a.x, b.x, s);
        s = fmaf(a.y, b.y, s);
        s = fmaf(a.z, b.z, s);
        s = fmaf(a.w, b.w, s);
      }
    }
  }
#pragma unroll
  for (int x = TR / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
  if (in && threadIdx.x % TR == 0) P.delta[(size_t)(row % P.Hq) * P.Nq + row / P.Hq] = s;
}

// ------------------------------------------------------------ host
bool a16(const void* p) { return (uintptr_t)p % 16 == 0; }

// Whether equal rows have tiles to cut (the table kernel's rule on their heaviest tile).
bool worth_cutting(const SmxP& P, int l) {
  const int tile = P.tile[l], nt = ((l == 2 ? P.Tk : P.T) + tile - 1) / tile;
  int64_t total = 0;
  int most = 0;
  for (int t = 0; t < nt; t++) {
    const int nb = blocks_of(l == 2, P.causal, t, tile, P.xb[l], P.G, P.T, P.Tk);
    total += nb;
    most = nb > most ? nb : most;
  }
  return pieces_in(most, piece_blocks(total * P.B, l == 2 ? P.Hkv : P.Hq, P.target[l], P.xb[l])) > 1;
}

bool offsets_ok(const int32_t* c, int n, int64_t end) {
  if (c[0] != 0 || c[n] != end) return false;
  for (int i = 0; i < n; i++)
    if (c[i + 1] < c[i]) return false;
  return true;
}

kda_status check(const kda_softmax_problem* p, SmxP* out) {
  if (!p) return KDA_ERR_INVALID_ARG;
  if (p->B <= 0 || p->T <= 0 || p->Tk <= 0 || p->Hq <= 0 || p->Hkv <= 0) return KDA_ERR_INVALID_ARG;
  if (p->dtype != KDA_BF16 && p->dtype != KDA_F32) return KDA_ERR_INVALID_ARG;
  if ((p->causal != 0 && p->causal != 1) || !isfinite(p->scale)) return KDA_ERR_INVALID_ARG;
  if (p->Hq > 4096 || p->Hq % p->Hkv != 0) return KDA_ERR_INVALID_ARG;
  const int64_t nq = (int64_t)p->B * p->T, nk = (int64_t)p->B * p->Tk;
  // (tile counts times heads fit a grid, and a tile's last row an int)
  const int64_t most = p->dtype == KDA_F32 ? (int64_t)1 << 29 : (int64_t)1 << 30;  // (three parts' rows in one map)
  if (nq > most || nk > most || nq * p->Hq > ((int64_t)1 << 36) ||
      nk * p->Hkv > ((int64_t)1 << 36))
    return KDA_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return KDA_ERR_UNSUPPORTED;
  SmxP P = {};
  P.rows = p->cu_seqlens == nullptr;
  if (P.rows) {
    if (p->cu_seqlens_k || p->cu_seqlens_host || p->cu_seqlens_k_host) return KDA_ERR_INVALID_ARG;
    P.n_docs = p->B;
  } else {
    if (p->n_docs <= 0 || p->n_docs > (1 << 24)) return KDA_ERR_INVALID_ARG;
    if (!p->cu_seqlens_k && (p->T != p->Tk || p->cu_seqlens_k_host)) return KDA_ERR_INVALID_ARG;
    if ((uintptr_t)p->cu_seqlens % 4 != 0 || (uintptr_t)p->cu_seqlens_k % 4 != 0) return KDA_ERR_ALIGNMENT;
    if (p->cu_seqlens_host && !offsets_ok(p->cu_seqlens_host, p->n_docs, nq)) return KDA_ERR_BAD_SEQLENS;
    if (p->cu_seqlens_k_host && !offsets_ok(p->cu_seqlens_k_host, p->n_docs, nk)) return KDA_ERR_BAD_SEQLENS;
    P.n_docs = p->n_docs;
    P.cu = p->cu_seqlens;
    P.cuk = p->cu_seqlens_k ? p->cu_seqlens_k : p->cu_seqlens;
  }
  P.Nq = (int)nq;
  P.Nk = (int)nk;
  P.B = p->B;
  P.T = p->T;
  P.Tk = p->Tk;
  P.Hq = p->Hq;
  P.Hkv = p->Hkv;
  P.G = p->Hq / p->Hkv;
  P.causal = p->causal;
  P.scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->D);
  P.scale2 = P.scale * LOG2E;
  const int parts = p->dtype == KDA_F32 ? 3 : 1;
  for (int l = 0; l < 3; l++) P.tile[l] = tc_tile(p->D, parts, l);
  // Cut tiles: where whole tiles would be fewer than four for each of 152 SMs, and some could have more than a few
  // blocks; a CTA's load is the average of one CTA per SM (half of that, at D = 64 with its two CTAs, cut tiles of the
  // packed 300M step whose join took what it gave; twice as many pieces for either head dim lost 3 to 10%).
  const int wave = SMS;
  for (int l = 0; l < 3; l++) {
    const int H = l == 2 ? P.Hkv : P.Hq, other = l == 2 ? (P.rows ? P.T : P.Nq) : P.rows ? P.Tk : P.Nk;
    P.xb[l] = tc_block(p->D, parts, l);
    if ((int64_t)max_tiles(P, l) * H <= 4 * wave && (int64_t)other * (l == 2 ? P.G : 1) > 1024 &&
        (!P.rows || P.B <= 1024)) {
      P.target[l] = wave;
      P.pieces[l] = piece_room(wave, H);
      if (P.rows && !worth_cutting(P, l)) P.target[l] = P.pieces[l] = 0;
    }
  }
  for (int l = 0; l < 3; l++)  // (documents, most of them empty, times heads: a grid each)
    if ((int64_t)max_tiles(P, l) * (l == 2 ? P.Hkv : P.Hq) > 2147483647) return KDA_ERR_INVALID_ARG;
  uint32_t tag = 0x536d61u;
  for (const int32_t v : {P.B, P.T, P.Tk, P.Hq, P.Hkv, p->D, p->dtype, P.causal, P.n_docs, P.rows,
                          (int32_t)(p->cu_seqlens_k != nullptr)})
    tag = (tag ^ (uint32_t)v) * 16777619u;
  uint32_t sb;
  static_assert(sizeof(sb) == sizeof(P.scale), "");
  memcpy(&sb, &P.scale, sizeof(sb));
  tag = (tag ^ sb) * 16777619u;
  P.tag = (int32_t)(tag | 1u);
  *out = P;
  return KDA_OK;
}

// Workspace: error word, saved-problem tag and tile counts; the tables; what a saving forward keeps.
size_t layout(SmxP& P, int D, int dtype, bool bwd, void* base) {
  unsigned char* w = (unsigned char*)base;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  P.err = (int32_t*)w;
  P.wtag = (int32_t*)(w + 4);
  P.counts = (int32_t*)(w + 8);
  for (int l = 0; l < (bwd ? 3 : 1); l++) {
    if (!P.rows || P.target[l]) {
      P.pre[l] = (int32_t*)(w + take(((size_t)P.n_docs + 1) * sizeof(int32_t)));
      P.list[l] = (int4*)(w + take((size_t)max_tiles(P, l) * 2 * sizeof(int4)));
    }
    if (P.target[l]) {
      const size_t rows = (size_t)P.pieces[l] * (l == 2 ? P.Hkv : P.Hq) * P.tile[l];
      P.joins[l] = (int4*)(w + take((size_t)P.pieces[l] * sizeof(int4)));
      if (l == 0) P.pl = (float*)(w + take(rows * sizeof(float)));
      P.po[l] = (float*)(w + take(rows * (l == 2 ? 2 : 1) * D * sizeof(float)));
    }
  }
  if (bwd) {
    P.lse2 = (float*)(w + take((size_t)P.Hq * P.Nq * sizeof(float)));
    P.delta = (float*)(w + take((size_t)P.Hq * P.Nq * sizeof(float)));
    if (dtype == KDA_BF16) P.res = (bf16*)(w + take((size_t)P.Nq * P.Hq * D * sizeof(bf16)));
  }
  if (dtype == KDA_F32) {
    const size_t nq = 3 * (size_t)P.Nq * P.Hq * D * sizeof(bf16), nk = 3 * (size_t)P.Nk * P.Hkv * D * sizeof(bf16);
    P.pq = (bf16*)(w + take(nq));
    P.pk = (bf16*)(w + take(nk));
    P.pv = (bf16*)(w + take(nk));
    if (bwd) P.pg = (bf16*)(w + take(nq));
  }
  return o;
}

template <int D, typename T>
cudaError_t launch_delta(const SmxP& P, const void* o, const void* dO, void* dq, void* dk, void* dv, cudaStream_t st) {
  const int64_t rows = (int64_t)P.Nq * P.Hq, per = 256 / (D / 8), grid = (rows + per - 1) / per;
  if (grid > 2147483647) return cudaErrorInvalidValue;
  prof_begin(K_SMX_DELTA, st);
  const cudaError_t e = launch_pdl(smx_delta_kernel<D, T>, dim3((unsigned)grid), dim3(256), 0, st, P, (const T*)o,
                                   (const T*)dO, (T*)dq, (T*)dk, (T*)dv);
  prof_end(K_SMX_DELTA, st);
  return e;
}

template <int D, typename T>
cudaError_t launch_join_grads(const SmxP& P, void* dq, void* dk, void* dv, cudaStream_t st) {
  prof_begin(K_SMX_JOIN_GRADS, st);
  const cudaError_t e = launch_pdl(smx_join_grads_kernel<D, T>, dim3(4 * SMS, P.target[2] ? 3 : 1), dim3(256), 0, st, P,
                                   (T*)dq, (T*)dk, (T*)dv);
  prof_end(K_SMX_JOIN_GRADS, st);
  return e;
}

template <int D, typename T>
cudaError_t launch_join(const SmxP& P, void* o, float* lse, cudaStream_t st) {
  const int64_t most = (int64_t)(P.pieces[0] / 2) * P.Hq * (P.tile[0] / 8);  // (a cut tile has two pieces at least)
  const int64_t grid = most < 8 * SMS ? most : 8 * SMS;
  prof_begin(K_SMX_JOIN_ROWS, st);
  const cudaError_t e = launch_pdl(smx_join_rows_kernel<D, T>, dim3((unsigned)grid), dim3(256), 0, st, P, (T*)o, lse);
  prof_end(K_SMX_JOIN_ROWS, st);
  return e;
}

cudaError_t launch_table(const SmxP& P, cudaStream_t st) {
  prof_begin(K_SMX_TABLE, st);
  const cudaError_t e = launch_pdl(smx_table_kernel, dim3(P.save ? 3 : 1), dim3(TT), 0, st, P);
  prof_end(K_SMX_TABLE, st);
  return e;
}

}  // namespace
}  // namespace smx
}  // namespace kda

using namespace kda;
using namespace kda::smx;

extern "C" KDA_API size_t kda_softmax_workspace_size(const kda_softmax_problem* p, int for_backward) {
  SmxP P;
  if (check(p, &P) != KDA_OK) return 0;
  return layout(P, p->D, p->dtype, for_backward != 0, nullptr);
}

extern "C" KDA_API kda_status kda_softmax_fwd(const kda_softmax_problem* p, const void* q, const void* k,
                                              const void* v, void* o, float* lse, int save_for_backward,
                                              void* workspace, size_t workspace_bytes, cudaStream_t st) {
  SmxP P;
  const kda_status s = check(p, &P);
  if (s != KDA_OK) return s;
  if (!q || !k || !v || !o || !lse) return KDA_ERR_INVALID_ARG;
  if (!a16(q) || !a16(k) || !a16(v) || !a16(o) || !a16(lse)) return KDA_ERR_ALIGNMENT;
  P.save = save_for_backward != 0;
  if (!workspace || workspace_bytes < layout(P, p->D, p->dtype, P.save, workspace)) return KDA_ERR_WORKSPACE;
  if ((uintptr_t)workspace % 256 != 0) return KDA_ERR_ALIGNMENT;
  if ((P.list[0] || P.list[1] || P.list[2]) && launch_table(P, st) != cudaSuccess) return KDA_ERR_CUDA;
  cudaError_t e;
  if (p->dtype == KDA_F32) {
    const float* x[3] = {(const float*)q, (const float*)k, (const float*)v};
    bf16* const parts[3] = {P.pq, P.pk, P.pv};
    const int64_t nk = (int64_t)P.Nk * P.Hkv * p->D, n[3] = {(int64_t)P.Nq * P.Hq * p->D, nk, nk};
    e = launch_split(3, x, parts, n, st);
    if (e == cudaSuccess) e = launch_tc_fwd(P, p->D, 3, P.pq, P.pk, P.pv, o, lse, st);
  } else {
    e = launch_tc_fwd(P, p->D, 1, q, k, v, o, lse, st);
  }
  if (e == cudaSuccess && P.target[0]) {
    if (p->dtype == KDA_F32)
      e = p->D == 64 ? launch_join<64, float>(P, o, lse, st) : launch_join<128, float>(P, o, lse, st);
    else
      e = p->D == 64 ? launch_join<64, bf16>(P, o, lse, st) : launch_join<128, bf16>(P, o, lse, st);
  }
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" KDA_API kda_status kda_softmax_bwd(const kda_softmax_problem* p, const void* q, const void* k,
                                              const void* v, const void* o, const void* dO, void* dq, void* dk,
                                              void* dv, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  SmxP P;
  const kda_status s = check(p, &P);
  if (s != KDA_OK) return s;
  if (!q || !k || !v || !o || !dO || !dq || !dk || !dv) return KDA_ERR_INVALID_ARG;
  for (const void* x : {q, k, v, o, dO, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!a16(x)) return KDA_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < layout(P, p->D, p->dtype, true, workspace)) return KDA_ERR_WORKSPACE;
  if ((uintptr_t)workspace % 256 != 0) return KDA_ERR_ALIGNMENT;
  cudaError_t e;
  if (p->dtype == KDA_F32)
    e = p->D == 64 ? launch_delta<64, float>(P, o, dO, dq, dk, dv, st) : launch_delta<128, float>(P, o, dO, dq, dk, dv, st);
  else
    e = p->D == 64 ? launch_delta<64, bf16>(P, o, dO, dq, dk, dv, st) : launch_delta<128, bf16>(P, o, dO, dq, dk, dv, st);
  if (e != cudaSuccess) return KDA_ERR_CUDA;
  if (p->dtype == KDA_BF16) {
    e = launch_tc_bwd(P, p->D, 1, q, k, v, dO, dq, dk, dv, st);
  } else {
    const float* x[1] = {(const float*)dO};
    bf16* const parts[1] = {P.pg};
    const int64_t n[1] = {(int64_t)P.Nq * P.Hq * p->D};
    e = launch_split(1, x, parts, n, st);
    if (e == cudaSuccess)
      e = p->D == 64 ? launch_tc_bwd(P, 64, 3, P.pq, P.pk, P.pv, P.pg, dq, dk, dv, st)
                     : launch_f32_bwd(P, (float*)dq, (float*)dk, (float*)dv, st);
  }
  if (e == cudaSuccess && (P.target[1] || P.target[2])) {
    if (p->dtype == KDA_F32)
      e = p->D == 64 ? launch_join_grads<64, float>(P, dq, dk, dv, st) : launch_join_grads<128, float>(P, dq, dk, dv, st);
    else
      e = p->D == 64 ? launch_join_grads<64, bf16>(P, dq, dk, dv, st) : launch_join_grads<128, bf16>(P, dq, dk, dv, st);
  }
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
