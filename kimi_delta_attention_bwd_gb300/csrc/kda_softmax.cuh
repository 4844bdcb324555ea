// Softmax attention with grouped heads: declarations shared by its kernels, all
// on the tensor cores (tables and entries: kda_softmax.cu, forward and backward:
// kda_softmax_tc.cu, the backward of fp32 io at D = 128: kda_softmax_f32.cu).
#pragma once
#include "kda_internal.cuh"
#include "../../include/kda.h"

#include <limits.h>

namespace kda {
namespace smx {

using bf16 = __nv_bfloat16;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct SmxP {
  int Nq, Nk, B, T, Tk, Hq, Hkv, G, n_docs, causal, rows;  // rows: documents are the rows of T queries, Tk keys
  int save, tag;
  float scale, scale2;  // scale2 = scale log2(e): exponentials are powers of two
  const int32_t *cu, *cuk;
  int32_t *err, *wtag, *counts;  // counts[l]: entries of list l; counts[3 + l]: its cut tiles
  int32_t* pre[3];               // [n_docs + 1] first tile of each document
  int4* list[3];                 // two int4 a tile, see Tile; 0: forward's queries, 1: dq's queries, 2: dk and dv's keys
                                 // (nullptr: equal rows, whose tiles follow from their number)
  // Tiles that are cut into pieces along the other side, see smx_table_kernel.  Per list: rows of a block of that
  // side, how many CTAs to aim at (0: no tile is cut), room for how many pieces, the cut tiles (first row, rows, first
  // piece, pieces), and the pieces' fp32 results [piece][head][tile][D]: o and its log2 sums (pl); dq; dk, then dv.
  int xb[3], target[3], pieces[3];
  int4* joins[3];
  float *po[3], *pl;
  int tile[3];                   // rows a tile
  float *lse2, *delta;           // [Hq][Nq]: log2 of the rows' sums, saved by the forward; sum_d o dO
  bf16* res;                     // [Nq, Hq, D] what rounding o to bf16 left, saved by the forward
  bf16 *pq, *pk, *pv, *pg;       // fp32 io: parts of q, k, v (the forward's) and dO
};

// Rows t * tile .. of a document's queries (or keys): its first query, queries, first key, keys.
// Blocks j0 .. j1 - 1 of the other side (keys; for dk and dv queries, head after head) are taken, as piece `piece` (-1: all).
struct Tile {
  int q0, Lq, k0, Lk, t, j0, j1, piece;
};

// Keys that query i of a document sees, as a bound on their index; queries that key j does not reach.
__host__ __device__ inline int keys_of(int causal, int i, int Lq, int Lk) {
  if (!causal) return Lk;
  const int n = i + 1 + Lk - Lq;
  return n < 0 ? 0 : n > Lk ? Lk : n;
}
__host__ __device__ inline int first_query(int causal, int j, int Lq, int Lk) {
  if (!causal) return 0;
  const int i = j - (Lk - Lq);
  return i < 0 ? 0 : i > Lq ? Lq : i;
}

// Tile x of list l, the heavy ones first; false past the last.  by_key: the tiles are of keys.  The backward's lists are
// the forward's: none is read from a workspace that another problem's forward filled.
__device__ __forceinline__ bool tile_of(const SmxP& P, int l, int x, bool by_key, Tile& t) {
  t.j0 = 0;
  t.j1 = INT_MAX;
  t.piece = -1;
  if (!P.list[l]) {
    const int nt = ((by_key ? P.Tk : P.T) + P.tile[l] - 1) / P.tile[l], i = x / P.B, b = x - i * P.B;
    if (i >= nt) return false;
    t.t = by_key ? i : nt - 1 - i;
    t.q0 = b * P.T;
    t.k0 = b * P.Tk;
    t.Lq = P.T;
    t.Lk = P.Tk;
    return true;
  }
  const int tag = l > 0 ? *P.wtag : P.tag;
  if (x >= P.counts[l] || tag != P.tag) return false;
  const int4 a = P.list[l][2 * (size_t)x], b = P.list[l][2 * (size_t)x + 1];
  t.q0 = a.x;
  t.Lq = a.y;
  t.k0 = a.z;
  t.Lk = a.w;
  t.t = b.x;
  t.j0 = b.y;
  t.j1 = b.z;
  t.piece = b.w;
  return true;
}

// Blocks of the other side that tile t of a document has.
__host__ __device__ inline int blocks_of(bool by_key, int causal, int t, int tile, int xb, int G, int Lq, int Lk) {
  if (by_key) return ((Lq + xb - 1) / xb - first_query(causal, t * tile, Lq, Lk) / xb) * G;
  const int end = (t + 1) * tile < Lq ? (t + 1) * tile : Lq;
  return (keys_of(causal, end - 1, Lq, Lk) + xb - 1) / xb;
}

// The tiles of a list in the documents' order: offsets, the documents' first tiles.
struct Tiles {
  const int32_t *cu, *cuk, *pre;
  int n, tile, xb, G, causal;  // n: documents
  bool by_key;
  struct Found {
    int4 doc;
    int t, nb;  // tile of the document; its blocks of the other side
  };
  __host__ __device__ Found find(int x) const {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    Found f;
    f.t = x - pre[lo];
    f.doc = make_int4(cu[lo], cu[lo + 1] - cu[lo], cuk[lo], cuk[lo + 1] - cuk[lo]);
    f.nb = blocks_of(by_key, causal, f.t, tile, xb, G, f.doc.y, f.doc.w);
    return f;
  }
  // Blocks of tiles first, first + step, .. below end: 600 tiles of millions of blocks pass 32 bits.
  __host__ __device__ int64_t blocks(int first, int end, int step) const {
    int64_t sum = 0;
    for (int x = first; x < end; x += step) sum += find(x).nb;
    return sum;
  }
};
// Blocks of a piece: the load that `target` CTAs have on average of a list's blocks with H heads, 512 rows at least.
__host__ __device__ inline int64_t piece_blocks(int64_t blocks, int H, int target, int xb) {
  const int64_t per = (blocks * H + target - 1) / target, least = 512 / xb;
  return per > least ? per : least;
}
// Pieces of a tile of nb blocks: one up to 1.5 times that load.
__host__ __device__ inline int pieces_in(int nb, int64_t per) { return nb > per + per / 2 ? (int)((nb + per - 1) / per) : 1; }
// Room for the pieces of all cut tiles: a tile of q > 1.5 loads has ceil(q) pieces, at most 1.5 q, and all tiles' q sum to
// at most target / H.
__host__ __device__ inline int piece_room(int target, int H) { return (target + H - 1) / H * 3 / 2 + 2; }

// The backward's kernels read only what a forward of the same problem saved.
__device__ __forceinline__ bool saved(const SmxP& P) {
  if (*P.wtag == P.tag && *P.err == KDA_OK) return true;
  if (*P.wtag != P.tag && blockIdx.x == 0 && threadIdx.x == 0) *P.err = KDA_ERR_WORKSPACE;
  return false;
}

// Tensor-core kernels.  parts = 1: bf16 io; 3: fp32 io, its inputs as three bf16 arrays one behind the other
// (launch_split); their backward at D = 128 is launch_f32_bwd.  Rows of list l's tiles: tc_tile, of their blocks: tc_block.
constexpr int tc_block(int D, int parts, int l) {
  return D == 64 ? 64 : parts == 3 ? (l == 0 ? 64 : 32) : 128;
}
constexpr int tc_tile(int D, int parts, int l) { return l > 0 || (parts == 3 && D == 128) ? 128 : 256; }
cudaError_t launch_tc_fwd(const SmxP& P, int D, int parts, const void* q, const void* k, const void* v, void* o,
                          float* lse, cudaStream_t st);
cudaError_t launch_tc_bwd(const SmxP& P, int D, int parts, const void* q, const void* k, const void* v, const void* dO,
                          void* dq, void* dk, void* dv, cudaStream_t st);
// Up to three fp32 arrays (their sizes multiples of 8) into their parts.
cudaError_t launch_split(int n, const float* const* x, bf16* const* parts, const int64_t* values, cudaStream_t st);

cudaError_t launch_f32_bwd(const SmxP& P, float* dq, float* dk, float* dv, cudaStream_t st);  // (of the parts in P)

// Upper bound on the entries of list l: its tiles, and the pieces of those that are cut.
inline int max_tiles(const SmxP& P, int l) {
  const int n = l == 2 ? P.Nk : P.Nq, t = P.tile[l], more = P.pieces[l];
  if (P.rows) return P.B * (((l == 2 ? P.Tk : P.T) + t - 1) / t) + more;
  const int64_t m = (int64_t)n / t + P.n_docs;
  return (int)(m < n ? m : n) + more;  // (every tile has a row)
}

}  // namespace smx
}  // namespace kda
