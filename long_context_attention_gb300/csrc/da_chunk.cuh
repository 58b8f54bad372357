// Chunks of new tokens over the paged cache: the host-side problem, the plan of
// a call, the line of work that the CTAs share, and where partial results lie.
// Shared by the kernels of both types (paged_chunk_f32.cu, paged_chunk_bf16.cu).
//
// Rows.  A row is one query of one query head.  The n new tokens of a sequence
// take n8 = n rounded up to 8 rows for each of its query heads, head by head.
// A column tile is up to `edge` rows that a CTA works on at once:
//   wide   (n > edge / 2): `edge` successive queries of one query head;
//   narrow (n <= edge / 2): all n8 rows of edge / n8 heads of one key head, so
//          that the key head's keys are read once for them.
// Key tiles are `edge` keys.
//
// The line.  A segment is what shares keys and totals: one query head of a wide
// sequence, one key head of a narrow one.  Each begins with `head` units (what
// beginning a piece costs), then has its key tiles, each worth the column tiles
// that see it.  The segments of all sequences lie on a line, every CTA takes an
// equal stretch of it, and the tiles of a segment that begin in the stretch are a
// piece.  A piece walks its column tiles in the queries' order, and its key tiles
// inside each, so that a key's total passes from query to query in one CTA.
//
// Partial results of a piece: those of a segment's first piece lie in the rows'
// own places (a), those of the piece a CTA continues in the CTA's places (b).
// They are joined in the line's order: equal calls give equal bits.
//
// Slices.  Every CTA has places for the rows of a sequence's new tokens (b), so that
// long parts go by slices of up to kChunkSlice of them: a chunk is what two halves of
// it are, one after the other.
//
// Values that are not finite.  A query's share of a key that it does not see is 0, and 0
// times infinity or NaN would be NaN.  So such elements of new tokens' values are cleared
// where they enter the products, and added to the outputs of the rows that see them; a
// flag a sequence and a bit a token and key head (chunk_join) say whether there are any.
#pragma once

#include "da_paged.h"
#include "da_ptx.cuh"

namespace da {

// One call.
struct PagedChunk {
  dilution_attn_paged_cache c;
  const void *q;
  void *out;
  const int32_t *cu;   // [S + 1]
  int N, max_new, max_len;
  int first;           // of each sequence's new tokens the first of this slice, which has up to max_new
  int all_new;         // new tokens of a sequence, at most
  HeadScale hs;
  float eps;
  bool earlier;
  int *status;
  uint8_t *ws;
};

// A sequence as the kernels see it (n = 0: nothing to do, or not valid).
struct ChunkSeq {
  int len, n, row0, tok0;   // length, new tokens, n8 of the sequences before, first token
};

// a / b of numbers that are mostly short: a 64-bit division takes several times as long.
DA_HD long long chunk_div(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// Equal cut of the line.
struct ChunkCut {
  long long total, base;
  int ctas, rem;
  DA_HD long long first(int cta) const { return cta * base + (cta < rem ? cta : rem); }
  DA_HD int cta_of(long long unit) const {
    const long long cut = rem * (base + 1);
    return (int)(unit < cut ? chunk_div(unit, base + 1) : rem + chunk_div(unit - cut, base));
  }
};
DA_HD ChunkCut chunk_cut(long long total, int ctas) {
  ChunkCut c;
  c.total = total;
  c.ctas = (int)(ctas < total ? ctas : total);
  if (c.ctas < 1) c.ctas = 1;
  c.base = chunk_div(total, c.ctas);
  c.rem = (int)(total - c.base * c.ctas);
  if (c.base < 1) c.base = 1;   // an empty line
  return c;
}

// What the units are: of a narrow key tile (its copies), of a column tile at a key
// tile, of 8 of its rows there, of a segment, and of each of its column tiles.
struct ChunkCost {
  int keys, tile, rows8, head, head_tile;
};

struct ChunkPlan {
  int edge, G, page_shift;
  int ctas_keys, ctas_values;
  ChunkCost cost;
  long long rows;        // rows of all heads, at most
  int cta_rows;          // rows of a CTA's places
  size_t seq_off, cum_off, odd_off, map_off, ml_a, ml_b, nl, acc_a, acc_b, total;
  size_t logits;         // q . k of (token, query head) and key, where they are kept
  int logits_ld;         // their keys (0: not kept)
  int logits_seq;        // tokens that each sequence has of them (0: as many as are new, one behind the other)
};
constexpr int kChunkFold = 4;       // up to so many new tokens leave room for second terms in their eight rows
constexpr int kChunkLogits = 128;   // their keys are a multiple of this, a key tile of bf16

// New tokens of a sequence in a slice.  (One prompt of 131072 tokens, 12 / 4 heads, d = 128:
// a workspace of 0.73 GB, in fp32 1.39; all at once 11.7 and 22.2, for 84.5 ms where the slices
// take 87.9.  32768 tokens 6.8 and 7.2 ms, in fp32 142 and 140; 12 heads of d = 64, 131072
// tokens 69.6 and 69.9.)
constexpr int kChunkSlice = 8192;

inline ChunkPlan chunk_plan(int S, int Hq, int Hkv, int d, long long N, int max_new, int page_size, int edge, int ctas_keys,
                            int ctas_values, ChunkCost cost) {
  ChunkPlan w{};
  w.edge = edge;
  w.G = Hq / Hkv;
  while ((1 << w.page_shift) < page_size) ++w.page_shift;
  w.ctas_keys = ctas_keys;
  w.ctas_values = ctas_values;
  w.cost = cost;
  if (N > (long long)S * max_new) N = (long long)S * max_new;   // (more are padding, or another slice's)
  const long long busy = N < S ? N : S;   // sequences with new tokens
  w.rows = (N + 7 * busy) * Hq;
  const int narrow = (int)round_up(max_new < edge / 2 ? max_new : edge / 2, 8) * w.G;
  const int wide = max_new > edge / 2 ? (int)round_up(max_new, 8) : 0;
  w.cta_rows = narrow > wide ? narrow : wide;
  const long long b_keys = (long long)ctas_keys * w.cta_rows, b_values = (long long)ctas_values * w.cta_rows;
  auto next = [](size_t off, long long bytes) { return (size_t)round_up((int64_t)off + bytes, 256); };
  w.seq_off = kStatusBytes;
  w.cum_off = next(w.seq_off, ((long long)S + 1) * (long long)sizeof(ChunkSeq));   // (the last: how many rows a head)
  w.odd_off = next(w.cum_off, ((long long)S + 1) * 8);
  w.map_off = next(w.odd_off, (long long)S * 4);
  w.ml_a = next(w.map_off, w.rows / 8 / w.G);
  w.ml_b = next(w.ml_a, w.rows * 8);
  w.nl = next(w.ml_b, b_keys * 8);
  w.acc_a = next(w.nl, w.rows * 4);
  w.acc_b = next(w.acc_a, w.rows * acc_stride(d) * 4);
  w.total = next(w.acc_b, b_values * acc_stride(d) * 4);
  return w;
}

// The segments of a sequence (all alike).
struct ChunkShape {
  int len, n, n8, P;       // P: place of the first query
  int tiles, cols;         // key tiles, column tiles
  int flat;                // key tiles before this one are seen by every column tile
  int segs, step;          // segments; rows of a column tile
  bool wide;
  long long w, w1, head, units;   // of a flat key tile; of a column tile there; before the first; of the segment

  DA_HD void set(int len_, int n_, int Hq, int Hkv, int edge, const ChunkCost &c) {
    len = len_;
    n = n_;
    n8 = (n + 7) & ~7;
    P = len - n;
    tiles = (len + edge - 1) / edge;
    wide = n > edge / 2;
    const int G = Hq / Hkv;
    if (wide) {
      segs = Hq;
      step = edge;
      cols = (n + edge - 1) / edge;
      flat = (P + edge - 1) / edge;
      w1 = c.tile + c.rows8 * (edge / 8);
      w = w1 * cols;
    } else {
      segs = Hkv;
      step = edge / n8 * n8;
      cols = (G * n8 + step - 1) / step;
      flat = tiles;
      w = c.keys + (long long)c.tile * cols + (long long)c.rows8 * G * (n8 / 8);
      w1 = 0;
    }
    head = c.head + (long long)c.head_tile * cols;
    units = pos(tiles);
  }
  // Place of key tile t in the segment: tile flat + j is not seen by the first j column tiles.
  DA_HD long long pos(int t) const {
    const long long j = t > flat ? t - flat : 0;
    return head + t * w - w1 * (j * (j - 1) / 2);
  }
  // The first key tile (or `tiles`) at place u or behind it.
  DA_HD int first_at(long long u) const {
    if (u <= head) return 0;
    if (u > pos(tiles - 1)) return tiles;
    const long long t = chunk_div(u - head + w - 1, w);   // exact while the tiles are flat
    if (t <= flat) return (int)t;
    int lo = flat, hi = tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (pos(mid) >= u)
        hi = mid;
      else
        lo = mid + 1;
    }
    return lo;
  }
  // Column tile b: the key tiles that it sees, and the first one that sees key tile t.
  DA_HD int seen(int b, int edge) const {
    const int last = wide ? P + (n < (b + 1) * edge ? n : (b + 1) * edge) : len;
    return (last + edge - 1) / edge;
  }
  DA_HD int col0(int t) const { return wide && t > flat ? t - flat : 0; }
};

#if defined(__CUDACC__)
struct ChunkLine {
  const ChunkSeq *seq;    // [S + 1]
  const long long *cum;   // [S + 1] units of the sequences before
};
__device__ __forceinline__ ChunkLine chunk_line(const PagedChunk &p, const ChunkPlan &w) {
  return ChunkLine{reinterpret_cast<const ChunkSeq *>(p.ws + w.seq_off),
                   reinterpret_cast<const long long *>(p.ws + w.cum_off)};
}
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkLine &l, int s) {
  const int4 v = __ldcg(reinterpret_cast<const int4 *>(l.seq + s));
  return ChunkSeq{v.x, v.y, v.z, v.w};
}

// Whether a new token of the sequence has a value that is not finite.
__device__ __forceinline__ int *chunk_odd(const PagedChunk &p, const ChunkPlan &w) { return reinterpret_cast<int *>(p.ws + w.odd_off); }
// Of which eight of them (from row0 + 8 i of the rows of a head) and key head.
__device__ __forceinline__ uint8_t *chunk_odd_map(const PagedChunk &p, const ChunkPlan &w, int row, int hkv) {
  return p.ws + w.map_off + (size_t)(row / 8) * p.c.Hkv + hkv;
}
__device__ __forceinline__ bool chunk_not_finite(uint32_t x) { return (x & 0x7f800000u) == 0x7f800000u; }   // bits of a float
// Of 16 bytes of values, bf16 or fp32: zeros for what is not finite; whether there was any.
__device__ __forceinline__ bool chunk_clear(uint4 &v, bool half) {
  bool any = false;
  uint32_t *x[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (chunk_not_finite(*x[i])) any = true, *x[i] &= half ? 0xffffu : 0u;
    if (half && chunk_not_finite(*x[i] << 16)) any = true, *x[i] &= 0xffff0000u;
  }
  return any;
}
// What is not finite of columns c .. c + 3 of token t's values, onto a.
template <int D, typename E>
__device__ __forceinline__ void chunk_see(const PagedChunk &p, int sh, int s, int hkv, int t, int c, float4 &a) {
  const int page = __ldcg(p.c.page_table + (size_t)s * p.c.max_pages + (t >> sh));
  if ((unsigned)page >= (unsigned)p.c.num_pages) return;
  const E *at = static_cast<const E *>(p.c.v_pages) +
                ((((size_t)page * p.c.Hkv + hkv) << sh) + (t & ((1 << sh) - 1))) * D + c;
  uint4 x;
  if constexpr (sizeof(E) == 4) {
    x = __ldcg(reinterpret_cast<const uint4 *>(at));
  } else {
    const uint2 y = __ldcg(reinterpret_cast<const uint2 *>(at));
    x = make_uint4(y.x << 16, y.x & 0xffff0000u, y.y << 16, y.y & 0xffff0000u);
  }
  if (chunk_not_finite(x.x)) a.x += __uint_as_float(x.x);
  if (chunk_not_finite(x.y)) a.y += __uint_as_float(x.y);
  if (chunk_not_finite(x.z)) a.z += __uint_as_float(x.z);
  if (chunk_not_finite(x.w)) a.w += __uint_as_float(x.w);
}

// The last sequence with cum <= u (one with units, for u on the line).  A warp's
// lanes look at 32 places at once.
__device__ __forceinline__ int chunk_find(const ChunkLine &l, int S, long long u, int lane) {
  int lo = 0, n = S;   // in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool le = lane * step < n && __ldcg(l.cum + at) <= u;
    const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;   // cum does not decrease
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Pieces of a CTA's stretch; every warp walks them for itself, all lanes alike.
struct ChunkWalk {
  ChunkShape g;
  ChunkSeq q;
  int s, seg;            // sequence, segment of it
  int tile, end;         // key tiles of the piece (tile >= end: none left)
  long long base, to;    // the segment's place; the stretch's end
  __device__ __forceinline__ void load(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l) {
    q = chunk_seq(l, s);
    g.set(q.len, q.n, p.c.Hq, p.c.Hkv, w.edge, w.cost);
  }
  __device__ void start(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l, const ChunkCut &cut, int lane) {
    tile = end = 0;
    const long long from = cut.first(blockIdx.x);
    to = (int)blockIdx.x < cut.ctas ? cut.first(blockIdx.x + 1) : 0;
    if (from >= to || from >= cut.total) return;
    s = chunk_find(l, p.c.S, from, lane);
    load(p, w, l);
    base = __ldcg(l.cum + s);
    seg = (int)chunk_div(from - base, g.units);
    base += seg * g.units;
    tile = g.first_at(from - base);
    end = min(g.first_at(to - base), g.tiles);
    if (tile >= end) settle(p, w, l);
  }
  __device__ __forceinline__ bool any() const { return tile < end; }
  __device__ void next(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l) {
    tile = end;
    settle(p, w, l);
  }
  // The next segment's first piece, if its first tile lies in the stretch.
  __device__ void settle(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l) {
    if (tile < g.tiles) {   // the stretch ends inside the segment
      end = tile;
      return;
    }
    base += g.units;
    tile = end = 0;
    if (base >= to) return;
    if (++seg == g.segs) {
      seg = 0;
      do {   // on to the next sequence with new tokens: the line goes on
        ++s;
        q = chunk_seq(l, s);
      } while (q.n == 0);
      g.set(q.len, q.n, p.c.Hq, p.c.Hkv, w.edge, w.cost);
    }
    end = g.first_at(to - base);
  }
  // First row of the segment in the rows' own places.
  __device__ __forceinline__ long long row0(const PagedChunk &p, const ChunkPlan &w) const {
    return (long long)q.row0 * p.c.Hq + (long long)seg * (g.wide ? 1 : w.G) * g.n8;
  }
  __device__ __forceinline__ int hkv(const ChunkPlan &w) const { return g.wide ? seg / w.G : seg; }
};

// The kept logits of a sequence's query.
__device__ __forceinline__ float *chunk_logits(const PagedChunk &p, const ChunkPlan &w, int s, int tok0, int query, int hq) {
  const size_t token = w.logits_seq > 0 ? (size_t)s * w.logits_seq + query : (size_t)tok0 + query;
  return reinterpret_cast<float *>(p.ws + w.logits) + (token * p.c.Hq + hq) * (size_t)w.logits_ld;
}

// The place of the piece's row r (of the segment) among `stride` floats a row.
__device__ __forceinline__ float *chunk_place(const PagedChunk &p, size_t a, size_t b, long long row0, int cta_rows, int tile,
                                              int cta, int r, int stride) {
  return reinterpret_cast<float *>(p.ws + (tile == 0 ? a : b)) +
         ((tile == 0 ? row0 : (long long)cta * cta_rows) + r) * stride;
}

// Where sums of share v lie, from the place of a row that is a multiple of eight: eight
// rows' 16-byte pieces beside each other (`piece`: columns 4 piece ..), then their sums
// of shares.  A warp with a row a lane so writes 4 lines at a time, and not 32, while the
// next column tile's products wait (16 prompts of d = 128: values 860 -> 811 us).
DA_HD constexpr int chunk_acc(int d, int row, int piece) { return row / 8 * 8 * acc_stride(d) + (piece * 8 + row % 8) * 4; }
DA_HD constexpr int chunk_acc_sum(int d, int row) { return row / 8 * 8 * acc_stride(d) + 8 * d + row % 8; }

// Eight rows (of one query head and one column tile), found by their number among
// all rows of the call: their sequence, query head, first query and segment.  All
// lanes of a warp call it alike.  false: behind the last row.
struct ChunkRows {
  ChunkShape g;
  ChunkSeq q;
  int s, hq, i;          // sequence, query head, first query
  int r;                 // first row of the eight in the segment
  int seen;              // key tiles that their column tile sees
  long long base, row0;  // the segment's place on the line; its first row
};
// The last sequence whose first row, of `heads` heads, is at or before this one (see chunk_find).
__device__ __forceinline__ int chunk_seq_of(const ChunkLine &l, int S, int heads, long long row, int lane) {
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool le = lane * step < n && (long long)__ldcg(&l.seq[at].row0) * heads <= row;
    const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}
__device__ __forceinline__ bool chunk_rows(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l, long long row, int lane,
                                           ChunkRows &x) {
  const int lo = chunk_seq_of(l, p.c.S, p.c.Hq, row, lane);
  x.s = lo;
  x.q = chunk_seq(l, lo);
  if (x.q.n == 0) return false;   // (of the sequences that begin there the last one: behind the last row)
  x.g.set(x.q.len, x.q.n, p.c.Hq, p.c.Hkv, w.edge, w.cost);
  const long long at = row - (long long)x.q.row0 * p.c.Hq;
  x.hq = (int)chunk_div(at, x.g.n8);
  if (x.hq >= p.c.Hq) return false;
  x.i = (int)(at - (long long)x.hq * x.g.n8);
  const int seg = x.g.wide ? x.hq : x.hq / w.G;
  x.row0 = (long long)x.q.row0 * p.c.Hq + (long long)seg * (x.g.wide ? 1 : w.G) * x.g.n8;
  x.r = (int)(row - x.row0);
  x.seen = x.g.seen(x.r / x.g.step, w.edge);
  x.base = __ldcg(l.cum + lo) + seg * x.g.units;
  return true;
}
// The pieces that the rows' column tile takes part in, 32 CTAs at a time: the first
// key tile of CTA `cta`'s piece, or -1.
struct ChunkPieces {
  int first = 0, last = -1;   // CTAs
  __device__ __forceinline__ void find(const ChunkRows &x, const ChunkCut &cut) {
    first = cut.cta_of(x.base + x.g.pos(0));
    last = cut.cta_of(x.base + x.g.pos(x.seen - 1));
  }
  __device__ __forceinline__ int tile(const ChunkRows &x, const ChunkCut &cut, int cta) const {
    if (cta > last) return -1;
    const int t = cta == first ? 0 : x.g.first_at(cut.first(cta) - x.base);
    return t < x.seen && x.base + x.g.pos(t) < cut.first(cta + 1) ? t : -1;
  }
};
#endif  // __CUDACC__

}  // namespace da
