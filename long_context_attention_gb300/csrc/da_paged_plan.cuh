// The paged decode step's plan: workspace layout, the line of work units
// that the CTAs share, and where each row's partial results lie.  Shared by the
// streaming kernels (paged_decode_bf16.cu, paged_decode_f32.cu) and those of a
// prefix with many rows (paged_prefix_bf16.cu).
#pragma once

#include "da_paged.h"
#include "da_ptx.cuh"

namespace da {

constexpr int kPgtMaxSeqs = 704;                  // lengths kept in shared memory (a larger batch goes in parts)
// Keys per stage (16 KB of K or V) and rows of a segment at most.
DA_HD constexpr int pgt_tile(int d, int dtype = DA_BF16) { return (dtype == DA_BF16 ? 8192 : 4096) / d; }
constexpr int kPgtRowTile = 16;
// Rows of a prefix's segment in bf16 at d = 64, if no segment has more and the keys
// stay in L2 until they are read again: 9 to 16 rows are a product more for every 16
// keys and two exponentials a lane instead of one.  16 x 12 heads x 2048 + 300 / 8192
// + 300 / 32768 (50 MB of keys): 17.5 / 23.5 / 44.1 us a step, with 16 rows 20.5 / 27.3 /
// 46.6; 12 x 12 x 65536 (101 MB) 75.6 against 67.5; at d = 128 37.3 against 32.4 for 96
// rows x 2 heads x 16384.
constexpr int kPgtPreRows = 8;
constexpr int64_t kPgtPreBytes = 64ll << 20;
DA_HD constexpr int pgt_warps(int d) { return pgt_tile(d) / 16; }    // pgt_keys: consumer warps, 16 keys of a stage each
DA_HD constexpr int pgt_threads(int d) { return 32 * pgt_warps(d) + 32; }   // and the producer warp
constexpr int kPgtMaxCtas = 2 * 152;              // two resident CTAs on each SM

constexpr int kPgtHead = 4;   // units of a segment before its first tile (a piece costs ~2 us beside its tiles' 0.5 us)

// Which kernels take a shared prefix.  The streaming kernels work on 16 rows (of
// the batch's sequences x query heads of one key head) at a time and read the
// prefix's keys from L2 once per 16 rows; the tcgen05 kernels take 64 rows, but
// are two launches more.  Device time of a step, tcgen05 against streaming, in us
// (rows x key heads x keys; below 4 M pairs and above 6 M measured on other inputs):
//   d = 64:  96 x 12 x 16384 (19 M pairs) 77 / 111, 64 x 12 x 8192 (6.3 M) 46.7 / 55.3,
//            40 x 8 x 16384 (5.2 M) 45.7 / 45.7, 46 x 12 x 9216 (5.1 M) 48.1 / 52.1,
//            24 x 12 x 16384 (4.7 M) 46.6 / 46.6, 64 x 2 x 36864 (4.7 M) 41.3 / 40.3,
//            46 x 12 x 8192 (4.5 M) 45.4 / 46.9, 64 x 1 x 70016 (4.5 M) 48.2 / 37.7,
//            24 x 12 x 14592 (4.2 M) 45.4 / 40.3, 17 x 8 x 30848 (4.2 M) 58.3 / 47.6,
//            17 x 12 x 16384 (3.3 M) 38.1 / 35.8, 44 x 2 x 37824 (3.3 M) 36.1 / 30.0;
//   d = 128: 40 x 8 x 16384 (5.2 M) 57.3 / 66.2, 24 x 12 x 16384 (4.7 M) 62.8 / 66.1,
//            96 x 4 x 12288 (4.7 M) 43.8 / 42.9, 64 x 2 x 36864 (4.7 M) 50.4 / 49.3,
//            64 x 1 x 73728 (4.7 M) 59.2 / 47.2, 24 x 12 x 14592 (4.2 M) 59.4 / 59.4,
//            96 x 2 x 16384 (3.1 M) 37.4 / 33.0.
// With many key heads the sides meet between 4.2 and 4.7 M pairs; with one key head or
// 17 rows of a segment's 64 the streaming kernels are still faster just above the bound.
constexpr int kPgxMinRows = 17;
constexpr int64_t kPgxMinPairs = 4ll << 20;
enum PgxUse { kPgxAuto, kPgxNever, kPgxAlways };
constexpr int kPgxRows = 64;      // rows of a segment there, at most
constexpr int kPgxTile = 128;     // keys of a tile
constexpr int kPgxCtas = 152;     // pgx_values: one CTA an SM
constexpr int kPgxKeyCtas = 304;  // pgx_keys: two
// Beginning and ending a piece there costs about as much as this many tiles (8 us
// of normalisers, queries and first copies, 3 us of sums; a tile 1 to 2 us; pgx_keys
// 3 us and 1 us): a segment takes as many units before its first tile, so that a
// CTA with two pieces gets fewer tiles (steps with 32 x 16 heads x 32768 / 64 x 12
// x 131072 / 32 x 12 x 32768: 76.8 / 255.6 / 70.9 us, with 5 81.0 / 257.0 / 72.8, with
// 10 78.0 / 254.9 / 69.5).
constexpr int kPgxHead = 8;

// Equal cut of `total` units into stretches of base or base + 1.
struct PgtCut {
  int total, ctas, base, rem;
  DA_HD int first(int cta) const { return cta < ctas ? cta * base + (cta < rem ? cta : rem) : total; }
  DA_HD int cta_of(int unit) const {   // total > 0
    const int cut = rem * (base + 1);
    return unit < cut ? unit / (base + 1) : rem + (unit - cut) / base;
  }
};
DA_HD PgtCut pgt_cut(int total, int ctas) {   // no stretch without a unit
  PgtCut c;
  c.total = total;
  c.ctas = ctas < total ? ctas : total;
  if (c.ctas < 1) c.ctas = 1;
  c.base = total / c.ctas;
  c.rem = total - c.base * c.ctas;
  return c;
}

// Host plan of a call; slots and scratch offsets.
struct PgtPlan {
  int ctas, tile, page_shift, G, own_rows, own_groups, prefix_groups, prefix_tiles, own_segs, prefix_segs, Lp;
  int logit_key0;                    // key of the logits' first column
  int wide;                          // the prefix goes to the tcgen05 kernels: 64-row segments, their own cuts
  int pre_rows;                      // rows of a prefix slot
  int x_groups, x_rows, x_tiles, x_segs;   // segments of the tcgen05 kernels: groups of equally many rows
  PgtCut x_keys, x_values;
  size_t logit_off, own_ml_off, own_acc_off, pre_ml_off, pre_acc_off, total;
};

inline PgtPlan pgt_plan(int S, int Hq, int Hkv, int d, int max_len, int prefix_len, int page_size, int dtype,
                        PgxUse use = kPgxAuto) {
  PgtPlan w;
  w.page_shift = 0;
  while ((1 << w.page_shift) < page_size) ++w.page_shift;
  w.G = Hq / Hkv;
  w.own_rows = w.G < kPgtRowTile ? w.G : kPgtRowTile;
  w.own_groups = (w.G + kPgtRowTile - 1) / kPgtRowTile;
  w.tile = pgt_tile(d, dtype);
  w.own_segs = S * Hkv * w.own_groups;
  const int rows = S * w.G;
  w.wide = dtype == DA_BF16 && prefix_len > 0 && rows >= kPgxMinRows && use != kPgxNever &&
           (use == kPgxAlways || (int64_t)rows * Hkv * prefix_len >= kPgxMinPairs);
  const bool narrow = prefix_len > 0 && !w.wide;
  w.prefix_tiles = narrow ? (prefix_len + w.tile - 1) / w.tile : 0;
  const bool few = use == kPgxAuto && dtype == DA_BF16 && d == 64 && w.own_rows <= kPgtPreRows &&
                   (int64_t)Hkv * prefix_len * d * 2 <= kPgtPreBytes;
  w.pre_rows = w.wide ? kPgxRows : few ? kPgtPreRows : kPgtRowTile;   // (the workspace is that of the most rows)
  w.prefix_groups = narrow ? (rows + w.pre_rows - 1) / w.pre_rows : 0;
  w.prefix_segs = Hkv * w.prefix_groups;
  w.x_tiles = w.wide ? (prefix_len + kPgxTile - 1) / kPgxTile : 0;
  w.x_groups = w.wide ? (rows + kPgxRows - 1) / kPgxRows : 0;
  w.x_rows = w.wide ? (rows + w.x_groups - 1) / w.x_groups : 0;
  w.x_segs = Hkv * w.x_groups;
  w.x_keys = pgt_cut(w.x_segs * (w.x_tiles + kPgxHead), kPgxKeyCtas);
  w.x_values = pgt_cut(w.x_segs * (w.x_tiles + kPgxHead), kPgxCtas);
  w.logit_key0 = w.wide ? prefix_len : 0;
  const int64_t own_tiles = (max_len - prefix_len + w.tile - 1) / w.tile;
  const int64_t most = w.own_segs * (own_tiles > 0 ? own_tiles + kPgtHead : 0) +
                       (int64_t)w.prefix_segs * (w.prefix_tiles + kPgtHead);   // units of the line
  w.ctas = (int)(most < 1 ? 1 : most > kPgtMaxCtas ? kPgtMaxCtas : most);
  w.Lp = (int)round_up(max_len - w.logit_key0, 16);
  // slots for the most CTAs: their size depends on the prefix's presence alone
  const int64_t own_slots = kPgtMaxCtas + w.own_segs;
  const int64_t pre_slots = prefix_len > 0 ? kPgtMaxCtas + w.prefix_segs + w.x_segs : 0;
  auto next = [](size_t off, int64_t bytes) { return (size_t)round_up((int64_t)off + bytes, 256); };
  w.logit_off = kStatusBytes;
  w.own_ml_off = next(w.logit_off, (int64_t)S * Hq * w.Lp * 4);
  w.own_acc_off = next(w.own_ml_off, own_slots * w.own_rows * 8);
  w.pre_ml_off = next(w.own_acc_off, own_slots * w.own_rows * acc_stride(d) * 4);
  w.pre_acc_off = next(w.pre_ml_off, pre_slots * w.pre_rows * 8);
  w.total = next(w.pre_acc_off, pre_slots * w.pre_rows * acc_stride(d) * 4);
  return w;
}

#if defined(__CUDACC__)
// ------------------------------------------------------------------ device plan
// Lengths of the sequences and the units of one of their segments, summed, in
// shared memory.
struct PgtLens {
  int len[kPgtMaxSeqs];
  int cum[kPgtMaxSeqs + 1];   // of the sequences before
  int warp_sum[32];
};

// All threads of the block: fills L; ends with a block barrier.
template <int THREADS>
__device__ void pgt_load_lens(const PagedDecode &p, const PgtPlan &w, PgtLens &L, int *status) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, S = p.c.S;
  const int per = (S + THREADS - 1) / THREADS;
  const int s0 = min(tid * per, S), s1 = min(s0 + per, S);
  int sum = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = paged_len(p, s, status);
    L.len[s] = n;
    L.cum[s] = sum;
    if (n > p.prefix_len) sum += kPgtHead + (n - p.prefix_len + w.tile - 1) / w.tile;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) L.warp_sum[warp] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int i = 0; i < warp; ++i) base += L.warp_sum[i];
  for (int s = s0; s < s1; ++s) L.cum[s] += base;
  if (tid == THREADS - 1) L.cum[S] = base + sum;
  __syncthreads();
}

// The line: the prefix's segments first, then each sequence's; and its cut.
struct PgtLine {
  int prefix;          // units of the prefix
  int per_own;         // segments of one sequence
  PgtCut cut;
};
__device__ __forceinline__ PgtLine pgt_line(const PagedDecode &p, const PgtPlan &w, const PgtLens &L) {
  PgtLine t;
  t.per_own = p.c.Hkv * w.own_groups;
  t.prefix = w.prefix_segs > 0 ? w.prefix_segs * (w.prefix_tiles + kPgtHead) : 0;
  t.cut = pgt_cut(t.prefix + L.cum[p.c.S] * t.per_own, w.ctas);
  return t;
}

// One piece of a segment.
struct PgtSeg {
  int s;                     // its sequence; -1: the prefix
  int hkv, row0, nrows;      // rows row0 .. of the sequence's group / of the batch
  int key0, end;             // the piece's first key and the segment's end
  int n;                     // tiles of the piece (0: none left)
  int seg;                   // its number among the prefix's or the sequences' segments
  int run;                   // tiles of the CTA's pieces before this one
  int unit, tiles, stop;     // place of its first tile, tiles of the segment, the stretch's end
  __device__ __forceinline__ void row(int G, int r, int &seq, int &hq) const {
    if (s >= 0) {
      seq = s;
      hq = hkv * G + row0 + r;
    } else {
      seq = (row0 + r) / G;
      hq = hkv * G + (row0 + r) % G;
    }
  }
  // Rows, keys and piece from s, seg, unit and the piece's first tile.
  __device__ __forceinline__ void fill(const PagedDecode &p, const PgtPlan &w, const PgtLine &t, const PgtLens &L,
                                       int tile) {
    const int left = tiles - tile;
    n = min(left, stop - unit);
    if (s < 0) {
      hkv = seg / w.prefix_groups;
      row0 = seg % w.prefix_groups * w.pre_rows;
      nrows = min(w.pre_rows, p.c.S * w.G - row0);
      key0 = tile * w.tile;
      end = p.prefix_len;
    } else {
      const int h = seg - s * t.per_own;
      hkv = h / w.own_groups;
      row0 = h % w.own_groups * kPgtRowTile;
      nrows = min(kPgtRowTile, w.G - row0);
      key0 = p.prefix_len + tile * w.tile;
      end = L.len[s];
    }
  }
  // The first piece of the stretch [from, to).
  __device__ void start(const PagedDecode &p, const PgtPlan &w, const PgtLine &t, const PgtLens &L, int from, int to) {
    stop = to;
    run = 0;
    n = 0;
    if (from >= to) return;
    int u;   // place inside the segment
    if (from < t.prefix) {
      s = -1;
      tiles = w.prefix_tiles;
      seg = from / (tiles + kPgtHead);
      u = from - seg * (tiles + kPgtHead);
    } else {
      const int x = from - t.prefix, q = x / t.per_own;
      int lo = 0, hi = p.c.S - 1;   // the last sequence with cum <= q: one with units of its own
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (L.cum[mid] <= q)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int units = L.cum[lo + 1] - L.cum[lo], r = x - L.cum[lo] * t.per_own, h = r / units;
      s = lo;
      tiles = units - kPgtHead;
      seg = lo * t.per_own + h;
      u = r - h * units;
    }
    const int tile = max(0, u - kPgtHead);
    unit = from + (tile + kPgtHead - u);
    fill(p, w, t, L, tile);
  }
  // The piece after this one.
  __device__ void next(const PagedDecode &p, const PgtPlan &w, const PgtLine &t, const PgtLens &L) {
    run += n;
    unit += n + kPgtHead;   // the next segment's first tile, if this piece ends its segment
    if (unit >= stop) {
      n = 0;
      return;
    }
    ++seg;
    if (s < 0 ? seg == w.prefix_segs : seg == (s + 1) * t.per_own) {   // on to the next sequence with keys of its own
      int k = s + 1;
      while (L.cum[k + 1] == L.cum[k]) ++k;   // there is one: the line goes on
      s = k;
      seg = k * t.per_own;
      tiles = L.cum[k + 1] - L.cum[k] - kPgtHead;
    }
    fill(p, w, t, L, 0);
  }
};

// Slots of the pieces of row (s, hq): the prefix's and its own.
struct PgtPieces {
  int pre0, npre, pre_row;   // first slot, count, row inside the slot
  int own0, nown, own_row;
};
// `values`: of the second pass (the tcgen05 kernels cut the two passes differently).
__device__ __forceinline__ PgtPieces pgt_pieces(const PagedDecode &p, const PgtPlan &w, const PgtLine &t,
                                                const PgtLens &L, int s, int hq, bool values) {
  PgtPieces r{0, 0, 0, 0, 0, 0};
  if (L.len[s] == 0) return r;
  const int hkv = hq / w.G, g = hq % w.G;
  if (w.wide) {
    const int R = s * w.G + g, seg = hkv * w.x_groups + R / w.x_rows;
    const PgtCut &c = values ? w.x_values : w.x_keys;
    const int first = seg * (w.x_tiles + kPgxHead) + kPgxHead;
    const int c0 = c.cta_of(first), c1 = c.cta_of(first + w.x_tiles - 1);
    r.pre0 = c0 + seg;
    r.npre = c1 - c0 + 1;
    r.pre_row = R % w.x_rows;
  } else if (w.prefix_tiles > 0) {
    const int R = s * w.G + g, seg = hkv * w.prefix_groups + R / w.pre_rows;
    const int a = seg * (w.prefix_tiles + kPgtHead) + kPgtHead;
    const int c0 = t.cut.cta_of(a), c1 = t.cut.cta_of(a + w.prefix_tiles - 1);
    r.pre0 = c0 + seg;
    r.npre = c1 - c0 + 1;
    r.pre_row = R % w.pre_rows;
  }
  const int units = L.cum[s + 1] - L.cum[s];
  if (units > 0) {
    const int h = hkv * w.own_groups + g / kPgtRowTile;
    const int a = t.prefix + L.cum[s] * t.per_own + h * units + kPgtHead;
    const int c0 = t.cut.cta_of(a), c1 = t.cut.cta_of(a + units - kPgtHead - 1);
    r.own0 = c0 + s * t.per_own + h;
    r.nown = c1 - c0 + 1;
    r.own_row = g % kPgtRowTile;
  }
  return r;
}

// lse2 of row (s, hq), by WIDTH neighbouring lanes (the same value in each): its
// pieces' (max, sum) joined.  All lanes of the warp call it.
template <int WIDTH>
__device__ __forceinline__ float pgt_row_lse(const PagedDecode &p, const PgtPlan &w, const PgtLine &t,
                                             const PgtLens &L, int s, int hq, int lane) {
  const PgtPieces pc = pgt_pieces(p, w, t, L, s, hq, false);
  const float2 *pre = reinterpret_cast<const float2 *>(p.ws + w.pre_ml_off);
  const float2 *own = reinterpret_cast<const float2 *>(p.ws + w.own_ml_off);
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int c = lane % WIDTH; c < pc.npre + pc.nown; c += WIDTH) {
    const float2 ml = __ldcg(c < pc.npre ? pre + (size_t)(pc.pre0 + c) * w.pre_rows + pc.pre_row
                                         : own + (size_t)(pc.own0 + c - pc.npre) * w.own_rows + pc.own_row);
    const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
    l = l * ex2_approx(m - ms) + ml.y * ex2_approx(ml.x - ms);
    m = mn;
  }
  __syncwarp();
#pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const float mn = fmaxf(m, m2), ms = mn == -INFINITY ? 0.f : mn;
    l = l * ex2_approx(m - ms) + l2 * ex2_approx(m2 - ms);
    m = mn;
  }
  return m + log2f(l);
}

// ------------------------------------------------------------------ tensor pieces
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The order of a 16-key group: column c of the first 8 (half 0) and the last 8
// (half 1) columns is key 4 (c / 2) + 2 half + c % 2, so that a thread's four
// columns (2t, 2t + 1 of both halves) are keys 4t .. 4t + 3.
__device__ __forceinline__ int group_key(int c, int half) { return 4 * (c >> 1) + 2 * half + (c & 1); }

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Kernels of one decode step, in launch order (see launch_after):
//   pgt_keys    waits for everything before the step, then lets its successor begin;
//   pgx_keys    needs nothing of pgt_keys; it waits for it before it ends;
//   pgt_values  waits for the keys' kernels, then lets its successor begin;
//   pgx_values  so begins after the keys' kernels; waits for pgt_values before it ends;
//   pgt_combine waits for its predecessor, and with it for all of them.
// What they read before a wait of their own, of the caller's or of each other's, is
// in L2 by then, and they read it there (__ldcg, asynchronous copies): an SM's L1 may
// hold what it saw before.
#endif  // __CUDACC__

}  // namespace da
