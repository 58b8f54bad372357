// Chunks over the paged cache on CUDA cores, fp32 arithmetic throughout (TF32
// products would miss the type's accuracy).
//
// Mathematics: query i of a sequence's n new ones (its last n tokens; place P + i)
// and query head h, over the keys t <= P + i:
//   x = q . k_t tau / sqrt(d) log2 e,  p = 2^(x - lse2),
//   total_t += p,  share = p / (total_t + eps)  (the total before p with the
//   earlier demand only),  out = sum share v / sum share.
//   ckf_keys    (max, sum 2^(x - max)) of every row over a piece's keys;
//   ckf_values  shares and totals, sums of share v and share over them.
//
// What bounds it: the fp32 units (three products of d a pair) once a key is seen
// by a dozen rows.  A tile is 64 rows by 64 keys, 256 threads with 4 x 4 products
// each, 8 reads of 16 bytes for 32 packed multiply-adds; warps without rows leave the
// products out.  K and V have a place each, filled by asynchronous copies as soon as
// the tile before has been read (rings of three to six places, one barrier a tile: as
// long, and 5 us more a call to fill).  A key's total runs over the rows of a tile: four
// threads a key take 16 rows each, after they have exchanged the sums of their bids
// (one thread a key left 3/4 of the block idle).
#include "da_chunk.cuh"

namespace da {

constexpr int kCkfEdge = 64;
constexpr int kCkfThreads = 256;
// CTAs an SM, where no column tile of the call has more than `most` rows: up to 8 and up
// to 16 have kernels of their own, with registers for as many (one kernel for all: 4 % more for
// many rows; us of 8 x 12 x 8001 with 3 tokens 195, as a part of one kernel 229, as up to 16
// rows 282; 2 x 12 x 131072 with 4 tokens 648, 774, 980; 8 x 12 x 8001 with 14 tokens 265, in one
// kernel 292; d = 128, 4 x 12 x 8001 with 14 tokens 270, in one kernel 356, three CTAs 401).  Two for
// many rows at d = 128 too, which their bids' place over K makes room for (4 sequences of 1001 ..
// 8001 with 301 .. 3 tokens 492 -> 395, 4 prompts of 2000 tokens 2829 -> 2788).
constexpr int ckf_ctas(int d, int most) { return most <= 8 || (most <= 16 && d == 64) ? 3 : 2; }
static int ckf_most(int Hq, int Hkv, int max_new) {
  const long long rows = (long long)(Hq / Hkv) * round_up(max_new, 8);
  return rows <= 8 ? 8 : rows <= 16 ? 16 : kCkfEdge;
}

ChunkPlan chunk_plan_f32(int S, int Hq, int Hkv, int d, long long N, int max_new, int page_size) {
  const int ctas = 152 * ckf_ctas(d, ckf_most(Hq, Hkv, max_new));
  return chunk_plan(S, Hq, Hkv, d, N, max_new, page_size, kCkfEdge, ctas, ctas, ChunkCost{4, 4, 1, 8, 4});
}

template <int D, int ROWS = kCkfEdge>
struct Ckf {
  static constexpr int kLd = D + 4;            // floats of a staged row: lanes of different rows read different banks
  static constexpr int kLdP = kCkfEdge + 4;
  static constexpr bool kOver = D == 128 && ROWS == kCkfEdge;   // bids over K, once it has been read: two CTAs fit
  static constexpr int kSmemBytes = (ROWS * (kLd + (kOver ? 0 : kLdP)) + 2 * kCkfEdge * kLd + 4 * kCkfEdge) * 4;
};

// A column tile: row c of it is query head hq(c), query i(c).
struct CkfCols {
  int r0, rows;          // first row of the segment; rows
  int hq0, n8, i0, n;    // wide: n8 = 0
  __device__ __forceinline__ CkfCols(const ChunkWalk &k, const ChunkPlan &w, int b) {
    r0 = b * k.g.step;
    n = k.g.n;
    if (k.g.wide) {
      n8 = 0;
      hq0 = k.seg;
      i0 = r0;
      rows = min(k.g.step, n - r0);
    } else {
      n8 = k.g.n8;
      hq0 = k.seg * w.G + r0 / n8;
      i0 = 0;
      rows = min(k.g.step, w.G * n8 - r0);
    }
  }
  __device__ __forceinline__ int head(int c) const { return n8 ? hq0 + c / n8 : hq0; }
  __device__ __forceinline__ int query(int c) const { return n8 ? c % n8 : i0 + c; }
  __device__ __forceinline__ bool valid(int c) const { return c < rows && query(c) < n; }
};

template <int D, int ROWS>
__device__ __forceinline__ void ckf_queries(const PagedChunk &p, const ChunkWalk &k, const CkfCols &t, float *sQ) {
  for (int e = threadIdx.x; e < ROWS * (D / 4); e += kCkfThreads) {
    const int c = e / (D / 4), x = e % (D / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t.valid(c))
      v = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) +
                                                  ((size_t)(k.q.tok0 + t.query(c)) * p.c.Hq + t.head(c)) * D) + x);
    *reinterpret_cast<float4 *>(sQ + c * Ckf<D>::kLd + 4 * x) = v;
  }
}

// The rows of a key tile that a thread copies, kCkfThreads / (d / 4) apart: their pages
// (-1 past the sequence's end), and asynchronous copies of K or V from them: one group.
// Zeros past the end and where there is no page (recorded).
template <int D>
struct CkfPages {
  static constexpr int STEP = kCkfThreads / (D / 4), ROWS = kCkfEdge / STEP;
  int page[ROWS];
  __device__ __forceinline__ void find(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, int tile) {
    const int32_t *table = p.c.page_table + (size_t)k.s * p.c.max_pages;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int key = tile * kCkfEdge + threadIdx.x / (D / 4) + i * STEP;
      page[i] = key < k.g.len ? __ldcg(table + (key >> w.page_shift)) : -1;
    }
  }
  __device__ __forceinline__ void copy(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, const void *pages, int tile,
                                       float *to) const {
    const int sh = w.page_shift, ps = 1 << sh, hkv = k.hkv(w), x = threadIdx.x % (D / 4);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = threadIdx.x / (D / 4) + i * STEP, key = tile * kCkfEdge + j;
      const bool ok = (unsigned)page[i] < (unsigned)p.c.num_pages;
      if (!ok && key < k.g.len) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      const float *from = static_cast<const float *>(pages);
      if (ok) from += ((((size_t)page[i] * p.c.Hkv + hkv) << sh) + (key & (ps - 1))) * D + 4 * x;
      cp_async16_fill(smem_u32(to + j * Ckf<D>::kLd + 4 * x), from, ok);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};
// The thread's own copies of a tile of V, once landed: of the sequence's new tokens only
// what is finite.
template <int D>
__device__ __forceinline__ void ckf_clear(const ChunkWalk &k, int tile, float *sV) {
  for (int j = threadIdx.x / (D / 4); j < kCkfEdge; j += CkfPages<D>::STEP) {
    uint4 *v = reinterpret_cast<uint4 *>(sV + j * Ckf<D>::kLd + threadIdx.x % (D / 4) * 4);
    uint4 x = *v;
    if (tile * kCkfEdge + j >= k.g.P && chunk_clear(x, false)) *v = x;
  }
}
template <int N>
__device__ __forceinline__ void ckf_landed() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Where the total of (key, query head) lies; null without one.
__device__ __forceinline__ float *ckf_total(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, int key, int hq) {
  if (key >= k.g.len) return nullptr;
  const int sh = w.page_shift;
  const int page = __ldcg(p.c.demand_table + (size_t)k.s * p.c.max_pages + (key >> sh));
  if ((unsigned)page >= (unsigned)p.c.num_demand_pages) {
    atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    return nullptr;
  }
  return p.c.demand_pages + ((((size_t)page * p.c.Hq + hq) << sh) + (key & ((1 << sh) - 1)));
}

// A thread's part of a tile.  Many rows: 4 rows (4 ty ..) by 4 keys (tx + 16 j).  Up to
// 16 rows: 4 rows (4 (ty % 4) ..) by one key (16 (ty / 4) + tx), so that all warps work
// (as many rows: 64 keys by 8 rows in one warp, 223 us for 4 sequences of 1001 .. 8001).
// Up to 8 rows: 2 rows by one key.
// Neighbouring lanes have the same key and two groups of rows: half a warp's 16-byte reads
// of K then fall on 8 places, once over the banks (16 keys a half-warp: twice).
template <int MAX>   // rows: 64, or few: 16, 8
struct CkfPart {
  static constexpr bool kFew = MAX <= 16;
  static constexpr int kKeys = kFew ? 1 : 4, kRows = MAX == 8 ? 2 : 4;
  int row, key;   // its first row and key
  int tx;         // 0 .. 15
  __device__ __forceinline__ CkfPart() {
    const int ty = threadIdx.x / 32 * 2 + threadIdx.x % 2;
    tx = threadIdx.x % 32 / 2;
    row = kFew ? kRows * (ty % 4) : 4 * ty;
    key = kFew ? 16 * (ty / 4) + tx : tx;
  }
};

// q . k of the thread's part.
template <int D, int MAX>
__device__ __forceinline__ void ckf_products(const float *sQ, const float *sK, float (&x)[CkfPart<MAX>::kRows][CkfPart<MAX>::kKeys]) {
  constexpr int NK = CkfPart<MAX>::kKeys, NR = CkfPart<MAX>::kRows;
  const CkfPart<MAX> t;
  float2 acc[NR][NK];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int j = 0; j < NK; ++j) acc[r][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int e = 0; e < D; e += 4) {
    float4 kv[NK];
#pragma unroll
    for (int j = 0; j < NK; ++j) kv[j] = *reinterpret_cast<const float4 *>(sK + (t.key + 16 * j) * Ckf<D>::kLd + e);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float4 q = *reinterpret_cast<const float4 *>(sQ + (t.row + r) * Ckf<D>::kLd + e);
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        acc[r][j] = ffma2(make_float2(q.x, q.y), make_float2(kv[j].x, kv[j].y), acc[r][j]);
        acc[r][j] = ffma2(make_float2(q.z, q.w), make_float2(kv[j].z, kv[j].w), acc[r][j]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int j = 0; j < NK; ++j) x[r][j] = acc[r][j].x + acc[r][j].y;
}

// The rows of a thread's part: scale, last key that each sees (-1: none), -lse2.
template <int MAX>
struct CkfRows {
  static constexpr int NR = CkfPart<MAX>::kRows;
  float c2[NR], nl[NR];
  int last[NR];
  __device__ __forceinline__ CkfRows(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, const CkfCols &t, bool first) {
    const CkfPart<MAX> part;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int c = part.row + r;
      last[r] = t.valid(c) ? k.g.P + t.query(c) : -1;
      c2[r] = last[r] >= 0 ? head_c2(p.hs, k.s * p.c.Hq + t.head(c), first ? p.status : nullptr) : 0.f;
      nl[r] = !first && last[r] >= 0
                  ? __ldcg(reinterpret_cast<const float *>(p.ws + w.nl) + k.row0(p, w) + t.r0 + c) : 0.f;
    }
  }
};

__device__ __forceinline__ void ckf_merge(float &m, float &sum, float m2, float s2) {
  const float mn = fmaxf(m, m2), ms = mn == -INFINITY ? 0.f : mn;
  sum = sum * ex2_approx(m - ms) + s2 * ex2_approx(m2 - ms);
  m = mn;
}

template <int D, int MAX, int PLACES>
__device__ __forceinline__ void ckf_keys_tile(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, const CkfCols &t, int end,
                                              float *smem) {
  using C = Ckf<D>;
  constexpr int NK = CkfPart<MAX>::kKeys, NR = CkfPart<MAX>::kRows;
  constexpr bool FEW = CkfPart<MAX>::kFew;
  float *sQ = smem, *sK = sQ + PLACES * C::kLd;   // two key tiles
  float2 *s_ml = reinterpret_cast<float2 *>(sK + 2 * kCkfEdge * C::kLd);
  const CkfPart<MAX> part;
  const int tx = part.tx, kg = threadIdx.x / 64;
  const bool work = FEW || threadIdx.x / 32 * 8 < t.rows;   // uniform over the warp
  CkfPages<D> pages;
  pages.find(p, w, k, k.tile);
  pages.copy(p, w, k, p.c.k_pages, k.tile, sK);
  if (k.tile + 1 < end) pages.find(p, w, k, k.tile + 1);
  ckf_queries<D, PLACES>(p, k, t, sQ);
  const CkfRows<MAX> rows(p, w, k, t, true);
  float m[NR], sum[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) m[r] = -INFINITY, sum[r] = 0.f;
  for (int tile = k.tile; tile < end; ++tile) {
    float *now = sK + ((tile - k.tile) & 1) * kCkfEdge * C::kLd;
    if (tile + 1 < end) {   // into the place of the tile before this one, which has been read
      pages.copy(p, w, k, p.c.k_pages, tile + 1, sK + ((tile + 1 - k.tile) & 1) * kCkfEdge * C::kLd);
      if (tile + 2 < end) pages.find(p, w, k, tile + 2);
      ckf_landed<1>();
    } else {
      ckf_landed<0>();
    }
    __syncthreads();
    if (work) {
      float x[NR][NK];
      ckf_products<D, MAX>(sQ, now, x);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float mn = m[r];
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          x[r][j] = tile * kCkfEdge + part.key + 16 * j <= rows.last[r] ? x[r][j] * rows.c2[r] : -INFINITY;
          mn = fmaxf(mn, x[r][j]);
        }
        const float ms = mn == -INFINITY ? 0.f : mn;
        sum[r] *= ex2_approx(m[r] - ms);
#pragma unroll
        for (int j = 0; j < NK; ++j) sum[r] += ex2_approx(x[r][j] - ms);
        m[r] = mn;
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int o = 16; o > 1; o >>= 1)
      ckf_merge(m[r], sum[r], __shfl_xor_sync(0xffffffffu, m[r], o), __shfl_xor_sync(0xffffffffu, sum[r], o));
  auto put = [&](int row, float2 ml) {
    *reinterpret_cast<float2 *>(chunk_place(p, w.ml_a, w.ml_b, k.row0(p, w), w.cta_rows, k.tile, blockIdx.x, t.r0 + row, 2)) = ml;
  };
  if constexpr (FEW) {   // four threads a row, each with a fourth of the keys
    if (tx == 0)
#pragma unroll
      for (int r = 0; r < NR; ++r) s_ml[kg * 16 + part.row + r] = make_float2(m[r], sum[r]);
    __syncthreads();
    if (threadIdx.x < 16 && t.valid(threadIdx.x)) {
      float2 a = s_ml[threadIdx.x];
#pragma unroll
      for (int g = 1; g < 4; ++g) ckf_merge(a.x, a.y, s_ml[g * 16 + threadIdx.x].x, s_ml[g * 16 + threadIdx.x].y);
      put(threadIdx.x, a);
    }
  } else {
    if (tx == 0)
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if (rows.last[r] >= 0) put(part.row + r, make_float2(m[r], sum[r]));
  }
}

template <int D, int MOST>
__global__ void __launch_bounds__(kCkfThreads, ckf_ctas(D, MOST)) ckf_keys(PagedChunk p, ChunkPlan w) {
  extern __shared__ __align__(16) float ckf_smem[];
  pdl_wait();
  pdl_launch_dependents();
  const ChunkLine l = chunk_line(p, w);
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_keys);
  ChunkWalk k;
  for (k.start(p, w, l, cut, threadIdx.x % 32); k.any(); k.next(p, w, l))
    for (int b = k.g.col0(k.tile); b < k.g.cols; ++b) {
      const CkfCols t(k, w, b);
      const int end = min(k.end, k.g.seen(b, kCkfEdge));
      __syncthreads();
      if constexpr (MOST <= 16) {
        ckf_keys_tile<D, MOST, MOST>(p, w, k, t, end, ckf_smem);
      } else {
        if (t.rows <= 16)
          ckf_keys_tile<D, 16, MOST>(p, w, k, t, end, ckf_smem);
        else
          ckf_keys_tile<D, MOST, MOST>(p, w, k, t, end, ckf_smem);
      }
    }
}

// bid / den, den > 0 (a reciprocal within an ulp); 0 without a bid, whatever den.
__device__ __forceinline__ float ckf_share(float bid, float den) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(den));
  return bid > 0.f ? bid * r : bid;
}

template <int D, int MAX, int PLACES>
__device__ __forceinline__ void ckf_values_tile(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, const CkfCols &t, int end,
                                                float *smem) {
  using C = Ckf<D, PLACES>;
  constexpr bool OVER = C::kOver;
  constexpr int NV = D / 64, NK = CkfPart<MAX>::kKeys, NR = CkfPart<MAX>::kRows;   // 4-column groups, keys and rows of a thread
  constexpr bool FEW = CkfPart<MAX>::kFew;
  float *sQ = smem, *sK = sQ + PLACES * C::kLd, *sV = sK + kCkfEdge * C::kLd, *sP = OVER ? sK : sV + kCkfEdge * C::kLd,
        *sPart = OVER ? sV + kCkfEdge * C::kLd : sP + PLACES * C::kLdP;
  const CkfPart<MAX> part;
  const int tid = threadIdx.x, tx = part.tx;
  const bool work = FEW || tid / 32 * 8 < t.rows;   // uniform over the warp
  const int j0 = FEW ? tid / 64 * 16 : 0, j1 = FEW ? j0 + 16 : kCkfEdge;   // keys of the thread's value products
  CkfPages<D> pages;
  pages.find(p, w, k, k.tile);
  pages.copy(p, w, k, p.c.k_pages, k.tile, sK);
  pages.copy(p, w, k, p.c.v_pages, k.tile, sV);
  if (k.tile + 1 < end) pages.find(p, w, k, k.tile + 1);
  ckf_queries<D, PLACES>(p, k, t, sQ);
  const CkfRows<MAX> rows(p, w, k, t, false);
  const bool odd = __ldcg(chunk_odd(p, w) + k.s) != 0;
  float num[NR][4 * NV], sum[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    sum[r] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * NV; ++e) num[r][e] = 0.f;
  }
  const int key_l = tid % kCkfEdge, quarter = tid / kCkfEdge;
  const bool several = t.n8 != 0, mine_too = !several || quarter * t.n8 < t.rows;
  float *col = sP + key_l;
  for (int tile = k.tile; tile < end; ++tile) {
    const int key = tile * kCkfEdge + key_l;
    // the total of this thread's (first) head: one head, or head `quarter` of several
    float *at = mine_too ? ckf_total(p, w, k, key, t.hq0 + (several ? quarter : 0)) : nullptr;
    const float before = at != nullptr ? __ldcg(at) : 0.f;
    ckf_landed<1>();   // K (V is the newer group)
    __syncthreads();
    float x[NR][NK];
    if (work) ckf_products<D, MAX>(sQ, sK, x);
    if constexpr (OVER) __syncthreads();   // K has been read
    if (work) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const bool sees = tile * kCkfEdge + part.key + 16 * j <= rows.last[r];
          sP[(part.row + r) * C::kLdP + part.key + 16 * j] = sees ? ex2_approx(fmaf(x[r][j], rows.c2[r], rows.nl[r])) : 0.f;
        }
    }
    __syncthreads();
    if (!OVER && tile + 1 < end) pages.copy(p, w, k, p.c.k_pages, tile + 1, sK);
    if (!several) {   // one head: 16 rows a thread
      const int n = min(16, t.rows - 16 * quarter);
      float mine = 0.f, run = 0.f;   // the rows' bids, summed apart from the total: it would take their last bits
#pragma unroll 4
      for (int c = 0; c < n; ++c) mine += col[(16 * quarter + c) * C::kLdP];
      sPart[quarter * kCkfEdge + key_l] = mine;
      __syncthreads();
      for (int i = 0; i < quarter; ++i) run += sPart[i * kCkfEdge + key_l];
#pragma unroll 4
      for (int c = 0; c < n; ++c) {
        const float bid = col[(16 * quarter + c) * C::kLdP], after = run + bid;
        col[(16 * quarter + c) * C::kLdP] = ckf_share(bid, before + (p.earlier ? run : after) + p.eps);
        run = after;
      }
      if (quarter == 3 && at != nullptr) __stcg(at, before + run);
    } else {
      float held = before;
      for (int h = quarter; h * t.n8 < t.rows; h += kCkfThreads / kCkfEdge) {
        if (h != quarter) {
          at = ckf_total(p, w, k, key, t.hq0 + h);
          held = at != nullptr ? __ldcg(at) : 0.f;
        }
        float run = 0.f;
#pragma unroll 4
        for (int c = h * t.n8; c < h * t.n8 + t.n; ++c) {
          const float bid = col[c * C::kLdP], after = run + bid;
          col[c * C::kLdP] = ckf_share(bid, held + (p.earlier ? run : after) + p.eps);
          run = after;
        }
        if (at != nullptr) __stcg(at, held + run);
      }
    }
    if (!OVER && tile + 1 < end)
      ckf_landed<1>();   // V (the next K is the newer group)
    else
      ckf_landed<0>();
    if (odd && (tile + 1) * kCkfEdge > k.g.P) ckf_clear<D>(k, tile, sV);
    __syncthreads();
    if (work) {
#pragma unroll 4
      for (int j = j0; j < j1; j += 4) {
        float4 sh[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          sh[r] = *reinterpret_cast<const float4 *>(sP + (part.row + r) * C::kLdP + j);
          if ((j - j0) / 4 == tx) sum[r] += (sh[r].x + sh[r].y) + (sh[r].z + sh[r].w);
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) {
          float4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4 *>(sV + (j + i) * C::kLd + 64 * e + 4 * tx);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float s4[4] = {sh[r].x, sh[r].y, sh[r].z, sh[r].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float2 &lo = *reinterpret_cast<float2 *>(&num[r][4 * e]), &hi = *reinterpret_cast<float2 *>(&num[r][4 * e + 2]);
              lo = ffma2(make_float2(s4[i], s4[i]), make_float2(v[i].x, v[i].y), lo);
              hi = ffma2(make_float2(s4[i], s4[i]), make_float2(v[i].z, v[i].w), hi);
            }
          }
        }
      }
    }
    __syncthreads();
    if (tile + 1 < end) {
      if (OVER) pages.copy(p, w, k, p.c.k_pages, tile + 1, sK);
      pages.copy(p, w, k, p.c.v_pages, tile + 1, sV);
      if (tile + 2 < end) pages.find(p, w, k, tile + 2);
    }
  }
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
  float *to = chunk_place(p, w.acc_a, w.acc_b, k.row0(p, w), w.cta_rows, k.tile, blockIdx.x, t.r0, acc_stride(D));
  if constexpr (FEW) {   // the four fourths of the keys, in order
    constexpr int LD = D + 4;
    float *stage = sK;   // [fourth][16 rows][d, sum]; the tile's K and V have been read
    static_assert(4 * 16 * LD <= 2 * kCkfEdge * C::kLd, "stage");
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float *row = stage + (tid / 64 * 16 + part.row + r) * LD;
#pragma unroll
      for (int e = 0; e < NV; ++e)
        *reinterpret_cast<float4 *>(row + 64 * e + 4 * tx) =
            make_float4(num[r][4 * e], num[r][4 * e + 1], num[r][4 * e + 2], num[r][4 * e + 3]);
      if (tx == 0) row[D] = sum[r];
    }
    __syncthreads();
    for (int i = tid; i < (t.rows + 7) / 8 * 8 * (D + 1); i += kCkfThreads) {   // eight rows after eight, as they lie
      const int r8 = i / (8 * (D + 1)) * 8, e = i % (8 * (D + 1)), r = r8 + (e < 8 * D ? e / 4 % 8 : e - 8 * D),
                c = e < 8 * D ? e / 32 * 4 + e % 4 : D;
      float a = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g) a += stage[(g * 16 + r) * LD + c];
      if (t.valid(r)) to[c < D ? chunk_acc(D, r, c / 4) + c % 4 : chunk_acc_sum(D, r)] = a;
    }
  } else if (work) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (rows.last[r] < 0) continue;
      const int row = part.row + r;
#pragma unroll
      for (int e = 0; e < NV; ++e)
        *reinterpret_cast<float4 *>(to + chunk_acc(D, row, 16 * e + tx)) =
            make_float4(num[r][4 * e], num[r][4 * e + 1], num[r][4 * e + 2], num[r][4 * e + 3]);
      if (tx == 0) to[chunk_acc_sum(D, row)] = sum[r];
    }
  }
}

template <int D, int MOST>
__global__ void __launch_bounds__(kCkfThreads, ckf_ctas(D, MOST)) ckf_values(PagedChunk p, ChunkPlan w) {
  extern __shared__ __align__(16) float ckf_smem[];
  pdl_wait();
  pdl_launch_dependents();
  const ChunkLine l = chunk_line(p, w);
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_values);
  ChunkWalk k;
  for (k.start(p, w, l, cut, threadIdx.x % 32); k.any(); k.next(p, w, l))
    for (int b = k.g.col0(k.tile); b < k.g.cols; ++b) {
      const CkfCols t(k, w, b);
      const int end = min(k.end, k.g.seen(b, kCkfEdge));
      __syncthreads();
      if constexpr (MOST <= 16) {
        ckf_values_tile<D, MOST, MOST>(p, w, k, t, end, ckf_smem);
      } else {
        if (t.rows <= 16)
          ckf_values_tile<D, 16, MOST>(p, w, k, t, end, ckf_smem);
        else
          ckf_values_tile<D, MOST, MOST>(p, w, k, t, end, ckf_smem);
      }
    }
}

cudaError_t launch_chunk_plan(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);      // paged_chunk.cu
cudaError_t launch_chunk_join(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);
cudaError_t launch_chunk_combine(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);

template <int D, int MOST>
static int launch_ckf(const PagedChunk &p, cudaStream_t stream) {
  constexpr int bytes = Ckf<D, MOST>::kSmemBytes;
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return (cudaFuncSetAttribute(ckf_keys<D, MOST>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
            cudaFuncSetAttribute(ckf_values<D, MOST>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  const ChunkPlan w = chunk_plan_f32(p.c.S, p.c.Hq, p.c.Hkv, D, p.N, p.max_new, p.c.page_size);
  if (launch_chunk_plan(p, w, stream) != cudaSuccess ||
      launch_after(ckf_keys<D, MOST>, w.ctas_keys, kCkfThreads, bytes, stream, p, w) != cudaSuccess ||
      launch_chunk_join(p, w, stream) != cudaSuccess ||
      launch_after(ckf_values<D, MOST>, w.ctas_values, kCkfThreads, bytes, stream, p, w) != cudaSuccess ||
      launch_chunk_combine(p, w, stream) != cudaSuccess)
    return DA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int launch_chunk_f32(const PagedChunk &p, cudaStream_t stream) {
  switch (ckf_most(p.c.Hq, p.c.Hkv, p.max_new)) {
    case 8: return p.c.d == 128 ? launch_ckf<128, 8>(p, stream) : launch_ckf<64, 8>(p, stream);
    case 16: return p.c.d == 128 ? launch_ckf<128, 16>(p, stream) : launch_ckf<64, 16>(p, stream);
    default: return p.c.d == 128 ? launch_ckf<128, kCkfEdge>(p, stream) : launch_ckf<64, kCkfEdge>(p, stream);
  }
}
}  // namespace da
