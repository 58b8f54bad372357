// Eviction from the paged cache by accumulated demand.
//
// Definition: the score of token t for a key head is the sum of its query heads'
// totals, added in fp32 in the heads' order; the first `sinks` and the last
// `recent` tokens and those whose score is NaN score +infinity.  Of each key head
// the m = min(length, keep) tokens with the highest scores stay, equal scores by
// the lower place.  They keep their order and become tokens 0 .. m - 1.
//
// evict_select: a cluster per (sequence, key head), its scores in the CTAs' shared
// memory as integers of the same order.  The m-th highest is found by three counts
// of 11, 11 and 10 bits, the CTAs' counts summed through distributed shared
// memory; then each CTA writes the places of its tokens that stay.
//
// evict_place: rows to their new places in the same pages.  Row r takes the row of
// token list[r] >= r, so a block that takes rows in order, has read a batch before it
// writes it, and is alone on its bytes, never overwrites what is still to be read.
// Blocks are therefore alone on a slice of a head's rows of keys or values (down to
// 32 bytes, a sector) or on the totals of a query head, for all rows.  (Not kept,
// 4 x 4 heads x 32768 of 131072 rows, a slice 150 us: a cluster a head, whole rows,
// a cluster barrier a batch 207; chunks of rows on any block, with a flag each that
// it has been read, 232 to 1100.)
//
// evict_move: rows to other pages; blocks take chunk after chunk by tickets.
//
// evict_small: all of it for up to 512 tokens a sequence in one launch, a block per
// (sequence, key head).
//
// What bounds it: HBM (4 bytes a total, then the rows that stay, once each way).
#include "da_evict.h"
#include "da_ptx.cuh"

namespace da {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kCopies = 4;   // of the counts: neighbouring lanes' scores fall into few bins

EvictWorkspace evict_workspace(int S, int Hkv, int max_keep, int max_len) {
  EvictWorkspace w;
  const int64_t items = (int64_t)S * Hkv;
  // CTAs of a cluster: up to 8 while the GPU has room and each still has 1024 keys
  int c = 1;
  while (c < kEvictCtas && ((items * c < 152 && max_len > c * 1024) || max_len > c * kEvictKeys / 3)) c *= 2;
  w.cluster = c;
  w.slice = (int)round_up((max_len + c - 1) / c, 32);
  w.shared = w.slice <= kEvictKeys;
  auto next = [](size_t off, int64_t bytes) { return (size_t)round_up((int64_t)off + bytes, 256); };
  w.info_off = kStatusBytes;
  w.list_off = next(w.info_off, (int64_t)S * 8);
  w.flag_off = next(w.list_off, items * max_keep * 4);
  w.total_chunks = (max_keep + kEvictTotals - 1) / kEvictTotals;
  w.key_off = next(w.flag_off, 4);
  w.total = next(w.key_off, w.shared ? 0 : items * c * w.slice * 4);
  return w;
}

// Scores as integers of the same order; NaN as +infinity, -0 as 0.
__device__ __forceinline__ uint32_t ev_key(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xff800000u;
  if (u == 0x80000000u) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select(EvictArgs a, EvictWorkspace w, int page_shift) {
  extern __shared__ uint32_t sel_keys[];
  __shared__ __align__(16) uint32_t s_hist[kCopies + 1][kBins];   // the first pass's (the third's in its first copy); the second's
  __shared__ uint32_t s_above[kSelWarps], s_equal[kSelWarps], s_count[2], s_pick[2];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t rank = cluster_rank(), C = (uint32_t)w.cluster;
  pdl_wait();
  pdl_launch_dependents();
  const int item = blockIdx.x / w.cluster, s = item / a.c.Hkv, h = item % a.c.Hkv, G = a.c.Hq / a.c.Hkv;
  const int len = __ldcg(a.c.seq_lens + s), keep = __ldcg(a.keep + s);
  const bool good = len >= 0 && len <= a.max_len && keep >= 0 && min(len, keep) <= a.max_keep;
  const int m = good ? min(len, keep) : 0;
  if (h == 0 && rank == 0 && tid == 0) {
    if (!good) atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
    reinterpret_cast<int2 *>(a.ws + w.info_off)[s] = make_int2(m, good ? m : len);
  }
  if (blockIdx.x == 0 && tid == 0) *reinterpret_cast<int32_t *>(a.ws + w.flag_off) = 0;   // evict_move's ticket
  int32_t *list = (a.kept != nullptr ? a.kept : reinterpret_cast<int32_t *>(a.ws + w.list_off)) + (size_t)item * a.max_keep;
  if (a.kept != nullptr)
    for (int i = m + (int)rank * kSelThreads + tid; i < a.max_keep; i += (int)C * kSelThreads) list[i] = -1;
  if (m == 0) return;   // (the same in every CTA of the cluster)
  const int per = (int)round_up((len + w.cluster - 1) / w.cluster, 32);
  const int t0 = min((int)rank * per, len), cnt = min(len - t0, per);
  if (m == len) {
    for (int i = tid; i < cnt; i += kSelThreads) list[t0 + i] = t0 + i;
    return;
  }
  uint32_t *keys = w.shared ? sel_keys
                            : reinterpret_cast<uint32_t *>(a.ws + w.key_off) + ((size_t)item * w.cluster + rank) * w.slice;
  const int32_t *dtab = a.c.demand_table + (size_t)s * a.c.max_pages;
  const int ps = 1 << page_shift;
  for (int i = tid; i < (kCopies + 1) * kBins; i += kSelThreads) s_hist[0][i] = 0;
  __syncthreads();
  // four tokens a thread, which lie in one page; the totals of four query heads on their
  // way at once
  auto page_of = [&](int i) { return i < cnt ? __ldcg(dtab + ((t0 + i) >> page_shift)) : 0; };
  int page = page_of(4 * tid);
#pragma unroll 2
  for (int i = 4 * tid; i < cnt; i += 4 * kSelThreads) {
    const int t = t0 + i, next = page_of(i + 4 * kSelThreads);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if ((unsigned)page < (unsigned)a.c.num_demand_pages) {
      const float *at = a.c.demand_pages + ((((size_t)page * a.c.Hq + (size_t)h * G) << page_shift) + (t & (ps - 1)));
      for (int g = 0; g < G; g += 4) {
        float4 f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + e < G) f[e] = __ldcg(reinterpret_cast<const float4 *>(at + ((size_t)(g + e) << page_shift)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (g + e >= G) break;
          const float x[4] = {f[e].x, f[e].y, f[e].z, f[e].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = g + e == 0 ? x[k] : __fadd_rn(v[k], x[k]);
        }
      }
    } else {
      atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
    }
    page = next;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e >= cnt) break;
      const uint32_t key = ev_key(t + e < a.sinks || t + e >= len - a.recent ? INFINITY : v[e]);
      keys[i + e] = key;
      atomicAdd(&s_hist[lane % kCopies][key >> 21], 1u);
    }
  }
  __syncthreads();
  // three counts: the digits of the m-th highest key, and how many keys equal to it stay
  uint32_t prefix = 0, need = (uint32_t)m;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    uint32_t *hist = s_hist[pass == 1 ? kCopies : 0];
    if (pass > 0) {
      const int above = pass == 1 ? 21 : 10;
      for (int i = tid; i < cnt; i += kSelThreads) {
        const uint32_t key = keys[i];
        if (key >> above == prefix) atomicAdd(&hist[(key >> shift) & (uint32_t)(bins - 1)], 1u);
      }
    } else {
      for (int i = tid; i < kBins; i += kSelThreads)
#pragma unroll
        for (int k = 1; k < kCopies; ++k) hist[i] += hist[k * kBins + i];
    }
    if (C > 1)
      cluster_sync();
    else
      __syncthreads();
    // thread i: 4 bins from the top.  (A CTA reads its peers' counts 16 bytes at a time: word
    // by word, 18 us for 8 CTAs.)
    const int bin0 = bins - 4 - 4 * tid;   // the lowest of the thread's
    uint32_t c[4] = {0, 0, 0, 0};
    if (bin0 >= 0) {
      if (C > 1) {
#pragma unroll 8
        for (uint32_t r = 0; r < C; ++r) {
          const uint4 x = ld_peer4(hist + bin0, r);
          c[0] += x.w, c[1] += x.z, c[2] += x.y, c[3] += x.x;
        }
      } else {
        const uint4 x = *reinterpret_cast<const uint4 *>(hist + bin0);
        c[0] = x.w, c[1] = x.z, c[2] = x.y, c[3] = x.x;
      }
    }
    const uint32_t sum = c[0] + c[1] + c[2] + c[3];
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_above[warp] = inc;
    __syncthreads();
    uint32_t before = inc - sum;
    for (int i = 0; i < warp; ++i) before += s_above[i];
    if (before < need && need <= before + sum) {   // one thread
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (before < need && need <= before + c[j]) {
          s_pick[0] = (uint32_t)(bin0 + 3 - j);
          s_pick[1] = need - before;
          break;
        }
        before += c[j];
      }
    }
    __syncthreads();
    prefix = prefix << (pass == 2 ? 10 : 11) | s_pick[0];
    need = s_pick[1];
    // the first pass's counts are not read any more once every CTA has passed the second's barrier
    if (pass == 1) {
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[0][i] = 0;
      __syncthreads();
    }
  }
  // tokens above the key, and equal ones, before each warp's run of the CTA's keys
  const int run = (int)round_up((cnt + kSelWarps - 1) / kSelWarps, 32);
  const int r0 = min(warp * run, cnt), r1 = min(r0 + run, cnt);
  uint32_t above = 0, equal = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    const uint32_t key = keys[i];
    above += key > prefix;
    equal += key == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) s_above[warp] = above, s_equal[warp] = equal;
  __syncthreads();
  if (tid == 0) {
    uint32_t x = 0, y = 0;
    for (int i = 0; i < kSelWarps; ++i) {
      const uint32_t xa = s_above[i], ya = s_equal[i];
      s_above[i] = x, s_equal[i] = y;
      x += xa, y += ya;
    }
    s_count[0] = x, s_count[1] = y;
  }
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  uint32_t na = s_above[warp], ne = s_equal[warp];
  for (uint32_t r = 0; r < rank; ++r) na += ld_peer(&s_count[0], r), ne += ld_peer(&s_count[1], r);
  for (int i = r0; i < r1; i += 32) {
    const bool in = i + lane < r1;
    const uint32_t key = in ? keys[i + lane] : 0u;
    const uint32_t ba = __ballot_sync(0xffffffffu, in && key > prefix), be = __ballot_sync(0xffffffffu, in && key == prefix);
    const uint32_t lt = (1u << lane) - 1u;
    const uint32_t xa = na + __popc(ba & lt), xe = ne + __popc(be & lt);
    if (in && (key > prefix || (key == prefix && xe < need))) list[xa + min(xe, need)] = t0 + i + lane;
    na += __popc(ba);
    ne += __popc(be);
  }
  if (C > 1) cluster_sync();   // no CTA leaves while a peer may read it
}

// ------------------------------------------------------------------------- the rows
constexpr int kMoveThreads = 256;
constexpr int kMoveBlocks = 3 * 152;   // resident
constexpr int kMoveLoads = 8;   // of a thread: 16 bytes, or a total
static_assert(kMoveThreads * kMoveLoads == kEvictTotals && kMoveThreads * kMoveLoads * 16 == kEvictRows * 256, "a block's share");

// Row numbers (page, row in it) of a place in a sequence; -1 without a page (recorded).
__device__ __forceinline__ long long ev_row(const int32_t *table, int t, int sh, int num_pages, int *status) {
  const int page = __ldg(table + (t >> sh));
  if ((unsigned)page >= (unsigned)num_pages) {
    atomicCAS(status, DA_OK, DA_ERR_INVALID);
    return -1;
  }
  return ((long long)page << sh) | (t & ((1 << sh) - 1));
}

// 0, once the loads behind `words` have returned: a barrier that says "read" must not
// overtake them.
__device__ __forceinline__ int ev_arrived(uint32_t words) {
  uint32_t same;
  asm volatile("mov.b32 %0, %1;" : "=r"(same) : "r"(words));
  return (int)(same ^ words);
}

template <typename V>
__device__ __forceinline__ V ev_load(const uint8_t *p) { return __ldcg(reinterpret_cast<const V *>(p)); }
__device__ __forceinline__ uint32_t ev_words(const uint4 &v) { return v.x | v.y | v.z | v.w; }
__device__ __forceinline__ uint32_t ev_words(float v) { return __float_as_uint(v); }

// A head's rows, or a query head's totals: where they come from and go.
struct MoveHead {
  const int32_t *list, *src, *dst;
  int s, h, m;
  __device__ __forceinline__ MoveHead(const EvictArgs &a, const EvictWorkspace &w, int s_, int h_, bool totals) : s(s_), h(h_) {
    m = __ldcg(reinterpret_cast<const int2 *>(a.ws + w.info_off) + s).x;
    list = (a.kept != nullptr ? a.kept : reinterpret_cast<const int32_t *>(a.ws + w.list_off)) +
           ((size_t)s * a.c.Hkv + (totals ? h / (a.c.Hq / a.c.Hkv) : h)) * a.max_keep;
    src = (totals ? a.c.demand_table : a.c.page_table) + (size_t)s * a.c.max_pages;
    dst = a.dst_page_table == nullptr ? src : (totals ? a.dst_demand_table : a.dst_page_table) + (size_t)s * a.dst_max_pages;
  }
};
// Of its row r, which takes token t's: both rows in the pool; false where nothing moves.
__device__ __forceinline__ bool ev_rows(const MoveHead &k, int t, int r, int sh, int num_pages, int *status, long long &from,
                                        long long &to) {
  from = ev_row(k.src, t, sh, num_pages, status);
  to = ev_row(k.dst, r, sh, num_pages, status);
  return from >= 0 && to >= 0 && from != to;
}

// 2048 totals: rows r0 .. + 2047 of those before `end`.
struct MoveTotals {
  float v[kMoveLoads];
  float *to[kMoveLoads];
  __device__ __forceinline__ void read(const EvictArgs &a, const MoveHead &k, int r0, int end, int sh) {
    int t[kMoveLoads];
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) {
      const int r = r0 + (int)threadIdx.x + u * kMoveThreads;
      t[u] = r < end ? __ldcg(k.list + r) : -1;
    }
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) {
      const int r = r0 + (int)threadIdx.x + u * kMoveThreads;
      long long i, o;
      to[u] = nullptr;
      if (t[u] >= 0 && ev_rows(k, t[u], r, sh, a.c.num_demand_pages, a.status, i, o)) {
        const int in_page = (1 << sh) - 1;   // of the pool: page, head, row
        v[u] = __ldcg(a.c.demand_pages + ((((size_t)(i >> sh) * a.c.Hq + k.h) << sh) + (size_t)(i & in_page)));
        to[u] = a.c.demand_pages + ((((size_t)(o >> sh) * a.c.Hq + k.h) << sh) + (size_t)(o & in_page));
      }
    }
  }
  __device__ __forceinline__ void write() {
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u)
      if (to[u] != nullptr) *to[u] = v[u];
  }
};

// 16-byte pieces of rows of keys and values, each thread's of a batch.
template <int THREADS>
struct MovePieces {
  uint8_t *k, *v;        // the pools, at the key head's first row
  size_t page_bytes;
  int row_bytes, half, shift, page_shift;
  __device__ __forceinline__ MovePieces(const EvictArgs &a, int h, int sh) : page_shift(sh) {
    row_bytes = a.c.d * (a.c.dtype == DA_BF16 ? 2 : 4);
    half = row_bytes / 16;                 // powers of two
    shift = __ffs(2 * half) - 1;
    page_bytes = ((size_t)a.c.Hkv * row_bytes) << sh;
    k = reinterpret_cast<uint8_t *>(a.c.k_pages) + (((size_t)h * row_bytes) << sh);
    v = reinterpret_cast<uint8_t *>(a.c.v_pages) + (((size_t)h * row_bytes) << sh);
  }
  __device__ __forceinline__ int row(int u) const { return ((int)threadIdx.x + u * THREADS) >> shift; }
  __device__ __forceinline__ uint4 *at(long long row, int u) const {
    const int piece = ((int)threadIdx.x + u * THREADS) & (2 * half - 1);
    return reinterpret_cast<uint4 *>((piece < half ? k : v) + (size_t)(row >> page_shift) * page_bytes +
                                     (size_t)(row & ((1 << page_shift) - 1)) * row_bytes) +
           (piece & (half - 1));
  }
};

// Rows from .. m - 1 of a head, in place: `lanes` threads with one V each for a row's
// slice, a batch of kMoveLoads steps at a time.  The next batch's places are found
// while one is on its way.  (With two batches on their way, 128 registers spill: 189 us
// where one takes 150.)
template <typename V>
struct MovePlace {
  uint8_t *pool;           // at the head's first row and the thread's bytes
  size_t page_bytes;
  int row_bytes, sh, num_pages, step, row0, m;   // rows of a step; the thread's first row
  int *status;
  const int32_t *list, *table;
  __device__ __forceinline__ uint8_t *at(int page, int t) const {
    return pool + (size_t)page * page_bytes + (size_t)((t & ((1 << sh) - 1)) * row_bytes);
  }
  __device__ __forceinline__ int row(int b, int u) const { return row0 + (b * kMoveLoads + u) * step; }
  __device__ __forceinline__ void tokens(int b, int (&t)[kMoveLoads]) const {
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) t[u] = row(b, u) < m ? __ldcg(list + row(b, u)) : -1;
  }
  __device__ __forceinline__ void pages(int b, const int (&t)[kMoveLoads], int (&from)[kMoveLoads], int (&to)[kMoveLoads]) const {
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) {
      from[u] = t[u] >= 0 ? __ldg(table + (t[u] >> sh)) : 0;
      to[u] = t[u] >= 0 ? __ldg(table + (row(b, u) >> sh)) : 0;
    }
  }
  // to: -1 where nothing moves
  __device__ __forceinline__ void read(int b, const int (&t)[kMoveLoads], const int (&from)[kMoveLoads], int (&to)[kMoveLoads],
                                       V (&v)[kMoveLoads]) const {
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) {
      const bool have = t[u] >= 0, ok = (unsigned)from[u] < (unsigned)num_pages && (unsigned)to[u] < (unsigned)num_pages;
      if (have && !ok) atomicCAS(status, DA_OK, DA_ERR_INVALID);
      if (have && ok && t[u] != row(b, u))
        v[u] = ev_load<V>(at(from[u], t[u]));
      else
        to[u] = -1;
    }
  }
  __device__ __forceinline__ void run() const {
    const int batches = (m - row0 + (int)threadIdx.x / ((int)blockDim.x / step) + kMoveLoads * step - 1) / (kMoveLoads * step);
    int t[kMoveLoads], from[kMoveLoads], to[kMoveLoads];
    tokens(0, t);
    pages(0, t, from, to);
#pragma unroll 1
    for (int b = 0; b < batches; ++b) {
      V v[kMoveLoads];
      uint8_t *out[kMoveLoads];
      read(b, t, from, to, v);
#pragma unroll
      for (int u = 0; u < kMoveLoads; ++u) out[u] = to[u] >= 0 ? at(to[u], row(b, u)) : nullptr;
      tokens(b + 1, t);
      pages(b + 1, t, from, to);
      uint32_t words = 0;
#pragma unroll
      for (int u = 0; u < kMoveLoads; ++u)
        if (out[u] != nullptr) words |= ev_words(v[u]);
      __syncthreads_or(ev_arrived(words));   // the batch has been read
#pragma unroll
      for (int u = 0; u < kMoveLoads; ++u)
        if (out[u] != nullptr) *reinterpret_cast<V *>(out[u]) = v[u];
    }
  }
};

__global__ void __launch_bounds__(kMoveThreads, 2) evict_place(EvictArgs a, EvictWorkspace w, int sh, int slices) {
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, G = a.c.Hq / a.c.Hkv, parts = 2 * slices + G;
  const int item = blockIdx.x / parts, part = blockIdx.x % parts;
  const bool totals = part >= 2 * slices;
  const int s = item / a.c.Hkv, hkv = item % a.c.Hkv;
  const MoveHead k(a, w, s, totals ? hkv * G + part - 2 * slices : hkv, totals);
  if (part == 0 && hkv == 0 && tid == 0) a.new_lens[s] = __ldcg(reinterpret_cast<const int2 *>(a.ws + w.info_off) + s).y;
  // the first row that moves: list[r] - r does not decrease
  int from = 0;
  for (int n = k.m; n > 0;) {
    const int step = (n + kMoveThreads - 1) / kMoveThreads, r = from + tid * step;
    const int same = __syncthreads_count(tid * step < n && __ldcg(k.list + r) == r);
    if (same == 0) break;
    const int skip = (same - 1) * step + 1;
    from += skip;
    n = min(step - 1, n - skip);
  }
  if (from >= k.m) return;
  if (totals) {
    MovePlace<float> x{reinterpret_cast<uint8_t *>(a.c.demand_pages) + (((size_t)k.h * 4) << sh), ((size_t)a.c.Hq * 4) << sh, 4, sh,
                       a.c.num_demand_pages, kMoveThreads, from + tid, k.m, a.status, k.list, k.src};
    x.run();
  } else {
    const int row_bytes = a.c.d * (a.c.dtype == DA_BF16 ? 2 : 4), bytes = row_bytes / slices, lanes = bytes / 16;   // powers of two
    uint8_t *pool = reinterpret_cast<uint8_t *>(part < slices ? a.c.k_pages : a.c.v_pages);
    MovePlace<uint4> x{pool + (((size_t)k.h * row_bytes) << sh) + part % slices * bytes + tid % lanes * 16,
                       ((size_t)a.c.Hkv * row_bytes) << sh, row_bytes, sh, a.c.num_pages, kMoveThreads / lanes, from + tid / lanes, k.m,
                       a.status, k.list, k.src};
    x.run();
  }
}

// To other pages.  The next chunk's places are found while the one at hand is on its
// way: ticket, list, tables and rows one after the other took 10 us a chunk.
constexpr int kMoveSeqs = 1024;   // sequences whose chunks are counted; more take equally many each
__global__ void __launch_bounds__(kMoveThreads, 3) evict_move(EvictArgs a, EvictWorkspace w, int sh) {
  __shared__ int s_cum[kMoveSeqs + 1];                   // chunks of a key head before each sequence
  __shared__ int s_warp[kMoveThreads / 32];
  __shared__ long long s_from[2][kEvictRows], s_to[2][kEvictRows];
  __shared__ int s_ticket[2];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, S = a.c.S, Hkv = a.c.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  int32_t *counter = reinterpret_cast<int32_t *>(a.ws + w.flag_off);
  const int rows = kEvictRows * 128 / (a.c.d * (a.c.dtype == DA_BF16 ? 2 : 4));   // of a chunk
  const int2 *info = reinterpret_cast<const int2 *>(a.ws + w.info_off);
  for (int s = blockIdx.x * kMoveThreads + tid; s < S; s += gridDim.x * kMoveThreads) a.new_lens[s] = __ldcg(info + s).y;
  const bool counted = S <= kMoveSeqs;
  if (counted) {
    constexpr int PER = kMoveSeqs / kMoveThreads;
    int c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = tid * PER + i;
      c[i] = sum;
      if (s < S) sum += (__ldcg(info + s).x + rows - 1) / rows;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int base = inc - sum;
    for (int i = 0; i < warp; ++i) base += s_warp[i];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (tid * PER + i <= S) s_cum[tid * PER + i] = base + c[i];
    if (tid == kMoveThreads - 1 && S == kMoveSeqs) s_cum[S] = base + sum;
  }
  if (tid == 0) {
    s_ticket[0] = atomicAdd(counter, 1);
    s_ticket[1] = atomicAdd(counter, 1);
  }
  __syncthreads();
  const int most = (int)((a.max_keep < a.max_len ? a.max_keep : a.max_len) + rows - 1) / rows;
  const long long chunks = (long long)Hkv * (counted ? s_cum[S] : (long long)S * most);
  const long long tickets = chunks + (long long)S * a.c.Hq * w.total_chunks;
  int cs = 0, ch = 0, cr = 0, ct = -1;                   // of the next chunk: sequence, key head, this thread's row and its token
  auto find = [&](int ticket) {
    ct = -1;
    if (ticket >= chunks) return;
    int first, each = most;
    if (counted) {
      int lo = 0, hi = S - 1;                             // the last sequence whose chunks begin at or before
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if ((long long)Hkv * s_cum[mid] <= ticket)
          lo = mid;
        else
          hi = mid - 1;
      }
      cs = lo;
      first = Hkv * s_cum[lo];
      each = s_cum[lo + 1] - s_cum[lo];
    } else {
      cs = ticket / (Hkv * most);
      first = cs * Hkv * most;
    }
    ch = (ticket - first) / each;
    cr = (ticket - first) % each * rows + tid;
    const MoveHead k(a, w, cs, ch, false);
    if (tid < rows && cr < k.m) ct = __ldcg(k.list + cr);
  };
  auto places = [&](int buf) {
    if (tid >= rows) return;
    long long i = -1, o = -1;
    const bool moves = ct >= 0 && ev_rows(MoveHead(a, w, cs, ch, false), ct, cr, sh, a.c.num_pages, a.status, i, o);
    s_from[buf][tid] = moves ? i : -1;
    s_to[buf][tid] = o;
  };
  int now = s_ticket[0];
  find(now);
  places(0);
  for (int turn = 0; now < tickets; ++turn) {
    const int buf = turn & 1, next = s_ticket[buf ^ 1];
    __syncthreads();                                      // the chunk's places are there
    if (now >= chunks) {
      const int item = (int)((now - chunks) / w.total_chunks), r0 = (int)((now - chunks) % w.total_chunks) * kEvictTotals;
      const MoveHead k(a, w, item / a.c.Hq, item % a.c.Hq, true);
      MoveTotals t;
      t.read(a, k, r0, min(k.m, r0 + kEvictTotals), sh);
      if (tid == 0) s_ticket[buf] = atomicAdd(counter, 1);
      t.write();
    } else {
      const MovePieces<kMoveThreads> x(a, ch, sh);
      uint4 v[kMoveLoads];
#pragma unroll
      for (int u = 0; u < kMoveLoads; ++u) {
        const long long i = s_from[buf][x.row(u)];
        if (i >= 0) v[u] = __ldcg(x.at(i, u));
      }
      find(next);                                         // (its list is on its way)
      if (tid == 0) s_ticket[buf] = atomicAdd(counter, 1);   // (of the chunk after the next)
      if (next < chunks) places(buf ^ 1);
#pragma unroll
      for (int u = 0; u < kMoveLoads; ++u)
        if (s_from[buf][x.row(u)] >= 0) *x.at(s_to[buf][x.row(u)], u) = v[u];
    }
    now = next;
    __syncthreads();                                      // the places have been read
  }
}

// Up to kSmallKeys tokens a sequence.  Thread t has token t; the m-th highest score is
// found bit by bit, a count over the block each.  (Every score compared with every other:
// 4 us of one SM's instructions for 500.)  Then rows in order, a batch read before it is written, so that in place nothing is overwritten
// that is still to be read (see evict_place).
constexpr int kSmallKeys = 512, kSmallThreads = kSmallKeys, kSmallLoads = 8;
__global__ void __launch_bounds__(kSmallThreads) evict_small(EvictArgs a, int sh) {
  __shared__ int s_list[kSmallKeys], s_warp[kSmallThreads / 32];
  __shared__ int s_page[4][kSmallKeys / 16];   // of keys and values, of totals: from, and where to
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int s = blockIdx.x / a.c.Hkv, h = blockIdx.x % a.c.Hkv, G = a.c.Hq / a.c.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  // tables and lengths at once: one after the other they were 1.3 us
  const bool same = a.dst_page_table == nullptr;
  if (tid < 4 * (kSmallKeys / 16)) {
    const int which = tid / (kSmallKeys / 16), i = tid % (kSmallKeys / 16);
    const int tokens = which < 2 || same ? a.max_len : min(a.max_keep, a.max_len), width = which < 2 || same ? a.c.max_pages : a.dst_max_pages;
    const int32_t *table = which == 0 || (same && which == 2) ? a.c.page_table
                           : which == 1 || same               ? a.c.demand_table
                           : which == 2                       ? a.dst_page_table
                                                              : a.dst_demand_table;
    s_page[which][i] = i << sh < tokens ? __ldcg(table + (size_t)s * width + i) : -1;
  }
  const int len = __ldcg(a.c.seq_lens + s), keep = __ldcg(a.keep + s);
  const bool good = len >= 0 && len <= a.max_len && keep >= 0 && min(len, keep) <= a.max_keep;
  const int m = good ? min(len, keep) : 0;
  __syncthreads();
  if (h == 0 && tid == 0) {
    if (!good) atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
    a.new_lens[s] = good ? m : len;   // (no other block reads it: see launch_evict)
  }
  int32_t *kept = a.kept != nullptr ? a.kept + (size_t)blockIdx.x * a.max_keep : nullptr;
  if (kept != nullptr)
    for (int i = m + tid; i < a.max_keep; i += kSmallThreads) kept[i] = -1;
  if (m == 0) return;
  const int in_page = (1 << sh) - 1;
  uint32_t key = 0;   // below every score
  if (tid < len && m < len) {
    const int page = s_page[1][tid >> sh];
    float v = 0.f;
    if ((unsigned)page < (unsigned)a.c.num_demand_pages) {
      const float *at = a.c.demand_pages + ((((size_t)page * a.c.Hq + (size_t)h * G) << sh) + (tid & in_page));
      for (int g = 0; g < G; g += 4) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + e < G) f[e] = __ldcg(at + ((size_t)(g + e) << sh));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g + e < G) v = g + e == 0 ? f[e] : __fadd_rn(v, f[e]);
      }
    } else {
      atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
    }
    key = ev_key(tid < a.sinks || tid >= len - a.recent ? INFINITY : v);
  }
  // the m-th highest key, bit by bit from the top, until just m are at least as high
  uint32_t least = 0;
  if (m < len) {
    for (int bit = 31; bit >= 0; --bit) {
      const int n = __syncthreads_count(key >= (least | 1u << bit));
      if (n >= m) least |= 1u << bit;
      if (n == m) break;
    }
  }
  const bool above = tid < len && key > least, equal = tid < len && key == least;
  const unsigned va = __ballot_sync(0xffffffffu, above), ve = __ballot_sync(0xffffffffu, equal), lt = (1u << lane) - 1u;
  if (lane == 0) s_warp[warp] = __popc(va) << 16 | __popc(ve);
  __syncthreads();
  int na = 0, ne = 0, all = 0;   // before this warp, and all that are above
  for (int i = 0; i < kSmallThreads / 32; ++i) {
    const int n = s_warp[i];
    all += n >> 16;
    if (i < warp) na += n >> 16, ne += n & 0xffff;
  }
  na += __popc(va & lt);
  ne += __popc(ve & lt);
  const int need = m - all;      // equal ones that stay, the first of them
  if (above || (equal && ne < need)) {
    const int place = na + min(ne, need);
    s_list[place] = tid;
    if (kept != nullptr) kept[place] = tid;
  }
  __syncthreads();
  // the row of a place: -1 without a page (recorded)
  auto row_of = [&](int table, int t, int num_pages) -> long long {
    const int page = s_page[table][t >> sh];
    if ((unsigned)page < (unsigned)num_pages) return ((long long)page << sh) | (t & in_page);
    atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
    return -1;
  };
  const MovePieces<kSmallThreads> x(a, h, sh);
  const int rows = kSmallThreads * kSmallLoads >> x.shift;   // of a batch
  for (int r0 = 0, g = 0; r0 < m || g < G; r0 += rows, g += 4) {
    uint4 v[kSmallLoads];
    uint4 *out[kSmallLoads];
    float f[4];
    float *to[4];
    uint32_t words = 0;
#pragma unroll
    for (int u = 0; u < kSmallLoads; ++u) {
      const int r = r0 + x.row(u);
      out[u] = nullptr;
      if (r >= m) continue;
      const int t = s_list[r];
      const long long i = row_of(0, t, a.c.num_pages), o = row_of(2, r, a.c.num_pages);
      if (i < 0 || o < 0 || i == o) continue;
      v[u] = __ldcg(x.at(i, u));
      out[u] = x.at(o, u);
    }
    // four query heads' totals, a row a thread
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = nullptr;
    if (g < G && tid < m) {
      const long long i = row_of(1, s_list[tid], a.c.num_demand_pages), o = row_of(3, tid, a.c.num_demand_pages);
      if (i >= 0 && o >= 0 && i != o) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (g + e >= G) break;
          const size_t head = (size_t)h * G + g + e;
          f[e] = __ldcg(a.c.demand_pages + ((((size_t)(i >> sh) * a.c.Hq + head) << sh) + (size_t)(i & in_page)));
          to[e] = a.c.demand_pages + ((((size_t)(o >> sh) * a.c.Hq + head) << sh) + (size_t)(o & in_page));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kSmallLoads; ++u)
      if (out[u] != nullptr) words |= ev_words(v[u]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (to[e] != nullptr) words |= ev_words(f[e]);
    __syncthreads_or(ev_arrived(words));   // the batch has been read
#pragma unroll
    for (int u = 0; u < kSmallLoads; ++u)
      if (out[u] != nullptr) *out[u] = v[u];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (to[e] != nullptr) *to[e] = f[e];
  }
}

// Whether `n` 32-bit words at a and at b share bytes.
static bool words_meet(const void *a, const void *b, int64_t n) {
  const intptr_t d = reinterpret_cast<intptr_t>(a) - reinterpret_cast<intptr_t>(b);
  return d < 4 * n && -d < 4 * n;
}

int launch_evict(const EvictArgs &a, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return cudaFuncSetAttribute(evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictKeys * 4) != cudaSuccess
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  const EvictWorkspace w = evict_workspace(a.c.S, a.c.Hkv, a.max_keep < a.max_len ? a.max_keep : a.max_len, a.max_len);
  int sh = 0;
  while ((1 << sh) < a.c.page_size) ++sh;
  const int rows = kEvictRows * 128 / (a.c.d * (a.c.dtype == DA_BF16 ? 2 : 4));
  const int64_t items = (int64_t)a.c.S * a.c.Hkv, totals = (int64_t)a.c.S * a.c.Hq, most = a.max_keep < a.max_len ? a.max_keep : a.max_len;
  const int64_t tickets = items * ((most + rows - 1) / rows) + totals * w.total_chunks;
  if (tickets > 0x7F000000 || items * w.cluster > 0x7FFFFFFF || items * 64 + totals > 0x7FFFFFFF)
    return DA_ERR_UNSUPPORTED;
  // One launch for short sequences whose rows are up to 96 MB, unless the lengths are
  // written where blocks still read them (us of one launch / two, half of about 500
  // tokens kept: 12 key heads of d = 64, 1 sequence 12.9 / 16.0, 8 12.9 / 24.2; d = 128, 64 x 4
  // 27.3 / 38.5, 64 x 12 (100 MB) 67.6 / 67.6, in fp32 (200 MB) 106.5 / 98.3).
  const int64_t row_bytes2 = 2 * a.c.d * (a.c.dtype == DA_BF16 ? 2 : 4);
  if (a.max_len <= kSmallKeys && items * most * row_bytes2 <= 96ll << 20 && !words_meet(a.new_lens, a.c.seq_lens, a.c.S) && !words_meet(a.new_lens, a.keep, a.c.S))
    return launch_after(evict_small, dim3((unsigned)items), kSmallThreads, 0, stream, a, sh) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.c.S * a.c.Hkv * w.cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = w.shared ? (size_t)w.slice * 4 : 0;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)w.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // (see launch_after)
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, evict_select, a, w, sh) != cudaSuccess) return DA_ERR_CUDA;
  if (a.dst_page_table == nullptr) {
    const int row_bytes = a.c.d * (a.c.dtype == DA_BF16 ? 2 : 4);
    int slices = 1;
    while (items * 2 * slices < 4 * 152 && row_bytes / slices > 32) slices *= 2;
    return launch_after(evict_place, dim3((unsigned)(items * (2 * slices + a.c.Hq / a.c.Hkv))), kMoveThreads, 0, stream, a, w, sh,
                        slices) == cudaSuccess
               ? DA_OK
               : DA_ERR_CUDA;
  }
  const int64_t blocks = tickets < 1 ? 1 : tickets < kMoveBlocks ? tickets : kMoveBlocks;
  return launch_after(evict_move, dim3((unsigned)blocks), kMoveThreads, 0, stream, a, w, sh) == cudaSuccess ? DA_OK
                                                                                                          : DA_ERR_CUDA;
}

}  // namespace da
