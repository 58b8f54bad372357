// Chunks over the paged cache in bf16: tcgen05 kernels.
//
// Mathematics: as paged_chunk_f32.cu.
//   ckx_keys    (max, sum 2^(x - max)) of every row over a piece's key tiles;
//   ckx_values  p = 2^(x - lse2), total += p, share = p / (total + eps), and the
//               sums of share v and share over them.
//
// What bounds it: with many rows the demand's arithmetic (an exponential, half a
// reciprocal and a running sum a pair), as in the prompt's sweep (fwd_bf16.cu); with
// few the pages, which both passes bring once for all rows of a key head.
//
// ckx_keys: S[row, key] = Q K^T (M = 128 rows, N = 128 keys), one thread a row with
// a running maximum and sum; two warpgroups take alternate key tiles.
//
// ckx_values: S^T[key, row] = K Q^T (M = 128 keys), one thread a key, which walks
// the rows of the column tile with the key's total in a register; kG warpgroups take
// the key tiles of a piece in turn, each always the same ones, so that a total
// comes back to the thread that left it.  The shares, rounded to bf16 once (the
// product's operands have one type; 2^-8 of each share, and numerator and sum hold
// the same ones), go to shared memory as the MN-major A operand of
// D[row, :] += share^T [V | 1].  Shares of drafted and single tokens keep 2^-16, as in a
// decode step: what the rounding left is a second term, of up to 4 tokens in the rows that
// round them up to 8 (chunk_combine adds them), else, where several heads have up to 64 rows in
// all, in the places of the other 64, for a second product (mixed batch of 48: 353 -> 359
// us).  Unlike the prompt's sweep, the rows stay and the keys
// stream: D stays in TMEM over a piece's key tiles and leaves once, as a partial
// result of fixed place, so that equal calls give equal bits.
//
// Roles: demand (or reduction) warpgroups, a warpgroup that takes D out, and
// control warps: a producer that walks the CTA's pieces, describes each column tile
// in a small ring that every role reads, and brings Q, K and V by TMA; one MMA issuer
// a demand warpgroup.  Waits are bounded; rows of missing or invalid pages are
// filled with zeros by reading past the pool's end.
#include "da_chunk.cuh"

#include <cuda.h>
#include <cuda_bf16.h>

namespace da {

bool make_page_map(CUtensorMap *m, const void *base, int64_t num, int page_size, int rows, int d, int dtype);   // fwd_bf16.cu
bool make_rows_map(CUtensorMap *m, const void *base, int64_t n, int heads, int d, int rows);

constexpr int kCkxEdge = 128;
constexpr int kCkxKeyCtas = 304, kCkxValueCtas = 152;
constexpr uint32_t kCkxHalf = 128 * 128;   // 128 rows x 64 bf16
static_assert(kChunkLogits == kCkxEdge, "kept logits are whole key tiles");

bool chunk_few(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len);   // paged_chunk_few.cu
cudaError_t launch_chunk_few(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);

ChunkPlan chunk_plan_bf16(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len, int page_size) {
  // a unit is 8 rows of a key tile, about 40 ns
  ChunkPlan w = chunk_plan(S, Hq, Hkv, d, N, max_new, page_size, kCkxEdge, kCkxKeyCtas, kCkxValueCtas,
                           ChunkCost{d == 128 ? 28 : 14, 3, 1, 64, 16});
  if (chunk_few(S, Hq, Hkv, d, N, max_new, max_len)) {   // behind what every call needs
    w.logits = w.total;
    w.logits_ld = (int)round_up(max_len, kChunkLogits);
    w.logits_seq = N > (long long)S * max_new ? max_new : 0;   // (padded: no room for so many tokens)
  }
  return w;
}

// A column tile of a piece, as the producer describes it.
struct CkxTile {
  float *place;        // its rows' partial results
  float c2;            // of one head's rows: the logits' scale
  int s, hkv, hq0;     // sequence, key head, query head of row 0
  int n8, n, i0;       // rows of a head (0: one head); queries; query of row 0
  int P, len;          // place of query 0; length
  int tok0;            // query 0 among all
  int rows;            // 0: no more
  int tile, end, t0;   // key tiles; number of the first among the CTA's
  bool odd;            // a row's sum is NaN: it must not reach the rows before it, nor totals that it does not see
  bool clear;          // new tokens have values that are not finite
  __device__ __forceinline__ int query(int c) const { return n8 ? c % n8 : i0 + c; }
  // a second term of the shares: in the rows from 4 on of each head's eight, in those from 64 on
  __device__ __forceinline__ bool folded() const { return n8 != 0 && n <= kChunkFold; }
  __device__ __forceinline__ bool two_terms() const { return n8 != 0 && n > kChunkFold && rows <= 64; }
};
constexpr int kCkxRing = 4;

__device__ __forceinline__ void ckx_drain(uint64_t *bar, uint32_t parity) {   // lets copies and products in flight land
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > 100ull * 1000ull * 1000ull) break;
}
__device__ __forceinline__ void ckx_release(uint64_t *bar, int lane) {   // after the last tcgen05.ld of a buffer
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ uint64_t ckx_kmajor(const uint8_t *tile) { return smem_desc(smem_u32(tile), 16, 1024); }

// One warp: this lane's page of key tile `tile`; the tile of K or V into `dst`.
__device__ __forceinline__ int ckx_page(const PagedChunk &p, int sh, int s, int len, int tile, int lane) {
  const int rows = min(1 << sh, kCkxEdge), key = tile * kCkxEdge + lane * rows;
  return lane * rows < kCkxEdge && key < len ? __ldcg(p.c.page_table + (size_t)s * p.c.max_pages + (key >> sh)) : -1;
}
template <int D>
__device__ __forceinline__ void ckx_load(const PagedChunk &p, int sh, const CUtensorMap *map, uint8_t *dst, uint64_t *bar,
                                         int len, int tile, int hkv, int page, int lane) {
  const int ps = 1 << sh, rows = min(ps, kCkxEdge), key = tile * kCkxEdge + lane * rows;
  if (lane == 0) mbar_arrive_expect_tx(bar, kCkxEdge * D * 2);
  __syncwarp();
  if (lane * rows < kCkxEdge) {
    const bool ok = (unsigned)page < (unsigned)p.c.num_pages;
    if (!ok && key < len) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    const int z = ok ? page * p.c.Hkv + hkv : max(p.c.num_pages * p.c.Hkv, 1);   // past the map's end: zeros
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      tma_load_3d(dst + h * kCkxHalf + lane * rows * 128, map, bar, h * 64, key & (ps - 1), z);
  }
}
// Q of a column tile: 8 rows a box (what lies behind a tile's last row is read by no one).
template <int D>
__device__ __forceinline__ void ckx_queries(const CUtensorMap *map, uint8_t *dst, uint64_t *bar, int tok0, int hq0, int n8,
                                            int i0, int rows, int lane) {
  const int boxes = (rows + 7) / 8;
  if (lane == 0) mbar_arrive_expect_tx(bar, boxes * 8 * D * 2);
  __syncwarp();
  if (lane < boxes) {
    const int c = 8 * lane, hq = n8 ? hq0 + c / n8 : hq0, token = tok0 + (n8 ? c % n8 : i0 + c);
#pragma unroll
    for (int h = 0; h < D / 64; ++h) tma_load_3d(dst + h * kCkxHalf + lane * 1024, map, bar, h * 64, token, hq);
  }
}

// The producer's walk: column tile after column tile.
struct CkxWalk {
  ChunkWalk k;
  int b, t0;
  __device__ __forceinline__ void start(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l, const ChunkCut &cut,
                                        int lane) {
    k.start(p, w, l, cut, lane);
    t0 = 0;
    b = k.any() ? k.g.col0(k.tile) : 0;
  }
  __device__ __forceinline__ CkxTile tile(const PagedChunk &p, const ChunkPlan &w, size_t place_a, size_t place_b,
                                          int stride) const {
    CkxTile x;
    x.rows = 0;
    x.odd = x.clear = false;
    if (!k.any()) return x;
    const int r0 = b * k.g.step;
    x.s = k.s;
    x.hkv = k.hkv(w);
    x.n = k.g.n;
    x.P = k.g.P;
    x.tok0 = k.q.tok0;
    x.len = k.g.len;
    if (k.g.wide) {
      x.n8 = 0;
      x.hq0 = k.seg;
      x.i0 = r0;
      x.rows = min(k.g.step, x.n - r0);
    } else {
      x.n8 = k.g.n8;
      x.hq0 = k.seg * w.G + r0 / x.n8;
      x.i0 = 0;
      x.rows = min(k.g.step, w.G * x.n8 - r0);
    }
    x.tile = k.tile;
    x.end = min(k.end, k.g.seen(b, kCkxEdge));
    x.t0 = t0;
    const long long row0 = k.row0(p, w);
    x.place = chunk_place(p, place_a, place_b, row0, w.cta_rows, k.tile, blockIdx.x, r0, stride);
    x.c2 = k.g.wide ? fmaxf(head_c2(p.hs, k.s * p.c.Hq + x.hq0, nullptr), 1e-30f) : 0.f;
    return x;
  }
  // -lse2 of the column tile's rows 4 lane ..
  __device__ __forceinline__ float4 nl(const PagedChunk &p, const ChunkPlan &w, const CkxTile &x, int lane) const {
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p.ws + w.nl) + k.row0(p, w) +
                                                             b * k.g.step) + lane);
    const int c = 4 * lane;
    return make_float4(c < x.rows ? v.x : -INFINITY, c + 1 < x.rows ? v.y : -INFINITY, c + 2 < x.rows ? v.z : -INFINITY,
                       c + 3 < x.rows ? v.w : -INFINITY);
  }
  __device__ __forceinline__ void next(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l, const CkxTile &x) {
    t0 += x.end - x.tile;
    if (++b < k.g.cols) return;
    k.next(p, w, l);
    if (k.any()) b = k.g.col0(k.tile);
  }
};

// ============================================================================ pass 1
template <int D>
struct CkxKeys {
  static constexpr int kThreads = 320;                 // 2 x 4 reduction warps, producer, MMA issuer
  static constexpr int kTB = kCkxEdge * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr uint32_t kOffK = kTB, kOffRing = kOffK + kStages * kTB, kOffMl = kOffRing + kCkxRing * sizeof(CkxTile);
  static constexpr uint32_t kOffBar = kOffMl + 128 * 8;
  static constexpr int kSmemBytes = 1024 + kOffBar + 512;
  static constexpr int kTmemCols = 256;                // two S buffers of 128 columns; two CTAs an SM
};

// KEEP: the logits are kept for a second pass that does not read the keys again
// (paged_chunk_few.cu).
template <int D, bool KEEP>
__global__ void __launch_bounds__(CkxKeys<D>::kThreads, 2)
    ckx_keys(PagedChunk p, ChunkPlan w, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap) {
  using C = CkxKeys<D>;
  extern __shared__ __align__(1024) uint8_t ckx_smem_raw[];
  uint8_t *smem = ckx_smem_raw + ((1024u - (smem_u32(ckx_smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem, *sK = smem + C::kOffK;
  CkxTile *ring = reinterpret_cast<CkxTile *>(smem + C::kOffRing);
  float2 *s_ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
  uint64_t *r_full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *r_free = r_full + kCkxRing;
  uint64_t *q_full = r_free + kCkxRing, *q_empty = q_full + 1, *k_full = q_empty + 1, *k_empty = k_full + C::kStages;
  uint64_t *s_full = k_empty + C::kStages, *s_free = s_full + 2, *ml_full = s_free + 2, *ml_free = ml_full + 4;
  uint64_t *done = ml_free + 4;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    for (int i = 0; i < kCkxRing; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_free[i], 9);   // 8 reduction warps and the issuer
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ml_full[i], 1);
      mbar_init(&ml_free[i], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  pdl_wait();   // nothing before touches memory
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status};
  if (warp == 8) {
    // ---------------------------------------------------------------- producer
    const ChunkLine l = chunk_line(p, w);
    const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_keys);
    const int sh = w.page_shift;
    CkxWalk it;
    int i = 0, issued = 0;
    bool ok = true;
    for (it.start(p, w, l, cut, lane); ok; ++i) {
      const CkxTile x = it.tile(p, w, w.ml_a, w.ml_b, 2);
      ok = warp_wait(&r_free[i % kCkxRing], ((i / kCkxRing) & 1) ^ 1, wc);
      if (!ok) break;
      if (lane == 0) {
        ring[i % kCkxRing] = x;
        mbar_arrive(&r_full[i % kCkxRing]);
      }
      if (x.rows == 0) break;
      ok = warp_wait(q_empty, (i & 1) ^ 1, wc);
      if (!ok) break;
      ckx_queries<D>(&qmap, sQ, q_full, it.k.q.tok0, x.hq0, x.n8, x.i0, x.rows, lane);
      int page = ckx_page(p, sh, x.s, x.len, x.tile, lane);
      for (int j = x.tile; j < x.end; ++j, ++issued) {
        const int ahead = j + 1 < x.end ? ckx_page(p, sh, x.s, x.len, j + 1, lane) : -1;
        const int st = issued % C::kStages;
        ok = warp_wait(&k_empty[st], ((issued / C::kStages) & 1) ^ 1, wc);
        if (!ok) break;
        ckx_load<D>(p, sh, &kmap, sK + st * C::kTB, &k_full[st], x.len, j, x.hkv, page, lane);
        page = ahead;
      }
      it.next(p, w, l, x);
    }
    if (*abort_flag && lane == 0) {
      for (int t = issued > C::kStages ? issued - C::kStages : 0; t < issued; ++t)
        ckx_drain(&k_full[t % C::kStages], (t / C::kStages) & 1);
      if (i > 0) ckx_drain(q_full, (i - 1) & 1);
      ckx_drain(q_full, i & 1);
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, kCkxEdge, false, false);
      const uint64_t dQ = ckx_kmajor(sQ), dK = ckx_kmajor(sK);
      int t = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        ok = mbar_wait(&r_full[i % kCkxRing], (i / kCkxRing) & 1, wc);
        if (!ok) break;
        const CkxTile &x = ring[i % kCkxRing];
        const int rows = x.rows, tiles = x.end - x.tile;
        mbar_arrive(&r_free[i % kCkxRing]);
        if (rows == 0) break;
        ok = mbar_wait(q_full, i & 1, wc);
        for (int j = 0; ok && j < tiles; ++j, ++t) {
          const int st = t % C::kStages, b = t & 1;
          ok = mbar_wait(&k_full[st], (t / C::kStages) & 1, wc) && mbar_wait(&s_free[b], ((t >> 1) & 1) ^ 1, wc);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dKs = dK + (uint64_t)st * (C::kTB >> 4);
          MmaRun<0, 4, 2, 2, false>::go(tmem + b * 128, dQ, dKs, idesc, 0u);
          if constexpr (D == 128)
            MmaRun<0, 4, 2, 2, false>::go(tmem + b * 128, dQ + (kCkxHalf >> 4), dKs + (kCkxHalf >> 4), idesc, 1u);
          mma_commit(&s_full[b]);
          mma_commit(&k_empty[st]);
        }
        if (ok) mma_commit(q_empty);
      }
      mma_commit(done);
      ckx_drain(done, 0);
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- reduction
    const int g = warp / 4, quarter = warp % 4, c = quarter * 32 + lane;   // tile parity; row of the column tile
    const uint32_t ts = tmem + g * 128 + ((uint32_t)(quarter * 32) << 16);
    for (int i = 0;; ++i) {
      if (!warp_wait(&r_full[i % kCkxRing], (i / kCkxRing) & 1, wc)) break;
      const CkxTile &x = ring[i % kCkxRing];
      const int rows = x.rows, tiles = x.end - x.tile, t0 = x.t0, first = x.tile;
      const int q = x.query(c);
      const bool valid = c < rows && q < x.n;
      const int last = valid ? x.P + q : -1;   // the last key that the row sees
      float2 *to = reinterpret_cast<float2 *>(x.place) + c;
      float c2 = 1e-30f;
      if (valid)
        c2 = fmaxf(head_c2(p.hs, x.s * p.c.Hq + x.hq0 + (x.n8 ? c / x.n8 : 0), g == 0 ? p.status : nullptr), 1e-30f);
      float *kept = nullptr;
      if (KEEP && valid)
        kept = chunk_logits(p, w, x.s, x.tok0, q, x.hq0 + (x.n8 ? c / x.n8 : 0)) + first * kCkxEdge;
      __syncwarp();
      if (lane == 0) mbar_arrive(&r_free[i % kCkxRing]);
      if (rows == 0) break;
      const bool work = quarter * 32 < rows;   // uniform over the warp
      float m = -INFINITY;
      float2 l0 = make_float2(0.f, 0.f), l1 = make_float2(0.f, 0.f);
      auto take = [&](float (&v)[32], int left, int key) {   // 32 keys (from `key` of the piece), of which the row sees `left`
        if (KEEP && left > 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4 *>(kept + key + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        if (left < 32) {
          if (left <= 0) return;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= left) v[e] = -INFINITY;
        }
        float a[11];
#pragma unroll
        for (int e = 0; e < 10; ++e) a[e] = fmax3(v[3 * e], v[3 * e + 1], v[3 * e + 2]);
        a[10] = fmaxf(v[30], v[31]);
        const float top =
            fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmax3(a[6], a[7], fmax3(a[8], a[9], a[10])));
        // (no way out where top is -infinity: NaN does not show in it)
        const float mn = fmaxf(m, top * c2), ms = mn == -INFINITY ? 0.f : mn;
        const float f = ex2_approx(m - ms);
        m = mn;
        l0 = fmul2(l0, make_float2(f, f));
        l1 = fmul2(l1, make_float2(f, f));
        const float2 c2v = make_float2(c2, c2), nm = make_float2(-ms, -ms);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 x0 = ffma2(make_float2(v[2 * e], v[2 * e + 1]), c2v, nm);
          const float2 x1 = ffma2(make_float2(v[2 * e + 2], v[2 * e + 3]), c2v, nm);
          l0 = fadd2(l0, make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
          l1 = fadd2(l1, make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
        }
      };
      bool ok = true;
      for (int j = g ^ (t0 & 1); j < tiles; j += 2) {   // alternate tiles of the CTA
        const int t = t0 + j;
        ok = warp_wait(&s_full[g], (t >> 1) & 1, wc);
        if (!ok) break;
        tc_fence_after();
        if (work) {
          const int left = last + 1 - (first + j) * kCkxEdge;
          float a[32], b[32];
          tmem_ld32(ts, a);
          tmem_wait_ld_r(a);
          tmem_ld32(ts + 32, b);
          take(a, left, j * kCkxEdge);
          tmem_wait_ld_r(b);
          tmem_ld32(ts + 64, a);
          take(b, left - 32, j * kCkxEdge + 32);
          tmem_wait_ld_r(a);
          tmem_ld32(ts + 96, b);
          take(a, left - 64, j * kCkxEdge + 64);
          tmem_wait_ld_r(b);
          ckx_release(&s_free[g], lane);
          take(b, left - 96, j * kCkxEdge + 96);
        } else {
          ckx_release(&s_free[g], lane);
        }
      }
      if (!ok) break;
      // the two warpgroups' halves of a row meet in warpgroup 0
      const float sum = (l0.x + l0.y) + (l1.x + l1.y);
      if (g == 1) {
        if (!warp_wait(&ml_free[quarter], (i & 1) ^ 1, wc)) break;
        s_ml[c] = make_float2(m, sum);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ml_full[quarter]);
      } else {
        if (!warp_wait(&ml_full[quarter], i & 1, wc)) break;
        const float2 o = s_ml[c];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ml_free[quarter]);
        const float mn = fmaxf(m, o.x), ms = mn == -INFINITY ? 0.f : mn;
        if (valid) *to = make_float2(mn, sum * ex2_approx(m - ms) + o.y * ex2_approx(o.x - ms));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ============================================================================ pass 2
// Registers (setmaxnreg): the block's at launch, kRegsLaunch a thread, are dealt out
// anew to demand, epilogue and control warpgroups (checked on the host).
template <int D>
struct CkxVal {
  static constexpr int kG = D == 64 ? 3 : 2;           // demand warpgroups
  static constexpr int kThreads = (kG + 2) * 128;      // an epilogue and a control warpgroup
  static constexpr int kRegsDemand = D == 64 ? 128 : 168, kRegsEpi = D == 64 ? 40 : 72, kRegsCtl = D == 64 ? 56 : 72;
  static constexpr int kRegsLaunch = D == 64 ? 96 : 120;
  static constexpr int kRegsNeeded = 128 * (kG * kRegsDemand + kRegsEpi + kRegsCtl);
  static constexpr int kTB = kCkxEdge * D * 2;
  static constexpr int kStages = D == 64 ? 3 : 2;      // of K, and of V
  static constexpr int kLag = kG;                      // V behind K, in tiles
  static constexpr int kDrain = D == 64 ? 16 : 32;     // columns of D that the epilogue's registers hold
  // Barriers of what has landed: three rounds of stages, since those that wait for a
  // tile need not have seen the ones before it in its stage land, and a barrier's
  // parity tells a round from the next alone.  (The tile before it in its barrier has
  // been read: its stage was filled again since, before K of this one came.)
  static constexpr int kFull = 3 * kStages;
  static constexpr uint32_t kShBytes = 32 * 1024;      // a warpgroup's shares: 2 x 64 rows x 128 keys
  static constexpr int kQs = D == 64 ? 2 : 1;          // of Q
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffSh = kQs * kTB;
  static constexpr uint32_t kOffK = kOffSh + kG * kShBytes;      // behind the shares: see the second term's product
  static constexpr uint32_t kOffV = kOffK + kStages * kTB;
  static constexpr uint32_t kOffOnes = kOffV + kStages * kTB;    // above every V tile (positive offset)
  static constexpr uint32_t kOffRing = kOffOnes + 2048;
  static constexpr uint32_t kOffBar = kOffRing + kCkxRing * sizeof(CkxTile);
  static constexpr int kSmemBytes = kOffBar + 512;     // (the base is 1024-byte aligned)
  // TMEM: S^T of warpgroup g at 128 g; D (80 columns: values 0-63, share sum at 64);
  // at d = 128 values 64-127 behind it.
  static constexpr uint32_t kTmemD = kG * 128, kTmemDHi = kTmemD + 80;
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(kTmemDHi + D - 64 <= 512, "TMEM columns");
  static_assert(kRegsNeeded <= kThreads * kRegsLaunch && kThreads * kRegsLaunch <= 65536, "register split");
};
template <int N>
__device__ __forceinline__ void ckx_regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void ckx_regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// -lse2 of a column tile's rows lies in the ones block, in the 16-byte pieces that the
// product does not read: of its 16 rows of 128 bytes (swizzled as V) pieces 0 and 1
// are the ones, 2 and 3, or 4 and 5, hold the values of 8 rows, for every other
// column tile.  The place of values 4 i .. 4 i + 3 of column tile b.
__device__ __forceinline__ uint32_t ckx_nl_place(int i, int b) {
  return (uint32_t)((i >> 1) * 128 + (((2 + 2 * (b & 1) + (i & 1)) ^ ((i >> 1) & 7)) << 4));
}
// The same for constant i: bases[m] = block + ((2 + 2 (b & 1)) ^ 2 m) 16.
__device__ __forceinline__ float4 ckx_nl(const uint32_t (&bases)[4], int i) {
  const int row = i >> 1;
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(bases[(row & 7) >> 1] + (uint32_t)(row * 128 + (((i ^ row) & 1) << 4))));
  return v;
}
__device__ __forceinline__ void ckx_put(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The denominators' first part, up to 1e18, so that the product of two is finite; above that
// a bid (at most 1) does not change it, and 1e18 / it is a factor of the shares instead (0
// where it is infinite).  NaN stays.
constexpr float kCkxLarge = 1e18f;
struct CkxDen {
  float base, scale;
  __device__ __forceinline__ explicit CkxDen(float den) {
    const bool large = den > kCkxLarge;
    base = large ? kCkxLarge : den;
    scale = large ? rcp_approx(den * (1.f / kCkxLarge)) : 1.f;
  }
};

// 32 rows of one key (its logits; -infinity where a row does not see it): bids, then
// shares as bf16 pairs.  `added`: what the column tile's rows have added to the key's total so
// far, a sum of its own (a total of 1 would lose half of the bits of bids of 10^-5);
// base: the total before them, and eps.  One reciprocal serves two rows,
// 1 / (d0 d1), with d >= eps >= 1e-18.
// They go to the key's row of the warpgroup's shares: `to`, the places of its 16-byte
// pieces 0 .. 3 (of the first 32 rows of 64; of the second 64 bytes on or back).
template <int CHUNK>
__device__ __forceinline__ void ckx_bids(float (&x)[32], float c2, const uint32_t (&nl)[4]) {
  const float2 c2v = make_float2(c2, c2);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 n4 = ckx_nl(nl, 8 * CHUNK + i);
    const float2 x0 = ffma2(make_float2(x[4 * i], x[4 * i + 1]), c2v, make_float2(n4.x, n4.y));
    const float2 x1 = ffma2(make_float2(x[4 * i + 2], x[4 * i + 3]), c2v, make_float2(n4.z, n4.w));
    x[4 * i] = ex2_approx(x0.x);
    x[4 * i + 1] = ex2_approx(x0.y);
    x[4 * i + 2] = ex2_approx(x1.x);
    x[4 * i + 3] = ex2_approx(x1.y);
  }
}
template <int CHUNK, bool EARLIER>
__device__ __forceinline__ void ckx_shares(const float (&p)[32], float2 base, float &added, const uint32_t (&to)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {   // 8 rows
    float d[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (EARLIER) {
        d[c] = added;
        added += p[8 * q + c];
      } else {
        added += p[8 * q + c];
        d[c] = added;
      }
    }
    uint32_t pk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 dd = fadd2(make_float2(d[2 * i + 1], d[2 * i]), base);   // (swapped: each share takes the other's)
      const float r = rcp_approx(dd.x * dd.y);
      const float2 sh = fmul2(fmul2(make_float2(p[8 * q + 2 * i], p[8 * q + 2 * i + 1]), dd), make_float2(r, r));
      pk[i] = pack_bf16x2(sh.x, sh.y);
    }
    ckx_put(CHUNK == 0 ? to[q] : to[q] ^ 64u, pk[0], pk[1], pk[2], pk[3]);
  }
}

template <int D, bool EARLIER>
__global__ void __launch_bounds__(CkxVal<D>::kThreads, 1) __maxnreg__(CkxVal<D>::kRegsLaunch)
    ckx_values(PagedChunk p, ChunkPlan w, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
  using C = CkxVal<D>;
  constexpr int kG = C::kG;
  extern __shared__ __align__(1024) uint8_t ckx_smem_raw[];
  uint8_t *smem = ckx_smem_raw;
  if (smem_u32(ckx_smem_raw) & 1023u) {   // no room to align it: refuse rather than compute with misaligned operands
    pdl_wait();
    if (threadIdx.x == 0) atomicCAS(p.status, DA_OK, DA_ERR_UNSUPPORTED);
    return;
  }
  uint8_t *sQ = smem + C::kOffQ, *sK = smem + C::kOffK, *sV = smem + C::kOffV, *sSh = smem + C::kOffSh;
  CkxTile *ring = reinterpret_cast<CkxTile *>(smem + C::kOffRing);
  uint64_t *r_full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *r_free = r_full + kCkxRing;
  uint64_t *q_full = r_free + kCkxRing, *q_empty = q_full + C::kQs, *k_full = q_empty + C::kQs, *k_empty = k_full + C::kFull;
  uint64_t *v_full = k_empty + C::kStages, *v_empty = v_full + C::kFull, *s_full = v_empty + C::kStages;
  uint64_t *s_free = s_full + kG, *sh_full = s_free + kG, *sh_free = sh_full + kG, *d_full = sh_free + kG;
  uint64_t *d_free = d_full + 1, *turn = d_free + 1, *done = turn + 4;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + kG);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, wg = warp / 4;
  constexpr int kWarpCtl = (kG + 1) * 4;
  if (tid == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    for (int i = 0; i < kCkxRing; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_free[i], kG + 4 + 4 * kG);   // issuers, epilogue and demand warps
    }
    for (int i = 0; i < C::kQs; ++i) {
      mbar_init(&q_full[i], 2);     // the queries' bytes, and -lse2
      mbar_init(&q_empty[i], kG);   // one commit per issuer
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < C::kFull; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&turn[i], 1);
    for (int g = 0; g < kG; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&s_free[g], 4);
      mbar_init(&sh_full[g], 4);
      mbar_init(&sh_free[g], 1);
      mbar_init(&done[g], 1);
    }
    mbar_init(d_full, kG);    // one commit per issuer
    mbar_init(d_free, 4);     // phase i: D is free for column tile i
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int e = tid; e < 2048 / 4; e += C::kThreads)   // the ones beside V: bf16 1.0
    reinterpret_cast<uint32_t *>(smem + C::kOffOnes)[e] = 0x3F803F80u;
  fence_proxy_async_smem();
  if (warp == kWarpCtl) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  pdl_wait();   // nothing before touches memory
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status};

  if (wg == kG + 1) {
    ckx_regs_dec<C::kRegsCtl>();
    if (warp == kWarpCtl) {
      // -------------------------------------------------------------- producer
      // V follows K kLag tiles behind: a place for V is free a warpgroup's whole tile later
      // than one for K, and K is needed a tile earlier.  (One tile behind at d = 64: the
      // demand warps waited 2085 cycles a tile for S, 2048 queries at 131072.)
      const ChunkLine l = chunk_line(p, w);
      const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_values);
      const int sh = w.page_shift;
      CkxWalk it;
      int i = 0, nk = 0, nv = 0;
      bool ok = true;
      int v_len[C::kLag] = {}, v_tile[C::kLag] = {}, v_hkv[C::kLag] = {}, v_page[C::kLag] = {};   // V still to be brought
      int v_due = 0;
      bool part = false;   // in the column tile before, demand warps wait for V: see tile_ready
      int before = 0;      // its first key tile's number
      auto bring_v = [&]() {
        const int st = nv % C::kStages;
        if (!warp_wait(&v_empty[st], ((nv / C::kStages) & 1) ^ 1, wc)) return false;
        ckx_load<D>(p, sh, &vmap, sV + st * C::kTB, &v_full[nv % C::kFull], v_len[0], v_tile[0], v_hkv[0], v_page[0], lane);
        ++nv;
#pragma unroll
        for (int e = 1; e < C::kLag; ++e)
          v_len[e - 1] = v_len[e], v_tile[e - 1] = v_tile[e], v_hkv[e - 1] = v_hkv[e], v_page[e - 1] = v_page[e];
        --v_due;
        return true;
      };
      for (it.start(p, w, l, cut, lane); ok; ++i) {
        CkxTile x = it.tile(p, w, w.acc_a, w.acc_b, acc_stride(D));
        float4 nl = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x.rows > 0) {
          nl = it.nl(p, w, x, lane);
          x.clear = __ldcg(chunk_odd(p, w) + x.s) != 0;
        }
        ok = warp_wait(&r_free[i % kCkxRing], ((i / kCkxRing) & 1) ^ 1, wc);
        if (!ok) break;
        x.odd = __any_sync(0xffffffffu, isnan(nl.x + nl.y) || isnan(nl.z + nl.w));   // (no +infinity among them)
        if (lane == 0) {
          ring[i % kCkxRing] = x;
          mbar_arrive(&r_full[i % kCkxRing]);
        }
        if (x.rows == 0) {
          while (ok && v_due > 0) ok = bring_v();
          break;
        }
        int page = ckx_page(p, sh, x.s, x.len, x.tile, lane);
        // What follows waits for the demand warps of column tile i - 2, and those for the
        // products of what came before; of some tiles for V itself.
        while (ok && v_due > 0 && (part || nv < before)) ok = bring_v();
        if (!ok) break;
        part = x.end * kCkxEdge > (x.clear ? x.P + x.i0 : x.len);
        before = x.t0;
        const int qs = i % C::kQs;
        // every role is done with column tile i - 2, whose -lse2 this one's replace
        ok = (i < 2 || warp_wait(&r_free[(i - 2) % kCkxRing], ((i - 2) / kCkxRing) & 1, wc)) &&
             warp_wait(&q_empty[qs], ((i / C::kQs) & 1) ^ 1, wc);
        if (!ok) break;
        *reinterpret_cast<float4 *>(smem + C::kOffOnes + ckx_nl_place(lane, i)) = nl;
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[qs]);
        ckx_queries<D>(&qmap, sQ + qs * C::kTB, &q_full[qs], it.k.q.tok0, x.hq0, x.n8, x.i0, x.rows, lane);
        for (int j = x.tile; j < x.end; ++j) {
          const int ahead = j + 1 < x.end ? ckx_page(p, sh, x.s, x.len, j + 1, lane) : -1;
          const int st = nk % C::kStages;
          ok = warp_wait(&k_empty[st], ((nk / C::kStages) & 1) ^ 1, wc);
          if (!ok) break;
          ckx_load<D>(p, sh, &kmap, sK + st * C::kTB, &k_full[nk % C::kFull], x.len, j, x.hkv, page, lane);
          ++nk;
          if (v_due == C::kLag) ok = bring_v();
          if (!ok) break;
#pragma unroll
          for (int e = 0; e < C::kLag; ++e)
            if (e == v_due) v_len[e] = x.len, v_tile[e] = j, v_hkv[e] = x.hkv, v_page[e] = page;
          ++v_due;
          page = ahead;
        }
        it.next(p, w, l, x);
      }
      if (*abort_flag && lane == 0) {
        for (int t = nk > C::kStages ? nk - C::kStages : 0; t < nk; ++t)
          ckx_drain(&k_full[t % C::kFull], (t / C::kFull) & 1);
        for (int t = nv > C::kStages ? nv - C::kStages : 0; t < nv; ++t)
          ckx_drain(&v_full[t % C::kFull], (t / C::kFull) & 1);
        for (int t = i > C::kQs ? i - C::kQs : 0; t <= i; ++t) ckx_drain(&q_full[t % C::kQs], (t / C::kQs) & 1);
      }
    } else if (warp <= kWarpCtl + kG && lane == 0) {
      // -------------------------------------------------------------- MMA issuers
      // S of the warpgroup's next key tile goes before the value product of the one
      // at hand: its slot is free before the shares are written.  An issuer without
      // tiles in a column tile takes part in its barriers all the same, and after
      // those of the one before (d_free).
      const int g = warp - kWarpCtl - 1;
      const uint32_t idesc_pv = idesc_bf16(128, 80, true, true), idesc_hi = idesc_bf16(128, 64, true, true);
      const uint32_t ones = smem_u32(smem + C::kOffOnes);
      const uint64_t dQ = ckx_kmajor(sQ), dK = ckx_kmajor(sK);
      // share^T: 64-row blocks 16 KB apart, 8-key groups 1 KB apart
      const uint64_t dSh = smem_desc(smem_u32(sSh) + g * C::kShBytes, 16384, 1024);
      // Second terms lie where the first of rows 64 .. would; behind them the next warpgroup's
      // shares, or K: what that makes of rows 64 .. no one reads.
      static_assert(C::kOffK == C::kOffSh + kG * C::kShBytes && C::kStages * C::kTB >= 16384, "64 rows behind the last shares");
      int m = 0, mv = 0;          // tiles of this warpgroup: S issued, value products issued
      int vt = 0, vi = 0;         // the tile whose value product is due, its column tile
      int due = 0;                // 0, or of the following (each in a register: 4 % of 16 prompts of d = 128)
      constexpr int kDue = 1, kBegins = 2, kEnds = 4, kTwo = 8;
      bool ok = true;
      // D += share^T [V | 1], in the tiles' order (sums in another order would have other
      // last bits).  Once V of tile t is there, the product of t - kStages has been formed,
      // so that four barriers tell whose turn it is.
      auto values = [&]() {
        if (due == 0) return true;
        const int st = vt % C::kStages;
        if (!mbar_wait(d_free, vi & 1, wc) || !mbar_wait(&v_full[vt % C::kFull], (vt / C::kFull) & 1, wc) ||
            !mbar_wait(&sh_full[g], mv & 1, wc) ||
            (vt > 0 && !mbar_wait(&turn[(vt - 1) & 3], ((vt - 1) >> 2) & 1, wc)))
          return false;
        ++mv;
        tc_fence_after();
        const uint32_t v = smem_u32(sV) + st * C::kTB;
        uint32_t onto = due & kBegins ? 0u : 1u;
        const uint64_t last = dSh + (due & kTwo ? 16384 >> 4 : 0);
        for (uint64_t sh = dSh; sh <= last; sh += 16384 >> 4, onto = 1u) {
          MmaRun<0, 8, 128, 128 - (128ll << 16), false>::go(tmem + C::kTmemD, sh, smem_desc(v, ones - v, 1024), idesc_pv, onto);
          if constexpr (D == 128)
            MmaRun<0, 8, 128, 128, false>::go(tmem + C::kTmemDHi, sh, smem_desc(v + kCkxHalf, kCkxHalf, 1024), idesc_hi, onto);
        }
        mma_commit(&sh_free[g]);
        mma_commit(&v_empty[st]);
        if (due & kEnds) mma_commit(d_full);
        due = 0;
        tc_fence_before();
        mbar_arrive(&turn[vt & 3]);
        return true;
      };
      // Before the first S of column tile i, with a value product due: whichever can go
      // first.  The keys that S needs may come only after values whose place that very
      // product frees (5 tiles, then 3: the producer waits with V(5) for the product of
      // tile 2, before it brings K(7)).
      auto first_of = [&](int i, uint64_t *k_bar, uint32_t k_parity) {
        const unsigned long long began = globaltimer();
        while (!(mbar_test_wait(&q_full[i % C::kQs], (i / C::kQs) & 1) && mbar_test_wait(k_bar, k_parity) &&
                 mbar_test_wait(&s_free[g], (m & 1) ^ 1))) {
          if (mbar_test_wait(d_free, vi & 1) && mbar_test_wait(&v_full[vt % C::kFull], (vt / C::kFull) & 1) &&
              mbar_test_wait(&sh_full[g], mv & 1) && (vt == 0 || mbar_test_wait(&turn[(vt - 1) & 3], ((vt - 1) >> 2) & 1)))
            return values();
          if (*abort_flag) return false;
          if (globaltimer() - began > wc.limit_ns) {
            raise_timeout(wc, k_bar);
            return false;
          }
          __nanosleep(40);
        }
        return true;
      };
      for (int i = 0; ok; ++i) {
        ok = mbar_wait(&r_full[i % kCkxRing], (i / kCkxRing) & 1, wc);
        if (!ok) break;
        const CkxTile &x = ring[i % kCkxRing];
        const int rows = x.rows, tiles = x.end - x.tile, t0 = x.t0;
        const bool terms = x.two_terms();
        mbar_arrive(&r_free[i % kCkxRing]);
        if (rows == 0) break;
        const uint32_t idesc_s = idesc_bf16(128, (rows + 15) & ~15, false, false);
        for (int j = g; ok && j < tiles; j += kG, ++m) {
          const int t = t0 + j, st = t % C::kStages;
          if (j == g && due != 0) ok = first_of(i, &k_full[t % C::kFull], (t / C::kFull) & 1);
          ok = ok && mbar_wait(&q_full[i % C::kQs], (i / C::kQs) & 1, wc) && mbar_wait(&k_full[t % C::kFull], (t / C::kFull) & 1, wc) &&
               mbar_wait(&s_free[g], (m & 1) ^ 1, wc);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dKs = dK + (uint64_t)st * (C::kTB >> 4), dQs = dQ + (uint64_t)(i % C::kQs) * (C::kTB >> 4);
          MmaRun<0, 4, 2, 2, false>::go(tmem + g * 128, dKs, dQs, idesc_s, 0u);
          if constexpr (D == 128)
            MmaRun<0, 4, 2, 2, false>::go(tmem + g * 128, dKs + (kCkxHalf >> 4), dQs + (kCkxHalf >> 4), idesc_s, 1u);
          mma_commit(&s_full[g]);
          mma_commit(&k_empty[st]);
          if (j + kG >= tiles) mma_commit(&q_empty[i % C::kQs]);   // its last S of the column tile
          ok = values();
          vt = t;
          vi = i;
          due = kDue | (j == 0 ? kBegins : 0) | (j + kG >= tiles ? kEnds : 0) | (terms ? kTwo : 0);
        }
        if (!ok) break;
        if (g >= tiles) {
          ok = mbar_wait(&q_full[i % C::kQs], (i / C::kQs) & 1, wc);
          if (!ok) break;
          mma_commit(&q_empty[i % C::kQs]);
          ok = values() && mbar_wait(d_free, i & 1, wc);
          if (ok) mma_commit(d_full);
        }
      }
      if (ok) values();
      mma_commit(&done[g]);
      ckx_drain(&done[g], 0);
    }
  } else if (wg == kG) {
    // ---------------------------------------------------------------- epilogue
    ckx_regs_dec<C::kRegsEpi>();
    const int quarter = warp % 4, c = quarter * 32 + lane;
    const uint32_t td = tmem + C::kTmemD + ((uint32_t)(quarter * 32) << 16);
    ckx_release(d_free, lane);
    for (int i = 0;; ++i) {
      if (!warp_wait(&r_full[i % kCkxRing], (i / kCkxRing) & 1, wc)) break;
      const CkxTile &x = ring[i % kCkxRing];
      const int rows = x.rows;
      float *to = x.place + chunk_acc(D, c, 0), *to_sum = x.place + chunk_acc_sum(D, c);
      __syncwarp();
      if (lane == 0) mbar_arrive(&r_free[i % kCkxRing]);
      if (rows == 0) break;
      if (!warp_wait(d_full, i & 1, wc)) break;
      tc_fence_after();
      float sums[8];   // alike
      tmem_ld8(td + 64, sums);
      tmem_wait_ld_r8(sums);
#pragma unroll
      for (int e = 0; e < D; e += C::kDrain) {
        float a[C::kDrain / 8][8];
        const uint32_t at = td + (e < 64 ? e : C::kTmemDHi - C::kTmemD + e - 64);
#pragma unroll
        for (int k = 0; k < C::kDrain / 8; ++k) tmem_ld8(at + 8 * k, a[k]);
#pragma unroll
        for (int k = 0; k < C::kDrain / 8; ++k) tmem_wait_ld_r8(a[k]);
        if (e + C::kDrain == D) ckx_release(d_free, lane);   // read: the next column tile's products while these are written
        if (c < rows) {
          float4 *o = reinterpret_cast<float4 *>(to + 8 * e);
#pragma unroll
          for (int k = 0; k < C::kDrain / 8; ++k) {
            o[16 * k] = make_float4(a[k][0], a[k][1], a[k][2], a[k][3]);
            o[16 * k + 8] = make_float4(a[k][4], a[k][5], a[k][6], a[k][7]);
          }
        }
        __syncwarp();
      }
      if (c < rows) *to_sum = sums[0];
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- demand
    ckx_regs_inc<C::kRegsDemand>();
    const int g = wg, quarter = warp % 4, key_l = quarter * 32 + lane, swz = key_l & 7;   // key of the tile
    const uint32_t ts = tmem + g * 128 + ((uint32_t)(quarter * 32) << 16);
    // this key's row of the warpgroup's shares: 64-row blocks 16 KB apart, pieces swizzled by the key
    const uint32_t sh_row = smem_u32(sSh) + g * C::kShBytes + (key_l / 8) * 1024 + (key_l % 8) * 128;
    const int sh = w.page_shift, ps = 1 << sh;
    const size_t page_totals = (size_t)p.c.Hq << sh;
    int m = 0;   // the warpgroup's tiles so far
    for (int i = 0;; ++i) {
      if (!warp_wait(&r_full[i % kCkxRing], (i / kCkxRing) & 1, wc)) break;
      const CkxTile &x = ring[i % kCkxRing];
      const int rows = x.rows, end = x.end, len = x.len;
      if (rows == 0) break;
      const int whole = x.clear ? x.P + x.i0 : len;   // keys whose values need no care: see tile_ready
      bool ok = true;
      const uint32_t ones = smem_u32(smem + C::kOffOnes);
      // the page of this thread's key in tile j, for the totals (-1: none), and its place
      const int32_t *const table = p.c.demand_table + (size_t)x.s * p.c.max_pages;
      float *const pool = p.c.demand_pages + ((size_t)x.hq0 << sh);   // of query head hq0
      auto page_of = [&](int j) {
        const int key = j * kCkxEdge + key_l;
        return key < len ? __ldcg(table + (key >> sh)) : -1;
      };
      auto total_at = [&](int page, int j) -> float * {
        const int key = j * kCkxEdge + key_l;
        if ((unsigned)page < (unsigned)p.c.num_demand_pages) return pool + page * page_totals + (key & (ps - 1));
        if (key < len) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
        return nullptr;
      };
      // The tile's S, and in a sequence's last tile zeros in the rows of V past its end,
      // which may hold anything: 0 times that is not 0.  Of keys that not every row sees too
      // (where a flag says so), or that two terms of a share would make inf - inf of.
      auto tile_ready = [&](int j) {
        if (!warp_wait(&s_full[g], m & 1, wc)) return false;
        tc_fence_after();
        if ((j + 1) * kCkxEdge > whole) {
          const int t = x.t0 + (j - x.tile), st = t % C::kStages;
          if (!warp_wait(&v_full[t % C::kFull], (t / C::kFull) & 1, wc)) return false;
          const int key = j * kCkxEdge + key_l;
          uint8_t *row = sV + st * C::kTB + key_l * 128;
          if (key >= whole) {
#pragma unroll 1
            for (int e = 0; e < D / 8; ++e) {
              uint4 *v = reinterpret_cast<uint4 *>(row + (e >> 3) * kCkxHalf + ((e & 7) << 4));
              uint4 y = *v;
              chunk_clear(y, true);
              *v = key < len ? y : make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        return true;
      };
      int j = x.tile + g;
      float *at = j < end ? total_at(page_of(j), j) : nullptr;
      float total = at != nullptr ? __ldcg(at) : 0.f;
      if (x.n8 == 0 && !x.odd) {
        // one head
        const int first = x.P + x.i0;   // place of row 0
        const float c2 = x.c2;
        for (; j < end; j += kG, ++m) {
          const float den = total + p.eps;
          if (__any_sync(0xffffffffu, den > kCkxLarge)) break;
          const int next_page = j + kG < end ? page_of(j + kG) : -1;
          float *next_at = nullptr;
          float next_total = 0.f;
          ok = tile_ready(j);
          if (!ok) break;
          if (j + kG < end) {
            next_at = total_at(next_page, j + kG);
            if (next_at != nullptr) next_total = __ldcg(next_at);
          }
          const bool mask = (j + 1) * kCkxEdge - 1 > first || rows < kCkxEdge;
          const float2 base = make_float2(den, den);
          float added = 0.f;
          uint32_t nl[4], to[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) nl[e] = ones + (((2 + 2 * (i & 1)) ^ (2 * e)) << 4), to[e] = sh_row + ((e ^ swz) << 4);
          // 64 rows at a time; not unrolled: the code of all 128 misses the instruction cache
          const int halves = rows > 64 ? 2 : 1;
#pragma unroll 1
          for (int half = 0; half < halves; ++half) {
            float a[32], b[32];
            tmem_ld32(ts + 64 * half, a);
            tmem_ld32(ts + 64 * half + 32, b);
            tmem_wait_ld_r(a);
            tmem_wait_ld_r(b);
            if (half + 1 == halves) ckx_release(&s_free[g], lane);   // the next tile's S while these rows are formed
            if (mask) {   // rows lo .. rows - 1 see the key
              const int key = j * kCkxEdge + key_l;
              const int lo = (key < len ? min(max(key - first, 0), rows) : rows) - 64 * half, n = rows - 64 * half - lo;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if ((unsigned)(e - lo) >= (unsigned)n) a[e] = -INFINITY;
                if ((unsigned)(32 + e - lo) >= (unsigned)n) b[e] = -INFINITY;
              }
            }
            ckx_bids<0>(a, c2, nl);
            if (half == 0) {   // the product of the tile before has read the shares
              ok = warp_wait(&sh_free[g], (m & 1) ^ 1, wc);
              if (!ok) break;
            }
            ckx_shares<0, EARLIER>(a, base, added, to);
            ckx_bids<1>(b, c2, nl);
            ckx_shares<1, EARLIER>(b, base, added, to);
#pragma unroll
            for (int e = 0; e < 4; ++e) nl[e] += 1024, to[e] += 16384;
          }
          if (!ok) break;
          if (at != nullptr) __stcg(at, total + added);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh_full[g]);
          at = next_at;
          total = next_total;
        }
      }
      if (ok && j < end) {
        // several heads of n8 rows: 8 rows at a time, a head's total from its first rows to its last.
        // (Or one head's, where a row's sum or a key's total needs the care that this loop takes: in
        // the other a least value for every pair's denominators costs 4 %, bids set to zero after
        // they are formed as much, and their scale 4 % too.)
        const int groups = (rows + 7) / 8, n8 = x.n8 ? x.n8 : 8 * groups, per = n8 / 8, n = x.n8 ? x.n : rows, P = x.P + x.i0,
                  head0 = x.s * p.c.Hq + x.hq0;
        const bool two = x.two_terms(), fold = x.folded();
        for (; j < end; j += kG, ++m) {
          const int next_page = j + kG < end ? page_of(j + kG) : -1;
          float *next_at = nullptr;
          float next_total = 0.f;
          ok = tile_ready(j);
          if (!ok) break;
          if (j + kG < end) {
            next_at = total_at(next_page, j + kG);
            if (next_at != nullptr) next_total = __ldcg(next_at);
          }
          const int key = j * kCkxEdge + key_l;
          const int lo = key < len ? min(max(key - P, 0), n) : n;   // queries lo .. n - 1 see the key
          float *head_at = at;
          float head_next = 0.f, added = 0.f, c2 = 0.f;
          int q = 0;   // query of the group's first row
          CkxDen den(total + p.eps);
          float v[8];
          tmem_ld8(ts, v);
          for (int u = 0, h = 0; u < groups; ++u) {
            if (q == 0) {
              c2 = fmaxf(head_c2(p.hs, head0 + h, nullptr), 1e-30f);
              if (u + per < groups && head_at != nullptr) head_next = __ldcg(head_at + ps);
            }
            float nlv[8];
            *reinterpret_cast<float4 *>(nlv) = *reinterpret_cast<const float4 *>(smem + C::kOffOnes + ckx_nl_place(2 * u, i));
            *reinterpret_cast<float4 *>(nlv + 4) =
                *reinterpret_cast<const float4 *>(smem + C::kOffOnes + ckx_nl_place(2 * u + 1, i));
            tmem_wait_ld_r8(v);
            float bid[8], d[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 y = ffma2(make_float2(v[e], v[e + 1]), make_float2(c2, c2), make_float2(nlv[e], nlv[e + 1]));
              bid[e] = (unsigned)(q + e - lo) < (unsigned)(n - lo) ? ex2_approx(y.x) : 0.f;
              bid[e + 1] = (unsigned)(q + e + 1 - lo) < (unsigned)(n - lo) ? ex2_approx(y.y) : 0.f;
            }
            if (u + 1 < groups)
              tmem_ld8(ts + 8 * (u + 1), v);
            else
              ckx_release(&s_free[g], lane);
            uint32_t pk[4], pk2[4];
            const float2 b2 = make_float2(den.base, den.base);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              d[e] = added;
              added += bid[e];
              if (!EARLIER) d[e] = added;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 dd = fadd2(make_float2(d[2 * e + 1], d[2 * e]), b2);
              if (!EARLIER) dd.x = fminf(dd.x, 2e18f);   // a NaN of the later row alone (else: both are below)
              const float r = rcp_approx(dd.x * dd.y);
              const float2 one = fmul2(fmul2(make_float2(bid[2 * e], bid[2 * e + 1]), dd), make_float2(r, r));
              const float2 s2 = fmul2(one, make_float2(den.scale, den.scale));   // (after r: both in one would underflow)
              pk[e] = pack_bf16x2(s2.x, s2.y);
              pk2[e] = pack_bf16x2(s2.x - __uint_as_float(pk[e] << 16), s2.y - __uint_as_float(pk[e] & 0xffff0000u));
            }
            if (fold) pk[2] = pk2[0], pk[3] = pk2[1];
            if (u == 0) {   // the product of the tile before has read the shares
              ok = warp_wait(&sh_free[g], (m & 1) ^ 1, wc);
              if (!ok) break;
            }
            ckx_put(sh_row + (u >> 3) * 16384 + (((u & 7) ^ swz) << 4), pk[0], pk[1], pk[2], pk[3]);
            if (two) ckx_put(sh_row + 16384 + ((u ^ swz) << 4), pk2[0], pk2[1], pk2[2], pk2[3]);
            q += 8;
            if (q == n8) {   // the head's last rows
              q = 0;
              ++h;
              if (head_at != nullptr) {
                __stcg(head_at, total + added);
                head_at += ps;
              }
              total = head_next;
              den = CkxDen(total + p.eps);
              added = 0.f;
            }
          }
          if (!ok) break;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh_full[g]);
          at = next_at;
          total = next_total;
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&r_free[i % kCkxRing]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpCtl) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================================ host
cudaError_t launch_chunk_plan(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);   // paged_chunk.cu
cudaError_t launch_chunk_join(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);
cudaError_t launch_chunk_combine(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);

// A register split larger than what the block is launched with would never
// resolve: refuse unless the compiled register count covers it.
template <int D, bool EARLIER>
static int ckx_prepare_values() {
  using C = CkxVal<D>;
  if (cudaFuncSetAttribute(ckx_values<D, EARLIER>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
    return DA_ERR_CUDA;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, ckx_values<D, EARLIER>) != cudaSuccess) return DA_ERR_CUDA;
  return fa.numRegs * C::kThreads < C::kRegsNeeded || fa.numRegs > C::kRegsDemand || fa.numRegs < C::kRegsEpi
             ? DA_ERR_UNSUPPORTED
             : DA_OK;
}

template <int D>
static int launch_ckx(const PagedChunk &p, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int prep = once.run([] {
    if (cudaFuncSetAttribute(ckx_keys<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, CkxKeys<D>::kSmemBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(ckx_keys<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, CkxKeys<D>::kSmemBytes) !=
            cudaSuccess)
      return DA_ERR_CUDA;
    const int st = ckx_prepare_values<D, false>();
    return st != DA_OK ? st : ckx_prepare_values<D, true>();
  });
  if (prep != DA_OK) return prep;
  const ChunkPlan w = chunk_plan_bf16(p.c.S, p.c.Hq, p.c.Hkv, D, p.N, p.max_new, p.max_len, p.c.page_size);
  const int64_t num = (int64_t)p.c.num_pages * p.c.Hkv;
  CUtensorMap qm, km, vm;
  // (an empty pool has no pages to map: every page id then fails its check)
  if (!make_rows_map(&qm, p.q, p.N, p.c.Hq, D, 8) ||
      !make_page_map(&km, p.c.k_pages, num > 0 ? num : 1, p.c.page_size, kCkxEdge, D, DA_BF16) ||
      !make_page_map(&vm, p.c.v_pages, num > 0 ? num : 1, p.c.page_size, kCkxEdge, D, DA_BF16))
    return DA_ERR_CUDA;
  using V = CkxVal<D>;
  const bool few = w.logits_ld > 0;
  if (launch_chunk_plan(p, w, stream) != cudaSuccess ||
      launch_after(few ? ckx_keys<D, true> : ckx_keys<D, false>, w.ctas_keys, CkxKeys<D>::kThreads, CkxKeys<D>::kSmemBytes, stream,
                   p, w, qm, km) != cudaSuccess ||
      launch_chunk_join(p, w, stream) != cudaSuccess ||
      (few         ? launch_chunk_few(p, w, stream)
       : p.earlier ? launch_after(ckx_values<D, true>, w.ctas_values, V::kThreads, V::kSmemBytes, stream, p, w, qm, km, vm)
                   : launch_after(ckx_values<D, false>, w.ctas_values, V::kThreads, V::kSmemBytes, stream, p, w, qm, km, vm)) !=
          cudaSuccess ||
      launch_chunk_combine(p, w, stream) != cudaSuccess)
    return DA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int launch_chunk_bf16(const PagedChunk &p, cudaStream_t stream) {
  return p.c.d == 128 ? launch_ckx<128>(p, stream) : launch_ckx<64>(p, stream);
}

}  // namespace da
