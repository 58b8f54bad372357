// Decode step over a shared prefix with many query rows: tcgen05 kernels.
//
// Mathematics: as paged_decode_bf16.cu, for the part of every sequence that lies in
// the shared prefix.  A segment is 64 rows (sequence, query head) of one key
// head; the prefix's keys and values are read once per pass for all of them.
//   pgx_keys    (max, sum 2^(x - max)) of every row over the CTA's key tiles;
//   pgx_values  p = 2^(x - lse2), share = p / (D + p + eps), D += p, and the
//               sums of share v and share over the CTA's key tiles.
//
// What bounds it: HBM, by the demand: 8 bytes for every (row, key) against the
// 4 d bytes a key costs for all rows.  The logits are therefore not kept
// between the passes (another 8 bytes each) but formed twice, which the tensor
// cores do for less than the demand takes to arrive; K is read twice.
//
// pgx_keys: S[row, key] = Q K^T with M = 128, N = 128.  The 64 rows stand twice
// in the M dimension; TMEM lanes 0-63 reduce keys 0-63 of a tile and lanes
// 64-127 keys 64-127, so that all threads work.  One thread per lane keeps a
// running maximum and sum; two warpgroups take alternate tiles.
//
// pgx_values: S^T[key, row] = K Q^T (M = 128 keys, N = 64 rows), one thread per
// key.  The demand of a tile lies in shared memory, [row][key]; every warp
// brings that of its own 32 keys by 16-byte asynchronous copies, 8 rows at a
// time, two groups ahead, into the place of rows it has just written back (32 KB
// an SM; 64 KB left the values one stage at d = 128, which then came too late:
// 95 us for 32 x 16 heads x 32768).  The shares go to shared memory as the MN-major A
// operand of D[row, :] += share^T [V | 1]: rows 0-63 of M = 128 hold the shares
// rounded to bf16, rows 64-127 what the rounding left (2^-16 relative in all;
// the second term costs no instruction).  Two pairs of warpgroups take alternate
// tiles, the warpgroups of a pair 32 rows each: four warps a scheduler hide the
// latency of each other's exponentials and shared-memory reads.
// (With the demand in registers, 4-byte loads and stores and fully unrolled
// rows, a (row, key) pair took 30 instructions, the instruction cache missed, and
// 64 rows x 12 heads x 131072 keys took 269 us; with one warpgroup a tile 237 us.)
//
// Roles: warps 0-15 demand, then a warp each for K copies, V copies, MMA issue
// and the demand-page table of the next tiles.  Waits are bounded; rows of
// missing or invalid pages are filled with zeros by reading past the pool's end;
// a key past the prefix's end has the logit -infinity, and so no bid and no share.
#include "da_paged_plan.cuh"

#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

namespace da {

bool make_page_map(CUtensorMap *m, const void *base, int64_t num, int page_size, int rows, int d,
                   int dtype);   // fwd_bf16.cu

constexpr uint32_t kXHalf = 128 * 128;        // 128 rows x 64 bf16
constexpr uint32_t kXQHalf = kPgxRows * 128;  // 64 rows x 64 bf16
constexpr uint32_t kNoDemand = 0xFFFFFFFFu;
constexpr int kTabPitch = 72, kTabWords = 8 * kTabPitch;   // a demand-page table (no bank conflicts between entries)

__device__ __forceinline__ uint64_t x_kmajor(const uint8_t *tile) { return smem_desc(smem_u32(tile), 16, 1024); }

__device__ __forceinline__ void x_drain(uint64_t *bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > 100ull * 1000ull * 1000ull) break;
}
__device__ __forceinline__ void x_release(uint64_t *bar, int lane) {   // after the last tcgen05.ld of a buffer
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Pieces of a CTA's stretch of the segments' units.
struct XPiece {
  int hkv, row0, nrows;   // rows of the batch
  int seg, tile, n;       // segment, first key tile, tiles
  int run;                // tiles of the pieces before
  // pgx_values deals a piece's rows out to both halves of its 64 places, so that
  // the warps of both have as many (80 rows as 64 + 16, filled from the first place
  // on, took 93.5 us a step of 40 x 8 heads x 52736, as 40 + 40 dealt out 89.5).
  // The row in a place; nrows or above: none.
  __device__ __forceinline__ int half() const { return (nrows + 15) / 16 * 8; }   // rows of the first half
  __device__ __forceinline__ int row_at(int place) const {
    return place >= 32 ? half() + place - 32 : place < half() ? place : kPgxRows;
  }
};
struct XWalk {
  XPiece c;
  int at, to;
  __device__ __forceinline__ void set(const PagedDecode &p, const PgtPlan &w) {
    c.n = 0;
    if (at >= to) return;
    const int units = w.x_tiles + kPgxHead;   // a segment: its head, then its tiles
    c.seg = at / units;
    c.tile = max(at - c.seg * units - kPgxHead, 0);
    at = c.seg * units + kPgxHead + c.tile;   // the piece's first tile
    c.n = max(min(w.x_tiles - c.tile, to - at), 0);
    c.hkv = c.seg / w.x_groups;
    c.row0 = c.seg % w.x_groups * w.x_rows;
    c.nrows = min(w.x_rows, p.c.S * w.G - c.row0);
  }
  __device__ __forceinline__ void start(const PagedDecode &p, const PgtPlan &w, const PgtCut &cut) {
    at = cut.first(blockIdx.x);
    to = cut.first(blockIdx.x + 1);
    c.run = 0;
    set(p, w);
  }
  __device__ __forceinline__ void next(const PagedDecode &p, const PgtPlan &w) {
    at += c.n;
    c.run += c.n;
    set(p, w);
  }
};

// One warp: key tile `tile` of the prefix for key head hkv into `dst`.  Pages
// past the prefix's end, or not in the pool, are read past the pool's end:
// zeros.  `page` is this lane's page of the tile (x_page), fetched beforehand.
__device__ __forceinline__ int x_page(const PagedDecode &p, const PgtPlan &w, int tile, int lane) {
  const int rows = min(1 << w.page_shift, kPgxTile);
  const int key = tile * kPgxTile + lane * rows;
  return lane * rows < kPgxTile && key < p.prefix_len ? __ldcg(p.prefix_table + (key >> w.page_shift)) : -1;
}
template <int D>
__device__ __forceinline__ void x_load(const PagedDecode &p, const PgtPlan &w, const CUtensorMap *map, uint8_t *dst,
                                       uint64_t *bar, int tile, int hkv, int page, int lane) {
  const int ps = 1 << w.page_shift, rows = min(ps, kPgxTile);
  const int key = tile * kPgxTile + lane * rows;
  if (lane == 0) mbar_arrive_expect_tx(bar, kPgxTile * D * 2);
  __syncwarp();
  if (lane * rows < kPgxTile) {
    const bool ok = (unsigned)page < (unsigned)p.c.num_pages;
    if (!ok && key < p.prefix_len) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    const int z = ok ? page * p.c.Hkv + hkv : max(p.c.num_pages * p.c.Hkv, 1);   // past the map's end: zeros
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      tma_load_3d(dst + h * kXHalf + lane * rows * 128, map, bar, h * 64, key & (ps - 1), z);
  }
}

// Query row r of a piece, as 16-byte piece i (zeros past the piece's rows).
template <int D>
__device__ __forceinline__ uint4 x_query(const PagedDecode &p, const PgtPlan &w, const XPiece &c, int r, int i) {
  if (r >= c.nrows) return make_uint4(0u, 0u, 0u, 0u);
  const int R = c.row0 + r, s = R / w.G, hq = c.hkv * w.G + R % w.G;
  return __ldcg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)s * p.c.Hq + hq) * D) + i);
}

// ============================================================================ pass 1
template <int D>
struct XKeys {
  static constexpr int kThreads = 320;                 // 2 x 4 reduction warps (alternate tiles), copies, MMA
  static constexpr int kTB = kPgxTile * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kSmemBytes = 1024 + kTB + kStages * kTB + 256;
  static constexpr int kTmemCols = 256;                // two S buffers of 128 columns; two CTAs an SM
};

template <int D>
__global__ void __launch_bounds__(XKeys<D>::kThreads, 2)
    pgx_keys(PagedDecode p, PgtPlan w, const __grid_constant__ CUtensorMap kmap) {
  using C = XKeys<D>;
  extern __shared__ __align__(1024) uint8_t x_smem_raw[];
  uint8_t *smem = x_smem_raw + ((1024u - (smem_u32(x_smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem, *sK = smem + C::kTB;
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::kTB + C::kStages * C::kTB);
  uint64_t *k_full = q_full + 1, *k_empty = k_full + C::kStages, *s_full = k_empty + C::kStages, *s_free = s_full + 2;
  uint64_t *done = s_free + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  __shared__ float2 s_ml[3][kPgxRows];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
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
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status, p.dbg.limit_ns[kPagedPrefixKeys]};
  XWalk it;
  it.start(p, w, w.x_keys);
  if (warp == 8) {
    int issued = 0;
    for (; it.c.n > 0; it.next(p, w)) {
      int page = x_page(p, w, it.c.tile, lane);
      bool ok = true;
      for (int k = 0; k < it.c.n; ++k, ++issued) {
        const int ahead = k + 1 < it.c.n ? x_page(p, w, it.c.tile + k + 1, lane) : -1;
        const int s = issued % C::kStages;
        ok = warp_wait(&k_empty[s], ((issued / C::kStages) & 1) ^ 1, wc);
        if (!ok) break;
        x_load<D>(p, w, &kmap, sK + s * C::kTB, &k_full[s], it.c.tile + k, it.c.hkv, page, lane);
        page = ahead;
      }
      if (!ok) break;
    }
    if (*abort_flag && lane == 0)
      for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
        x_drain(&k_full[i % C::kStages], (i / C::kStages) & 1);
  } else if (warp == 9) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, kPgxTile, false, false);
      const uint64_t dQ = x_kmajor(sQ), dK = x_kmajor(sK);
      int t = 0, piece = 0;
      bool ok = true;
      for (; ok && it.c.n > 0; it.next(p, w), ++piece) {
        ok = mbar_wait(q_full, piece & 1, wc);
        for (int k = 0; ok && k < it.c.n; ++k, ++t) {
          const int s = t % C::kStages, b = t & 1;
          ok = mbar_wait(&k_full[s], (t / C::kStages) & 1, wc) && mbar_wait(&s_free[b], ((t >> 1) & 1) ^ 1, wc);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dKs = dK + (uint64_t)s * (C::kTB >> 4);
          MmaRun<0, 4, 2, 2, false>::go(tmem + b * 128, dQ, dKs, idesc, 0u);
          if constexpr (D == 128)
            MmaRun<0, 4, 2, 2, false>::go(tmem + b * 128, dQ + (kXHalf >> 4), dKs + (kXHalf >> 4), idesc, 1u);
          mma_commit(&s_full[b]);
          if (t > 0 || (int)blockIdx.x != p.dbg.stall_block[kPagedPrefixKeys])   // (test hook: one stage is kept)
            mma_commit(&k_empty[s]);
        }
      }
      mma_commit(done);
      x_drain(done, 0);
    }
  } else {
    const int g = warp / 4, row = tid % 128, r = row % kPgxRows, half = row / kPgxRows;   // TMEM lane; query row; keys 64 half ..
    for (; it.c.n > 0; it.next(p, w)) {
      // the rows, twice, as the K-major A operand (every product of the piece
      // before has completed: the warpgroups saw their last tiles and met)
      for (int e = tid; e < 128 * (D / 8); e += 256) {
        const int rr = e / (D / 8), i = e % (D / 8);
        *reinterpret_cast<uint4 *>(sQ + (i >> 3) * kXHalf + rr * 128 + (((i & 7) ^ (rr & 7)) << 4)) =
            x_query<D>(p, w, it.c, rr % kPgxRows, i);
      }
      fence_proxy_async_smem();
      named_bar_sync(1, 256);
      if (tid == 0) mbar_arrive(q_full);
      float c2 = 1e-30f;
      if (r < it.c.nrows) {
        const int R = it.c.row0 + r, s = R / w.G;
        c2 = fmaxf(head_c2(p.hs, s * p.c.Hq + it.c.hkv * w.G + R % w.G, tid < 64 ? p.status : nullptr), 1e-30f);
      }
      const bool work = (row & 32) < it.c.nrows;   // uniform over the warp: its 32 rows hold at least one
      float m = -INFINITY;
      float2 l0 = make_float2(0.f, 0.f), l1 = make_float2(0.f, 0.f);
      auto take = [&](float (&x)[32], int left) {   // 32 keys, of which `left` come before the prefix's end
        if (left < 32) {
          if (left <= 0) return;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= left) x[e] = -INFINITY;
        }
        float a[11];
#pragma unroll
        for (int e = 0; e < 10; ++e) a[e] = fmax3(x[3 * e], x[3 * e + 1], x[3 * e + 2]);
        a[10] = fmaxf(x[30], x[31]);
        const float top =
            fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmax3(a[6], a[7], fmax3(a[8], a[9], a[10])));
        if (top == -INFINITY) return;
        const float mn = fmaxf(m, top * c2);
        const float f = ex2_approx(m - mn);
        m = mn;
        l0 = fmul2(l0, make_float2(f, f));
        l1 = fmul2(l1, make_float2(f, f));
        const float2 c2v = make_float2(c2, c2), nm = make_float2(-mn, -mn);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 x0 = ffma2(make_float2(x[2 * e], x[2 * e + 1]), c2v, nm);
          const float2 x1 = ffma2(make_float2(x[2 * e + 2], x[2 * e + 3]), c2v, nm);
          l0 = fadd2(l0, make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
          l1 = fadd2(l1, make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
        }
      };
      const int tiles = __any_sync(0xffffffffu, *abort_flag != 0) ? 0 : it.c.n;
      for (int k = g ^ (it.c.run & 1); k < tiles; k += 2) {   // the warpgroup's tiles: alternate over the whole run
        const int t = it.c.run + k, b = g;
        if (!warp_wait(&s_full[b], (t >> 1) & 1, wc)) break;
        tc_fence_after();
        if (work) {
          const uint32_t ta = tmem + b * 128 + half * 64 + ((uint32_t)(warp % 4 * 32) << 16);
          const int left = p.prefix_len - (it.c.tile + k) * kPgxTile - half * 64;
          float x[32];
          tmem_ld32(ta, x);
          tmem_wait_ld_r(x);
          take(x, left);
          tmem_ld32(ta + 32, x);
          tmem_wait_ld_r(x);
          x_release(&s_free[b], lane);
          take(x, left - 32);
        } else {
          x_release(&s_free[b], lane);
        }
      }
      // a row's four parts: two halves of the keys, two warpgroups
      const float l = (l0.x + l0.y) + (l1.x + l1.y);
      const int part = 2 * g + half;
      if (part > 0) s_ml[part - 1][r] = make_float2(m, l);
      named_bar_sync(1, 256);
      if (part == 0 && r < it.c.nrows) {
        float M = m;
#pragma unroll
        for (int i = 0; i < 3; ++i) M = fmaxf(M, s_ml[i][r].x);
        const float ms = M == -INFINITY ? 0.f : M;
        float sum = l * ex2_approx(m - ms);
#pragma unroll
        for (int i = 0; i < 3; ++i) sum += s_ml[i][r].y * ex2_approx(s_ml[i][r].x - ms);
        reinterpret_cast<float2 *>(p.ws + w.pre_ml_off)[(size_t)(blockIdx.x + it.c.seg) * w.pre_rows + r] =
            make_float2(M, sum);
      }
      named_bar_sync(1, 256);
    }
    if (tid == 0) pdl_wait();   // this kernel ends after its predecessor: whoever waits for it waits for both
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
template <int D>
struct XVal {
  static constexpr int kDemandWarps = 16;              // warpgroup x: tiles of parity x & 1, rows 32 (x >> 1) ..
  static constexpr int kThreads = 640;                 // and a warp each for K, V, MMA and the table
  static constexpr int kTB = kPgxTile * D * 2;
  static constexpr int kKStages = D == 64 ? 3 : 1;     // K: each stage is free as soon as its S is formed
  static constexpr int kVStages = D == 64 ? 3 : 2;
  static constexpr uint32_t kShBytes = 32 * 1024;      // a warpgroup's shares: 2 x 64 rows x 128 keys
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kPgxRows * D * 2;
  static constexpr uint32_t kOffV = kOffK + kKStages * kTB;
  static constexpr uint32_t kOffSh = kOffV + kVStages * kTB;
  static constexpr uint32_t kOffOnes = kOffSh + 2 * kShBytes;   // above every V tile (positive offset)
  static constexpr uint32_t kOffDem = kOffOnes + 2048;          // demand: 16 warps x 2 x [8 rows][32 keys]
  static constexpr uint32_t kOffTab = kOffDem + 16 * 2048;      // 4 tables [up to 8 pages][64 rows, padded]
  static constexpr uint32_t kOffRow = kOffTab + 4 * kTabWords * 4;       // c2, then -lse2, of the rows
  static constexpr uint32_t kOffBar = kOffRow + kPgxRows * 8;
  static constexpr int kSmemBytes = 1024 + kOffBar + 512;
  // TMEM: S^T of warpgroup g at 64 g; D at 128 (80 columns: values 0-63, share
  // sum at 64); at d = 128 values 64-127 at 208.
  static constexpr uint32_t kTmemD = 128, kTmemDHi = 208;
  static constexpr int kLd = D + 5;                    // floats per row of the low terms' stage
};

template <int D, bool EARLIER>
__global__ void __launch_bounds__(XVal<D>::kThreads, 1)
    pgx_values(PagedDecode p, PgtPlan w, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap) {
  using C = XVal<D>;
  extern __shared__ __align__(1024) uint8_t x_smem_raw[];
  uint8_t *smem = x_smem_raw + ((1024u - (smem_u32(x_smem_raw) & 1023u)) & 1023u);
  uint8_t *sQ = smem + C::kOffQ, *sK = smem + C::kOffK, *sV = smem + C::kOffV, *sSh = smem + C::kOffSh;
  uint32_t *sTab = reinterpret_cast<uint32_t *>(smem + C::kOffTab);
  float *sC2 = reinterpret_cast<float *>(smem + C::kOffRow), *sNl = sC2 + kPgxRows;
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
  uint64_t *k_full = q_full + 1, *k_empty = k_full + C::kKStages, *v_full = k_empty + C::kKStages,
           *v_empty = v_full + C::kVStages, *s_full = v_empty + C::kVStages, *s_free = s_full + 2, *sh_full = s_free + 2,
           *sh_free = sh_full + 2, *tab_full = sh_free + 2, *tab_free = tab_full + 4, *d_full = tab_free + 4,
           *d_free = d_full + 1, *done = d_free + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  __shared__ PgtLens L;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 8);
      mbar_init(&sh_full[i], 8);
      mbar_init(&sh_free[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&tab_full[i], 1);
      mbar_init(&tab_free[i], 8);
    }
    mbar_init(d_full, 1);
    mbar_init(d_free, 4);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  for (int e = tid; e < 2048 / 4; e += C::kThreads)   // the ones beside V: bf16 1.0
    reinterpret_cast<uint32_t *>(smem + C::kOffOnes)[e] = 0x3F803F80u;
  fence_proxy_async_smem();
  if (warp == C::kDemandWarps + 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pgt_load_lens<C::kThreads>(p, w, L, nullptr);   // ends with a block barrier
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.status};
  XWalk it;
  it.start(p, w, w.x_values);
  if (warp == C::kDemandWarps || warp == C::kDemandWarps + 1) {
    // ------------------------------------------------------------ K and V copies
    const bool isk = warp == C::kDemandWarps;
    const CUtensorMap *map = isk ? &kmap : &vmap;
    uint8_t *ring = isk ? sK : sV;
    uint64_t *full = isk ? k_full : v_full, *empty = isk ? k_empty : v_empty;
    const int stages = isk ? C::kKStages : C::kVStages;
    int issued = 0;
    for (; it.c.n > 0; it.next(p, w)) {
      int page = x_page(p, w, it.c.tile, lane);
      bool ok = true;
      for (int k = 0; k < it.c.n; ++k, ++issued) {
        const int ahead = k + 1 < it.c.n ? x_page(p, w, it.c.tile + k + 1, lane) : -1;
        const int s = issued % stages;
        ok = warp_wait(&empty[s], ((issued / stages) & 1) ^ 1, wc);
        if (!ok) break;
        x_load<D>(p, w, map, ring + s * C::kTB, &full[s], it.c.tile + k, it.c.hkv, page, lane);
        page = ahead;
      }
      if (!ok) break;
    }
    if (*abort_flag && lane == 0)
      for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
        x_drain(&full[i % stages], (i / stages) & 1);
  } else if (warp == C::kDemandWarps + 2) {
    // ------------------------------------------------------------ MMA issue
    // S(0), S(1), then S(k + 2) before PV(k): the buffer of S(k) is free once
    // its warpgroup has read it, before it has written the shares of k.
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16(128, kPgxRows, false, false);
      const uint32_t idesc_pv = idesc_bf16(128, 80, true, true), idesc_hi = idesc_bf16(128, 64, true, true);
      const uint32_t ones = smem_u32(smem + C::kOffOnes);
      const uint64_t dQ = x_kmajor(sQ), dK = x_kmajor(sK);
      int piece = 0;
      bool ok = true;
      for (; ok && it.c.n > 0; it.next(p, w), ++piece) {
        const int n = it.c.n, run = it.c.run;
        auto scores = [&](int k) {
          const int t = run + k, s = t % C::kKStages, g = t & 1;
          if (!mbar_wait(&k_full[s], (t / C::kKStages) & 1, wc) || !mbar_wait(&s_free[g], ((t >> 1) & 1) ^ 1, wc))
            return false;
          tc_fence_after();
          const uint64_t dKs = dK + (uint64_t)s * (C::kTB >> 4);
          MmaRun<0, 4, 2, 2, false>::go(tmem + g * 64, dKs, dQ, idesc_s, 0u);
          if constexpr (D == 128)
            MmaRun<0, 4, 2, 2, false>::go(tmem + g * 64, dKs + (kXHalf >> 4), dQ + (kXQHalf >> 4), idesc_s, 1u);
          mma_commit(&s_full[g]);
          mma_commit(&k_empty[s]);
          return true;
        };
        ok = mbar_wait(q_full, piece & 1, wc) && scores(0) && (n < 2 || scores(1));
        for (int k = 0; ok && k < n; ++k) {
          if (k + 2 < n && !scores(k + 2)) {
            ok = false;
            break;
          }
          const int t = run + k, s = t % C::kVStages, g = t & 1;
          ok = mbar_wait(&v_full[s], (t / C::kVStages) & 1, wc) && mbar_wait(&sh_full[g], (t >> 1) & 1, wc) &&
               (k > 0 || mbar_wait(d_free, (piece & 1) ^ 1, wc));
          if (!ok) break;
          tc_fence_after();
          // share^T: 64-row blocks (rounded, remainder) 16 KB apart, 8-key groups 1 KB apart;
          // [V | 1]: the second 64-column block is the ones (descriptor's leading offset)
          const uint64_t dSh = smem_desc(smem_u32(sSh) + g * C::kShBytes, 16384, 1024);
          const uint32_t v = smem_u32(sV) + s * C::kTB;
          MmaRun<0, 8, 128, 128 - (128ll << 16), false>::go(tmem + C::kTmemD, dSh, smem_desc(v, ones - v, 1024),
                                                            idesc_pv, k > 0 ? 1u : 0u);
          if constexpr (D == 128)
            MmaRun<0, 8, 128, 128, false>::go(tmem + C::kTmemDHi, dSh, smem_desc(v + kXHalf, kXHalf, 1024), idesc_hi,
                                              k > 0 ? 1u : 0u);
          mma_commit(&sh_free[g]);
          mma_commit(&v_empty[s]);
        }
        if (ok) mma_commit(d_full);
      }
      mma_commit(done);
      x_drain(done, 0);
    }
  } else if (warp == C::kDemandWarps + 3) {
    // ------------------------------------------------------------ demand pages
    // Table of a tile: for every row and page (or the tile's part of one), its place
    // in the demand pool in units of 16 floats.  One warp issues about one
    // instruction every 6 cycles, and the demand warps wait for the table first, so
    // it is short: with an entry for every 16 keys they waited 4200 of the 6700
    // cycles between their tiles.
    const int sh = w.page_shift, ps = 1 << sh;
    const uint32_t page_places = (uint32_t)p.c.Hq << (sh - 4);
    bool ok = true;
    auto tiles = [&](auto entries) {
      constexpr int E = decltype(entries)::value, KEYS = kPgxTile / E;
      for (; ok && it.c.n > 0; it.next(p, w)) {
        const int32_t *dtab[2];
        uint32_t head[2];
        bool on[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = it.c.row_at(lane + 32 * h), R = it.c.row0 + r, s = r < it.c.nrows ? R / w.G : 0;
          on[h] = r < it.c.nrows && L.len[s] > 0;          // idle slots and rows past the piece's have no demand
          dtab[h] = p.c.demand_table + (size_t)s * p.c.max_pages;
          head[h] = (uint32_t)(it.c.hkv * w.G + R % w.G) << (sh - 4);
        }
        int id[2][E];
        auto fetch = [&](int k) {
          const int key0 = (it.c.tile + k) * kPgxTile;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < E; ++e)
              id[h][e] = on[h] && k < it.c.n && key0 + KEYS * e < p.prefix_len ? __ldcg(dtab[h] + ((key0 + KEYS * e) >> sh)) : -1;
        };
        fetch(0);
        for (int k = 0; k < it.c.n; ++k) {
          const int t = it.c.run + k, b = t & 3, key0 = (it.c.tile + k) * kPgxTile;
          ok = warp_wait(&tab_free[b], ((t >> 2) & 1) ^ 1, wc);
          if (!ok) break;
          const uint32_t part = E == 1 ? (uint32_t)(key0 & (ps - 1)) >> 4 : 0u;   // the tile's place in its page
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < E; ++e) {
              uint32_t at = kNoDemand;
              if ((unsigned)id[h][e] < (unsigned)p.c.num_demand_pages)
                at = (uint32_t)id[h][e] * page_places + (head[h] + part);
              else if (on[h] && key0 + KEYS * e < p.prefix_len)
                atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
              sTab[b * kTabWords + e * kTabPitch + lane + 32 * h] = at;
            }
          fetch(k + 1);
          __syncwarp();
          if (lane == 0 && (t > 0 || (int)blockIdx.x != p.dbg.stall_block[kPagedPrefixValues]))   // (test hook: a table
            mbar_arrive(&tab_full[b]);                                                            // is not handed over)
        }
      }
    };
    if (sh >= 7)
      tiles(std::integral_constant<int, 1>());
    else if (sh == 6)
      tiles(std::integral_constant<int, 2>());
    else if (sh == 5)
      tiles(std::integral_constant<int, 4>());
    else
      tiles(std::integral_constant<int, 8>());
  } else {
    // ------------------------------------------------------------ demand warpgroups
    const int g = warp / 4 & 1, rh = warp / 8, quarter = warp % 4;   // tile parity, row half, TMEM quarter
    const int key_l = quarter * 32 + lane;                           // key inside the tile
    const PgtLine line = pgt_line(p, w, L);
    const uint32_t ts = tmem + g * 64 + 32 * rh + ((uint32_t)(quarter * 32) << 16);
    uint8_t *sh_row = sSh + g * C::kShBytes + (key_l / 8) * 1024 + (key_l % 8) * 128;
    // the warp's demand: lane -> row 4 j + lane / 8, keys 4 (lane % 8) .. of the warp's 32
    float *const dem = reinterpret_cast<float *>(smem + C::kOffDem + warp * 2048);
    const int dr = lane / 8, dk = 4 * (lane % 8);
    // its 16-key group: entry (group >> es) of the table, and the rest of the place
    const int group = (quarter * 32 + dk) >> 4, es = min(w.page_shift - 4, 3);
    const uint32_t *tab_lane = sTab + (group >> es) * kTabPitch + 32 * rh + dr;
    float *const pool = p.c.demand_pages + 16 * (group & ((1 << es) - 1)) + (dk & 15);
    float *const slot = dem + dr * 32 + dk;
    float *const mine = dem + lane;                  // this thread's key: row r of a group at 32 r
    int piece = 0;
    for (; it.c.n > 0; it.next(p, w), ++piece) {
      const int n = it.c.n;
      // rows: scale and normaliser (a row without a sequence bids nothing)
      {
        static_assert(4 * C::kDemandWarps == kPgxRows, "8 lanes a row");
        const int place = warp * 4 + lane / 8, r = it.c.row_at(place);
        const int R = it.c.row0 + min(r, it.c.nrows - 1), s = R / w.G;
        const int hq = it.c.hkv * w.G + R % w.G;
        const float lse = pgt_row_lse<8>(p, w, line, L, s, hq, lane);
        const bool on = r < it.c.nrows && L.len[s] > 0;
        if (lane % 8 == 0) {
          sC2[place] = on ? fmaxf(head_c2(p.hs, s * p.c.Hq + hq, nullptr), 1e-30f) : 1e-30f;
          sNl[place] = on ? -lse : -INFINITY;
        }
      }
      for (int e = tid; e < kPgxRows * (D / 8); e += 512) {   // Q: the K-major B operand
        const int r = e / (D / 8), i = e % (D / 8);
        *reinterpret_cast<uint4 *>(sQ + (i >> 3) * kXQHalf + r * 128 + (((i & 7) ^ (r & 7)) << 4)) =
            x_query<D>(p, w, it.c, it.c.row_at(r), i);
      }
      fence_proxy_async_smem();
      named_bar_sync(1, 512);
      if (tid == 0) mbar_arrive(q_full);
      const bool dead = __any_sync(0xffffffffu, *abort_flag != 0);
      const int k0 = (g ^ (it.c.run & 1));           // the warpgroup's first tile: alternate over the whole run
      // 8-row groups of the half with rows
      const int groups = (max(0, rh == 0 ? min(it.c.half(), it.c.nrows) : it.c.nrows - it.c.half()) + 7) / 8;
      for (int i = groups; i < 4; ++i) {   // rows past them: no share (the products before are done)
        const int to = ((4 * rh + i) ^ (key_l & 7)) << 4;
        *reinterpret_cast<uint4 *>(sh_row + to) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(sh_row + 16384 + to) = make_uint4(0u, 0u, 0u, 0u);
      }
      // The places of the lane's demand, for the tile at hand and the next.
      uint32_t at[8], at_next[8];
      auto places = [&](uint32_t (&a)[8], const uint32_t *tab, bool valid) {
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = valid ? tab[4 * j] : kNoDemand;
      };
      // 8 rows of a tile's demand: one group of copies, into place c & 1; zeros
      // where there is none.
      auto bring = [&](const uint32_t (&a)[8], int c) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float *to = slot + (8 * (c & 1) + 4 * j) * 32;
          if (a[2 * c + j] != kNoDemand)
            cp_async16(to, pool + (size_t)a[2 * c + j] * 16);
          else
            *reinterpret_cast<float4 *>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      bool ok = !dead;
      if (ok && k0 < n) {
        const int t = it.c.run + k0;
        ok = warp_wait(&tab_full[t & 3], (t >> 2) & 1, wc);
        places(at, tab_lane + (t & 3) * kTabWords, ok);
        bring(at, 0);
        bring(at, 1);
      }
      for (int k = k0; ok && k < n; k += 2) {
        const int t = it.c.run + k;
        const bool more = k + 2 < n;
        // infinity: a key past the prefix's end, which bids nothing
        const float eps = (it.c.tile + k) * kPgxTile + key_l < p.prefix_len ? p.eps : INFINITY;
        const float2 eps2 = make_float2(eps, eps);
        ok = !more || warp_wait(&tab_full[(t + 2) & 3], ((t + 2) >> 2) & 1, wc);
        places(at_next, tab_lane + ((t + 2) & 3) * kTabWords, more && ok);
        ok = ok && warp_wait(&s_full[g], (t >> 1) & 1, wc) &&
             // the product of this pair's previous tile has read the shares
             warp_wait(&sh_free[g], ((t >> 1) & 1) ^ 1, wc);
        if (!ok) break;
        tc_fence_after();
        if (groups < 1) x_release(&s_free[g], lane);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");   // this group's copies have landed
          if (c < groups) {
            float x[8];
            tmem_ld8(ts + 8 * c, x);
            __syncwarp();                                        // .. those of every lane
            tmem_wait_ld_r8(x);
            if (c == groups - 1) x_release(&s_free[g], lane);    // the next tile's S may be formed
            // A place past the prefix's end has the logit 0 of a row of zeros: where all of a
            // query's logits lie below -89 its bid would be 2^128 and its share infinity x 0.
            if (__any_sync(0xffffffffu, eps == INFINITY)) {
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = eps == INFINITY ? -INFINITY : x[e];
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 sc = *reinterpret_cast<const float4 *>(sC2 + 32 * rh + 8 * c + 4 * q);
              const float4 nl = *reinterpret_cast<const float4 *>(sNl + 32 * rh + 8 * c + 4 * q);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = 4 * q + 2 * e;
                float *m0 = mine + (8 * (c & 1) + r) * 32;
                const float2 y = ffma2(make_float2(x[r], x[r + 1]), e ? make_float2(sc.z, sc.w) : make_float2(sc.x, sc.y),
                                       e ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y));
                const float2 bid = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                const float2 d = make_float2(m0[0], m0[32]);
                const float2 nd = fadd2(d, bid);
                m0[0] = nd.x;
                m0[32] = nd.y;
                const float2 den = fadd2(EARLIER ? d : nd, eps2);
                const float2 sh = fmul2(bid, make_float2(rcp_approx(den.x), rcp_approx(den.y)));
                const uint32_t h2 = pack_bf16x2(sh.x, sh.y);
                const float2 rest = ffma2(make_float2(__uint_as_float(h2 << 16), __uint_as_float(h2 & 0xffff0000u)),
                                          make_float2(-1.f, -1.f), sh);
                hi[2 * q + e] = h2;
                lo[2 * q + e] = pack_bf16x2(rest.x, rest.y);
              }
            }
            const int to = ((4 * rh + c) ^ (key_l & 7)) << 4;    // rows 32 rh + 8 c ..: a 16-byte piece of each block
            *reinterpret_cast<uint4 *>(sh_row + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(sh_row + 16384 + to) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            __syncwarp();                                        // the new demand of every lane's key
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 d4 = *reinterpret_cast<const float4 *>(slot + (8 * (c & 1) + 4 * j) * 32);
              if (at[2 * c + j] != kNoDemand) *reinterpret_cast<float4 *>(pool + (size_t)at[2 * c + j] * 16) = d4;
            }
          }
          // two groups on, over what this lane has just written back
          if (c < 2)
            bring(at, c + 2);
          else
            bring(at_next, c - 2);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh_full[g]);
          mbar_arrive(&tab_free[t & 3]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) at[j] = at_next[j];
      }
      cp_async_wait_all();
      // the piece's sums: TMEM lanes 0-63 hold the rounded shares' products, 64-127 the remainders'
      named_bar_sync(1, 512);
      if (warp < 4) {
        float *stage = reinterpret_cast<float *>(sSh);
        const bool have = warp_wait(d_full, piece & 1, wc);
        tc_fence_after();
        const uint32_t td = tmem + C::kTmemD + ((uint32_t)(quarter * 32) << 16);
        const int place = key_l % kPgxRows, r = it.c.row_at(place);
        float *part = reinterpret_cast<float *>(p.ws + w.pre_acc_off) +
                      ((size_t)(blockIdx.x + it.c.seg) * w.pre_rows + r) * acc_stride(D);
        auto column = [&](int c) { return td + (D == 128 && c >= 64 ? C::kTmemDHi - C::kTmemD + c - 64 : c); };
        if (have && quarter >= 2) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float x[32];
            tmem_ld32(column(c), x);
            tmem_wait_ld_r(x);
#pragma unroll
            for (int e = 0; e < 32; ++e) stage[place * C::kLd + c + e] = x[e];
          }
          float s1;
          tmem_ld1(td + 64, s1);
          tmem_wait_ld();
          asm volatile("" : "+f"(s1));
          stage[place * C::kLd + D] = s1;
        }
        named_bar_sync(2, 128);
        if (have && quarter < 2) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            float x[32];
            tmem_ld32(column(c), x);
            tmem_wait_ld_r(x);
            if (r < it.c.nrows) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4 *>(part + c + e) =
                    make_float4(x[e] + stage[place * C::kLd + c + e], x[e + 1] + stage[place * C::kLd + c + e + 1],
                                x[e + 2] + stage[place * C::kLd + c + e + 2], x[e + 3] + stage[place * C::kLd + c + e + 3]);
            }
          }
          float s1;
          tmem_ld1(td + 64, s1);
          tmem_wait_ld();
          asm volatile("" : "+f"(s1));
          if (r < it.c.nrows) part[D] = s1 + stage[place * C::kLd + D];
        }
        x_release(d_free, lane);
      }
      named_bar_sync(1, 512);
    }
    if (tid == 0) pdl_wait();   // (see launch_after) this kernel ends after its predecessor
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kDemandWarps + 2) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================================ host
static bool x_map(const PagedDecode &p, const void *pages, CUtensorMap *m) {
  const int64_t num = (int64_t)p.c.num_pages * p.c.Hkv;
  return make_page_map(m, pages, num > 0 ? num : 1, p.c.page_size, kPgxTile, p.c.d, DA_BF16);
}

template <int D>
static int pgx_prepare() {
  static PerDeviceOnce once;
  return once.run([] {
    return (cudaFuncSetAttribute(pgx_keys<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, XKeys<D>::kSmemBytes) !=
                cudaSuccess ||
            cudaFuncSetAttribute(pgx_values<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 XVal<D>::kSmemBytes) != cudaSuccess ||
            cudaFuncSetAttribute(pgx_values<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 XVal<D>::kSmemBytes) != cudaSuccess)
               ? DA_ERR_CUDA
               : DA_OK;
  });
}

template <int D>
static int launch_keys_t(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream) {
  CUtensorMap km;
  if (pgx_prepare<D>() != DA_OK || !x_map(p, p.c.k_pages, &km)) return DA_ERR_CUDA;
  return launch_after(pgx_keys<D>, w.x_keys.ctas, XKeys<D>::kThreads, XKeys<D>::kSmemBytes, stream, p, w, km) ==
                 cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

template <int D>
static int launch_values_t(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream) {
  CUtensorMap km, vm;
  if (pgx_prepare<D>() != DA_OK || !x_map(p, p.c.k_pages, &km) || !x_map(p, p.c.v_pages, &vm)) return DA_ERR_CUDA;
  const cudaError_t e = p.earlier ? launch_after(pgx_values<D, true>, w.x_values.ctas, XVal<D>::kThreads,
                                                 XVal<D>::kSmemBytes, stream, p, w, km, vm)
                                  : launch_after(pgx_values<D, false>, w.x_values.ctas, XVal<D>::kThreads,
                                                 XVal<D>::kSmemBytes, stream, p, w, km, vm);
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int launch_pgx_keys(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream) {
  return p.c.d == 128 ? launch_keys_t<128>(p, w, stream) : launch_keys_t<64>(p, w, stream);
}
int launch_pgx_values(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream) {
  return p.c.d == 128 ? launch_values_t<128>(p, w, stream) : launch_values_t<64>(p, w, stream);
}

}  // namespace da
