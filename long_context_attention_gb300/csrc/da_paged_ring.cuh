// The ring of 16 KB stages that one warp fills with key or value tiles by TMA, for
// the streaming kernels of the paged decode step in both types.
#pragma once

#include "da_paged_plan.cuh"

#include <cuda.h>

namespace da {

constexpr int kStageBytes = 16384;

// Byte offset of 16-byte piece `piece` of row `row` in a staged tile of TILE rows:
// boxes of 128 bytes a row by TILE rows, pieces swizzled by the row.
template <int TILE>
__device__ __forceinline__ uint32_t tile_off(int row, int piece) {
  return (uint32_t)((piece >> 3) * TILE * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

struct PgtRing {
  uint64_t full[8], empty[8];
  volatile int abort_word;
  __device__ __forceinline__ void init(int stages, int arrivals) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], arrivals);   // one per consumer of a tile
    }
    abort_word = 0;
    fence_mbar_init();
  }
};

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
  asm volatile(
      "{\n\t.reg .b64 pol;\n\t"
      "createpolicy.fractional.L2::evict_first.b64 pol, 1.0;\n\t"
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], pol;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Let the copies in flight land before the CTA exits after a timeout.
__device__ __forceinline__ void drain(uint64_t *full, int stages, int issued) {
  for (int st = issued > stages ? issued - stages : 0; st < issued; ++st) {
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(&full[st % stages], (uint32_t)((st / stages) & 1)))
      if (globaltimer() - t0 > 100ull * 1000ull * 1000ull) break;
  }
}

// Producer warp: fills the ring with the tiles of the stretch [from, to) of K or
// V.  Lane i brings page piece i of a tile.  One warp issues about one
// dependent instruction every 5 cycles, and a tile has 0.7 us at HBM rate, so
// the loop is short: no divisions, one table entry per lane, fetched a tile
// ahead.
// A tile is TILE rows of 16384 / TILE bytes; XSTEP: elements in 128 bytes.  AFTER_WAIT:
// the kernel has waited for its predecessor (see launch_after).  Otherwise its
// consumers wait before they free a slot, so that from the second round on entries
// may come from L1 (all from L2: 531 us for 8 x 12 x 131072, so 519).
template <int TILE, int XSTEP, bool AFTER_WAIT>
__device__ void produce(const PagedDecode &p, const PgtPlan &w, const PgtLine &line, const PgtLens &L, PgtRing &ring,
                        const CUtensorMap *map, uint32_t base, int stages, int from, int to, const WaitCtx &wc) {
  constexpr int BOXES = kStageBytes / (TILE * 128);
  const int lane = threadIdx.x % 32, sh = w.page_shift, ps = 1 << sh;
  const int rows = min(ps, TILE);
  int slot = 0;
  uint32_t parity = 1;
  PgtSeg g;
  int issued = 0;
  for (g.start(p, w, line, L, from, to); g.n > 0; g.next(p, w, line, L)) {
    const int32_t *table = g.s >= 0 ? p.c.page_table + (size_t)g.s * p.c.max_pages : p.prefix_table;
    int key = g.key0 + lane * rows;                                   // this lane's piece
    const int limit = lane * rows < TILE ? g.end : 0;                 // lanes past the tile bring nothing
    auto entry = [&](int at, bool l1) { return l1 ? table[at >> sh] : __ldcg(table + (at >> sh)); };
    int page = key < limit ? entry(key, AFTER_WAIT) : -1;
    for (int k = 0; k < g.n; ++k, ++issued) {
      const int ahead = k + 1 < g.n && key + TILE < limit ? entry(key + TILE, AFTER_WAIT || issued > stages) : -1;
      if (!warp_wait(&ring.empty[slot], parity, wc)) {
        if (lane == 0) drain(ring.full, stages, issued);
        return;
      }
      const bool ok = (unsigned)page < (unsigned)p.c.num_pages;
      const uint32_t have = __ballot_sync(0xffffffffu, ok);
      if (!ok && key < limit) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[slot], (uint32_t)(__popc(have) * rows) * (BOXES * 128));
      __syncwarp();
      if (ok) {
        const uint32_t dst = base + slot * kStageBytes + lane * rows * 128;
#pragma unroll
        for (int x = 0; x < BOXES; ++x)
          tma_page(dst + x * TILE * 128, map, &ring.full[slot], x * XSTEP, key & (ps - 1), page * p.c.Hkv + g.hkv);
      }
      page = ahead;
      key += TILE;
      if (++slot == stages) {
        slot = 0;
        parity ^= 1;
      }
    }
  }
  if (ring.abort_word && lane == 0) drain(ring.full, stages, issued);
}

extern __shared__ __align__(1024) uint8_t pgt_smem_raw[];
__device__ __forceinline__ uint8_t *pgt_smem_base() {   // the swizzle counts from 1024-byte boundaries
  return pgt_smem_raw + ((1024u - (smem_u32(pgt_smem_raw) & 1023u)) & 1023u);
}

// fwd_bf16.cu: a pool of `num` pages (per key head) of page_size rows of d
// elements as a tensor map, copied a page (at most `rows` rows) by 128 bytes at a time.
bool make_page_map(CUtensorMap *m, const void *base, int64_t num, int page_size, int rows, int d, int dtype);

}  // namespace da
