// Decode step over the paged cache in bf16: streaming tensor-core kernels.
//
// Mathematics, for one query head against the keys of its sequence: p = softmax(x),
// share = p / (D + p + eps) of each key's demand total D (D + eps with the earlier
// demand only), out = sum share v / sum share, D += p.  Two passes over the keys,
// joined by the softmax normaliser that a share needs:
//   pgt_keys    x = q . k (tau / sqrt(d) log2 e) of every key into a scratch of
//               4 bytes per (row, key), and each piece's (max, sum 2^(x - max));
//   pgt_values  lse2 from the pieces, p = 2^(x - lse2), share = p / (D + p +
//               eps), D += p, and each piece's sum share v and sum share;
//   pgt_combine out = sum of the pieces' numerators / sum of their share sums,
//               in a fixed order (equal bits from equal calls).
//
// What bounds it: HBM.  K and V are read once, D is read and written once, the
// logits stay mostly in L2.  So the layout serves the copies: whole pages (or
// a tile's rows of one) arrive by TMA with a 128-byte swizzle into a ring of stages
// of 16 KB (128 keys at d = 64, 64 at d = 128) that one producer warp fills, and
// in pgt_values every thread keeps its logits and demand in flight two tiles ahead.
//
// Tensor cores: m16n8k16 (bf16, fp32 sums).  A decode step has few query rows
// per key head, so the tensor rate is not what bounds it; the M = 16 rows are
// the query heads that share a key head (padded), and one 16-key group costs a
// warp 8 + 16 instructions at d = 64.  Keys are taken in an order in which each
// thread holds 4 consecutive keys of a row: logits, demand and shares then move
// in 16-byte pieces, and the share of a key is already where the A operand of
// the value product wants it (no shuffles).  Shares enter that product as two
// bf16 terms (share rounded, and what rounding left), so they keep 2^-16
// relative; one term alone would double the output's rounding error.
//
// Work split: a segment is one sequence's own part or the shared prefix for one
// key head and up to 16 rows.  All segments lie on one line, each as kPgtHead
// units (what beginning a segment costs, in tiles) followed by its key tiles;
// every CTA takes an equal stretch of the line, so ragged lengths balance to a
// tile and many short sequences do not gather in one CTA (48 sequences of 1 ..
// 16384 tokens, d = 128: without the head units the SMs were busy 43 % of
// pgt_keys).  The part of a segment inside one stretch is a piece and leaves
// one partial result, in slot (CTA + segment), which grows along the line and
// is therefore unique.
#include "da_paged_ring.cuh"

#include <cuda_bf16.h>

namespace da {

constexpr int kPgtSmemPerCta = 100 * 1024;        // two CTAs an SM beside their static shared memory

// pgt_values for up to GE rows of a segment (1, 2, 4, 8 or 16).
template <int D, int GE>
struct PgtVal {
  static constexpr bool kWide = GE == 16;             // rows fill the M = 16 of the product
  static constexpr int kTile = pgt_tile(D);
  static constexpr int kGroups = kWide ? 1 : (8 / GE < kTile / 16 ? 8 / GE : kTile / 16);   // 16-key groups a step
  static constexpr int kStep = 16 * kGroups;          // keys a warp takes at a time
  static constexpr int kStepsPerTile = kTile / kStep;
  // Enough warps that the shares of a 16 KB tile take less than its 0.7 us at HBM rate.
  static constexpr int kWarps = D == 64 && GE >= 8 ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps + 32;
  static constexpr int kTileStride = kWarps / kStepsPerTile;   // tiles between a warp's steps
  static_assert(kWarps % kStepsPerTile == 0, "whole tiles");
  static constexpr int kAhead = kTileStride >= 2 ? 2 : 3;      // steps whose logits and demand are in flight or in use
  static constexpr int kHalves = kWide ? 2 : 1;
  static constexpr int kSideBytes = kAhead * kHalves * 1024;   // a warp's logits and demand
  static constexpr int kRedBytes = (kWide ? 16 : 8) * D * 4;   // a warp's numerators, in the same place afterwards
  static constexpr int kWarpBytes = kSideBytes > kRedBytes ? kSideBytes : kRedBytes;
  static constexpr int kRoom = (kPgtSmemPerCta - 1024 - kWarps * kWarpBytes) / 16384;
  // A multiple of the stride: every tile that passes through a slot then goes
  // to the same warps, which therefore see each phase of its barrier (a wait
  // that skips a phase cannot tell it from the one before it).
  static constexpr int kStages = (kRoom < 8 ? kRoom : 8) / kTileStride * kTileStride;
  static_assert(kStages >= 2 && kStages >= kTileStride, "a slot for every warp");
  static constexpr int kSmemBytes = 1024 + kStages * 16384 + kWarps * kWarpBytes;
};

// ------------------------------------------------------------------ pass 1: logits
// HH: halves of 8 rows in use (1 for up to 8 rows).
template <int D, int HH>
__global__ void __launch_bounds__(pgt_threads(D), 2)
    pgt_keys(PagedDecode p, PgtPlan w, const __grid_constant__ CUtensorMap kmap, int stages) {
  constexpr int KS = D / 16;   // k-steps
  constexpr int TILE = pgt_tile(D), WARPS = pgt_warps(D);
  __shared__ PgtLens L;
  __shared__ PgtRing ring;
  __shared__ float2 s_ml[WARPS][16];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) ring.init(stages, WARPS);
  pdl_wait();   // for everything before the step
  pdl_launch_dependents();
  pgt_load_lens<pgt_threads(D)>(p, w, L, blockIdx.x == 0 ? p.status : nullptr);
  const PgtLine line = pgt_line(p, w, L);
  const int from = line.cut.first(blockIdx.x), to = line.cut.first(blockIdx.x + 1);
  const WaitCtx wc{&ring.abort_word, p.status, p.dbg.limit_ns[kPagedKeys]};
  const uint32_t base = smem_u32(pgt_smem_base());
  if (warp == WARPS) {
    produce<pgt_tile(D), 64, true>(p, w, line, L, ring, &kmap, base, stages, from, to, wc);
    return;
  }
  const int gid = lane / 4, t = lane % 4;
  const bool keep = warp == 0 && (int)blockIdx.x == p.dbg.stall_block[kPagedKeys];   // test hook
  // lane -> the row it addresses: matrices (half 0, k 0-7), (half 0, k 8-15), (half 1, ..), (half 1, ..)
  const int row = warp * 16 + group_key(lane & 7, lane >> 4);
  int slot = 0;
  uint32_t parity = 0;
  PgtSeg g;
  for (g.start(p, w, line, L, from, to); g.n > 0; g.next(p, w, line, L)) {
    const int n = g.n;
    const int tiles = __any_sync(0xffffffffu, ring.abort_word != 0) ? 0 : n;   // a wait gave up: touch no barrier again
    // Q rows as the A operand; rows past the segment's are 0
    uint32_t qa[KS][4] = {};
    float c2[HH] = {};
    float *xrow[HH] = {};
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
      const int r = gid + 8 * hh;
      const bool ok = r < g.nrows;
      int s = 0, hq = 0;
      if (ok) {
        g.row(w.G, r, s, hq);
        c2[hh] = head_c2(p.hs, s * p.c.Hq + hq, (t == 0 && warp == 0) ? p.status : nullptr);
        xrow[hh] = reinterpret_cast<float *>(p.ws + w.logit_off) + ((size_t)s * p.c.Hq + hq) * w.Lp - w.logit_key0;
      }
      const uint32_t *qr =
          reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)s * p.c.Hq + hq) * D);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qa[ks][hh] = ok ? qr[ks * 8 + t] : 0u;
        qa[ks][2 + hh] = ok ? qr[ks * 8 + 4 + t] : 0u;
      }
    }
    float m[HH], l[HH];
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) m[hh] = -INFINITY, l[hh] = 0.f;
    const int first = g.key0 + warp * 16;   // this warp's 16 keys of the first tile
    // A wait that gave up ends the piece's loop but not the warp, which still
    // meets the others at the barriers below.
    for (int k = 0; k < tiles; ++k) {
      if (!warp_wait(&ring.full[slot], parity, wc)) break;
      const uint32_t tile = base + slot * kStageBytes;
      const int kg = first + k * TILE;
      if (kg < g.end) {
        float acc[2][4] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t bfr[4];
          ldsm_x4(tile + tile_off<pgt_tile(D)>(row, 2 * ks + ((lane >> 3) & 1)), bfr);
          mma16816(acc[0], qa[ks], bfr[0], bfr[1]);
          mma16816(acc[1], qa[ks], bfr[2], bfr[3]);
        }
        const int key = kg + 4 * t;
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) {
          if (gid + 8 * hh >= g.nrows) continue;
          float x[4] = {acc[0][2 * hh] * c2[hh], acc[0][2 * hh + 1] * c2[hh], acc[1][2 * hh] * c2[hh],
                        acc[1][2 * hh + 1] * c2[hh]};
          *reinterpret_cast<float4 *>(xrow[hh] + key) = make_float4(x[0], x[1], x[2], x[3]);
          if (kg + 16 > g.end) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + e >= g.end) x[e] = -INFINITY;
          }
          const float mn = fmaxf(m[hh], fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
          const float ms = mn == -INFINITY ? 0.f : mn;
          l[hh] = l[hh] * ex2_approx(m[hh] - ms) + (ex2_approx(x[0] - ms) + ex2_approx(x[1] - ms)) +
                  (ex2_approx(x[2] - ms) + ex2_approx(x[3] - ms));
          m[hh] = mn;
        }
      }
      __syncwarp();
      if (lane == 0 && !(keep && k == 0)) mbar_arrive(&ring.empty[slot]);
      if (++slot == stages) {
        slot = 0;
        parity ^= 1;
      }
    }
    // the piece's (max, sum) of each row: over the quad, then over the warps
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m[hh], o), l2 = __shfl_xor_sync(0xffffffffu, l[hh], o);
        const float mn = fmaxf(m[hh], m2), ms = mn == -INFINITY ? 0.f : mn;
        l[hh] = l[hh] * ex2_approx(m[hh] - ms) + l2 * ex2_approx(m2 - ms);
        m[hh] = mn;
      }
      if (t == 0) s_ml[warp][gid + 8 * hh] = make_float2(m[hh], l[hh]);
    }
    named_bar_sync(1, WARPS * 32);
    if (tid < g.nrows) {
      float M = -INFINITY, S = 0.f;
#pragma unroll
      for (int v = 0; v < WARPS; ++v) M = fmaxf(M, s_ml[v][tid].x);
      const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int v = 0; v < WARPS; ++v) S += s_ml[v][tid].y * ex2_approx(s_ml[v][tid].x - ms);
      const size_t at = (size_t)blockIdx.x + g.seg;
      float2 *ml = g.s >= 0 ? reinterpret_cast<float2 *>(p.ws + w.own_ml_off) + at * w.own_rows
                            : reinterpret_cast<float2 *>(p.ws + w.pre_ml_off) + at * w.pre_rows;
      ml[tid] = make_float2(M, S);
    }
    named_bar_sync(1, WARPS * 32);
  }
}

// ------------------------------------------------------------------ pass 2: shares
// Lane (g, t) of a warp holds 4 consecutive keys of one row.  With GE rows the
// 8 values of g are GE rows x kGroups groups of 16 keys, so that few query heads
// per key head still use every lane for the exponentials and reciprocals: group
// q's shares sit in rows q GE .. of the A operand, the other rows are 0 for its
// product, and the rows of equal query head are added once per piece.  Rows
// 8-15 of the operand take what rounding the shares to bf16 left (the second
// term costs no instructions).  With 9 to 16 rows (GE = 16) the second term is
// a product of its own.
//
// Each thread brings the logits and demand of its own keys itself, by 16-byte
// asynchronous copies into its own place in shared memory one or two steps
// ahead: nothing to hand over between warps, and no registers held by bytes in
// flight.  A warp takes every kTileStride-th tile's step (8 x 12 x 131072 keys,
// d = 64: 4 of 32 lanes at work and 250 instructions per 16 keys took 365 us).
template <int D, int GE>
__global__ void __launch_bounds__(PgtVal<D, GE>::kThreads, 2)
    pgt_values(PagedDecode p, PgtPlan w, const __grid_constant__ CUtensorMap vmap) {
  using V = PgtVal<D, GE>;
  constexpr int NT = D / 8;    // n-tiles of the value product
  constexpr int TILE = V::kTile, WARPS = V::kWarps, HH = V::kHalves, AHEAD = V::kAhead;
  constexpr int STRIDE = V::kTileStride * TILE;   // keys between a warp's steps
  __shared__ PgtLens L;
  __shared__ PgtRing ring;
  __shared__ float s_lse[16];
  __shared__ float s_sum[WARPS][16];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) ring.init(V::kStages, V::kStepsPerTile);
  pgt_load_lens<V::kThreads>(p, w, L, nullptr);
  const PgtLine line = pgt_line(p, w, L);
  const int from = line.cut.first(blockIdx.x), to = line.cut.first(blockIdx.x + 1);
  const WaitCtx wc{&ring.abort_word, p.status, p.dbg.limit_ns[kPagedValues]};
  uint8_t *const smem = pgt_smem_base();
  const uint32_t base = smem_u32(smem);
  if (warp == WARPS) {   // the values do not depend on the first pass
    produce<pgt_tile(D), 64, false>(p, w, line, L, ring, &vmap, base, V::kStages, from, to, wc);
    return;
  }
  uint8_t *const mine = smem + V::kStages * 16384 + warp * V::kWarpBytes;
  float *const stash = reinterpret_cast<float *>(mine) + lane * 8;   // this thread's logits and demand: [AHEAD][HH]
  const float *const logits = reinterpret_cast<const float *>(p.ws + w.logit_off);
  const int gid = lane / 4, t = lane % 4, sh = w.page_shift, ps = 1 << sh;
  const int q = V::kWide ? 0 : gid / GE, r0 = V::kWide ? gid : gid % GE;   // the lane's group and row
  const int sub = warp % V::kStepsPerTile * V::kStep;    // the warp's keys inside a tile
  const bool keep = warp == 0 && (int)blockIdx.x == p.dbg.stall_block[kPagedValues];   // test hook
  // lane -> row: matrices (k half 0, n 0-7), (k half 1, n 0-7), (k half 0, n 8-15), (k half 1, n 8-15)
  const int vrow = sub + group_key(lane & 7, (lane >> 3) & 1);
  bool waited = false;
  PgtSeg g;
  for (g.start(p, w, line, L, from, to); g.n > 0; g.next(p, w, line, L)) {
    const int n = g.n;
    // the warp's first tile of the piece: tile x of the CTA's run goes to the
    // warps x % kTileStride, whatever the pieces
    const int tile0 = (warp / V::kStepsPerTile + V::kTileStride - g.run % V::kTileStride) % V::kTileStride;
    int steps = n > tile0 ? (n - tile0 + V::kTileStride - 1) / V::kTileStride : 0;
    if (__any_sync(0xffffffffu, ring.abort_word != 0)) steps = 0;    // a wait gave up: touch no barrier again
    const int step0 = g.key0 + tile0 * TILE + sub;                   // its first key
    const int key0 = step0 + 16 * q + 4 * t;                         // the lane's first key
    // the lane's rows: logits, demand table, demand pool of its query head
    const float *xrow[HH];
    const int32_t *dtab[HH];
    float *dpool[HH];
    bool on[HH];
    const size_t page_floats = (size_t)p.c.Hq << sh;
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
      const int r = r0 + 8 * hh;
      int s = 0, hq = 0;
      on[hh] = r < g.nrows && q < V::kGroups;
      if (on[hh]) g.row(w.G, r, s, hq);
      on[hh] = on[hh] && L.len[s] > 0;                 // an idle slot bids nothing
      xrow[hh] = logits + ((size_t)s * p.c.Hq + hq) * w.Lp + (key0 - w.logit_key0);
      dtab[hh] = p.c.demand_table + (size_t)s * p.c.max_pages;
      dpool[hh] = p.c.demand_pages + ((size_t)hq << sh);
    }
    auto demand_page = [&](int k, int hh, bool after_wait) -> int {   // of the lane's keys of step k
      const int key = key0 + k * STRIDE;
      const int32_t *at = dtab[hh] + (key >> sh);
      return on[hh] && k < steps && key < g.end ? (after_wait ? *at : __ldcg(at)) : -1;
    };
    auto demand_at = [&](int k, int hh, int pg) -> float * {
      return dpool[hh] + (size_t)pg * page_floats + ((key0 + k * STRIDE) & (ps - 1));
    };
    auto bring = [&](int k, const int (&pg)[HH]) {
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) {
        if (on[hh] && k < steps && key0 + k * STRIDE < g.end) {
          float *to = stash + ((k % AHEAD) * HH + hh) * 256;
          cp_async16(to, xrow[hh] + k * STRIDE);
          if ((unsigned)pg[hh] < (unsigned)p.c.num_demand_pages)
            cp_async16(to + 4, demand_at(k, hh, pg[hh]));
          else
            atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int pages[AHEAD + 1][HH];   // demand pages of steps k .. k + AHEAD
#pragma unroll
    for (int a = 0; a < AHEAD; ++a)
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) pages[a][hh] = demand_page(a, hh, waited);
    if (!waited) {   // the demand does not depend on the first pass: to L2 meanwhile
#pragma unroll
      for (int a = 0; a < AHEAD - 1; ++a)
#pragma unroll
        for (int hh = 0; hh < HH; ++hh)
          if ((unsigned)pages[a][hh] < (unsigned)p.c.num_demand_pages) prefetch_l2(demand_at(a, hh, pages[a][hh]));
      pdl_wait();
      pdl_launch_dependents();
      waited = true;
    }
#pragma unroll
    for (int a = 0; a < AHEAD - 1; ++a) bring(a, pages[a]);
    // lse2 of the rows: 8 lanes join a row's pieces
    for (int r4 = warp * 4; r4 < g.nrows; r4 += WARPS * 4) {
      const int r = r4 + lane / 8;
      int s = 0, hq = 0;
      g.row(w.G, min(r, g.nrows - 1), s, hq);
      const float v = pgt_row_lse<8>(p, w, line, L, s, hq, lane);
      if (lane % 8 == 0 && r < g.nrows) s_lse[r] = v;
    }
    named_bar_sync(1, WARPS * 32);
    float lse[HH], sum[HH] = {};
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) lse[hh] = on[hh] ? s_lse[r0 + 8 * hh] : 0.f;
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    // A wait that gave up ends the piece's loop but not the warp (see pgt_keys).
    for (int k = 0; k < steps; ++k) {
      bring(k + AHEAD - 1, pages[AHEAD - 1]);
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) pages[AHEAD][hh] = demand_page(k + AHEAD, hh, true);
      asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");   // step k's have landed
      const int left = g.end - (step0 + k * STRIDE);     // keys of the step before the end
      const int valid = left - 16 * q - 4 * t;           // of the lane's four
      uint32_t hi[HH][2], lo[HH][2];
#pragma unroll
      for (int hh = 0; hh < HH; ++hh) {
        hi[hh][0] = hi[hh][1] = lo[hh][0] = lo[hh][1] = 0u;
        if (on[hh] && valid > 0) {
          const float *from = stash + ((k % AHEAD) * HH + hh) * 256;
          const float4 x = *reinterpret_cast<const float4 *>(from);
          const float4 d = *reinterpret_cast<const float4 *>(from + 4);
          const float xe[4] = {x.x, x.y, x.z, x.w}, de[4] = {d.x, d.y, d.z, d.w};
          float nd[4], share[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float bid = ex2_approx(xe[e] - lse[hh]);
            nd[e] = de[e] + bid;
            const float den = (p.earlier ? de[e] : nd[e]) + p.eps;
            share[e] = bid * rcp_approx(den);
          }
          if (valid < 4) {
#pragma unroll
            for (int e = 1; e < 4; ++e)
              if (e >= valid) share[e] = 0.f;
          }
          sum[hh] += (share[0] + share[1]) + (share[2] + share[3]);
          if ((unsigned)pages[0][hh] < (unsigned)p.c.num_demand_pages) {
            float *dst = demand_at(k, hh, pages[0][hh]);
            if (valid >= 4) {
              *reinterpret_cast<float4 *>(dst) = make_float4(nd[0], nd[1], nd[2], nd[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 3; ++e)
                if (e < valid) dst[e] = nd[e];
            }
          }
          // columns 2t, 2t + 1 of the first 8 are keys 4t, 4t + 1, of the last 8 keys 4t + 2, 4t + 3
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float s0 = share[2 * half], s1 = share[2 * half + 1];
            const uint32_t h2 = pack_bf16x2(s0, s1);
            hi[hh][half] = h2;
            lo[hh][half] = pack_bf16x2(s0 - __uint_as_float(h2 << 16), s1 - __uint_as_float(h2 & 0xffff0000u));
          }
        }
      }
#pragma unroll
      for (int a = 0; a < AHEAD; ++a)
#pragma unroll
        for (int hh = 0; hh < HH; ++hh) pages[a][hh] = pages[a + 1][hh];
      const int st = g.run + tile0 + k * V::kTileStride;       // the tile's place in the ring
      const int slot = st % V::kStages;
      if (!warp_wait(&ring.full[slot], (uint32_t)((st / V::kStages) & 1), wc)) break;
      const uint32_t tile = base + slot * 16384;
      if (left > 0 && left < V::kStep) {   // rows past the end may hold anything: 0 times NaN is NaN
        const int fill = (-left) & 15;     // up to the end of their group; later groups are left out
        for (int j = lane; j < fill * (D / 8); j += 32) {
          const int r = sub + left + j / (D / 8);
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(tile + tile_off<pgt_tile(D)>(r, j % (D / 8))), "r"(0u)
                       : "memory");
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
#pragma unroll
      for (int gg = 0; gg < V::kGroups; ++gg) {
        if (16 * gg >= left) break;
        uint32_t a1[4], a2[4];
        if constexpr (V::kWide) {
          a1[0] = hi[0][0], a1[1] = hi[HH - 1][0], a1[2] = hi[0][1], a1[3] = hi[HH - 1][1];
          a2[0] = lo[0][0], a2[1] = lo[HH - 1][0], a2[2] = lo[0][1], a2[3] = lo[HH - 1][1];
        } else {
          const bool here = V::kGroups == 1 || q == gg;
          a1[0] = here ? hi[0][0] : 0u, a1[1] = here ? lo[0][0] : 0u;
          a1[2] = here ? hi[0][1] : 0u, a1[3] = here ? lo[0][1] : 0u;
        }
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t bfr[4];
          ldsm_x4_t(tile + tile_off<pgt_tile(D)>(vrow + 16 * gg, j + (lane >> 4)), bfr);
          mma16816(acc[j], a1, bfr[0], bfr[1]);
          mma16816(acc[j + 1], a1, bfr[2], bfr[3]);
          if constexpr (V::kWide) {
            mma16816(acc[j], a2, bfr[0], bfr[1]);
            mma16816(acc[j + 1], a2, bfr[2], bfr[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0 && !(keep && k == 0)) mbar_arrive(&ring.empty[slot]);
    }
    cp_async_wait_all();
    __syncwarp();
    // the piece's numerators and share sums: each warp's rows into its own
    // place, then the parts of a query head added in a fixed order
    float *const red = reinterpret_cast<float *>(mine);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float *to = red + gid * D + 8 * j + 2 * t;
      if constexpr (V::kWide) {
        *reinterpret_cast<float2 *>(to) = make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2 *>(to + 8 * D) = make_float2(acc[j][2], acc[j][3]);
      } else {
        *reinterpret_cast<float2 *>(to) = make_float2(acc[j][0] + acc[j][2], acc[j][1] + acc[j][3]);
      }
    }
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) sum[hh] += __shfl_xor_sync(0xffffffffu, sum[hh], o);
      if (t == 0) s_sum[warp][gid + 8 * hh] = sum[hh];
    }
    named_bar_sync(1, WARPS * 32);
    const size_t at = (size_t)blockIdx.x + g.seg;
    float *part = g.s >= 0 ? reinterpret_cast<float *>(p.ws + w.own_acc_off) + at * w.own_rows * acc_stride(D)
                           : reinterpret_cast<float *>(p.ws + w.pre_acc_off) + at * w.pre_rows * acc_stride(D);
    for (int j = tid; j < g.nrows * D; j += WARPS * 32) {
      const int r = j / D, e = j % D;
      float a = 0.f;
#pragma unroll
      for (int v = 0; v < WARPS; ++v)
#pragma unroll
        for (int gg = 0; gg < V::kGroups; ++gg)
          a += reinterpret_cast<const float *>(smem + V::kStages * 16384 + v * V::kWarpBytes)[(gg * GE + r) * D + e];
      part[r * acc_stride(D) + e] = a;
    }
    if (tid < g.nrows) {
      float a = 0.f;
#pragma unroll
      for (int v = 0; v < WARPS; ++v)
#pragma unroll
        for (int gg = 0; gg < V::kGroups; ++gg) a += s_sum[v][gg * GE + tid];
      part[tid * acc_stride(D) + D] = a;
    }
    named_bar_sync(1, WARPS * 32);
  }
  if (!waited) {
    pdl_wait();
    pdl_launch_dependents();
  }
}

// ------------------------------------------------------------------ join
constexpr int kPgtCombThreads = 256;

// One block a row: thread (way, e) adds 4 columns of every WAYS-th piece, then
// the ways are added in order.
template <typename E, int D>
__global__ void __launch_bounds__(kPgtCombThreads) pgt_combine(PagedDecode p, PgtPlan w) {
  constexpr int COLS = D / 4, WAYS = kPgtCombThreads / COLS;
  __shared__ PgtLens L;
  __shared__ float4 s_a[WAYS][COLS];
  __shared__ float s_r[WAYS];
  const int tid = threadIdx.x, e = tid % COLS, way = tid / COLS;
  pgt_load_lens<kPgtCombThreads>(p, w, L, nullptr);
  const PgtLine line = pgt_line(p, w, L);
  const int s = blockIdx.x / p.c.Hq, hq = blockIdx.x % p.c.Hq;
  const PgtPieces pc = pgt_pieces(p, w, line, L, s, hq, true);
  const float *pre = reinterpret_cast<const float *>(p.ws + w.pre_acc_off) + pc.pre_row * acc_stride(D);
  const float *own = reinterpret_cast<const float *>(p.ws + w.own_acc_off) + pc.own_row * acc_stride(D);
  pdl_wait();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float rs = 0.f;
#pragma unroll 2
  for (int c = way; c < pc.npre + pc.nown; c += WAYS) {
    const float *pa = c < pc.npre ? pre + (size_t)(pc.pre0 + c) * w.pre_rows * acc_stride(D)
                                  : own + (size_t)(pc.own0 + c - pc.npre) * w.own_rows * acc_stride(D);
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(pa + 4 * e));
    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    rs += __ldcg(pa + D);
  }
  s_a[way][e] = a;
  if (e == 0) s_r[way] = rs;
  __syncthreads();
  if (tid < D) {
    const float *col = reinterpret_cast<const float *>(&s_a[0][0]) + tid;
    float sum = 0.f, tot = 0.f;
#pragma unroll
    for (int v = 0; v < WAYS; ++v) {
      sum += col[v * D];
      tot += s_r[v];
    }
    static_cast<E *>(p.out)[(size_t)blockIdx.x * D + tid] = (E)(L.len[s] > 0 ? sum / tot : 0.f);   // rounds to nearest
  }
}

cudaError_t launch_combine(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream) {
  const int grid = p.c.S * p.c.Hq;
  if (p.c.dtype == DA_BF16)
    return p.c.d == 128 ? launch_after(pgt_combine<__nv_bfloat16, 128>, grid, kPgtCombThreads, 0, stream, p, w)
                        : launch_after(pgt_combine<__nv_bfloat16, 64>, grid, kPgtCombThreads, 0, stream, p, w);
  return p.c.d == 128 ? launch_after(pgt_combine<float, 128>, grid, kPgtCombThreads, 0, stream, p, w)
                      : launch_after(pgt_combine<float, 64>, grid, kPgtCombThreads, 0, stream, p, w);
}

// ------------------------------------------------------------------ host
// paged_prefix_bf16.cu: the two passes over a prefix with many rows.
int launch_pgx_keys(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream);
int launch_pgx_values(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream);

size_t pgt_workspace(int S, int Hq, int Hkv, int d, int max_len, int prefix_len, int dtype) {
  if (S > kPgtMaxSeqs) S = kPgtMaxSeqs;
  // enough for either way of taking a prefix, so that the size depends on the prefix's presence alone
  const size_t a = pgt_plan(S, Hq, Hkv, d, max_len, prefix_len, 16, dtype, kPgxNever).total;
  const size_t b = pgt_plan(S, Hq, Hkv, d, max_len, prefix_len, 16, dtype, kPgxAlways).total;
  return a > b ? a : b;
}
// Units on the line at most (int arithmetic on the device).
bool pgt_fits(int S, int Hq, int Hkv, int d, int max_len, int prefix_len, int dtype) {
  if (S > kPgtMaxSeqs) S = kPgtMaxSeqs;
  const int64_t G = Hq / Hkv, tile = pgt_tile(d, dtype), rt = kPgtRowTile, rows = (S * G + kPgtPreRows - 1) / kPgtPreRows;
  const int64_t own = (max_len - prefix_len + tile - 1) / tile + kPgtHead;
  const int64_t pre = (prefix_len + tile - 1) / tile + kPgtHead;
  return S * (int64_t)Hkv * ((G + rt - 1) / rt) * own + (prefix_len > 0 ? Hkv * rows * pre : 0) < 0x7FFF0000ll;
}

template <int D, int GE>
static int launch_pgt_t(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream) {
  using V = PgtVal<D, GE>;
  constexpr int HH = GE > 8 ? 2 : 1;
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return (cudaFuncSetAttribute(pgt_keys<D, HH>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgtSmemPerCta) !=
                cudaSuccess ||
            cudaFuncSetAttribute(pgt_values<D, GE>, cudaFuncAttributeMaxDynamicSharedMemorySize, V::kSmemBytes) !=
                cudaSuccess)
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  CUtensorMap km, vm;
  const int64_t num = (int64_t)p.c.num_pages * p.c.Hkv;
  // an empty pool has no pages to map; every page id then fails its check, and no copy is issued
  if (!make_page_map(&km, p.c.k_pages, num > 0 ? num : 1, p.c.page_size, pgt_tile(D), D, DA_BF16) ||
      !make_page_map(&vm, p.c.v_pages, num > 0 ? num : 1, p.c.page_size, pgt_tile(D), D, DA_BF16))
    return DA_ERR_CUDA;
  // Stages of pgt_keys: 4 leave room for the next kernel's CTAs to begin beside
  // the last of this one.  A step with 4 / 6 stages, us: 8 x 12 x 131072 519 / 525,
  // three query heads a key head 204 / 206, 8 x 12 x 65536 at d = 128 499 / 502, 48
  // ragged at d = 128 38.3 / 39.0.  With a prefix its CTAs are few and short: 16 x 12 x
  // 2048 + 300 17.8 / 17.4, 64 x 12 x 131072 + 1000 261.2 / 260.9, 16 x 8192 + 300 with
  // shared heads 20.6 / 20.5, 32 x 16 heads x 32768 at d = 128 76.3 / 76.4, 8 x 12 x 16384
  // at d = 128 29.6 / 30.1.
  const int k_stages = p.prefix_len == 0 ? 4 : 6;
  constexpr int k_most = 1024 + 6 * kStageBytes;
  static_assert(k_most <= kPgtSmemPerCta, "two CTAs an SM");
  if (launch_after(pgt_keys<D, HH>, w.ctas, pgt_threads(D), 1024 + k_stages * kStageBytes, stream, p, w, km, k_stages) !=
      cudaSuccess)
    return DA_ERR_CUDA;
  if (w.wide) {
    const int st = launch_pgx_keys(p, w, stream);
    if (st != DA_OK) return st;
  }
  if (launch_after(pgt_values<D, GE>, w.ctas, V::kThreads, V::kSmemBytes, stream, p, w, vm) != cudaSuccess)
    return DA_ERR_CUDA;
  if (w.wide) {
    const int st = launch_pgx_values(p, w, stream);
    if (st != DA_OK) return st;
  }
  if (launch_combine(p, w, stream) != cudaSuccess)
    return DA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

template <int D>
static int launch_pgt_d(const PagedDecode &p, cudaStream_t stream) {
  const PgtPlan w = pgt_plan(p.c.S, p.c.Hq, p.c.Hkv, D, p.max_len, p.prefix_len, p.c.page_size, DA_BF16);
  int rows = w.own_rows;                                 // the most rows of a segment
  if (w.prefix_segs > 0) rows = p.c.S * w.G < w.pre_rows ? p.c.S * w.G : w.pre_rows;
  if (rows <= 1) return launch_pgt_t<D, 1>(p, w, stream);
  if (rows <= 2) return launch_pgt_t<D, 2>(p, w, stream);
  if (rows <= 4) return launch_pgt_t<D, 4>(p, w, stream);
  if (rows <= 8) return launch_pgt_t<D, 8>(p, w, stream);
  return launch_pgt_t<D, 16>(p, w, stream);
}

// paged_small_bf16.cu: short calls in one launch.
int small_cluster(int S, int Hq, int Hkv, int d, int max_len);
int launch_paged_small_bf16(const PagedDecode &p, int csize, cudaStream_t stream);
// paged_decode_f32.cu
int launch_paged_f32(const PagedDecode &p, cudaStream_t stream);

int launch_paged_decode(const PagedDecode &a, cudaStream_t stream) {
  const bool bf16 = a.c.dtype == DA_BF16;
  const int cluster = bf16 ? small_cluster(a.c.S, a.c.Hq, a.c.Hkv, a.c.d, a.max_len) : 0;
  if (cluster > 0) return launch_paged_small_bf16(a, cluster, stream);
  for (int s0 = 0; s0 < a.c.S; s0 += kPgtMaxSeqs) {   // the kernels keep the lengths of one part in shared memory
    PagedDecode p = a;
    const size_t rows = (size_t)s0 * a.c.Hq, skip = rows * a.c.d * (bf16 ? 2 : 4);
    p.c.S = a.c.S - s0 < kPgtMaxSeqs ? a.c.S - s0 : kPgtMaxSeqs;
    p.c.page_table += (size_t)s0 * a.c.max_pages;
    p.c.demand_table += (size_t)s0 * a.c.max_pages;
    p.c.seq_lens += s0;
    p.q = static_cast<const uint8_t *>(a.q) + skip;
    p.out = static_cast<uint8_t *>(a.out) + skip;
    if (a.hs.tau_bh != nullptr) p.hs.tau_bh = a.hs.tau_bh + rows;
    const int st = !bf16           ? launch_paged_f32(p, stream)
                   : a.c.d == 128 ? launch_pgt_d<128>(p, stream)
                                  : launch_pgt_d<64>(p, stream);
    if (st != DA_OK) return st;
  }
  return DA_OK;
}

}  // namespace da
