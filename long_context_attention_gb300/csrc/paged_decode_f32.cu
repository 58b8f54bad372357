// Decode step over the paged cache in fp32: streaming kernels on CUDA cores.
//
// The operator is that of decode.cu for sequences of different lengths whose keys
// and values are scattered over pages, with Hq / Hkv query heads sharing a key
// head and an optional prefix that the whole batch shares:
//   x_k = q . k_k tau / sqrt(d) log2 e,  p_k = 2^(x_k - lse2),
//   share_k = p_k / (D_k + p_k + eps),  out = sum share_k v_k / sum share_k,
//   D_k += p_k.
// Everything in fp32 (TF32 products would miss the type's accuracy).  The passes,
// the line of work, the page ring and the join are those of paged_decode_bf16.cu.
//
// What bounds it: HBM up to about 4 rows a key head, then the fp32 units and the
// shared-memory reads of the products.
//
// A warp takes 32 keys at a time.  pgf_keys: a lane forms the products of up to 4
// keys and 4 rows (16 rows: 8 lanes of keys by 4 of rows), so that 8 reads of 16
// bytes, one shared-memory cycle each, feed 32 packed multiply-adds.  (A key a lane
// and 8 rows a segment took 12 cycles for 16: 32 x 16 heads x 44928 keys, d = 128,
// 281 us, now 180; the step 554 and 391.)  pgf_values: shares by key, then by column: a lane owns d / 32
// columns of the numerators and walks the keys, 4 at a time, whose shares are
// broadcast.  4 x 12 x 4001 .. 16001 keys: 97 us with plain loads and no ring.
#include "da_paged_ring.cuh"

namespace da {

constexpr int kPgfSmemPerCta = 100 * 1024;   // two CTAs an SM
constexpr int kPgfWarps = 4;
constexpr int kPgfThreads = 32 * kPgfWarps + 32;

// A warp's steps: 32 keys of every kStride-th tile (see PgtVal on the ring).
template <int D>
struct PgfSteps {
  static constexpr int kTile = pgt_tile(D, DA_F32);   // 64 or 32 keys
  static constexpr int kPerTile = kTile / 32;
  static constexpr int kStride = kPgfWarps / kPerTile;
};

// Lanes of pgf_keys: kRowLanes of rows by kKeyLanes of keys.
template <int R>   // rows of a segment at most (1, 2, 4, 8, 16)
struct PgfBlock {
  static constexpr int kRowLanes = R > 4 ? R / 4 : 1, kKeyLanes = 32 / kRowLanes;
  static constexpr int kRows = R / kRowLanes, kKeys = 32 / kKeyLanes;   // of a lane: rows j kRowLanes + .., keys i kKeyLanes + ..
};

template <int D, int R>
__global__ void __launch_bounds__(kPgfThreads, 2)
    pgf_keys(PagedDecode p, PgtPlan w, const __grid_constant__ CUtensorMap kmap) {
  using T = PgfSteps<D>;
  using B = PgfBlock<R>;
  constexpr int TILE = T::kTile, STAGES = (kPgfSmemPerCta - 1024) / kStageBytes / T::kStride * T::kStride;
  static_assert(STAGES <= 8 && STAGES >= T::kStride, "ring");
  __shared__ PgtLens L;
  __shared__ PgtRing ring;
  __shared__ __align__(16) float s_q[R][D + 4];   // (padded: the lanes of different rows read different banks)
  __shared__ float s_c2[R];
  __shared__ float2 s_ml[kPgfWarps][R];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) ring.init(STAGES, T::kPerTile);
  pdl_wait();
  pdl_launch_dependents();
  pgt_load_lens<kPgfThreads>(p, w, L, blockIdx.x == 0 ? p.status : nullptr);
  const PgtLine line = pgt_line(p, w, L);
  const int from = line.cut.first(blockIdx.x), to = line.cut.first(blockIdx.x + 1);
  const WaitCtx wc{&ring.abort_word, p.status, p.dbg.limit_ns[kPagedKeys]};
  uint8_t *const smem = pgt_smem_base();
  if (warp == kPgfWarps) {
    produce<TILE, 32, true>(p, w, line, L, ring, &kmap, smem_u32(smem), STAGES, from, to, wc);
    return;
  }
  const bool keep = warp == 0 && (int)blockIdx.x == p.dbg.stall_block[kPagedKeys];   // test hook
  const int sub = warp % T::kPerTile * 32, kl = lane % B::kKeyLanes, rl = lane / B::kKeyLanes;
  PgtSeg g;
  for (g.start(p, w, line, L, from, to); g.n > 0; g.next(p, w, line, L)) {
    for (int i = tid; i < R * D; i += 32 * kPgfWarps) {
      const int r = i / D;
      float v = 0.f;
      if (r < g.nrows) {
        int s, hq;
        g.row(w.G, r, s, hq);
        v = static_cast<const float *>(p.q)[((size_t)s * p.c.Hq + hq) * D + i % D];
        if (i % D == 0) s_c2[r] = head_c2(p.hs, s * p.c.Hq + hq, p.status);
      }
      s_q[r][i % D] = v;
    }
    named_bar_sync(1, 32 * kPgfWarps);
    float m[B::kRows], l[B::kRows], *xrow[B::kRows];
#pragma unroll
    for (int j = 0; j < B::kRows; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.f;
      const int r = j * B::kRowLanes + rl;
      int s = 0, hq = 0;
      if (r < g.nrows) g.row(w.G, r, s, hq);
      xrow[j] = reinterpret_cast<float *>(p.ws + w.logit_off) + ((size_t)s * p.c.Hq + hq) * w.Lp;
    }
    const int tile0 = (warp / T::kPerTile + T::kStride - g.run % T::kStride) % T::kStride;
    int steps = g.n > tile0 ? (g.n - tile0 + T::kStride - 1) / T::kStride : 0;
    if (__any_sync(0xffffffffu, ring.abort_word != 0)) steps = 0;   // a wait gave up: touch no barrier again
    for (int k = 0; k < steps; ++k) {
      const int st = g.run + tile0 + k * T::kStride, slot = st % STAGES;
      if (!warp_wait(&ring.full[slot], (uint32_t)((st / STAGES) & 1), wc)) break;
      const int key = g.key0 + (tile0 + k * T::kStride) * TILE + sub + kl;   // the lane's first key
      if (key - kl < g.end) {
        const uint8_t *tile = smem + slot * kStageBytes;
        float2 acc[B::kKeys][B::kRows];
#pragma unroll
        for (int i = 0; i < B::kKeys; ++i)
#pragma unroll
          for (int j = 0; j < B::kRows; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int c = 0; c < D / 4; ++c) {
          float4 kv[B::kKeys];
#pragma unroll
          for (int i = 0; i < B::kKeys; ++i)
            kv[i] = *reinterpret_cast<const float4 *>(tile + tile_off<TILE>(sub + kl + i * B::kKeyLanes, c));
#pragma unroll
          for (int j = 0; j < B::kRows; ++j) {
            const float4 qv = *reinterpret_cast<const float4 *>(&s_q[j * B::kRowLanes + rl][4 * c]);
#pragma unroll
            for (int i = 0; i < B::kKeys; ++i) {
              acc[i][j] = ffma2(make_float2(kv[i].x, kv[i].y), make_float2(qv.x, qv.y), acc[i][j]);
              acc[i][j] = ffma2(make_float2(kv[i].z, kv[i].w), make_float2(qv.z, qv.w), acc[i][j]);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < B::kRows; ++j) {
          const int r = j * B::kRowLanes + rl;
          if (r >= g.nrows) break;
          const float c2 = s_c2[r];
          float x[B::kKeys], mn = m[j];
#pragma unroll
          for (int i = 0; i < B::kKeys; ++i) {
            const bool in = key + i * B::kKeyLanes < g.end;
            x[i] = in ? (acc[i][j].x + acc[i][j].y) * c2 : -INFINITY;
            if (in) xrow[j][key + i * B::kKeyLanes] = x[i];
            mn = fmaxf(mn, x[i]);
          }
          const float ms = mn == -INFINITY ? 0.f : mn;
          l[j] *= ex2_approx(m[j] - ms);
#pragma unroll
          for (int i = 0; i < B::kKeys; ++i) l[j] += ex2_approx(x[i] - ms);
          m[j] = mn;
        }
      }
      __syncwarp();
      if (lane == 0 && !(keep && k == 0)) mbar_arrive(&ring.empty[slot]);
    }
#pragma unroll
    for (int j = 0; j < B::kRows; ++j) {
#pragma unroll
      for (int o = B::kKeyLanes / 2; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m[j], o), l2 = __shfl_xor_sync(0xffffffffu, l[j], o);
        const float mn = fmaxf(m[j], m2), ms = mn == -INFINITY ? 0.f : mn;
        l[j] = l[j] * ex2_approx(m[j] - ms) + l2 * ex2_approx(m2 - ms);
        m[j] = mn;
      }
      if (kl == 0) s_ml[warp][j * B::kRowLanes + rl] = make_float2(m[j], l[j]);
    }
    named_bar_sync(1, 32 * kPgfWarps);
    if (tid < g.nrows) {
      float M = -INFINITY, S = 0.f;
#pragma unroll
      for (int v = 0; v < kPgfWarps; ++v) M = fmaxf(M, s_ml[v][tid].x);
      const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int v = 0; v < kPgfWarps; ++v) S += s_ml[v][tid].y * ex2_approx(s_ml[v][tid].x - ms);
      const size_t at = (size_t)blockIdx.x + g.seg;
      float2 *ml = g.s >= 0 ? reinterpret_cast<float2 *>(p.ws + w.own_ml_off) + at * w.own_rows
                            : reinterpret_cast<float2 *>(p.ws + w.pre_ml_off) + at * w.pre_rows;
      ml[tid] = make_float2(M, S);
    }
    named_bar_sync(1, 32 * kPgfWarps);
  }
}

// Each warp brings the logits and demand of its next step by 16-byte asynchronous
// copies into its own place, [row][32 keys] of each, two steps in turn; the shares
// take the logits' place, and the new demand goes back from the demand's.  16 rows
// are two warps' work, each with 8 rows of the same 32 keys: one warp's numerators of
// 16 rows do not fit the registers (32 x 16 heads x 44928, d = 128: 373 us with
// spills, 231 us so).
template <int D, int R>
struct PgfVal {
  static constexpr int kRows = R > 8 ? 8 : R;                       // of a warp
  static constexpr int kTile = pgt_tile(D, DA_F32), kSubs = kTile / 32;
  static constexpr int kPerTile = kSubs * (R / kRows);              // warps of a tile: by rows, then by keys
  static constexpr int kStride = kPgfWarps / kPerTile;              // tiles between a warp's steps (see PgtVal on the ring)
  static constexpr int kSide = 2 * 2 * kRows * 32 * 4;              // a warp's logits and demand, two steps
  static constexpr int kRed = kRows * D * 4;                        // its numerators, afterwards
  static constexpr int kWarpBytes = kSide > kRed ? kSide : kRed;
  static constexpr int kRoom = (kPgfSmemPerCta - 1024 - kPgfWarps * kWarpBytes) / kStageBytes;
  static constexpr int kStages = (kRoom < 8 ? kRoom : 8) / kStride * kStride;
  static_assert(kStages >= 2 && kStages >= kStride, "a slot for every warp");
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kPgfWarps * kWarpBytes;
};

template <int D, int ROWS>   // of a segment at most
__global__ void __launch_bounds__(kPgfThreads, 2)
    pgf_values(PagedDecode p, PgtPlan w, const __grid_constant__ CUtensorMap vmap) {
  using V = PgfVal<D, ROWS>;
  constexpr int R = V::kRows, TILE = V::kTile, STRIDE = V::kStride * TILE, NC = D / 32;   // NC: columns of a lane
  constexpr int PIECES = (R * 8 + 31) / 32;                                 // 16-byte pieces of a lane (rows x 8)
  __shared__ PgtLens L;
  __shared__ PgtRing ring;
  __shared__ float s_lse[ROWS];
  __shared__ float s_sum[kPgfWarps][R];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) ring.init(V::kStages, V::kPerTile);
  pgt_load_lens<kPgfThreads>(p, w, L, nullptr);
  const PgtLine line = pgt_line(p, w, L);
  const int from = line.cut.first(blockIdx.x), to = line.cut.first(blockIdx.x + 1);
  const WaitCtx wc{&ring.abort_word, p.status, p.dbg.limit_ns[kPagedValues]};
  uint8_t *const smem = pgt_smem_base();
  if (warp == kPgfWarps) {   // the values do not depend on the first pass
    produce<TILE, 32, false>(p, w, line, L, ring, &vmap, smem_u32(smem), V::kStages, from, to, wc);
    return;
  }
  uint8_t *const base = smem + V::kStages * kStageBytes;
  float *const mine = reinterpret_cast<float *>(base + warp * V::kWarpBytes);   // [2 steps][x, D][R][32]
  const int sh = w.page_shift, ps = 1 << sh, sub = warp % V::kSubs * 32;
  const int r0 = warp % V::kPerTile / V::kSubs * R;   // the warp's first row
  const bool keep = warp == 0 && (int)blockIdx.x == p.dbg.stall_block[kPagedValues];   // test hook
  const int pr = lane / 8, pk = 4 * (lane % 8);       // the lane's pieces: rows pr, pr + 4 of the warp's, keys pk .. of a step
  // byte offsets of the lane's columns in a tile, for key & 7 = 0 .. 7
  uint32_t col[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = lane * NC * 4 / 16;   // its 16-byte piece
    col[j] = (uint32_t)((c >> 3) * TILE * 128 + (((c & 7) ^ j) << 4) + (NC == 2 ? (lane & 1) * 8 : 0));
  }
  bool waited = false;
  PgtSeg g;
  for (g.start(p, w, line, L, from, to); g.n > 0; g.next(p, w, line, L)) {
    const int tile0 = (warp / V::kPerTile + V::kStride - g.run % V::kStride) % V::kStride;
    int steps = g.n > tile0 ? (g.n - tile0 + V::kStride - 1) / V::kStride : 0;
    if (__any_sync(0xffffffffu, ring.abort_word != 0)) steps = 0;   // a wait gave up: touch no barrier again
    const int step0 = g.key0 + tile0 * TILE + sub;                  // the warp's first key
    // the lane's pieces
    const float *xrow[PIECES];
    const int32_t *dtab[PIECES];
    float *dpool[PIECES];
    bool on[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int r = r0 + pr + 4 * i;
      int s = 0, hq = 0;
      on[i] = pr + 4 * i < R && r < g.nrows;
      if (on[i]) g.row(w.G, r, s, hq);
      on[i] = on[i] && L.len[s] > 0;   // an idle slot bids nothing
      xrow[i] = reinterpret_cast<const float *>(p.ws + w.logit_off) + ((size_t)s * p.c.Hq + hq) * w.Lp;
      dtab[i] = p.c.demand_table + (size_t)s * p.c.max_pages;
      dpool[i] = p.c.demand_pages + ((size_t)hq << sh);
    }
    auto demand_page = [&](int k, int i, bool after_wait) -> int {
      const int key = step0 + k * STRIDE + pk;
      const int32_t *at = dtab[i] + (key >> sh);
      return on[i] && k < steps && key < g.end ? (after_wait ? *at : __ldcg(at)) : -1;
    };
    auto bring = [&](int k, const int (&pg)[PIECES]) {
      float *x = mine + (k & 1) * (2 * R * 32);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int key = step0 + k * STRIDE + pk;
        if (on[i] && k < steps && key < g.end) {
          float *to = x + (pr + 4 * i) * 32 + pk;
          cp_async16(to, xrow[i] + key);
          if ((unsigned)pg[i] < (unsigned)p.c.num_demand_pages)
            cp_async16(to + R * 32, dpool[i] + (((size_t)pg[i] * p.c.Hq) << sh) + (key & (ps - 1)));
          else
            atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int pages[2][PIECES];   // demand pages of steps k and k + 1
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int i = 0; i < PIECES; ++i) pages[a][i] = demand_page(a, i, waited);
    if (!waited) {   // the demand does not depend on the first pass: to L2 meanwhile
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if ((unsigned)pages[0][i] < (unsigned)p.c.num_demand_pages)
          prefetch_l2(dpool[i] + (((size_t)pages[0][i] * p.c.Hq) << sh) + ((step0 + pk) & (ps - 1)));
      pdl_wait();
      pdl_launch_dependents();
      waited = true;
    }
    bring(0, pages[0]);
    // lse2 of the rows: 8 lanes join a row's pieces
    for (int r4 = warp * 4; r4 < g.nrows; r4 += kPgfWarps * 4) {
      const int r = r4 + lane / 8;
      int s = 0, hq = 0;
      g.row(w.G, min(r, g.nrows - 1), s, hq);
      const float v = pgt_row_lse<8>(p, w, line, L, s, hq, lane);
      if (lane % 8 == 0 && r < g.nrows) s_lse[r] = L.len[s] > 0 ? v : INFINITY;
    }
    named_bar_sync(1, 32 * kPgfWarps);
    float num[R][NC], sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sum[r] = 0.f;
#pragma unroll
      for (int e = 0; e < NC; ++e) num[r][e] = 0.f;
    }
    for (int k = 0; k < steps; ++k) {
      bring(k + 1, pages[1]);
      int next[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; ++i) next[i] = demand_page(k + 2, i, true);
      asm volatile("cp.async.wait_group 1;" ::: "memory");   // step k's have landed
      __syncwarp();
      float *x = mine + (k & 1) * (2 * R * 32), *dm = x + R * 32;
      const int left = g.end - (step0 + k * STRIDE);          // keys of the step before the end
      const bool in = lane < left;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r0 + r >= g.nrows) break;
        const float lse = s_lse[r0 + r];
        float share = 0.f;
        if (in && lse != INFINITY) {
          const float bid = ex2_approx(x[r * 32 + lane] - lse), d = dm[r * 32 + lane], nd = d + bid;
          dm[r * 32 + lane] = nd;
          share = bid / ((p.earlier ? d : nd) + p.eps);
        }
        x[r * 32 + lane] = share;
        sum[r] += share;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if ((unsigned)pages[0][i] < (unsigned)p.c.num_demand_pages) {   // (-1 where there is nothing)
          const int key = step0 + k * STRIDE + pk;
          const float4 v = *reinterpret_cast<const float4 *>(dm + (pr + 4 * i) * 32 + pk);
          float *to = dpool[i] + (((size_t)pages[0][i] * p.c.Hq) << sh) + (key & (ps - 1));
          if (pk + 4 <= left) {
            *reinterpret_cast<float4 *>(to) = v;
          } else {
            const float e4[3] = {v.x, v.y, v.z};
#pragma unroll
            for (int e = 0; e < 3; ++e)
              if (pk + e < left) to[e] = e4[e];
          }
        }
        pages[0][i] = pages[1][i];
        pages[1][i] = next[i];
      }
      const int st = g.run + tile0 + k * V::kStride, slot = st % V::kStages;
      if (!warp_wait(&ring.full[slot], (uint32_t)((st / V::kStages) & 1), wc)) break;
      const uint8_t *tile = smem + slot * kStageBytes + sub * 128;
      // columns: 4 keys at a time (rows past the end are left out: they may hold anything)
      auto take = [&](int key, const float (&sv)[R], uint32_t at) {
        float v[NC];
        if constexpr (NC == 2) {
          const float2 t2 = *reinterpret_cast<const float2 *>(tile + key * 128 + at);
          v[0] = t2.x, v[1] = t2.y;
        } else {
          const float4 t4 = *reinterpret_cast<const float4 *>(tile + key * 128 + at);
          v[0] = t4.x, v[1] = t4.y, v[NC - 2] = t4.z, v[NC - 1] = t4.w;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < NC; e += 2) {
            const float2 n2 = ffma2(make_float2(sv[r], sv[r]), make_float2(v[e], v[e + 1]), make_float2(num[r][e], num[r][e + 1]));
            num[r][e] = n2.x, num[r][e + 1] = n2.y;
          }
      };
      if (left >= 32) {
#pragma unroll
        for (int k4 = 0; k4 < 32; k4 += 4) {
          float4 sv[R];
#pragma unroll
          for (int r = 0; r < R; ++r)
            sv[r] = r0 + r < g.nrows ? *reinterpret_cast<const float4 *>(x + r * 32 + k4) : make_float4(0.f, 0.f, 0.f, 0.f);
          float s0[R], s1[R], s2[R], s3[R];
#pragma unroll
          for (int r = 0; r < R; ++r) s0[r] = sv[r].x, s1[r] = sv[r].y, s2[r] = sv[r].z, s3[r] = sv[r].w;
          take(k4, s0, col[k4 & 7]);
          take(k4 + 1, s1, col[(k4 + 1) & 7]);
          take(k4 + 2, s2, col[(k4 + 2) & 7]);
          take(k4 + 3, s3, col[(k4 + 3) & 7]);
        }
      } else {
#pragma unroll 1
        for (int kk = 0; kk < left; ++kk) {
          float sv[R];
#pragma unroll
          for (int r = 0; r < R; ++r) sv[r] = r0 + r < g.nrows ? x[r * 32 + kk] : 0.f;
          const int c = lane * NC * 4 / 16;
          take(kk, sv,
               (uint32_t)((c >> 3) * TILE * 128 + (((c & 7) ^ (kk & 7)) << 4) + (NC == 2 ? (lane & 1) * 8 : 0)));
        }
      }
      __syncwarp();
      if (lane == 0 && !(keep && k == 0)) mbar_arrive(&ring.empty[slot]);
    }
    cp_async_wait_all();
    __syncwarp();
    // the piece's numerators and share sums, over the warps in order
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < NC; ++e) mine[r * D + lane * NC + e] = num[r][e];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
      if (lane == 0) s_sum[warp][r] = sum[r];
    }
    named_bar_sync(1, 32 * kPgfWarps);
    const size_t at = (size_t)blockIdx.x + g.seg;
    float *part = g.s >= 0 ? reinterpret_cast<float *>(p.ws + w.own_acc_off) + at * w.own_rows * acc_stride(D)
                           : reinterpret_cast<float *>(p.ws + w.pre_acc_off) + at * w.pre_rows * acc_stride(D);
    for (int j = tid; j < g.nrows * D; j += 32 * kPgfWarps) {
      float a = 0.f;
#pragma unroll
      for (int v = 0; v < kPgfWarps; ++v)
        if (R == ROWS || v % V::kPerTile / V::kSubs == j / D / R)   // the warps of the row
          a += reinterpret_cast<const float *>(base + v * V::kWarpBytes)[j % (R * D)];
      part[j / D * acc_stride(D) + j % D] = a;
    }
    if (tid < g.nrows) {
      float a = 0.f;
#pragma unroll
      for (int v = 0; v < kPgfWarps; ++v)
        if (R == ROWS || v % V::kPerTile / V::kSubs == tid / R) a += s_sum[v][tid % R];
      part[tid * acc_stride(D) + D] = a;
    }
    named_bar_sync(1, 32 * kPgfWarps);
  }
  if (!waited) {
    pdl_wait();
    pdl_launch_dependents();
  }
}

cudaError_t launch_combine(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream);   // paged_decode_bf16.cu

template <int D, int R>
static int launch_pgf_t(const PagedDecode &p, const PgtPlan &w, cudaStream_t stream) {
  using T = PgfSteps<D>;
  constexpr int k_smem = 1024 + (kPgfSmemPerCta - 1024) / kStageBytes / T::kStride * T::kStride * kStageBytes;
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return (cudaFuncSetAttribute(pgf_keys<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, k_smem) != cudaSuccess ||
            cudaFuncSetAttribute(pgf_values<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PgfVal<D, R>::kSmemBytes) != cudaSuccess)
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  CUtensorMap km, vm;
  const int64_t num = (int64_t)p.c.num_pages * p.c.Hkv;
  // an empty pool has no pages to map; every page id then fails its check, and no copy is issued
  if (!make_page_map(&km, p.c.k_pages, num > 0 ? num : 1, p.c.page_size, T::kTile, D, DA_F32) ||
      !make_page_map(&vm, p.c.v_pages, num > 0 ? num : 1, p.c.page_size, T::kTile, D, DA_F32))
    return DA_ERR_CUDA;
  if (launch_after(pgf_keys<D, R>, w.ctas, kPgfThreads, k_smem, stream, p, w, km) != cudaSuccess ||
      launch_after(pgf_values<D, R>, w.ctas, kPgfThreads, PgfVal<D, R>::kSmemBytes, stream, p, w, vm) != cudaSuccess ||
      launch_combine(p, w, stream) != cudaSuccess)
    return DA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

template <int D>
static int launch_pgf_d(const PagedDecode &p, cudaStream_t stream) {
  const PgtPlan w = pgt_plan(p.c.S, p.c.Hq, p.c.Hkv, D, p.max_len, p.prefix_len, p.c.page_size, DA_F32);
  int rows = w.own_rows;   // the most rows of a segment
  if (w.prefix_segs > 0) rows = p.c.S * w.G < kPgtRowTile ? p.c.S * w.G : kPgtRowTile;
  if (rows <= 1) return launch_pgf_t<D, 1>(p, w, stream);
  if (rows <= 2) return launch_pgf_t<D, 2>(p, w, stream);
  if (rows <= 4) return launch_pgf_t<D, 4>(p, w, stream);
  if (rows <= 8) return launch_pgf_t<D, 8>(p, w, stream);
  return launch_pgf_t<D, 16>(p, w, stream);
}

int launch_paged_f32(const PagedDecode &p, cudaStream_t stream) {
  return p.c.d == 128 ? launch_pgf_d<128>(p, stream) : launch_pgf_d<64>(p, stream);
}

}  // namespace da
