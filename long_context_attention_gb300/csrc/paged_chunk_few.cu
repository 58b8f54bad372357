// Chunks of few rows over the paged cache in bf16: the second pass over kept logits.
//
// Mathematics: as paged_chunk_f32.cu.  A share enters the product as two bf16 terms (2^-16
// of itself, as in a decode step; one would double the output's rounding error), and the
// sums are those of the terms.
//
// What bounds it: HBM.  A key head's group has few rows (drafted tokens), so that the
// cache is read for little work, and half of what the kernel for many rows reads is K,
// for the logits that the first pass has had.  Here that pass keeps them (ckx_keys), 4
// bytes a row and key for K's 2 d.  A warp works alone, on every kWarps-th 32 keys: their
// values, logits and totals are copied asynchronously a step ahead; a lane has a key for
// bids, shares and totals; m16n8k16 forms share^T V (tcgen05's 128 rows would be mostly
// padding).  The warps' sums meet at a piece's end, in their order.
// 8 x 12 x 131072, 4 tokens, d = 64: 307 us, 6.2 TB/s of values, logits and totals;
// the first pass 288, 6.3 TB/s of keys and logits.
#include "da_chunk.cuh"
#include "da_paged_plan.cuh"

#include <cuda_bf16.h>

namespace da {

constexpr long long kChunkLogitBytes = 2ll << 30;
constexpr int kCklKeys = 32;   // of a step

template <int D, int ROWS>
struct Ckl {
  static constexpr int kWarps = D == 64 ? 16 : ROWS == 8 ? 10 : 8;     // what shared memory holds (16 of 8: 300 us for 557)
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kOffX = kCklKeys * D * 2;                       // a stage: values, logits, totals
  static constexpr int kOffT = kOffX + ROWS * kCklKeys * 4;
  static constexpr int kStage = kOffT + ROWS * kCklKeys * 4;
  static constexpr int kShRow = 80;                                    // bytes of a row of shares: 8 rows on all banks
  static constexpr int kShRows = 2 * ROWS;                             // their first terms, their second: up to 8 in one operand
  static constexpr int kWarp = 2 * kStage + kShRows * kShRow;
  static constexpr int kSmemBytes = kWarps * kWarp;
  static constexpr int kLd = D + 4;                                    // floats of a row of a warp's sums
  static_assert(kSmemBytes <= 231424 && ROWS * kLd * 4 <= kWarp, "shared memory");
};

// Whether a call's logits are kept: a key head's group has at most d / 8 rows, whose
// logits, written and read, are half of the bytes of K, and they take at most 2 GB of
// workspace.  Times in us of both second passes' calls (sequences x query / key heads x
// keys, new tokens; kept / not):
//   d = 64, 8 x 12/12 x 131072: 1 565 / 853, 4 612 / 857, 8 703 / 861; past the bound 16 1167 / 844;
//     8 x 12/4 x 32768: 1 93 / 129, 2 98 / 128; past the bound 5 (15 rows) 140 / 138;
//     64 x 12/12 x 4096: 4 199 / 275; past the bound 16 337 / 281; 1 x 12/12 x 16384: 4 42 / 50;
//   d = 128, 8 x 16/4 x 131072: 4 (16 rows) 575 / 648; 4 x 32/2 x 65536: 1 (16 rows) 143 / 251.
// (Past the bound: before shares had second terms.)
bool chunk_few(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len) {
  const long long tokens = N < (long long)S * max_new ? N : (long long)S * max_new;   // (more are padding)
  return max_new > 0 && (long long)(Hq / Hkv) * max_new * 8 <= d &&
         tokens * Hq * round_up(max_len, kChunkLogits) * 4 <= kChunkLogitBytes;
}
// Their room in a workspace that serves all calls within these bounds: of those with
// the most tokens and rows that keep them.
size_t chunk_few_room(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len, long long &tokens, int &most) {
  const int rows = d / 8 / (Hq / Hkv);
  most = max_new < rows ? max_new : rows;
  tokens = N < (long long)S * most ? N : (long long)S * most;
  const long long bytes = tokens * Hq * round_up(max_len, kChunkLogits) * 4;
  return (size_t)(bytes < kChunkLogitBytes ? bytes : kChunkLogitBytes);
}

template <int D, int ROWS>
__global__ void __launch_bounds__(Ckl<D, ROWS>::kThreads, 1) ckl_values(PagedChunk p, ChunkPlan w) {
  using C = Ckl<D, ROWS>;
  constexpr int PP = D / 8;   // 16-byte pieces of a row of V
  extern __shared__ __align__(128) uint8_t ckl_smem[];
  __shared__ float2 s_row[ROWS];       // scale, -lse2
  __shared__ uint64_t s_logits[ROWS];  // the row's logits
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  uint8_t *stages = ckl_smem + warp * C::kWarp, *shares = stages + 2 * C::kStage;
  const int sh = w.page_shift, ps = 1 << sh, G = w.G;
  const int ar = (lane & 7) + ((lane >> 3) & 1) * 8, ap = lane >> 4;   // of the products' operands: rows (keys), halves of 16
  auto piece = [](int r, int i) { return (uint32_t)((r * PP + (i ^ (r & 7))) << 4); };
  pdl_wait();
  pdl_launch_dependents();
  const ChunkLine l = chunk_line(p, w);
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_values);
  ChunkWalk k;
  for (k.start(p, w, l, cut, lane); k.any(); k.next(p, w, l)) {
    const int n = k.g.n, n8 = k.g.n8, R = G * n, hkv = k.seg, hq0 = hkv * G, P = k.g.P;
    const int key0 = k.tile * kChunkLogits, key1 = min(k.end * kChunkLogits, k.g.len), steps = (key1 - key0 + kCklKeys - 1) / kCklKeys;
    const long long row0 = k.row0(p, w);
    __syncthreads();   // the sums of the piece before have been read
    if (tid < R) {
      const int h = tid / n, q = tid % n;
      s_row[tid] = make_float2(fmaxf(head_c2(p.hs, k.s * p.c.Hq + hq0 + h, nullptr), 1e-30f),
                               __ldcg(reinterpret_cast<const float *>(p.ws + w.nl) + row0 + h * n8 + q));
      s_logits[tid] = reinterpret_cast<uint64_t>(chunk_logits(p, w, k.s, k.q.tok0, q, hq0 + h));
    }
    const bool odd = __ldcg(chunk_odd(p, w) + k.s) != 0;
    for (int e = lane; e < C::kShRows * C::kShRow / 4; e += 32) reinterpret_cast<uint32_t *>(shares)[e] = 0u;   // rows from R on stay 0
    __syncthreads();
    const int32_t *vtab = p.c.page_table + (size_t)k.s * p.c.max_pages, *dtab = p.c.demand_table + (size_t)k.s * p.c.max_pages;
    // this lane's key of step j: its pages
    int vpage = -1, dpage = -1;
    auto find = [&](int j) {
      const int key = key0 + j * kCklKeys + lane;
      vpage = dpage = -1;
      if (j < steps && key < key1) {
        vpage = __ldcg(vtab + (key >> sh));
        dpage = __ldcg(dtab + (key >> sh));
      }
    };
    auto copy = [&](int j, int st) {
      const uint32_t to = smem_u32(stages + st * C::kStage);
      const int first = key0 + j * kCklKeys, key = first + lane;
      const bool okv = (unsigned)vpage < (unsigned)p.c.num_pages, okd = (unsigned)dpage < (unsigned)p.c.num_demand_pages;
      if (key < key1 && !(okv && okd)) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      const uint64_t v = okv ? reinterpret_cast<uint64_t>(static_cast<const __nv_bfloat16 *>(p.c.v_pages) +
                                                          ((((size_t)vpage * p.c.Hkv + hkv) << sh) + (key & (ps - 1))) * D)
                             : 0;
      const uint64_t t = okd ? reinterpret_cast<uint64_t>(p.c.demand_pages + ((((size_t)dpage * p.c.Hq + hq0) << sh) + (key & (ps - 1))))
                             : 0;
#pragma unroll
      for (int u = 0; u < PP; ++u) {
        const int e = lane + 32 * u, r = e / PP, i = e % PP;
        const uint64_t from = __shfl_sync(0xffffffffu, v, r);
        cp_async16_fill(to + piece(r, i), reinterpret_cast<const void *>(from ? from + 16 * i : reinterpret_cast<uint64_t>(p.c.v_pages)), from != 0);
      }
      for (int r = lane / 8; r < R; r += 4)   // keys 4 (lane % 8) ..
        cp_async16_fill(to + C::kOffX + (r * 8 + lane % 8) * 16, reinterpret_cast<const void *>(s_logits[r] + 4 * first + lane % 8 * 16), true);
      // a page holds all keys of four
      const uint64_t four = __shfl_sync(0xffffffffu, t, lane % 8 * 4);
      for (int h = lane / 8; h < G; h += 4)
        cp_async16_fill(to + C::kOffT + (h * 8 + lane % 8) * 16,
                 reinterpret_cast<const void *>(four ? four + ((uint64_t)h << sh) * 4 : reinterpret_cast<uint64_t>(p.c.demand_pages)), four != 0);
    };
    float acc[D / 8][4], sums[ROWS];
#pragma unroll
    for (int e = 0; e < D / 8; ++e) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) sums[r] = 0.f;
    find(warp);
    if (warp < steps) copy(warp, 0);
    int page = dpage, st = 0;   // of the totals of the step at hand
    find(warp + C::kWarps);
    for (int j = warp; j < steps; j += C::kWarps) {
      const int key = key0 + j * kCklKeys + lane;
      uint8_t *now = stages + st * C::kStage;
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (odd && key0 + (j + 1) * kCklKeys > P) {   // the lane's own copies: no new token's values but finite ones
#pragma unroll 1
        for (int e = lane; e < kCklKeys * PP; e += 32) {
          uint4 *v = reinterpret_cast<uint4 *>(now + piece(e / PP, e % PP));
          uint4 x = *v;
          if (key0 + j * kCklKeys + e / PP >= P && chunk_clear(x, true)) *v = x;
        }
      }
      __syncwarp();   // the step's copies are there, and the step before has been read
      if (j + C::kWarps < steps) copy(j + C::kWarps, st ^ 1);
      float *at = (unsigned)page < (unsigned)p.c.num_demand_pages
                      ? p.c.demand_pages + ((((size_t)page * p.c.Hq + hq0) << sh) + (key & (ps - 1)))
                      : nullptr;
      page = dpage;
      find(j + 2 * C::kWarps);
      st ^= 1;
      const float *x = reinterpret_cast<const float *>(now + C::kOffX) + lane, *t = reinterpret_cast<const float *>(now + C::kOffT) + lane;
      float held = 0.f, added = 0.f;   // the rows' bids, summed apart from the total: it would take their last bits
      int h = 0, q = 0;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (r >= R) break;
        if (q == 0) held = key < key1 ? t[h * kCklKeys] : 0.f, added = 0.f;
        const float2 row = s_row[r];
        const float bid = key < key1 && key <= P + q ? ex2_approx(fmaf(x[r * kCklKeys], row.x, row.y)) : 0.f, before = added;
        added += bid;
        const float share = bid * rcp_approx(held + p.eps + (p.earlier ? before : added));
        const __nv_bfloat16 hi = __float2bfloat16_rn(share), lo = __float2bfloat16_rn(share - __bfloat162float(hi));
        *reinterpret_cast<__nv_bfloat16 *>(shares + r * C::kShRow + 2 * lane) = hi;
        *reinterpret_cast<__nv_bfloat16 *>(shares + (ROWS + r) * C::kShRow + 2 * lane) = lo;
        sums[r] += __bfloat162float(hi) + __bfloat162float(lo);
        if (++q == n) {
          if (at != nullptr) __stcg(at + ((size_t)h << sh), held + added);
          q = 0;
          ++h;
        }
      }
      __syncwarp();
#pragma unroll
      for (int ks = 0; ks < kCklKeys / 16; ++ks) {
        uint32_t a[4], a2[4];
        ldsm_x4(smem_u32(shares) + ar * C::kShRow + (2 * ks + ap) * 16, a);
        if constexpr (ROWS == 16) ldsm_x4(smem_u32(shares) + (16 + ar) * C::kShRow + (2 * ks + ap) * 16, a2);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t v[4];
          ldsm_x4_t(smem_u32(now) + piece(16 * ks + ar, 2 * c + ap), v);
          mma16816(acc[2 * c], a, v[0], v[1]);
          mma16816(acc[2 * c + 1], a, v[2], v[3]);
          if constexpr (ROWS == 16) {
            mma16816(acc[2 * c], a2, v[0], v[1]);
            mma16816(acc[2 * c + 1], a2, v[2], v[3]);
          }
        }
      }
      // (the next step's shares are written after its __syncwarp)
    }
    __syncwarp();   // (all copies have been waited for and read)
    float *mine = reinterpret_cast<float *>(stages);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      float *to = mine + lane / 4 * C::kLd + c * 8 + 2 * (lane % 4);
      if constexpr (ROWS == 16) {
        *reinterpret_cast<float2 *>(to) = make_float2(acc[c][0], acc[c][1]);
        *reinterpret_cast<float2 *>(to + 8 * C::kLd) = make_float2(acc[c][2], acc[c][3]);
      } else {
        *reinterpret_cast<float2 *>(to) = make_float2(acc[c][0] + acc[c][2], acc[c][1] + acc[c][3]);
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sums[r] += __shfl_xor_sync(0xffffffffu, sums[r], o);
      if (lane == 0) mine[r * C::kLd + D] = sums[r];
    }
    __syncthreads();
    float *to = chunk_place(p, w.acc_a, w.acc_b, row0, w.cta_rows, k.tile, blockIdx.x, 0, acc_stride(D));
    for (int e = tid; e < R * (D + 1); e += C::kThreads) {
      const int r = e / (D + 1), c = e % (D + 1), at = r / n * n8 + r % n;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < C::kWarps; ++i) sum += reinterpret_cast<const float *>(ckl_smem + i * C::kWarp)[r * C::kLd + c];
      to[c < D ? chunk_acc(D, at, c / 4) + c % 4 : chunk_acc_sum(D, at)] = sum;
    }
  }
}

template <int D, int ROWS>
static cudaError_t launch_ckl(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  using C = Ckl<D, ROWS>;
  static PerDeviceOnce once;
  if (once.run([] {
        return cudaFuncSetAttribute(ckl_values<D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) == cudaSuccess
                   ? DA_OK
                   : DA_ERR_CUDA;
      }) != DA_OK)
    return cudaErrorUnknown;
  return launch_after(ckl_values<D, ROWS>, w.ctas_values, C::kThreads, C::kSmemBytes, stream, p, w);
}
cudaError_t launch_chunk_few(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  if (p.c.d == 64) return launch_ckl<64, 8>(p, w, stream);
  return w.G * p.max_new <= 8 ? launch_ckl<128, 8>(p, w, stream) : launch_ckl<128, 16>(p, w, stream);
}

}  // namespace da
