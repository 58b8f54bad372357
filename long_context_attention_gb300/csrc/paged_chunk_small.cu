// Short chunks over the paged cache: one launch.
//
// Mathematics: as paged_chunk_f32.cu.  What bounds the call is latency: its five
// kernels take 32 us for 5 tokens x 12 heads x 500 keys (1.6 MB).  Here a cluster of up
// to 8 CTAs takes a (sequence, key head), 256 keys a CTA at most and up to 64 rows (the
// group's query heads by the new tokens, n8 rows a head); in fp32 128 keys and 32 rows:
//   keys, values and queries come into shared memory; S = Q K^T by m16n8k16
//   products, the logits stay in shared memory; every row's (max, sum) goes through
//   distributed shared memory; one thread a key walks the rows of each head with its
//   total; the shares, each as two bf16 terms (2^-16 of itself; one would double the
//   output's rounding error, as in a decode step), times V; the CTAs' numerators and sums
//   are added in the CTAs' order by the CTA that writes them.
// m16n8k16 and not tcgen05: the products are 1 % of the call.  fp32: all of it on CUDA
// cores, 4 rows by 4 keys, or columns, a thread.
#include "da_chunk.cuh"
#include "da_paged_plan.cuh"

#include <cuda_bf16.h>

namespace da {

constexpr int kCksKeys = 256, kCksRows = 64, kCksThreads = 256, kCksWarps = 8, kCksCluster = 8;
constexpr int kCksKeysF32 = 128, kCksRowsF32 = 32;

// CTAs per (sequence, key head), 0 where the call is not short enough: one wave of
// CTAs (one on each SM), two where there are up to 32 rows, four in fp32.  Device time
// of this kernel and of the five others in us (sequences x key heads x rows x keys):
//   bf16, d = 64: 1 x 12 x 8 x 500 9.4 / 26.6, 1 x 12 x 64 x 2048 25.0 / 39.8, 8 x 4 x 8 x
//   2048 (256 CTAs) 29.6 / 33.8, 38 x 8 x 32 x 256 (304) 30.3 / 42.5; past the bound
//   8 x 4 x 64 x 2048 (256) 69.3 / 42.9, at d = 128 80.5 / 47.9;
//   fp32: 1 x 12 x 8 x 500 10.0 / 30.3, 38 x 8 x 32 x 128 (304) 20.9 / 51.7, d = 128 43.7 / 82.3.
int chunk_small_cluster(int S, int Hq, int Hkv, int max_new, int max_len, int dtype) {
  const int64_t pairs = (int64_t)S * Hkv;
  const int keys = dtype == DA_BF16 ? kCksKeys : kCksKeysF32, rows = dtype == DA_BF16 ? kCksRows : kCksRowsF32;
  if ((int64_t)(Hq / Hkv) * round_up(max_new, 8) > rows || max_len < 1 || max_len > kCksCluster * keys) return 0;
  int c = 1;
  while (c * keys < max_len) c *= 2;
  const int waves = dtype == DA_F32 ? 4 : (Hq / Hkv) * round_up(max_new, 8) <= 32 ? 2 : 1;
  if (pairs * c > waves * 152) return 0;
  // more CTAs shorten each one's copies and products, down to 64 keys
  while (c < kCksCluster && pairs * c * 2 <= 152 && max_len > c * 64) c *= 2;
  return c;
}

// 16-byte piece i of row r of `pieces` pieces, swizzled by the row.
__device__ __forceinline__ uint32_t cks_off(int r, int i, int pieces) { return (uint32_t)((r * pieces + (i ^ (r & 7))) << 4); }

// One CTA's part: its sequence and key head, rows, and keys.
struct CksPart {
  int s, hkv, a, n, n8, rows, P, key0, cnt, fill;   // first token; cnt keys from key0 on, fill with those up to 16
  bool any;
  __device__ __forceinline__ CksPart(const PagedChunk &p, int G, int csize) {
    const int pair = blockIdx.x / csize, rank = (int)cluster_rank();
    s = pair / p.c.Hkv;
    hkv = pair % p.c.Hkv;
    const int len = __ldcg(p.c.seq_lens + s), b = __ldcg(p.cu + s + 1);
    a = __ldcg(p.cu + s);
    n = b - a;
    any = false;
    if (len < 0 || len > p.max_len || a < 0 || b < a || b > p.N || n > p.max_new || n > len) {
      if (hkv == 0 && rank == 0 && threadIdx.x == 0) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      return;
    }
    any = n > 0;
    n8 = (n + 7) & ~7;
    rows = G * n8;
    P = len - n;
    const int share = ((len + csize - 1) / csize + 15) & ~15;
    key0 = rank * share;
    cnt = max(0, min(share, len - key0));
    fill = (cnt + 15) & ~15;
  }
  // The last key that row r sees; -1: the row is none.
  __device__ __forceinline__ int last(int r) const { return r < rows && r % n8 < n ? P + r % n8 : -1; }
};

// After a cluster barrier: -lse2 of every row from the CTAs' (max, sum).
__device__ __forceinline__ void cks_join(const float2 *s_ml, float *s_nl, int rows, int csize) {
  if ((int)threadIdx.x >= rows) return;
  float m = -INFINITY, sum = 0.f;
  for (int c = 0; c < csize; ++c) {
    const float2 ml = ld_peer(s_ml + threadIdx.x, (uint32_t)c);
    const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
    sum = sum * ex2_approx(m - ms) + ml.y * ex2_approx(ml.x - ms);
    m = mn;
  }
  s_nl[threadIdx.x] = m == -INFINITY ? 0.f : -(m + log2f(sum));   // (a row that is none: its logits are -infinity)
}

// (max, sum) of every row of logits over the CTA's keys: a warp a row.
__device__ __forceinline__ void cks_stats(const float *sP, int ld, const CksPart &k, float2 *s_ml) {
  const int lane = threadIdx.x % 32;
  for (int r = threadIdx.x / 32; r < k.rows; r += kCksWarps) {
    float m = -INFINITY, sum = 0.f;
    for (int i = lane; i < k.fill; i += 32) m = fmaxf(m, sP[r * ld + i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ms = m == -INFINITY ? 0.f : m;
    for (int i = lane; i < k.fill; i += 32) sum += ex2_approx(sP[r * ld + i] - ms);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_ml[r] = make_float2(m, sum);
  }
}

// After a cluster barrier: whether a CTA of the cluster has cleared a value (last warp).
__device__ __forceinline__ void cks_any(const uint32_t *s_odd, uint32_t *s_any, int csize) {
  const int lane = threadIdx.x - (kCksThreads - 32);
  if (lane < 0) return;
  const uint32_t odd = __any_sync(0xffffffffu, lane < csize && ld_peer(s_odd, (uint32_t)lane) != 0);
  if (lane == 0) *s_any = odd;
}

// After a cluster barrier: out, the CTAs' numerators (`parts` blocks of `rows_max` rows
// of `stage` floats each) and sums added in order; a CTA writes its share of the pieces.
template <int D, typename E>
__device__ __forceinline__ void cks_out(const PagedChunk &p, const CksPart &k, int G, const float *num, int parts, int rows_max, int stage,
                                        const float *s_sum, int csize, int page_shift, bool odd) {
  for (int e = (int)cluster_rank() * kCksThreads + threadIdx.x; e < k.rows * (D / 4); e += csize * kCksThreads) {
    const int r = e / (D / 4), c = e % (D / 4), h = r / k.n8, q = r % k.n8;
    if (q >= k.n) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int i = 0; i < csize; ++i) {
      for (int part = 0; part < parts; ++part) {
        const float4 v = ld_peer4(num + (part * rows_max + r) * stage + 4 * c, (uint32_t)i);
        a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
      }
      sum += ld_peer(s_sum + r, (uint32_t)i);
    }
    if (odd)
      for (int t = k.P; t <= k.P + q; ++t) chunk_see<D, E>(p, page_shift, k.s, k.hkv, t, 4 * c, a);
    const size_t to = ((size_t)(k.a + q) * p.c.Hq + k.hkv * G + h) * D + 4 * c;
    if constexpr (sizeof(E) == 4)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to) = make_float4(a.x / sum, a.y / sum, a.z / sum, a.w / sum);
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + to) =
          make_uint2(pack_bf16x2(a.x / sum, a.y / sum), pack_bf16x2(a.z / sum, a.w / sum));
  }
}

template <int D>
struct Cks {
  static constexpr int kPieces = D / 8;
  static constexpr int kLd = kCksKeys + 4;              // floats of a row of logits
  static constexpr uint32_t kOffV = kCksKeys * D * 2, kOffQ = 2 * kOffV, kOffP = kOffQ + kCksRows * D * 2;
  static constexpr uint32_t kShBytes = kCksRows * kCksKeys * 2;   // shares: their first terms over K, their second
  static constexpr uint32_t kOffSh2 = 2 * kShBytes <= kOffV ? kShBytes : kOffP + kCksRows * kLd * 4;   // behind them, or last
  static constexpr int kSmemBytes = kOffP + kCksRows * kLd * 4 + (kOffSh2 > kOffP ? kShBytes : 0);
  static constexpr int kSplit = 128 / D;                // warps that share a 16-column tile of out: by keys
  static constexpr int kStage = D + 4;                  // floats of a row of numerators
  static_assert(kShBytes <= kOffV, "shares over K");
  static_assert(kSmemBytes <= 231424, "shared memory");
  static_assert(kSplit * kCksRows * kStage <= kCksRows * kLd, "numerators over the logits");
};

template <int D>
__global__ void __launch_bounds__(kCksThreads, 1) cks_chunk(PagedChunk p, int G, int page_shift, int csize) {
  using C = Cks<D>;
  constexpr int PP = C::kPieces;
  extern __shared__ __align__(128) uint8_t cks_smem[];
  const uint32_t sK = smem_u32(cks_smem), sV = sK + C::kOffV, sQ = sK + C::kOffQ, sSh = sK, sSh2 = sK + C::kOffSh2;
  float *sP = reinterpret_cast<float *>(cks_smem + C::kOffP);
  __shared__ float2 s_ml[kCksRows];                     // this CTA's (max, sum) of the rows
  __shared__ float s_nl[kCksRows], s_sum[kCksRows];
  __shared__ uint32_t s_odd, s_any;                          // values that are not finite: see da_chunk.cuh
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int ps = 1 << page_shift;
  pdl_wait();
  pdl_launch_dependents();
  const CksPart k(p, G, csize);
  if (!k.any) return;   // (the same in every CTA of the cluster)
  const int s = k.s, hkv = k.hkv, a = k.a, n = k.n, n8 = k.n8, rows = k.rows, key0 = k.key0, cnt = k.cnt, fill = k.fill;
  const int blocks = (rows + 15) / 16, key = key0 + tid;   // this thread's key, where tid < cnt
  // queries, keys, then values; rows from cnt on are zeros
  for (int e = tid; e < blocks * 16 * PP; e += kCksThreads) {
    const int r = e / PP, i = e % PP, h = r / n8, q = r % n8;
    const bool have = r < rows && q < n;
    cp_async16_fill(sQ + cks_off(r, i, PP),
             static_cast<const __nv_bfloat16 *>(p.q) + (have ? ((size_t)(a + q) * p.c.Hq + hkv * G + h) * D + 8 * i : 0), have);
  }
  {
    constexpr int STEP = kCksThreads / PP;
    const int i = tid % PP;
    const int32_t *table = p.c.page_table + (size_t)s * p.c.max_pages;
    for (int r0 = tid / PP; r0 < fill; r0 += 4 * STEP) {
      int page[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + j * STEP;
        page[j] = r < cnt ? __ldcg(table + ((key0 + r) >> page_shift)) : -1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + j * STEP;
        if (r >= fill) break;
        const bool ok = (unsigned)page[j] < (unsigned)p.c.num_pages;
        if (!ok && r < cnt) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
        const size_t at = ok ? ((((size_t)page[j] * p.c.Hkv + hkv) << page_shift) + ((key0 + r) & (ps - 1))) * D + 8 * i : 0;
        cp_async16_fill(sK + cks_off(r, i, PP), static_cast<const __nv_bfloat16 *>(p.c.k_pages) + at, ok);
        cp_async16_fill(sV + cks_off(r, i, PP), static_cast<const __nv_bfloat16 *>(p.c.v_pages) + at, ok);
      }
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  // the key's totals, of the first heads at once
  constexpr int HELD = 8;
  static_assert(HELD * 8 == kCksRows, "every head's");
  float *at = nullptr;
  float held[HELD];
  if (tid < cnt) {
    const int page = __ldcg(p.c.demand_table + (size_t)s * p.c.max_pages + (key >> page_shift));
    if ((unsigned)page < (unsigned)p.c.num_demand_pages)
      at = p.c.demand_pages + ((((size_t)page * p.c.Hq + hkv * G) << page_shift) + (key & (ps - 1)));
    else
      atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
  }
#pragma unroll
  for (int h = 0; h < HELD; ++h) held[h] = h < G && at != nullptr ? __ldcg(at + ((size_t)h << page_shift)) : 0.f;
  cp_async_wait_all();
  bool odd = false;   // of the thread's own copies
  for (int r = tid / PP; r < cnt; r += kCksThreads / PP) {
    if (key0 + r < k.P) continue;
    uint4 *v = reinterpret_cast<uint4 *>(cks_smem + C::kOffV + cks_off(r, tid % PP, PP)), x = *v;
    if (chunk_clear(x, true)) *v = x, odd = true;
  }
  odd = __syncthreads_or(odd);
  if (tid == 0) s_odd = odd;
  // logits: a warp takes 32 keys
  if (warp * 32 < fill) {
    float acc[4][4][4];
#pragma unroll
    for (int rb = 0; rb < 4; ++rb)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[rb][j][e] = 0.f;
    const int br = warp * 32 + (lane & 7) + ((lane >> 4) << 3), bp = (lane >> 3) & 1;   // keys x 16 elements of the second operand
    const int ar = (lane & 7) + ((lane >> 3) & 1) * 8, ap = lane >> 4;                  // rows x 16 elements of the first
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t kb[2][4];
      ldsm_x4(sK + cks_off(br, 2 * ks + bp, PP), kb[0]);
      ldsm_x4(sK + cks_off(br + 16, 2 * ks + bp, PP), kb[1]);
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) {
        if (rb >= blocks) break;
        uint32_t qa[4];
        ldsm_x4(sQ + cks_off(rb * 16 + ar, 2 * ks + ap, PP), qa);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[rb][j], qa, kb[j >> 1][2 * (j & 1)], kb[j >> 1][2 * (j & 1) + 1]);
      }
    }
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      if (rb >= blocks) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = rb * 16 + lane / 4 + (e >> 1) * 8, h = r / n8, last = k.last(r);
        const float c2 = last >= 0 ? fmaxf(head_c2(p.hs, s * p.c.Hq + hkv * G + h, p.status), 1e-30f) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = warp * 32 + j * 8 + 2 * (lane % 4) + (e & 1);
          sP[r * C::kLd + i] = i < cnt && key0 + i <= last ? acc[rb][j][e] * c2 : -INFINITY;
        }
      }
    }
  }
  __syncthreads();
  // (max, sum) of every row over the CTA's keys, then over the cluster's
  cks_stats(sP, C::kLd, k, s_ml);
  cluster_sync();
  cks_join(s_ml, s_nl, rows, csize);
  cks_any(&s_odd, &s_any, csize);
  __syncthreads();
  // shares and totals: a thread a key
  if (tid < fill) {
    __nv_bfloat16 *sh = reinterpret_cast<__nv_bfloat16 *>(cks_smem), *sh2 = sh + C::kOffSh2 / 2;
    auto put = [&](int r, float v) {
      const uint32_t i = cks_off(r, tid >> 3, kCksKeys / 8) / 2 + (tid & 7);
      sh[i] = __float2bfloat16_rn(v);
      sh2[i] = __float2bfloat16_rn(v - __bfloat162float(sh[i]));
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      if (h >= G) break;
      const float base = held[h] + p.eps;
      float added = 0.f;   // the rows' bids, summed apart from the total: it would take their last bits
#pragma unroll 4
      for (int q = 0; q < n; ++q) {
        const int r = h * n8 + q;
        const float x = sP[r * C::kLd + tid];
        const float bid = x == -INFINITY ? 0.f : ex2_approx(x + s_nl[r]), before = added;   // (none from a row that does not see the key, whatever its sum is)
        added += bid;
        put(r, bid * rcp_approx(base + (p.earlier ? before : added)));
      }
      for (int q = n; q < n8; ++q) put(h * n8 + q, 0.f);
      if (at != nullptr) __stcg(at + ((size_t)h << page_shift), held[h] + added);
    }
    for (int r = rows; r < blocks * 16; ++r) put(r, 0.f);
  }
  __syncthreads();
  // the sums of the shares' terms; numerators over the logits
  for (int r = warp; r < rows; r += kCksWarps) {
    float sum = 0.f;
    for (int i = lane; i < fill / 8; i += 32) {
      const uint32_t at = cks_off(r, i, kCksKeys / 8);
      const uint4 v = *reinterpret_cast<const uint4 *>(cks_smem + at), v2 = *reinterpret_cast<const uint4 *>(cks_smem + C::kOffSh2 + at);
      const uint32_t w[8] = {v2.x, v2.y, v2.z, v2.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += __uint_as_float(w[e] << 16) + __uint_as_float(w[e] & 0xffff0000u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_sum[r] = sum;
  }
  {
    const int tile = warp % (D / 16), part = warp / (D / 16);   // 16 columns; every kSplit-th 16 keys
    float acc[4][2][4];
#pragma unroll
    for (int rb = 0; rb < 4; ++rb)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[rb][j][e] = 0.f;
    const int ar = (lane & 7) + ((lane >> 3) & 1) * 8, ap = lane >> 4;   // rows (or keys) and halves of 16
    for (int i = 16 * part; i < fill; i += 16 * C::kSplit) {
      uint32_t vb[4];
      ldsm_x4_t(sV + cks_off(i + ar, 2 * tile + ap, PP), vb);
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) {
        if (rb >= blocks) break;
        uint32_t sa[4], sa2[4];
        const uint32_t off = cks_off(rb * 16 + ar, (i >> 3) + ap, kCksKeys / 8);
        ldsm_x4(sSh + off, sa);
        ldsm_x4(sSh2 + off, sa2);
        mma16816(acc[rb][0], sa, vb[0], vb[1]);
        mma16816(acc[rb][1], sa, vb[2], vb[3]);
        mma16816(acc[rb][0], sa2, vb[0], vb[1]);
        mma16816(acc[rb][1], sa2, vb[2], vb[3]);
      }
    }
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      if (rb >= blocks) break;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<float2 *>(sP + (part * kCksRows + rb * 16 + lane / 4 + (e >> 1) * 8) * C::kStage + tile * 16 + j * 8 +
                                      2 * (lane % 4)) = make_float2(acc[rb][j][e], acc[rb][j][e + 1]);
    }
  }
  cluster_sync();
  cks_out<D, __nv_bfloat16>(p, k, G, sP, C::kSplit, kCksRows, C::kStage, s_sum, csize, page_shift, s_any != 0);
  cluster_sync();   // no CTA leaves while a peer may read it
}

// ------------------------------------------------------------------------- fp32
template <int D>
struct CksF32 {
  static constexpr int kLd = D + 4;                     // floats of a staged row: lanes of different rows read different banks
  static constexpr int kLdP = kCksKeysF32 + 4;
  static constexpr int kOffV = kCksKeysF32 * kLd, kOffQ = 2 * kOffV, kOffP = kOffQ + kCksRowsF32 * kLd;
  static constexpr int kSmemBytes = (kOffP + kCksRowsF32 * kLdP) * 4;
};

template <int D>
__global__ void __launch_bounds__(kCksThreads, 1) cks_chunk_f32(PagedChunk p, int G, int page_shift, int csize) {
  using C = CksF32<D>;
  constexpr int PP = D / 4;
  extern __shared__ __align__(128) uint8_t cks_smem[];
  float *sK = reinterpret_cast<float *>(cks_smem), *sV = sK + C::kOffV, *sQ = sK + C::kOffQ, *sP = sK + C::kOffP;
  float *sNum = sK;                                     // numerators: over K
  __shared__ float2 s_ml[kCksRowsF32];
  __shared__ float s_nl[kCksRowsF32], s_sum[kCksRowsF32];
  __shared__ uint32_t s_odd, s_any;                          // as above
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, ps = 1 << page_shift;
  pdl_wait();
  pdl_launch_dependents();
  const CksPart k(p, G, csize);
  if (!k.any) return;   // (the same in every CTA of the cluster)
  for (int e = tid; e < kCksRowsF32 * PP; e += kCksThreads) {
    const int r = e / PP, i = e % PP;
    const bool have = k.last(r) >= 0;
    const size_t at = have ? ((size_t)(k.a + r % k.n8) * p.c.Hq + k.hkv * G + r / k.n8) * D + 4 * i : 0;
    cp_async16_fill(smem_u32(sQ + r * C::kLd + 4 * i), static_cast<const float *>(p.q) + at, have);
  }
  const int32_t *table = p.c.page_table + (size_t)k.s * p.c.max_pages;
  for (int e = tid; e < k.fill * PP; e += kCksThreads) {
    const int r = e / PP, i = e % PP;
    const int page = r < k.cnt ? __ldcg(table + ((k.key0 + r) >> page_shift)) : -1;
    const bool ok = (unsigned)page < (unsigned)p.c.num_pages;
    if (!ok && r < k.cnt) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    const size_t at = ok ? ((((size_t)page * p.c.Hkv + k.hkv) << page_shift) + ((k.key0 + r) & (ps - 1))) * D + 4 * i : 0;
    cp_async16_fill(smem_u32(sK + r * C::kLd + 4 * i), static_cast<const float *>(p.c.k_pages) + at, ok);
    cp_async16_fill(smem_u32(sV + r * C::kLd + 4 * i), static_cast<const float *>(p.c.v_pages) + at, ok);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  // the totals: a thread a key and every other head
  constexpr int HELD = kCksRowsF32 / 8 / 2;
  const int key_l = tid % kCksKeysF32, half = tid / kCksKeysF32;
  float *at = nullptr, held[HELD];
  if (key_l < k.cnt) {
    const int key = k.key0 + key_l, page = __ldcg(p.c.demand_table + (size_t)k.s * p.c.max_pages + (key >> page_shift));
    if ((unsigned)page < (unsigned)p.c.num_demand_pages)
      at = p.c.demand_pages + ((((size_t)page * p.c.Hq + k.hkv * G) << page_shift) + (key & (ps - 1)));
    else
      atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
  }
#pragma unroll
  for (int j = 0; j < HELD; ++j)
    held[j] = 2 * j + half < G && at != nullptr ? __ldcg(at + ((size_t)(2 * j + half) << page_shift)) : 0.f;
  cp_async_wait_all();
  bool odd = false;   // of the thread's own copies
  for (int r = tid / PP; r < k.cnt; r += kCksThreads / PP) {
    if (k.key0 + r < k.P) continue;
    uint4 *v = reinterpret_cast<uint4 *>(sV + r * C::kLd + tid % PP * 4), x = *v;
    if (chunk_clear(x, false)) *v = x, odd = true;
  }
  odd = __syncthreads_or(odd);
  if (tid == 0) s_odd = odd;
  const bool work = 4 * warp < k.rows;                  // rows 4 warp ..; keys lane + 32 j
  if (work) {
    float2 acc[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[r][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      float4 kv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4 *>(sK + (lane + 32 * j) * C::kLd + e);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 q = *reinterpret_cast<const float4 *>(sQ + (4 * warp + r) * C::kLd + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[r][j] = ffma2(make_float2(q.x, q.y), make_float2(kv[j].x, kv[j].y), acc[r][j]);
          acc[r][j] = ffma2(make_float2(q.z, q.w), make_float2(kv[j].z, kv[j].w), acc[r][j]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * warp + r, last = k.last(row);
      const float c2 = last >= 0 ? head_c2(p.hs, k.s * p.c.Hq + k.hkv * G + row / k.n8, p.status) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = lane + 32 * j;
        sP[row * C::kLdP + i] = i < k.cnt && k.key0 + i <= last ? (acc[r][j].x + acc[r][j].y) * c2 : -INFINITY;
      }
    }
  }
  __syncthreads();
  cks_stats(sP, C::kLdP, k, s_ml);
  cluster_sync();
  cks_join(s_ml, s_nl, k.rows, csize);
  cks_any(&s_odd, &s_any, csize);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    const int h = 2 * j + half;
    if (h >= G) break;
    float added = 0.f;   // the rows' bids, summed apart from the total: it would take their last bits
#pragma unroll 4
    for (int q = 0; q < k.n; ++q) {
      float *x = sP + (h * k.n8 + q) * C::kLdP + key_l;
      const float bid = key_l < k.fill && *x != -INFINITY ? ex2_approx(*x + s_nl[h * k.n8 + q]) : 0.f, before = added;
      added += bid;
      float r;
      asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(held[j] + (p.earlier ? before : added) + p.eps));
      *x = bid > 0.f ? bid * r : 0.f;
    }
    for (int q = k.n; q < k.n8; ++q) sP[(h * k.n8 + q) * C::kLdP + key_l] = 0.f;
    if (at != nullptr) __stcg(at + ((size_t)h << page_shift), held[j] + added);
  }
  __syncthreads();
  if (work) {
    constexpr int SPLIT = 128 / D;                      // lanes that share columns: every SPLIT-th 4 keys
    const int col = 4 * (lane % (D / 4)), part = lane / (D / 4);
    float2 num[4][2];
    float sum[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) num[r][0] = num[r][1] = make_float2(0.f, 0.f), sum[r] = 0.f;
#pragma unroll 2
    for (int i = 4 * part; i < k.fill; i += 4 * SPLIT) {
      float4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float4 *>(sV + (i + e) * C::kLd + col);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 sh = *reinterpret_cast<const float4 *>(sP + (4 * warp + r) * C::kLdP + i);
        const float s4[4] = {sh.x, sh.y, sh.z, sh.w};
        sum[r] += (sh.x + sh.y) + (sh.z + sh.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          num[r][0] = ffma2(make_float2(s4[e], s4[e]), make_float2(v[e].x, v[e].y), num[r][0]);
          num[r][1] = ffma2(make_float2(s4[e], s4[e]), make_float2(v[e].z, v[e].w), num[r][1]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (SPLIT == 2) {
        num[r][0].x += __shfl_xor_sync(0xffffffffu, num[r][0].x, 16);
        num[r][0].y += __shfl_xor_sync(0xffffffffu, num[r][0].y, 16);
        num[r][1].x += __shfl_xor_sync(0xffffffffu, num[r][1].x, 16);
        num[r][1].y += __shfl_xor_sync(0xffffffffu, num[r][1].y, 16);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 16);
      }
      const int row = 4 * warp + r;
      if (part == 0) *reinterpret_cast<float4 *>(sNum + row * C::kLd + col) =
          make_float4(num[r][0].x, num[r][0].y, num[r][1].x, num[r][1].y);
      if (lane == 0) s_sum[row] = sum[r];
    }
  }
  cluster_sync();
  cks_out<D, float>(p, k, G, sNum, 1, kCksRowsF32, C::kLd, s_sum, csize, page_shift, s_any != 0);
  cluster_sync();   // no CTA leaves while a peer may read it
}

template <typename Kernel>
static int launch_cks(Kernel kernel, int smem, const PagedChunk &p, int csize, cudaStream_t stream) {
  int shift = 0;
  while ((1 << shift) < p.c.page_size) ++shift;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.S * p.c.Hkv * csize));
  cfg.blockDim = dim3(kCksThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)csize;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // (see launch_after)
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, p.c.Hq / p.c.Hkv, shift, csize) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

template <int D>
static int launch_cks_d(const PagedChunk &p, int csize, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return (cudaFuncSetAttribute(cks_chunk<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cks<D>::kSmemBytes) != cudaSuccess ||
            cudaFuncSetAttribute(cks_chunk_f32<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, CksF32<D>::kSmemBytes) !=
                cudaSuccess)
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  return p.c.dtype == DA_BF16 ? launch_cks(cks_chunk<D>, Cks<D>::kSmemBytes, p, csize, stream)
                              : launch_cks(cks_chunk_f32<D>, CksF32<D>::kSmemBytes, p, csize, stream);
}

int launch_chunk_small(const PagedChunk &p, int csize, cudaStream_t stream) {
  return p.c.d == 128 ? launch_cks_d<128>(p, csize, stream) : launch_cks_d<64>(p, csize, stream);
}

}  // namespace da
