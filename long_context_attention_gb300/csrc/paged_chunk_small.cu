// Short chunks over the paged cache in bf16: one launch.
//
// Mathematics: as paged_chunk_f32.cu.  What bounds the call is latency: its five
// kernels take 32 us for 5 tokens x 12 heads x 500 keys (1.6 MB).  Here a cluster of up
// to 8 CTAs takes a (sequence, key head), 256 keys a CTA at most and up to 64 rows (the
// group's query heads by the new tokens, n8 rows a head):
//   keys, values and queries come into shared memory; S = Q K^T by m16n8k16
//   products, the logits stay in shared memory; every row's (max, sum) goes through
//   distributed shared memory; one thread a key walks the rows of each head with its
//   total; the shares, rounded to bf16 once as in paged_chunk_bf16.cu, times V; the
//   CTAs' numerators and sums are added in the CTAs' order by the CTA that writes them.
// m16n8k16 and not tcgen05: the products are 1 % of the call.
#include "da_chunk.cuh"
#include "da_paged_plan.cuh"

#include <cuda_bf16.h>

namespace da {

constexpr int kCksKeys = 256, kCksRows = 64, kCksThreads = 256, kCksWarps = 8, kCksCluster = 8;

// CTAs per (sequence, key head), 0 where the call is not short enough: few enough
// CTAs for two waves (one on each SM).
int chunk_small_cluster(int S, int Hq, int Hkv, int max_new, int max_len) {
  const int64_t pairs = (int64_t)S * Hkv;
  if ((int64_t)(Hq / Hkv) * round_up(max_new, 8) > kCksRows || max_len < 1 || max_len > kCksCluster * kCksKeys) return 0;
  int c = 1;
  while (c * kCksKeys < max_len) c *= 2;
  if (pairs * c > 2 * 152) return 0;
  // more CTAs shorten each one's copies and products, down to 64 keys
  while (c < kCksCluster && pairs * c * 2 <= 152 && max_len > c * 64) c *= 2;
  return c;
}

__device__ __forceinline__ uint32_t cks_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cks_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cks_peer(const void *local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 cks_peer2(const float2 *local, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cks_peer(local, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 cks_peer4(const float *local, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cks_peer(local, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void cks_copy(uint32_t dst, const void *src, bool have) {   // zeros where !have
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(have ? 16 : 0)
               : "memory");
}
// 16-byte piece i of row r of `pieces` pieces, swizzled by the row.
__device__ __forceinline__ uint32_t cks_off(int r, int i, int pieces) { return (uint32_t)((r * pieces + (i ^ (r & 7))) << 4); }

template <int D>
struct Cks {
  static constexpr int kPieces = D / 8;
  static constexpr int kLd = kCksKeys + 4;              // floats of a row of logits
  static constexpr uint32_t kOffV = kCksKeys * D * 2, kOffQ = 2 * kOffV, kOffP = kOffQ + kCksRows * D * 2;
  static constexpr int kSmemBytes = kOffP + kCksRows * kLd * 4;
  static constexpr int kSplit = 128 / D;                // warps that share a 16-column tile of out: by keys
  static constexpr int kStage = D + 4;                  // floats of a row of numerators
  static_assert(kCksRows * kCksKeys * 2 <= kOffV, "shares over K");
  static_assert(kSplit * kCksRows * kStage <= kCksRows * kLd, "numerators over the logits");
};

template <int D>
__global__ void __launch_bounds__(kCksThreads, 1) cks_chunk(PagedChunk p, int G, int page_shift, int csize) {
  using C = Cks<D>;
  constexpr int PP = C::kPieces;
  extern __shared__ __align__(128) uint8_t cks_smem[];
  const uint32_t sK = smem_u32(cks_smem), sV = sK + C::kOffV, sQ = sK + C::kOffQ, sSh = sK;   // shares: over K
  float *sP = reinterpret_cast<float *>(cks_smem + C::kOffP);
  __shared__ float2 s_ml[kCksRows];                     // this CTA's (max, sum) of the rows
  __shared__ float s_nl[kCksRows], s_sum[kCksRows];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t rank = cks_rank();
  const int pair = blockIdx.x / csize, s = pair / p.c.Hkv, hkv = pair % p.c.Hkv, ps = 1 << page_shift;
  pdl_wait();
  pdl_launch_dependents();
  const int len = __ldcg(p.c.seq_lens + s), a = __ldcg(p.cu + s), b = __ldcg(p.cu + s + 1), n = b - a;
  if (len < 0 || len > p.max_len || a < 0 || b < a || b > p.N || n > p.max_new || n > len) {
    if (hkv == 0 && rank == 0 && tid == 0) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    return;   // (the same in every CTA of the cluster)
  }
  if (n == 0) return;
  const int n8 = (n + 7) & ~7, rows = G * n8, P = len - n, blocks = (rows + 15) / 16;
  const int share = ((len + csize - 1) / csize + 15) & ~15;   // keys of each CTA
  const int key0 = (int)rank * share, cnt = max(0, min(share, len - key0)), fill = (cnt + 15) & ~15;
  const int key = key0 + tid;                           // this thread's, where tid < cnt
  // queries, keys, then values; rows from cnt on are zeros
  for (int e = tid; e < blocks * 16 * PP; e += kCksThreads) {
    const int r = e / PP, i = e % PP, h = r / n8, q = r % n8;
    const bool have = r < rows && q < n;
    cks_copy(sQ + cks_off(r, i, PP),
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
        cks_copy(sK + cks_off(r, i, PP), static_cast<const __nv_bfloat16 *>(p.c.k_pages) + at, ok);
        cks_copy(sV + cks_off(r, i, PP), static_cast<const __nv_bfloat16 *>(p.c.v_pages) + at, ok);
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
  __syncthreads();
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
        const int r = rb * 16 + lane / 4 + (e >> 1) * 8, h = r / n8, q = r % n8;
        const int last = r < rows && q < n ? P + q : -1;   // the last key that the row sees
        const float c2 = last >= 0 ? fmaxf(head_c2(p.hs, s * p.c.Hq + hkv * G + h, p.status), 1e-30f) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = warp * 32 + j * 8 + 2 * (lane % 4) + (e & 1);
          sP[r * C::kLd + k] = k < cnt && key0 + k <= last ? acc[rb][j][e] * c2 : -INFINITY;
        }
      }
    }
  }
  __syncthreads();
  // (max, sum) of every row over the CTA's keys, then over the cluster's
  for (int r = warp; r < rows; r += kCksWarps) {
    float m = -INFINITY, sum = 0.f;
    for (int k = lane; k < fill; k += 32) m = fmaxf(m, sP[r * C::kLd + k]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ms = m == -INFINITY ? 0.f : m;
    for (int k = lane; k < fill; k += 32) sum += ex2_approx(sP[r * C::kLd + k] - ms);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_ml[r] = make_float2(m, sum);
  }
  cks_sync();
  if (tid < rows) {
    float m = -INFINITY, sum = 0.f;
    for (int c = 0; c < csize; ++c) {
      const float2 ml = cks_peer2(&s_ml[tid], (uint32_t)c);
      const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
      sum = sum * ex2_approx(m - ms) + ml.y * ex2_approx(ml.x - ms);
      m = mn;
    }
    s_nl[tid] = m == -INFINITY ? 0.f : -(m + log2f(sum));   // (a row that is none: its logits are -infinity)
  }
  __syncthreads();
  // shares and totals: a thread a key
  if (tid < fill) {
    __nv_bfloat16 *sh = reinterpret_cast<__nv_bfloat16 *>(cks_smem);
    auto put = [&](int r, float v) {
      sh[cks_off(r, tid >> 3, kCksKeys / 8) / 2 + (tid & 7)] = __float2bfloat16_rn(v);
    };
#pragma unroll
    for (int h = 0; h < HELD; ++h) {
      if (h >= G) break;
      const float base = held[h] + p.eps;
      float added = 0.f;   // the rows' bids, summed apart from the total: it would take their last bits
#pragma unroll 4
      for (int q = 0; q < n; ++q) {
        const int r = h * n8 + q;
        const float bid = ex2_approx(sP[r * C::kLd + tid] + s_nl[r]), before = added;
        added += bid;
        put(r, bid * rcp_approx(base + (p.earlier ? before : added)));
      }
      for (int q = n; q < n8; ++q) put(h * n8 + q, 0.f);
      if (at != nullptr) __stcg(at + ((size_t)h << page_shift), held[h] + added);
    }
    for (int r = rows; r < blocks * 16; ++r) put(r, 0.f);
  }
  __syncthreads();
  // the sums of the rounded shares; numerators over the logits
  for (int r = warp; r < rows; r += kCksWarps) {
    float sum = 0.f;
    for (int i = lane; i < fill / 8; i += 32) {
      const uint4 v = *reinterpret_cast<const uint4 *>(cks_smem + cks_off(r, i, kCksKeys / 8));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += __uint_as_float(w[e] << 16) + __uint_as_float(w[e] & 0xffff0000u);
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
    for (int k = 16 * part; k < fill; k += 16 * C::kSplit) {
      uint32_t vb[4];
      ldsm_x4_t(sV + cks_off(k + ar, 2 * tile + ap, PP), vb);
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) {
        if (rb >= blocks) break;
        uint32_t sa[4];
        ldsm_x4(sSh + cks_off(rb * 16 + ar, (k >> 3) + ap, kCksKeys / 8), sa);
        mma16816(acc[rb][0], sa, vb[0], vb[1]);
        mma16816(acc[rb][1], sa, vb[2], vb[3]);
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
  cks_sync();
  // out: a CTA adds and writes its share of the rows' pieces
  for (int e = (int)rank * kCksThreads + tid; e < rows * (D / 4); e += csize * kCksThreads) {
    const int r = e / (D / 4), c = e % (D / 4), h = r / n8, q = r % n8;
    if (q >= n) continue;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    for (int k = 0; k < csize; ++k) {
#pragma unroll
      for (int part = 0; part < C::kSplit; ++part) {
        const float4 v = cks_peer4(sP + (part * kCksRows + r) * C::kStage + 4 * c, (uint32_t)k);
        num.x += v.x, num.y += v.y, num.z += v.z, num.w += v.w;
      }
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(cks_peer(&s_sum[r], (uint32_t)k)) : "memory");
      sum += x;
    }
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + ((size_t)(a + q) * p.c.Hq + hkv * G + h) * D + 4 * c) =
        make_uint2(pack_bf16x2(num.x / sum, num.y / sum), pack_bf16x2(num.z / sum, num.w / sum));
  }
  cks_sync();   // no CTA leaves while a peer may read it
}

template <int D>
static int launch_cks(const PagedChunk &p, int csize, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return cudaFuncSetAttribute(cks_chunk<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cks<D>::kSmemBytes) != cudaSuccess
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  int shift = 0;
  while ((1 << shift) < p.c.page_size) ++shift;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.S * p.c.Hkv * csize));
  cfg.blockDim = dim3(kCksThreads);
  cfg.dynamicSmemBytes = Cks<D>::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)csize;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // (see launch_after)
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, cks_chunk<D>, p, p.c.Hq / p.c.Hkv, shift, csize) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int launch_chunk_small(const PagedChunk &p, int csize, cudaStream_t stream) {
  return p.c.d == 128 ? launch_cks<128>(p, csize, stream) : launch_cks<64>(p, csize, stream);
}

}  // namespace da
