// Decode step over short paged caches in bf16: one launch.
//
// Mathematics: as paged_decode_bf16.cu.  A short step is bound by latency, not by
// bytes: three kernels that follow one another cost 12 us on the device and 10
// us of launches for 1 x 12 x 500 keys (0.2 us of copies).  Here a cluster of up
// to 8 CTAs takes one (sequence, key head): every CTA holds its share of the
// keys and values in shared memory, all copies issued at once; logits stay in
// the registers of the threads that will use them; the softmax's (max, sum) and
// the partial results pass between the CTAs through distributed shared memory.
//
// Tensor cores, key order and the two-term shares are those of
// paged_decode_bf16.cu: a warp takes groups of 16 keys, lane (g, t) the keys 4t ..
// 4t + 3 of row g (and g + 8).  A prefix's pages are read by every sequence: at
// these sizes they come from L2.
#include "da_paged_plan.cuh"

#include <cuda_bf16.h>

namespace da {

constexpr int kSmallThreads = 256;
constexpr int kSmallWarps = kSmallThreads / 32;
DA_HD constexpr int small_keys(int d) { return d == 64 ? 256 : 128; }   // keys a CTA can hold (32 KB of K, 32 KB of V)
constexpr int kSmallMaxCluster = 8;
constexpr int kSmallMaxCtas = 3 * 152;   // one wave: 3 CTAs on each SM

// CTAs per (sequence, key head), 0 where the call is not short enough.  One wave
// of CTAs, or two where one or two CTAs hold a sequence.  Device time of this
// kernel and of the three streaming ones, in us: 64 x 8 x 100 keys (512 CTAs of
// one) 13.7 against 16.5, 64 x 12 x 250 (768 of one) 17.3 against 23.6, 8 x 12 x
// 1000 (384 of four) 9.8 against 13.0; past the bound 8 x 12 x 2000 (768 of
// eight) 18.0 against 16.0, 16 x 8 x 2000 (1024 of eight) 25.8 against 18.7.
int small_cluster(int S, int Hq, int Hkv, int d, int max_len) {
  const int64_t pairs = (int64_t)S * Hkv;
  if (Hq / Hkv > 16 || max_len < 1 || max_len > kSmallMaxCluster * small_keys(d)) return 0;
  int c = 1;
  while (c * small_keys(d) < max_len) c *= 2;
  if (pairs * c > (c <= 2 ? 2 : 1) * kSmallMaxCtas) return 0;
  // more CTAs shorten each one's copies and products, down to 32 keys
  while (c < kSmallMaxCluster && pairs * c * 2 <= kSmallMaxCtas && max_len > c * 32) c *= 2;
  return c;
}

// Row r (d elements), 16-byte piece i of a chunk: pieces swizzled by the row.
template <int D>
__device__ __forceinline__ uint32_t small_off(int r, int i) {
  return (uint32_t)(r * D * 2 + ((i ^ (r & 7)) << 4));
}

template <int D, bool WIDE>   // WIDE: 9 to 16 rows
__global__ void __launch_bounds__(kSmallThreads)
    pgs_small(PagedDecode p, int G, int page_shift, int csize) {
  constexpr int KEYS = small_keys(D), PPR = D / 8, NT = D / 8, KS = D / 16;
  constexpr int HH = WIDE ? 2 : 1, ROWS = WIDE ? 16 : 8;
  constexpr int GROUPS = KEYS / 16 / kSmallWarps;   // 16-key groups of a warp at most
  extern __shared__ __align__(128) uint8_t small_smem[];
  uint8_t *sK = small_smem, *sV = small_smem + KEYS * D * 2;
  float *red = reinterpret_cast<float *>(small_smem);   // [warps][ROWS][D], over K once the logits are formed
  static_assert(kSmallWarps * ROWS * D * 4 <= 2 * KEYS * D * 2, "the warps' sums over K (and V, read by then)");
  __shared__ float s_m[kSmallWarps][16], s_l[kSmallWarps][16], s_sum[kSmallWarps][16];
  __shared__ float s_ml[2][16];                          // this CTA's (max, sum) of the rows
  __shared__ float s_all[2][kSmallMaxCluster][16];
  __shared__ float s_part[16][D + 1];                    // this CTA's numerators and share sums
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x / csize, s = pair / p.c.Hkv, hkv = pair % p.c.Hkv;
  const int ps = 1 << page_shift;
  pdl_wait();
  const int len = paged_len(p, s, hkv == 0 && rank == 0 && tid == 0 ? p.status : nullptr);
  const int share_keys = ((len + csize - 1) / csize + 15) & ~15;      // keys of each CTA
  const int key0 = rank * share_keys, nk = max(0, min(share_keys, len - key0)), fill = (nk + 15) & ~15;
  const int32_t *table = p.c.page_table + (size_t)s * p.c.max_pages;
  const int32_t *dtab = p.c.demand_table + (size_t)s * p.c.max_pages;
  // all keys, then all values; rows from nk on are zeros
  {
    constexpr int IT = KEYS * PPR / kSmallThreads;
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(p.c.k_pages);
    const __nv_bfloat16 *vp = static_cast<const __nv_bfloat16 *>(p.c.v_pages);
    const int i = tid % PPR, r0 = tid / PPR;
    constexpr int STEP = kSmallThreads / PPR;
    int page[IT];
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int r = r0 + j * STEP, key = key0 + r;
      page[j] = -1;
      if (r < nk) page[j] = (key < p.prefix_len ? p.prefix_table : table)[key >> page_shift];
    }
    size_t at[IT];
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int r = r0 + j * STEP, key = key0 + r;
      if (r < nk && (unsigned)page[j] >= (unsigned)p.c.num_pages) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      const bool ok = (unsigned)page[j] < (unsigned)p.c.num_pages;
      at[j] = ok ? ((((size_t)page[j] * p.c.Hkv + hkv) << page_shift) + (key & (ps - 1))) * D + i * 8 : 0;
      if (r < fill) cp_async16_fill(smem_u32(sK) + small_off<D>(r, i), kp + at[j], ok);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
    for (int j = 0; j < IT; ++j) {
      const int r = r0 + j * STEP;
      if (r < fill) cp_async16_fill(smem_u32(sV) + small_off<D>(r, i), vp + at[j], (unsigned)page[j] < (unsigned)p.c.num_pages);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // query rows as the A operand
  uint32_t qa[KS][4] = {};
  float c2[HH];
  bool on[HH];
#pragma unroll
  for (int hh = 0; hh < HH; ++hh) {
    const int r = g + 8 * hh;
    on[hh] = r < G;
    const int hq = hkv * G + (on[hh] ? r : 0);
    c2[hh] = head_c2(p.hs, s * p.c.Hq + hq, rank == 0 && on[hh] && t == 0 && warp == 0 ? p.status : nullptr);
    const uint32_t *qr =
        reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.q) + ((size_t)s * p.c.Hq + hq) * D);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qa[ks][hh] = on[hh] ? qr[ks * 8 + t] : 0u;
      qa[ks][2 + hh] = on[hh] ? qr[ks * 8 + 4 + t] : 0u;
    }
  }
  // the lane's demand: 4 keys of its rows in each of the warp's groups
  float *dp[GROUPS][HH];
  float4 dem[GROUPS][HH];
#pragma unroll
  for (int j = 0; j < GROUPS; ++j) {
    const int kl = 16 * (warp + j * kSmallWarps) + 4 * t, key = key0 + kl;
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
      dp[j][hh] = nullptr;
      dem[j][hh] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (on[hh] && kl < nk) {
        const int dpg = dtab[key >> page_shift];
        if ((unsigned)dpg < (unsigned)p.c.num_demand_pages) {
          dp[j][hh] = p.c.demand_pages + (((size_t)dpg * p.c.Hq + hkv * G + g + 8 * hh) << page_shift) + (key & (ps - 1));
          dem[j][hh] = *reinterpret_cast<const float4 *>(dp[j][hh]);
        } else {
          atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  __syncthreads();
  // logits of the warp's groups, in the lane layout of the shares
  float x[GROUPS][HH][4], m[HH], l[HH];
#pragma unroll
  for (int hh = 0; hh < HH; ++hh) m[hh] = -INFINITY, l[hh] = 0.f;
#pragma unroll
  for (int j = 0; j < GROUPS; ++j) {
    const int k16 = 16 * (warp + j * kSmallWarps);
    float acc[2][4] = {};
    if (k16 < nk) {
      const int row = k16 + group_key(lane & 7, lane >> 4);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t b[4];
        ldsm_x4(smem_u32(sK) + small_off<D>(row, 2 * ks + ((lane >> 3) & 1)), b);
        mma16816(acc[0], qa[ks], b[0], b[1]);
        mma16816(acc[1], qa[ks], b[2], b[3]);
      }
    }
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = acc[e >> 1][2 * hh + (e & 1)] * c2[hh];
        x[j][hh][e] = k16 + 4 * t + e < nk ? v : -INFINITY;
        m[hh] = fmaxf(m[hh], x[j][hh][e]);
      }
    }
  }
#pragma unroll
  for (int hh = 0; hh < HH; ++hh) {
    const float ms = m[hh] == -INFINITY ? 0.f : m[hh];
#pragma unroll
    for (int j = 0; j < GROUPS; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) l[hh] += ex2_approx(x[j][hh][e] - ms);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[hh], o), l2 = __shfl_xor_sync(0xffffffffu, l[hh], o);
      const float mn = fmaxf(m[hh], m2), mb = mn == -INFINITY ? 0.f : mn;
      l[hh] = l[hh] * ex2_approx(m[hh] - mb) + l2 * ex2_approx(m2 - mb);
      m[hh] = mn;
    }
    if (t == 0) {
      s_m[warp][g + 8 * hh] = m[hh];
      s_l[warp][g + 8 * hh] = l[hh];
    }
  }
  __syncthreads();
  if (tid < ROWS) {
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int v = 0; v < kSmallWarps; ++v) M = fmaxf(M, s_m[v][tid]);
    const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int v = 0; v < kSmallWarps; ++v) sum += s_l[v][tid] * ex2_approx(s_m[v][tid] - ms);
    s_ml[0][tid] = M;
    s_ml[1][tid] = sum;
  }
  cluster_sync();
  for (int i = tid; i < 2 * ROWS * csize; i += kSmallThreads) {
    const int which = i / (ROWS * csize), rest = i % (ROWS * csize);
    s_all[which][rest / ROWS][rest % ROWS] = ld_peer(&s_ml[which][rest % ROWS], rest / ROWS);
  }
  cp_async_wait_all();
  __syncthreads();   // the values of every thread, the peers' statistics
  float sum[HH];
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  float lse[HH];
#pragma unroll
  for (int hh = 0; hh < HH; ++hh) {
    sum[hh] = 0.f;
    const int r = g + 8 * hh;
    float M = -INFINITY, tot = 0.f;
    for (int c = 0; c < csize; ++c) M = fmaxf(M, s_all[0][c][r]);
    const float ms = M == -INFINITY ? 0.f : M;
    for (int c = 0; c < csize; ++c) tot += s_all[1][c][r] * ex2_approx(s_all[0][c][r] - ms);
    lse[hh] = ms + log2f(tot);
  }
#pragma unroll
  for (int j = 0; j < GROUPS; ++j) {
    const int k16 = 16 * (warp + j * kSmallWarps), valid = nk - k16 - 4 * t;
    if (k16 >= nk) break;
    uint32_t hi[HH][2], lo[HH][2];
#pragma unroll
    for (int hh = 0; hh < HH; ++hh) {
      const float de[4] = {dem[j][hh].x, dem[j][hh].y, dem[j][hh].z, dem[j][hh].w};
      float nd[4], sh[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float bid = ex2_approx(x[j][hh][e] - lse[hh]);
        nd[e] = de[e] + bid;
        sh[e] = on[hh] && e < valid ? bid * rcp_approx((p.earlier ? de[e] : nd[e]) + p.eps) : 0.f;
      }
      sum[hh] += (sh[0] + sh[1]) + (sh[2] + sh[3]);
      if (dp[j][hh] != nullptr) {
        if (valid >= 4) {
          *reinterpret_cast<float4 *>(dp[j][hh]) = make_float4(nd[0], nd[1], nd[2], nd[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (e < valid) dp[j][hh][e] = nd[e];
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float s0 = sh[2 * half], s1 = sh[2 * half + 1];
        const uint32_t h2 = pack_bf16x2(s0, s1);
        hi[hh][half] = h2;
        lo[hh][half] = pack_bf16x2(s0 - __uint_as_float(h2 << 16), s1 - __uint_as_float(h2 & 0xffff0000u));
      }
    }
    uint32_t a1[4], a2[4];
    if constexpr (WIDE) {
      a1[0] = hi[0][0], a1[1] = hi[HH - 1][0], a1[2] = hi[0][1], a1[3] = hi[HH - 1][1];
      a2[0] = lo[0][0], a2[1] = lo[HH - 1][0], a2[2] = lo[0][1], a2[3] = lo[HH - 1][1];
    } else {   // the second term in the unused rows
      a1[0] = hi[0][0], a1[1] = lo[0][0], a1[2] = hi[0][1], a1[3] = lo[0][1];
    }
    __syncwarp();
    const int row = k16 + group_key(lane & 7, (lane >> 3) & 1);
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t b[4];
      ldsm_x4_t(smem_u32(sV) + small_off<D>(row, n + (lane >> 4)), b);
      mma16816(acc[n], a1, b[0], b[1]);
      mma16816(acc[n + 1], a1, b[2], b[3]);
      if constexpr (WIDE) {
        mma16816(acc[n], a2, b[0], b[1]);
        mma16816(acc[n + 1], a2, b[2], b[3]);
      }
    }
  }
  __syncthreads();   // every warp has read its values: the sums may lie over them
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float *to = red + ((size_t)warp * ROWS + g) * D + 8 * n + 2 * t;
    if constexpr (WIDE) {
      *reinterpret_cast<float2 *>(to) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2 *>(to + 8 * D) = make_float2(acc[n][2], acc[n][3]);
    } else {
      *reinterpret_cast<float2 *>(to) = make_float2(acc[n][0] + acc[n][2], acc[n][1] + acc[n][3]);
    }
  }
#pragma unroll
  for (int hh = 0; hh < HH; ++hh) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) sum[hh] += __shfl_xor_sync(0xffffffffu, sum[hh], o);
    if (t == 0) s_sum[warp][g + 8 * hh] = sum[hh];
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += kSmallThreads) {
    const int r = i / D, e = i % D;
    float a = 0.f;
#pragma unroll
    for (int v = 0; v < kSmallWarps; ++v) a += red[((size_t)v * ROWS + r) * D + e];
    s_part[r][e] = a;
  }
  if (tid < G) {
    float a = 0.f;
#pragma unroll
    for (int v = 0; v < kSmallWarps; ++v) a += s_sum[v][tid];
    s_part[tid][D] = a;
  }
  cluster_sync();
  // each CTA joins an equal part of the outputs, over the CTAs in order
  for (int i = rank * kSmallThreads + tid; i < G * D; i += csize * kSmallThreads) {
    const int r = i / D, e = i % D;
    float a = 0.f, rs = 0.f;
    for (int c = 0; c < csize; ++c) {
      a += ld_peer(&s_part[r][e], c);
      rs += ld_peer(&s_part[r][D], c);
    }
    static_cast<__nv_bfloat16 *>(p.out)[((size_t)s * p.c.Hq + hkv * G + r) * D + e] =
        __float2bfloat16_rn(len > 0 ? a / rs : 0.f);
  }
  cluster_sync();   // no CTA leaves while a peer may read it
}

template <int D, bool WIDE>
static int launch_small_t(const PagedDecode &p, int csize, cudaStream_t stream) {
  constexpr int smem = 2 * small_keys(D) * D * 2;
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return cudaFuncSetAttribute(pgs_small<D, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  int shift = 0;
  while ((1 << shift) < p.c.page_size) ++shift;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.S * p.c.Hkv * csize));
  cfg.blockDim = dim3(kSmallThreads);
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
  return cudaLaunchKernelEx(&cfg, pgs_small<D, WIDE>, p, p.c.Hq / p.c.Hkv, shift, csize) == cudaSuccess ? DA_OK
                                                                                                        : DA_ERR_CUDA;
}

int launch_paged_small_bf16(const PagedDecode &p, int csize, cudaStream_t stream) {
  const bool wide = p.c.Hq / p.c.Hkv > 8;
  if (p.c.d == 128) return wide ? launch_small_t<128, true>(p, csize, stream) : launch_small_t<128, false>(p, csize, stream);
  return wide ? launch_small_t<64, true>(p, csize, stream) : launch_small_t<64, false>(p, csize, stream);
}

}  // namespace da
