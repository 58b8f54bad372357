// Chunks over the paged cache on CUDA cores, fp32 arithmetic throughout (TF32
// products would miss the type's accuracy).
//
// Mathematics: query i of a sequence's n new ones (its last n tokens; place P + i)
// and query head h, over the keys t <= P + i:
//   x = q . k_t tau / sqrt(d) log2 e,  p = 2^(x - lse2),
//   total_t += p,  share = p / (total_t + eps)  (the total before p with the
//   earlier demand only),  out = sum share v / sum share.
//   ckf_keys    (max, sum 2^(x - max)) of every row over a piece's keys;
//   ckf_values  shares and totals, sums of share v and share over them.
//
// What bounds it: the fp32 units (three products of d a pair) once a key is seen
// by a dozen rows.  A tile is 64 rows by 64 keys, 256 threads with 4 x 4 products
// each, 8 reads of 16 bytes for 32 packed multiply-adds; warps without rows leave the
// products out.  K and V have a place each, filled by asynchronous copies as soon as
// the tile before has been read.  A key's total runs over the rows of a tile: four
// threads a key take 16 rows each, after they have exchanged the sums of their bids
// (one thread a key left 3/4 of the block idle).
#include "da_chunk.cuh"

namespace da {

constexpr int kCkfEdge = 64;
constexpr int kCkfThreads = 256;
constexpr int ckf_ctas(int d) { return d == 64 ? 304 : 152; }   // two CTAs an SM, or one

ChunkPlan chunk_plan_f32(int S, int Hq, int Hkv, int d, long long N, int max_new, int page_size) {
  return chunk_plan(S, Hq, Hkv, d, N, max_new, page_size, kCkfEdge, ckf_ctas(d), ckf_ctas(d), ChunkCost{4, 4, 1, 8, 4});
}

template <int D>
struct Ckf {
  static constexpr int kLd = D + 4;            // floats of a staged row: lanes of different rows read different banks
  static constexpr int kLdP = kCkfEdge + 4;
  static constexpr int kSmemBytes = (3 * kCkfEdge * kLd + kCkfEdge * kLdP + 4 * kCkfEdge) * 4;
};

// A column tile: row c of it is query head hq(c), query i(c).
struct CkfCols {
  int r0, rows;          // first row of the segment; rows
  int hq0, n8, i0, n;    // wide: n8 = 0
  __device__ __forceinline__ CkfCols(const ChunkWalk &k, const ChunkPlan &w, int b) {
    r0 = b * k.g.step;
    n = k.g.n;
    if (k.g.wide) {
      n8 = 0;
      hq0 = k.seg;
      i0 = r0;
      rows = min(k.g.step, n - r0);
    } else {
      n8 = k.g.n8;
      hq0 = k.seg * w.G + r0 / n8;
      i0 = 0;
      rows = min(k.g.step, w.G * n8 - r0);
    }
  }
  __device__ __forceinline__ int head(int c) const { return n8 ? hq0 + c / n8 : hq0; }
  __device__ __forceinline__ int query(int c) const { return n8 ? c % n8 : i0 + c; }
  __device__ __forceinline__ bool valid(int c) const { return c < rows && query(c) < n; }
};

template <int D>
__device__ __forceinline__ void ckf_queries(const PagedChunk &p, const ChunkWalk &k, const CkfCols &t, float *sQ) {
  for (int e = threadIdx.x; e < kCkfEdge * (D / 4); e += kCkfThreads) {
    const int c = e / (D / 4), x = e % (D / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t.valid(c))
      v = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) +
                                                  ((size_t)(k.q.tok0 + t.query(c)) * p.c.Hq + t.head(c)) * D) + x);
    *reinterpret_cast<float4 *>(sQ + c * Ckf<D>::kLd + 4 * x) = v;
  }
}

// Asynchronous copies of key tile `tile` of K or V: one group.  Zeros past the
// sequence's end and where there is no page (recorded).  A thread's rows lie
// kCkfThreads / (d / 4) apart.
template <int D>
__device__ __forceinline__ void ckf_rows(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, const void *pages,
                                         int tile, float *to) {
  constexpr int STEP = kCkfThreads / (D / 4), ROWS = kCkfEdge / STEP;
  const int sh = w.page_shift, ps = 1 << sh, hkv = k.hkv(w);
  const int j0 = threadIdx.x / (D / 4), x = threadIdx.x % (D / 4);
  const int32_t *table = p.c.page_table + (size_t)k.s * p.c.max_pages;
  int page[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int key = tile * kCkfEdge + j0 + i * STEP;
    page[i] = key < k.g.len ? __ldcg(table + (key >> sh)) : -1;
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int j = j0 + i * STEP, key = tile * kCkfEdge + j;
    const bool ok = (unsigned)page[i] < (unsigned)p.c.num_pages;
    if (!ok && key < k.g.len) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    const float *from = static_cast<const float *>(pages);
    if (ok) from += ((((size_t)page[i] * p.c.Hkv + hkv) << sh) + (key & (ps - 1))) * D + 4 * x;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to + j * Ckf<D>::kLd + 4 * x)),
                 "l"(reinterpret_cast<uint64_t>(from)), "r"(ok ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void ckf_landed() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Where the total of (key, query head) lies; null without one.
__device__ __forceinline__ float *ckf_total(const PagedChunk &p, const ChunkPlan &w, const ChunkWalk &k, int key, int hq) {
  if (key >= k.g.len) return nullptr;
  const int sh = w.page_shift;
  const int page = __ldcg(p.c.demand_table + (size_t)k.s * p.c.max_pages + (key >> sh));
  if ((unsigned)page >= (unsigned)p.c.num_demand_pages) {
    atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    return nullptr;
  }
  return p.c.demand_pages + ((((size_t)page * p.c.Hq + hq) << sh) + (key & ((1 << sh) - 1)));
}

// Rows 4 ty .. by keys tx + 16 j: q . k.
template <int D>
__device__ __forceinline__ void ckf_products(const float *sQ, const float *sK, float (&x)[4][4]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float2 acc[4][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[r][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int e = 0; e < D; e += 4) {
    float4 kv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4 *>(sK + (tx + 16 * j) * Ckf<D>::kLd + e);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float4 q = *reinterpret_cast<const float4 *>(sQ + (4 * ty + r) * Ckf<D>::kLd + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[r][j] = ffma2(make_float2(q.x, q.y), make_float2(kv[j].x, kv[j].y), acc[r][j]);
        acc[r][j] = ffma2(make_float2(q.z, q.w), make_float2(kv[j].z, kv[j].w), acc[r][j]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[r][j] = acc[r][j].x + acc[r][j].y;
}

template <int D>
__global__ void __launch_bounds__(kCkfThreads, D == 64 ? 2 : 1) ckf_keys(PagedChunk p, ChunkPlan w) {
  using C = Ckf<D>;
  extern __shared__ __align__(16) float ckf_smem[];
  float *sQ = ckf_smem, *sK = sQ + kCkfEdge * C::kLd;   // two key tiles
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  pdl_wait();
  pdl_launch_dependents();
  const ChunkLine l = chunk_line(p, w);
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_keys);
  ChunkWalk k;
  for (k.start(p, w, l, cut, threadIdx.x % 32); k.any(); k.next(p, w, l)) {
    for (int b = k.g.col0(k.tile); b < k.g.cols; ++b) {
      const CkfCols t(k, w, b);
      const int end = min(k.end, k.g.seen(b, kCkfEdge));
      const bool work = threadIdx.x / 32 * 8 < t.rows;   // uniform over the warp
      __syncthreads();
      ckf_rows<D>(p, w, k, p.c.k_pages, k.tile, sK);
      ckf_queries<D>(p, k, t, sQ);
      float m[4], sum[4], c2[4];
      int last[4];   // the last key that the row sees
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int c = 4 * ty + r;
        m[r] = -INFINITY;
        sum[r] = 0.f;
        last[r] = t.valid(c) ? k.g.P + t.query(c) : -1;
        c2[r] = last[r] >= 0 ? head_c2(p.hs, k.s * p.c.Hq + t.head(c), p.status) : 0.f;
      }
      for (int tile = k.tile; tile < end; ++tile) {
        float *now = sK + ((tile - k.tile) & 1) * kCkfEdge * C::kLd;
        if (tile + 1 < end) {   // into the place of the tile before this one, which the barrier below follows
          ckf_rows<D>(p, w, k, p.c.k_pages, tile + 1, sK + ((tile + 1 - k.tile) & 1) * kCkfEdge * C::kLd);
          ckf_landed<1>();
        } else {
          ckf_landed<0>();
        }
        __syncthreads();
        if (work) {
          float x[4][4];
          ckf_products<D>(sQ, now, x);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float mn = m[r];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[r][j] = tile * kCkfEdge + tx + 16 * j <= last[r] ? x[r][j] * c2[r] : -INFINITY;
              mn = fmaxf(mn, x[r][j]);
            }
            const float ms = mn == -INFINITY ? 0.f : mn;
            sum[r] *= ex2_approx(m[r] - ms);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[r] += ex2_approx(x[r][j] - ms);
            m[r] = mn;
          }
        }
        __syncthreads();
      }
      if (!work) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          const float m2 = __shfl_xor_sync(0xffffffffu, m[r], o), s2 = __shfl_xor_sync(0xffffffffu, sum[r], o);
          const float mn = fmaxf(m[r], m2), ms = mn == -INFINITY ? 0.f : mn;
          sum[r] = sum[r] * ex2_approx(m[r] - ms) + s2 * ex2_approx(m2 - ms);
          m[r] = mn;
        }
        if (tx == 0 && last[r] >= 0)
          *reinterpret_cast<float2 *>(chunk_place(p, w.ml_a, w.ml_b, k.row0(p, w), w.cta_rows, k.tile, blockIdx.x,
                                                  t.r0 + 4 * ty + r, 2)) = make_float2(m[r], sum[r]);
      }
    }
  }
}

// bid / den, den > 0 (a reciprocal within an ulp); 0 without a bid, whatever den.
__device__ __forceinline__ float ckf_share(float bid, float den) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(den));
  return bid > 0.f ? bid * r : bid;
}

template <int D>
__global__ void __launch_bounds__(kCkfThreads, D == 64 ? 2 : 1) ckf_values(PagedChunk p, ChunkPlan w) {
  using C = Ckf<D>;
  constexpr int NV = D / 64;   // 4-column groups of a thread
  extern __shared__ __align__(16) float ckf_smem[];
  float *sQ = ckf_smem, *sK = sQ + kCkfEdge * C::kLd, *sV = sK + kCkfEdge * C::kLd, *sP = sV + kCkfEdge * C::kLd,
        *sPart = sP + kCkfEdge * C::kLdP;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  pdl_wait();
  pdl_launch_dependents();
  const ChunkLine l = chunk_line(p, w);
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_values);
  const float *nl_all = reinterpret_cast<const float *>(p.ws + w.nl);
  ChunkWalk k;
  for (k.start(p, w, l, cut, tid % 32); k.any(); k.next(p, w, l)) {
    for (int b = k.g.col0(k.tile); b < k.g.cols; ++b) {
      const CkfCols t(k, w, b);
      const int end = min(k.end, k.g.seen(b, kCkfEdge));
      const bool work = tid / 32 * 8 < t.rows;   // uniform over the warp
      __syncthreads();
      ckf_rows<D>(p, w, k, p.c.k_pages, k.tile, sK);
      ckf_rows<D>(p, w, k, p.c.v_pages, k.tile, sV);
      ckf_queries<D>(p, k, t, sQ);
      float c2[4], nl[4], num[4][4 * NV], sum[4];
      int last[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int c = 4 * ty + r;
        last[r] = t.valid(c) ? k.g.P + t.query(c) : -1;
        c2[r] = last[r] >= 0 ? head_c2(p.hs, k.s * p.c.Hq + t.head(c), nullptr) : 0.f;
        nl[r] = last[r] >= 0 ? __ldcg(nl_all + k.row0(p, w) + t.r0 + c) : 0.f;
        sum[r] = 0.f;
#pragma unroll
        for (int e = 0; e < 4 * NV; ++e) num[r][e] = 0.f;
      }
      // the totals of one head's keys are brought a tile ahead (their thread writes them
      // in this column tile's tile, and reads them in the next column tile's)
      const int key_l = tid % kCkfEdge, part = tid / kCkfEdge;
      for (int tile = k.tile; tile < end; ++tile) {
        const int key = tile * kCkfEdge + key_l;
        float *col = sP + key_l, *at = nullptr;
        float before = 0.f;
        if (t.n8 == 0) {
          at = ckf_total(p, w, k, key, t.hq0);
          if (at != nullptr) before = __ldcg(at);
        }
        ckf_landed<1>();   // K (V is the newer group)
        __syncthreads();
        if (work) {
          float x[4][4];
          ckf_products<D>(sQ, sK, x);
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool sees = tile * kCkfEdge + tx + 16 * j <= last[r];
              sP[(4 * ty + r) * C::kLdP + tx + 16 * j] = sees ? ex2_approx(fmaf(x[r][j], c2[r], nl[r])) : 0.f;
            }
        }
        __syncthreads();
        if (tile + 1 < end) ckf_rows<D>(p, w, k, p.c.k_pages, tile + 1, sK);
        if (t.n8 == 0) {   // one head: 16 rows a thread
          const int rows = min(16, t.rows - 16 * part);
          float mine = 0.f, run = 0.f;   // the rows' bids, summed apart from the total: it would take their last bits
          for (int c = 0; c < rows; ++c) mine += col[(16 * part + c) * C::kLdP];
          sPart[part * kCkfEdge + key_l] = mine;
          __syncthreads();
          for (int i = 0; i < part; ++i) run += sPart[i * kCkfEdge + key_l];
#pragma unroll 4
          for (int c = 0; c < rows; ++c) {
            const float bid = col[(16 * part + c) * C::kLdP], after = run + bid;
            col[(16 * part + c) * C::kLdP] = ckf_share(bid, before + (p.earlier ? run : after) + p.eps);
            run = after;
          }
          if (part == 3 && at != nullptr) __stcg(at, before + run);
        } else {
          for (int h = part; h * t.n8 < t.rows; h += kCkfThreads / kCkfEdge) {
            float *head_at = ckf_total(p, w, k, key, t.hq0 + h);
            const float held = head_at != nullptr ? __ldcg(head_at) : 0.f;
            float run = 0.f;
#pragma unroll 4
            for (int c = h * t.n8; c < h * t.n8 + t.n; ++c) {
              const float bid = col[c * C::kLdP], after = run + bid;
              col[c * C::kLdP] = ckf_share(bid, held + (p.earlier ? run : after) + p.eps);
              run = after;
            }
            if (head_at != nullptr) __stcg(head_at, held + run);
          }
        }
        if (tile + 1 < end)
          ckf_landed<1>();   // V (the next K is the newer group)
        else
          ckf_landed<0>();
        __syncthreads();
        if (work) {
#pragma unroll 4
          for (int j = 0; j < kCkfEdge; j += 4) {
            float4 sh[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              sh[r] = *reinterpret_cast<const float4 *>(sP + (4 * ty + r) * C::kLdP + j);
              if (j / 4 == tx) sum[r] += (sh[r].x + sh[r].y) + (sh[r].z + sh[r].w);
            }
#pragma unroll
            for (int e = 0; e < NV; ++e) {
              float4 v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4 *>(sV + (j + i) * C::kLd + 64 * e + 4 * tx);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float s4[4] = {sh[r].x, sh[r].y, sh[r].z, sh[r].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float2 &lo = *reinterpret_cast<float2 *>(&num[r][4 * e]), &hi = *reinterpret_cast<float2 *>(&num[r][4 * e + 2]);
                  lo = ffma2(make_float2(s4[i], s4[i]), make_float2(v[i].x, v[i].y), lo);
                  hi = ffma2(make_float2(s4[i], s4[i]), make_float2(v[i].z, v[i].w), hi);
                }
              }
            }
          }
        }
        __syncthreads();
        if (tile + 1 < end) ckf_rows<D>(p, w, k, p.c.v_pages, tile + 1, sV);
      }
      if (!work) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
        if (last[r] < 0) continue;
        float *to = chunk_place(p, w.acc_a, w.acc_b, k.row0(p, w), w.cta_rows, k.tile, blockIdx.x, t.r0 + 4 * ty + r,
                                acc_stride(D));
#pragma unroll
        for (int e = 0; e < NV; ++e)
          *reinterpret_cast<float4 *>(to + 64 * e + 4 * tx) =
              make_float4(num[r][4 * e], num[r][4 * e + 1], num[r][4 * e + 2], num[r][4 * e + 3]);
        if (tx == 0) to[D] = sum[r];
      }
    }
  }
}

cudaError_t launch_chunk_plan(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);      // paged_chunk.cu
cudaError_t launch_chunk_join(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);
cudaError_t launch_chunk_combine(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream);

template <int D>
static int launch_ckf(const PagedChunk &p, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return (cudaFuncSetAttribute(ckf_keys<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ckf<D>::kSmemBytes) !=
                cudaSuccess ||
            cudaFuncSetAttribute(ckf_values<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ckf<D>::kSmemBytes) !=
                cudaSuccess)
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  const ChunkPlan w = chunk_plan_f32(p.c.S, p.c.Hq, p.c.Hkv, D, p.N, p.max_new, p.c.page_size);
  if (launch_chunk_plan(p, w, stream) != cudaSuccess ||
      launch_after(ckf_keys<D>, w.ctas_keys, kCkfThreads, Ckf<D>::kSmemBytes, stream, p, w) != cudaSuccess ||
      launch_chunk_join(p, w, stream) != cudaSuccess ||
      launch_after(ckf_values<D>, w.ctas_values, kCkfThreads, Ckf<D>::kSmemBytes, stream, p, w) != cudaSuccess ||
      launch_chunk_combine(p, w, stream) != cudaSuccess)
    return DA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int launch_chunk_f32(const PagedChunk &p, cudaStream_t stream) {
  return p.c.d == 128 ? launch_ckf<128>(p, stream) : launch_ckf<64>(p, stream);
}
}  // namespace da
