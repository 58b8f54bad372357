// Chunks over the paged cache: what both types share.  chunk_plan_kernel lays
// the call's work on its line, chunk_join makes each row's normaliser of the first
// pass's pieces, chunk_combine its output of the second's.
//
// What bounds them: latency.  The plan is one block; the other two read a few
// pieces a row, (max, sum) and d + 1 floats each.
#include "da_chunk.cuh"

#include <cuda_bf16.h>

namespace da {

int launch_chunk_f32(const PagedChunk &p, cudaStream_t stream);
int launch_chunk_bf16(const PagedChunk &p, cudaStream_t stream);

// Lengths and new tokens of every sequence, checked once; rows and units before
// each.  What is not valid is recorded and has no new tokens, so that no later
// kernel meets it.
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ long long plan_scan(long long v, long long *warp_sum, long long &total) {   // exclusive
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  long long base = 0;
  total = 0;
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < warp) base += warp_sum[i];
    total += warp_sum[i];
  }
  __syncthreads();
  return base + inc - v;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(PagedChunk p, ChunkPlan w) {
  __shared__ long long warp_sum[kPlanThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  ChunkSeq *seq = reinterpret_cast<ChunkSeq *>(p.ws + w.seq_off);
  long long *cum = reinterpret_cast<long long *>(p.ws + w.cum_off);
  const int tid = threadIdx.x, S = p.c.S;
  const int per = (S + kPlanThreads - 1) / kPlanThreads, s0 = min(tid * per, S), s1 = min(s0 + per, S);
  const long long cap = w.rows / p.c.Hq;
  long long rows = 0, units = 0, total;
  for (int s = s0; s < s1; ++s) {
    const int len = __ldcg(p.c.seq_lens + s), a = __ldcg(p.cu + s), b = __ldcg(p.cu + s + 1);
    int n = b - a;
    if (len < 0 || len > p.max_len || a < 0 || b < a || b > p.N || n > p.max_new || n > len) {
      atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      n = 0;
    }
    seq[s] = ChunkSeq{n > 0 ? len : 0, n, 0, a};
    rows += (n + 7) & ~7;
  }
  rows = plan_scan(rows, warp_sum, total);
  if (tid == 0) seq[S] = ChunkSeq{0, 0, (int)(total < cap ? total : cap), 0};
  for (int s = s0; s < s1; ++s) {
    ChunkSeq q = seq[s];
    const int n8 = (q.n + 7) & ~7;
    q.row0 = (int)rows;
    if (rows + n8 > cap) {   // cu_tokens counts tokens twice
      if (q.n > 0) atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      q.n = 0;
      q.row0 = (int)cap;
    }
    rows += n8;
    seq[s] = q;
    if (q.n > 0) {
      ChunkShape g;
      g.set(q.len, q.n, p.c.Hq, p.c.Hkv, w.edge, w.cost);
      units += g.units * g.segs;
    }
  }
  units = plan_scan(units, warp_sum, total);
  if (tid == 0) cum[S] = total;
  for (int s = s0; s < s1; ++s) {
    const ChunkSeq q = seq[s];
    cum[s] = units;
    if (q.n > 0) {
      ChunkShape g;
      g.set(q.len, q.n, p.c.Hq, p.c.Hkv, w.edge, w.cost);
      units += g.units * g.segs;
    }
  }
}

// -lse2 of every row, from (max, sum) of its pieces.
__global__ void __launch_bounds__(256) chunk_join(PagedChunk p, ChunkPlan w) {
  pdl_wait();
  pdl_launch_dependents();
  const ChunkLine l = chunk_line(p, w);
  const long long rows = (long long)__ldcg(&l.seq[p.c.S].row0) * p.c.Hq;
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_keys);
  float *nl = reinterpret_cast<float *>(p.ws + w.nl);
  for (long long row = (long long)blockIdx.x * 256 + threadIdx.x; row < rows; row += (long long)gridDim.x * 256) {
    ChunkRow x;
    if (!chunk_row(p, w, l, row, x)) continue;
    float m = -INFINITY, sum = 0.f;
    chunk_pieces(x, cut, [&](int tile, int cta) {
      const float2 ml = __ldcg(
          reinterpret_cast<const float2 *>(chunk_place(p, w.ml_a, w.ml_b, x.row0, w.cta_rows, tile, cta, x.r, 2)));
      const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
      sum = sum * ex2_approx(m - ms) + ml.y * ex2_approx(ml.x - ms);
      m = mn;
    });
    nl[row] = -(m + log2f(sum));
  }
}

// out = numerators / shares, summed over the pieces in the line's order.
template <int D, typename E>
__global__ void __launch_bounds__(256) chunk_combine(PagedChunk p, ChunkPlan w) {
  constexpr int LANES = D / 4;   // of a row
  pdl_wait();
  pdl_launch_dependents();
  const ChunkLine l = chunk_line(p, w);
  const long long rows = (long long)__ldcg(&l.seq[p.c.S].row0) * p.c.Hq;
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_values);
  const int c = threadIdx.x % LANES;
  for (long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / LANES; row < rows;
       row += (long long)gridDim.x * 256 / LANES) {
    ChunkRow x;
    if (!chunk_row(p, w, l, row, x)) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    chunk_pieces(x, cut, [&](int tile, int cta) {
      const float *at = chunk_place(p, w.acc_a, w.acc_b, x.row0, w.cta_rows, tile, cta, x.r, acc_stride(D));
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(at) + c);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
      sum += __ldcg(at + D);
    });
    const size_t to = ((size_t)(x.q.tok0 + x.i) * p.c.Hq + x.hq) * D + 4 * c;
    a.x /= sum, a.y /= sum, a.z /= sum, a.w /= sum;
    if constexpr (sizeof(E) == 4)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to) = a;
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + to) =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

static int row_blocks(long long rows, int per_block) {
  const long long n = (rows + per_block - 1) / per_block, most = 152 * 8;
  return (int)(n < 1 ? 1 : n < most ? n : most);
}

cudaError_t launch_chunk_plan(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  return launch_after(chunk_plan_kernel, 1, kPlanThreads, 0, stream, p, w);
}
cudaError_t launch_chunk_join(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  return launch_after(chunk_join, row_blocks(w.rows, 256), 256, 0, stream, p, w);
}
cudaError_t launch_chunk_combine(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  const int blocks = row_blocks(w.rows, 256 / (p.c.d / 4));
  if (p.c.dtype == DA_F32)
    return p.c.d == 128 ? launch_after(chunk_combine<128, float>, blocks, 256, 0, stream, p, w)
                        : launch_after(chunk_combine<64, float>, blocks, 256, 0, stream, p, w);
  return p.c.d == 128 ? launch_after(chunk_combine<128, __nv_bfloat16>, blocks, 256, 0, stream, p, w)
                      : launch_after(chunk_combine<64, __nv_bfloat16>, blocks, 256, 0, stream, p, w);
}

// The plans of the types: edge, CTAs of the passes, costs (see the kernels).
ChunkPlan chunk_plan_f32(int S, int Hq, int Hkv, int d, long long N, int max_new, int page_size);
ChunkPlan chunk_plan_bf16(int S, int Hq, int Hkv, int d, long long N, int max_new, int page_size);

size_t chunk_workspace(int S, int Hq, int Hkv, int d, long long N, int max_new, int dtype) {
  return (dtype == DA_F32 ? chunk_plan_f32(S, Hq, Hkv, d, N, max_new, 16)
                          : chunk_plan_bf16(S, Hq, Hkv, d, N, max_new, 16)).total;
}

int launch_paged_chunk(const PagedChunk &p, cudaStream_t stream) {
  return p.c.dtype == DA_F32 ? launch_chunk_f32(p, stream) : launch_chunk_bf16(p, stream);
}

}  // namespace da
