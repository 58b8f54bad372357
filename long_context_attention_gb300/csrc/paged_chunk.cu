// Chunks over the paged cache: what both types share.  chunk_plan_kernel lays
// the call's work on its line, chunk_join makes each row's normaliser of the first
// pass's pieces and finds values that are not finite, chunk_combine its output of the
// second's.
//
// What bounds them: latency; the plan is one block, and the other two read a few
// pieces a row, (max, sum) and d + 1 floats each.  Over many rows chunk_combine comes to
// 5 TB/s (16 prompts of d = 128: 550 MB in 110 us).
#include "da_chunk.cuh"

#include <cuda_bf16.h>

namespace da {

int launch_chunk_f32(const PagedChunk &p, cudaStream_t stream);
int launch_chunk_bf16(const PagedChunk &p, cudaStream_t stream);
int chunk_small_cluster(int S, int Hq, int Hkv, int max_new, int max_len, int dtype);
int launch_chunk_small(const PagedChunk &p, int csize, cudaStream_t stream);

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

// One sequence, checked: its new tokens of this slice, or 0; its length up to them.
__device__ __forceinline__ ChunkSeq plan_seq(const PagedChunk &p, int s) {
  const int len = __ldcg(p.c.seq_lens + s), a = __ldcg(p.cu + s), b = __ldcg(p.cu + s + 1), n = b - a;
  if (len < 0 || len > p.max_len || a < 0 || b < a || b > p.N || n > p.all_new || n > len) {
    atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
    return ChunkSeq{0, 0, 0, a};
  }
  const int now = max(0, min(n - p.first, p.max_new));
  return ChunkSeq{now > 0 ? len - n + p.first + now : 0, now, 0, a + p.first};
}
__device__ __forceinline__ long long plan_units(const PagedChunk &p, const ChunkPlan &w, const ChunkSeq &q) {
  if (q.n == 0) return 0;
  ChunkShape g;
  g.set(q.len, q.n, p.c.Hq, p.c.Hkv, w.edge, w.cost);
  return g.units * g.segs;
}

// Up to 32 PER sequences by one warp: no block barriers (48 sequences 6.9 -> 5.1 us).
constexpr int kPlanFew = 4;   // of a lane
template <int PER>
__device__ __forceinline__ void plan_few(const PagedChunk &p, const ChunkPlan &w, ChunkSeq *seq, long long *cum) {
  const int lane = threadIdx.x, S = p.c.S;
  if (lane >= 32) return;
  const long long cap = w.rows / p.c.Hq;
  auto before = [&](long long v, long long &all) {   // the sum of the lanes before this one, and of all
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    all = __shfl_sync(0xffffffffu, inc, 31);
    return inc - v;
  };
  ChunkSeq q[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) q[i] = 32 * i + lane < S ? plan_seq(p, 32 * i + lane) : ChunkSeq{0, 0, 0, 0};
  long long rows = 0, units = 0, all;   // of the sequences before the 32 at hand: at most 128 x 2^30 rows
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = 32 * i + lane, n8 = (q[i].n + 7) & ~7;
    const long long at = rows + before(n8, all);
    rows += all;
    q[i].row0 = (int)(at < cap ? at : cap);
    if (at + n8 > cap && q[i].n > 0) {   // cu_tokens counts tokens twice
      atomicCAS(p.status, DA_OK, DA_ERR_INVALID);
      q[i].n = 0;
      q[i].row0 = (int)cap;
    }
    const long long first = units + before(plan_units(p, w, q[i]), all);
    units += all;
    if (s < S) {
      seq[s] = q[i];
      cum[s] = first;
      chunk_odd(p, w)[s] = 0;
    }
  }
  if (lane == 31) {
    seq[S] = ChunkSeq{0, 0, (int)(rows < cap ? rows : cap), 0};
    cum[S] = units;
  }
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(PagedChunk p, ChunkPlan w) {
  __shared__ long long warp_sum[kPlanThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  ChunkSeq *seq = reinterpret_cast<ChunkSeq *>(p.ws + w.seq_off);
  long long *cum = reinterpret_cast<long long *>(p.ws + w.cum_off);
  const int tid = threadIdx.x, S = p.c.S;
  if (S <= 32) {
    plan_few<1>(p, w, seq, cum);
    return;
  }
  if (S <= 32 * kPlanFew) {
    plan_few<kPlanFew>(p, w, seq, cum);
    return;
  }
  const int per = (S + kPlanThreads - 1) / kPlanThreads, s0 = min(tid * per, S), s1 = min(s0 + per, S);
  const long long cap = w.rows / p.c.Hq;
  long long rows = 0, units = 0, total;
  for (int s = s0; s < s1; ++s) {
    seq[s] = plan_seq(p, s);
    rows += (seq[s].n + 7) & ~7;
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
    units += plan_units(p, w, q);
  }
  units = plan_scan(units, warp_sum, total);
  if (tid == 0) cum[S] = total;
  for (int s = s0; s < s1; ++s) {
    const ChunkSeq q = seq[s];
    cum[s] = units;
    chunk_odd(p, w)[s] = 0;
    units += plan_units(p, w, q);
  }
}

constexpr int kRowWarps = 8;   // of a block
constexpr int kJoinCtas = 4, kCombineCtas = 2;   // blocks an SM (three of the second would not hold a row group's loads: 145 us for 110)

// A warp's rows: `run` times eight in succession, found once for each column tile.
template <typename F>
__device__ __forceinline__ void row_groups(const PagedChunk &p, const ChunkPlan &w, const ChunkLine &l, long long rows, int run,
                                           int blocks, int lane, F &&f) {
  for (long long r0 = 8ll * run * (blockIdx.x * kRowWarps + threadIdx.x / 32); r0 < rows; r0 += 8ll * run * blocks * kRowWarps) {
    ChunkRows x;
    bool known = false, fresh = false;
    for (long long row = r0; row < r0 + 8 * run && row < rows; row += 8) {
      if (known && x.i + 8 < x.g.n8 && (x.r + 8) / x.g.step == x.r / x.g.step) {
        x.i += 8;
        x.r += 8;
        fresh = false;
      } else {
        known = fresh = chunk_rows(p, w, l, row, lane, x);
      }
      if (known) f(x, row, fresh);
    }
  }
}

// Which of eight tokens (n of them are) of a key head have a value that is not finite: a bit each.
__device__ __forceinline__ unsigned values_odd(const PagedChunk &p, int sh, int s, int hkv, int t, int n, int lane) {
  const bool half = p.c.dtype == DA_BF16;
  const int pieces = p.c.d * (half ? 2 : 4) / 16;   // of 16 bytes: 8, 16 or 32
  int page = -1;
  if (lane < n) page = __ldcg(p.c.page_table + (size_t)s * p.c.max_pages + ((t + lane) >> sh));
  unsigned odd = 0;
#pragma unroll 4
  for (int e = lane; e < 8 * pieces; e += 32) {
    const int r = e / pieces, pg = __shfl_sync(0xffffffffu, page, r);
    if ((unsigned)pg >= (unsigned)p.c.num_pages) continue;
    uint4 v = __ldcg(reinterpret_cast<const uint4 *>(p.c.v_pages) +
                     ((((size_t)pg * p.c.Hkv + hkv) << sh) + ((t + r) & ((1 << sh) - 1))) * pieces + e % pieces);
    odd |= (unsigned)chunk_clear(v, half) << r;
  }
  return __reduce_or_sync(0xffffffffu, odd);
}

// -lse2 of every row, from (max, sum) of its pieces: a lane takes a row's every
// fourth piece.  Blocks from `blocks` on look through the new tokens' values meanwhile, eight
// tokens of a key head a warp (mixed batch of 48: 10 us less than the same warps before their
// rows).
__global__ void __launch_bounds__(32 * kRowWarps, kJoinCtas) chunk_join(PagedChunk p, ChunkPlan w, int run, int blocks) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 32, r = lane % 8, part = lane / 8;
  const ChunkLine l = chunk_line(p, w);
  const long long rows = (long long)__ldcg(&l.seq[p.c.S].row0) * p.c.Hq;
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_keys);
  float *nl = reinterpret_cast<float *>(p.ws + w.nl);
  if ((int)blockIdx.x >= blocks) {
    const long long of_keys = rows / w.G, step = 8ll * kRowWarps * (gridDim.x - blocks);
    for (long long row = 8ll * ((blockIdx.x - blocks) * kRowWarps + threadIdx.x / 32); row < of_keys; row += step) {
      const int s = chunk_seq_of(l, p.c.S, p.c.Hkv, row, lane);
      const ChunkSeq q = chunk_seq(l, s);
      if (q.n == 0) continue;   // (behind the last row)
      const int n8 = (q.n + 7) & ~7;
      const long long at = row - (long long)q.row0 * p.c.Hkv;
      const int hkv = (int)chunk_div(at, n8), i = (int)(at - (long long)hkv * n8);
      if (hkv >= p.c.Hkv) continue;
      const unsigned odd = values_odd(p, w.page_shift, s, hkv, q.len - q.n + i, min(q.n - i, 8), lane);
      if (lane > 0) continue;
      *chunk_odd_map(p, w, q.row0 + i, hkv) = (uint8_t)odd;
      if (odd != 0) chunk_odd(p, w)[s] = 1;
    }
    return;
  }
  ChunkPieces pc;
  int tile0 = -1;   // of the first 32 CTAs
  row_groups(p, w, l, rows, run, blocks, lane, [&](const ChunkRows &x, long long row, bool fresh) {
    if (fresh) {
      pc.find(x, cut);
      tile0 = pc.tile(x, cut, pc.first + lane);
    }
    const bool valid = x.i + r < x.q.n;
    float m = -INFINITY, sum = 0.f;
    for (int c = pc.first; c <= pc.last; c += 32) {
      const int tile = c == pc.first ? tile0 : pc.tile(x, cut, c + lane);
      const unsigned have = __ballot_sync(0xffffffffu, tile >= 0);
      for (int k = 0; k < __popc(have); k += 4) {
        const int from = k + part < __popc(have) ? __fns(have, 0, k + part + 1) : 0;
        const int t = __shfl_sync(0xffffffffu, tile, from);
        if (k + part < __popc(have) && valid) {
          const float2 ml = __ldcg(reinterpret_cast<const float2 *>(
              chunk_place(p, w.ml_a, w.ml_b, x.row0, w.cta_rows, t, c + from, x.r + r, 2)));
          const float mn = fmaxf(m, ml.x), ms = mn == -INFINITY ? 0.f : mn;
          sum = sum * ex2_approx(m - ms) + ml.y * ex2_approx(ml.x - ms);
          m = mn;
        }
      }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
      const float mn = fmaxf(m, m2), ms = mn == -INFINITY ? 0.f : mn;
      sum = sum * ex2_approx(m - ms) + s2 * ex2_approx(m2 - ms);
      m = mn;
    }
    if (part == 0 && valid) nl[row + r] = -(m + log2f(sum));
  });
}

// out = numerators / shares, summed over the pieces in the line's order.
template <int D, typename E>
__global__ void __launch_bounds__(32 * kRowWarps, kCombineCtas) chunk_combine(PagedChunk p, ChunkPlan w, int run) {
  constexpr int PER = D / 16;   // 16-byte pieces of a lane
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const ChunkLine l = chunk_line(p, w);
  const long long rows = (long long)__ldcg(&l.seq[p.c.S].row0) * p.c.Hq;
  const ChunkCut cut = chunk_cut(__ldcg(l.cum + p.c.S), w.ctas_values);
  ChunkPieces pc;
  int tile0 = -1;   // of the first 32 CTAs
  bool odd = false;
  row_groups(p, w, l, rows, run, gridDim.x, lane, [&](const ChunkRows &x, long long, bool fresh) {
    if (fresh) {
      pc.find(x, cut);
      tile0 = pc.tile(x, cut, pc.first + lane);
      odd = __ldcg(chunk_odd(p, w) + x.s) != 0;
    }
    const int r = lane % 8;                     // the lane's row
    const bool valid = x.i + r < x.q.n;
    // the second terms' sums of row r in row r + 4: see paged_chunk_bf16.cu
    const bool fold = sizeof(E) == 2 && w.logits_ld == 0 && x.q.n <= kChunkFold;
    const bool have_row = fold ? r % kChunkFold < x.q.n : valid;
    float4 a[PER];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = pc.first; c <= pc.last; c += 32) {
      const int tile = c == pc.first ? tile0 : pc.tile(x, cut, c + lane);
      for (unsigned have = __ballot_sync(0xffffffffu, tile >= 0); have; have &= have - 1) {
        const int from = __ffs(have) - 1, t = __shfl_sync(0xffffffffu, tile, from);
        const float *at = chunk_place(p, w.acc_a, w.acc_b, x.row0, w.cta_rows, t, c + from, x.r, acc_stride(D));
        if (!have_row) continue;
        float4 v[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = __ldcg(reinterpret_cast<const float4 *>(at + chunk_acc(D, r, lane / 8 + 4 * e)));
        sum += __ldcg(at + chunk_acc_sum(D, r));
#pragma unroll
        for (int e = 0; e < PER; ++e) a[e].x += v[e].x, a[e].y += v[e].y, a[e].z += v[e].z, a[e].w += v[e].w;
      }
    }
    if (fold) {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        a[e].x += __shfl_xor_sync(0xffffffffu, a[e].x, kChunkFold);
        a[e].y += __shfl_xor_sync(0xffffffffu, a[e].y, kChunkFold);
        a[e].z += __shfl_xor_sync(0xffffffffu, a[e].z, kChunkFold);
        a[e].w += __shfl_xor_sync(0xffffffffu, a[e].w, kChunkFold);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, kChunkFold);
    }
    if (odd) {   // what the rows see that is not finite, 32 times eight tokens at a time
      for (int i0 = 0; i0 <= x.i; i0 += 8 * 32) {
        const unsigned mine = i0 + 8 * lane <= x.i ? __ldcg(chunk_odd_map(p, w, x.q.row0 + i0 + 8 * lane, x.hq / w.G)) : 0u;
        for (unsigned have = __ballot_sync(0xffffffffu, mine != 0); have; have &= have - 1) {
          const int from = __ffs(have) - 1;
          for (unsigned bits = __shfl_sync(0xffffffffu, mine, from); bits; bits &= bits - 1) {
            const int i = i0 + 8 * from + __ffs(bits) - 1;
            if (valid && i <= x.i + r)
#pragma unroll
              for (int e = 0; e < PER; ++e)
                chunk_see<D, E>(p, w.page_shift, x.s, x.hq / w.G, x.g.P + i, lane / 8 * 4 + 16 * e, a[e]);
          }
        }
      }
    }
    if (!valid) return;
    // a normal reciprocal: one division does for the row
    const bool plain = sum >= 0x1p-100f && sum <= 0x1p100f;
    const float inv = plain ? 1.f / sum : 0.f;
    const size_t to = ((size_t)(x.q.tok0 + x.i + r) * p.c.Hq + x.hq) * D + lane / 8 * 4;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      float4 v = a[e];
      if (plain)
        v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
      else
        v.x /= sum, v.y /= sum, v.z /= sum, v.w /= sum;
      if constexpr (sizeof(E) == 4)
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to + 16 * e) = v;
      else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + to + 16 * e) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
  });
}

// Eight rows a warp where there are few, and where there are many up to 32 (16 prompts of
// d = 128, 325,000 rows: combine 122, 112, 110, 124 us at 8, 16, 32 and 64, join, without the
// blocks for values, 59, 43, 39, 48: a few rows find their segment again and again, many leave some warps far behind).
static int row_run(long long rows, int ctas) {
  const long long fill = 8ll * kRowWarps * 152 * ctas, run = (rows + fill - 1) / fill;
  return (int)(run < 1 ? 1 : run > 4 ? 4 : run);
}
static int row_blocks(long long rows, int ctas) {
  const long long each = 8ll * kRowWarps * row_run(rows, ctas), n = (rows + each - 1) / each, most = 152 * 64;
  return (int)(n < 1 ? 1 : n < most ? n : most);
}

cudaError_t launch_chunk_plan(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  return launch_after(chunk_plan_kernel, 1, p.c.S <= 32 * kPlanFew ? 32 : kPlanThreads, 0, stream, p, w);
}
cudaError_t launch_chunk_join(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  const int blocks = row_blocks(w.rows, kJoinCtas), of_keys = row_blocks(w.rows / w.G, kJoinCtas);
  return launch_after(chunk_join, blocks + of_keys, 32 * kRowWarps, 0, stream, p, w, row_run(w.rows, kJoinCtas), blocks);
}
template <typename E>
static cudaError_t launch_combine_t(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  return p.c.d == 128 ? launch_after(chunk_combine<128, E>, row_blocks(w.rows, kCombineCtas), 32 * kRowWarps, 0, stream, p, w, row_run(w.rows, kCombineCtas))
                      : launch_after(chunk_combine<64, E>, row_blocks(w.rows, kCombineCtas), 32 * kRowWarps, 0, stream, p, w, row_run(w.rows, kCombineCtas));
}
cudaError_t launch_chunk_combine(const PagedChunk &p, const ChunkPlan &w, cudaStream_t stream) {
  return p.c.dtype == DA_F32 ? launch_combine_t<float>(p, w, stream) : launch_combine_t<__nv_bfloat16>(p, w, stream);
}

// The plans of the types: edge, CTAs of the passes, costs (see the kernels).
ChunkPlan chunk_plan_f32(int S, int Hq, int Hkv, int d, long long N, int max_new, int page_size);
ChunkPlan chunk_plan_bf16(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len, int page_size);
size_t chunk_few_room(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len, long long &tokens, int &most);

// Enough for all calls within these bounds, those that keep their logits among them.
size_t chunk_workspace(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len, int dtype) {
  if (max_new > kChunkSlice) max_new = kChunkSlice;
  if (dtype == DA_F32) {   // up to 16 rows a key head have more CTAs
    const int few = 16 / (Hq / Hkv) / 8 * 8;
    const size_t all = chunk_plan_f32(S, Hq, Hkv, d, N, max_new, 16).total,
                 some = chunk_plan_f32(S, Hq, Hkv, d, N, max_new < few ? max_new : few, 16).total;
    return all > some ? all : some;
  }
  long long tokens;
  int most;
  const size_t room = chunk_few_room(S, Hq, Hkv, d, N, max_new, max_len, tokens, most);
  const size_t few = chunk_plan_bf16(S, Hq, Hkv, d, tokens, most, max_len, 16).total + room;
  const size_t all = chunk_plan_bf16(S, Hq, Hkv, d, N, max_new, max_len, 16).total;
  return all > few ? all : few;
}

int launch_paged_chunk(const PagedChunk &p, cudaStream_t stream) {
  const int c = chunk_small_cluster(p.c.S, p.c.Hq, p.c.Hkv, p.max_new, p.max_len, p.c.dtype);
  if (c > 0) return launch_chunk_small(p, c, stream);
  PagedChunk r = p;
  int st = DA_OK;
  do {
    r.max_new = p.max_new - r.first < kChunkSlice ? p.max_new - r.first : kChunkSlice;
    st = p.c.dtype == DA_F32 ? launch_chunk_f32(r, stream) : launch_chunk_bf16(r, stream);
    r.first += kChunkSlice;
  } while (st == DA_OK && r.first < p.max_new);
  return st;
}

}  // namespace da
