// Decode step over the paged cache, on CUDA cores (every type and layout).
//
// The operator of decode.cu for sequences of different lengths whose keys and
// values are scattered over pages, with Hq / Hkv query heads sharing a key
// head, and with an optional prefix that the whole batch shares:
//   x_k = q . k_k tau / sqrt(d) log2 e,  p_k = 2^(x_k - lse2),
//   share_k = p_k / (D_k + p_k + eps),  out = sum share_k v_k / sum share_k,
//   D_k += p_k.
// A share needs the finished softmax normaliser, so there are two passes:
// pgs_logits writes the logits and each chunk's (max, sum), pgs_update forms
// the shares and their sums, pgs_combine joins the chunks in a fixed order.
//
// Work is cut into (chunk of 256 keys, key head, rows): the rows of a
// sequence's own part are the query heads that share the key head; the rows
// of the prefix are those of the whole batch, 16 at a time, so a prefix key is
// read once for 16 rows.
#include "da_paged.h"
#include "da_ptx.cuh"

#include <cuda_bf16.h>

namespace da {

constexpr int kPgsThreads = 256;
constexpr int kPgsChunk = 256;   // keys per block, one per thread
constexpr int kPgsRows = 16;     // rows per block at most

// Workspace: status | logits [S Hq][Lp] | (max, sum) [S Hq][nchunk] | partial
// rows [S Hq][nchunk][d + 4].
struct PgsLayout {
  size_t logit_off, ml_off, acc_off, total;
  int Lp, prefix_chunks, own_chunks, nchunk;
};
DA_HD PgsLayout pgs_layout(int64_t rows, int max_len, int prefix_len, int d) {
  PgsLayout w;
  w.Lp = (int)round_up(max_len, 16);
  w.prefix_chunks = (prefix_len + kPgsChunk - 1) / kPgsChunk;
  w.own_chunks = (max_len - prefix_len + kPgsChunk - 1) / kPgsChunk;
  w.nchunk = (max_len + kPgsChunk - 1) / kPgsChunk + 1;   // for any prefix

  w.logit_off = kStatusBytes;
  w.ml_off = (size_t)round_up((int64_t)w.logit_off + rows * w.Lp * 4, 256);
  w.acc_off = (size_t)round_up((int64_t)w.ml_off + rows * w.nchunk * 8, 256);
  w.total = (size_t)round_up((int64_t)w.acc_off + rows * w.nchunk * acc_stride(d) * 4, 256);
  return w;
}
size_t pgs_workspace(int64_t rows, int max_len, int prefix_len, int d) {
  return pgs_layout(rows, max_len, prefix_len, d).total;
}

template <typename E>
struct PgsVec;
template <>
struct PgsVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void to_float(const uint4 &u, float *f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct PgsVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void to_float(const uint4 &u, float *f) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
};

// What a block works on: grid (chunk, key head, z).  z < S is a sequence's own
// part, z >= S + 16-row group of the prefix.
struct PgsBlock {
  int hkv, nrows, row0, key0, key_end, chunk;   // keys [key0, key_end)
  int s;                                        // own part: its sequence, prefix: -1
  // row r of the block is query row (sequence, query head)
  __device__ __forceinline__ void row(const PagedDecode &p, int G, int r, int &seq, int &hq) const {
    const int gr = s >= 0 ? r : row0 + r;
    seq = s >= 0 ? s : gr / G;
    hq = hkv * G + (s >= 0 ? row0 + r : gr % G);
  }
};

// Blocks of sequences whose own part needs more than 16 rows per key head
// split them: z = group * S + s.
__device__ __forceinline__ PgsBlock pgs_block(const PagedDecode &p, const PgsLayout &L, int G, int own_groups) {
  PgsBlock b;
  b.hkv = blockIdx.y;
  const int z = blockIdx.z, own = own_groups * p.c.S;
  if (z < own) {
    b.s = z % p.c.S;
    b.row0 = z / p.c.S * kPgsRows;
    b.nrows = min(G - b.row0, kPgsRows);
    b.chunk = L.prefix_chunks + blockIdx.x;
    b.key0 = p.prefix_len + blockIdx.x * kPgsChunk;
    b.key_end = (int)blockIdx.x < L.own_chunks
                    ? min(b.key0 + kPgsChunk, paged_len(p, b.s, threadIdx.x == 0 ? p.status : nullptr))
                    : -1;
  } else {
    b.s = -1;
    b.row0 = (z - own) * kPgsRows;
    b.nrows = min(p.c.S * G - b.row0, kPgsRows);
    b.chunk = blockIdx.x;
    b.key0 = blockIdx.x * kPgsChunk;
    b.key_end = min(b.key0 + kPgsChunk, p.prefix_len);
  }
  return b;
}

__device__ __forceinline__ int pgs_page(const PagedDecode &p, const PgsBlock &b, int key) {
  const int32_t *e = b.s >= 0 ? p.c.page_table + (size_t)b.s * p.c.max_pages + key / p.c.page_size
                              : p.prefix_table + key / p.c.page_size;
  return checked_page(e, p.c.num_pages, p.status);
}

template <typename E, int D>
__global__ void __launch_bounds__(kPgsThreads) pgs_logits(PagedDecode p, PgsLayout L, int own_groups) {
  constexpr int NV = PgsVec<E>::N;
  __shared__ __align__(16) float sq[kPgsRows][D];
  __shared__ int s_len[kPgsRows];
  __shared__ float s_c2[kPgsRows];
  __shared__ float2 s_ml[kPgsThreads / 32][kPgsRows];
  const int G = p.c.Hq / p.c.Hkv, tid = threadIdx.x;
  const PgsBlock b = pgs_block(p, L, G, own_groups);
  if (b.s >= 0 && (int)blockIdx.x >= L.own_chunks) return;
  if (b.s < 0 && (int)blockIdx.x >= L.prefix_chunks) return;
  if (b.key0 >= b.key_end) {   // nothing here: an empty chunk
    if (tid < b.nrows) {
      int s, hq;
      b.row(p, G, tid, s, hq);
      reinterpret_cast<float2 *>(p.ws + L.ml_off)[((size_t)s * p.c.Hq + hq) * L.nchunk + b.chunk] =
          make_float2(-INFINITY, 0.f);
    }
    return;
  }
  for (int i = tid; i < b.nrows * D; i += kPgsThreads) {
    int s, hq;
    b.row(p, G, i / D, s, hq);
    const E x = static_cast<const E *>(p.q)[((size_t)s * p.c.Hq + hq) * D + i % D];
    sq[i / D][i % D] = (float)x;
  }
  if (tid < b.nrows) {
    int s, hq;
    b.row(p, G, tid, s, hq);
    s_len[tid] = b.s >= 0 ? b.key_end : (paged_len(p, s, nullptr) > 0 ? b.key_end : 0);
    s_c2[tid] = head_c2(p.hs, s * p.c.Hq + hq, p.status);
  }
  __syncthreads();
  const int key = b.key0 + tid;
  int page = -1;
  if (key < b.key_end) page = pgs_page(p, b, key);
  float acc[kPgsRows];
#pragma unroll
  for (int r = 0; r < kPgsRows; ++r) acc[r] = 0.f;
  if (page >= 0) {
    const uint4 *kr = reinterpret_cast<const uint4 *>(
        static_cast<const E *>(p.c.k_pages) +
        (((size_t)page * p.c.Hkv + b.hkv) * p.c.page_size + key % p.c.page_size) * D);
#pragma unroll 4
    for (int i = 0; i < D / NV; ++i) {
      float kf[NV];
      PgsVec<E>::to_float(__ldg(kr + i), kf);
#pragma unroll
      for (int r = 0; r < kPgsRows; ++r) {
        if (r < b.nrows) {
#pragma unroll
          for (int e = 0; e < NV; ++e) acc[r] = fmaf(sq[r][i * NV + e], kf[e], acc[r]);
        }
      }
    }
  }
  const int warp = tid / 32, lane = tid % 32;
#pragma unroll
  for (int r = 0; r < kPgsRows; ++r) {
    if (r >= b.nrows) break;
    const bool ok = page >= 0 && key < s_len[r];
    float x = ok ? acc[r] * s_c2[r] : -INFINITY;
    if (key < s_len[r]) {
      int s, hq;
      b.row(p, G, r, s, hq);
      reinterpret_cast<float *>(p.ws + L.logit_off)[((size_t)s * p.c.Hq + hq) * L.Lp + key] = x;
    }
    float m = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = ok ? exp2f(x - m) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) s_ml[warp][r] = make_float2(m, l);
  }
  __syncthreads();
  if (tid < b.nrows) {
    float m = -INFINITY, l = 0.f;
    for (int w = 0; w < kPgsThreads / 32; ++w) m = fmaxf(m, s_ml[w][tid].x);
    for (int w = 0; w < kPgsThreads / 32; ++w)
      if (s_ml[w][tid].y != 0.f) l += s_ml[w][tid].y * exp2f(s_ml[w][tid].x - m);
    int s, hq;
    b.row(p, G, tid, s, hq);
    reinterpret_cast<float2 *>(p.ws + L.ml_off)[((size_t)s * p.c.Hq + hq) * L.nchunk + b.chunk] = make_float2(m, l);
  }
}

template <typename E, int D>
__global__ void __launch_bounds__(kPgsThreads) pgs_update(PagedDecode p, PgsLayout L, int own_groups) {
  constexpr int NV = PgsVec<E>::N;
  constexpr int LPR = D / NV, KPR = kPgsThreads / LPR;   // lanes per key, keys side by side
  constexpr int RB = 2;                                  // rows accumulated at a time
  __shared__ float s_share[kPgsRows][kPgsChunk];
  __shared__ float s_lse[kPgsRows];
  __shared__ int s_page[kPgsChunk];
  __shared__ float s_sum[kPgsThreads / 32][kPgsRows];
  __shared__ float s_red[RB][KPR][D + 1];
  const int G = p.c.Hq / p.c.Hkv, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const PgsBlock b = pgs_block(p, L, G, own_groups);
  if (b.s >= 0 && (int)blockIdx.x >= L.own_chunks) return;
  if (b.s < 0 && (int)blockIdx.x >= L.prefix_chunks) return;
  if (b.key0 >= b.key_end) return;
  // lse2 of the block's rows: one warp per row over the chunks' (max, sum)
  for (int r = warp; r < b.nrows; r += kPgsThreads / 32) {
    int s, hq;
    b.row(p, G, r, s, hq);
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws + L.ml_off) + ((size_t)s * p.c.Hq + hq) * L.nchunk;
    float m = -INFINITY, l = 0.f;
    for (int c = lane; c < L.prefix_chunks + L.own_chunks; c += 32) m = fmaxf(m, ml[c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int c = lane; c < L.prefix_chunks + L.own_chunks; c += 32)
      if (ml[c].y != 0.f) l += ml[c].y * exp2f(ml[c].x - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const bool active = b.s >= 0 || paged_len(p, s, nullptr) > 0;
    if (lane == 0) s_lse[r] = active ? m + log2f(l) : INFINITY;   // idle rows bid 0
  }
  const int key = b.key0 + tid;
  int page = -1;
  if (key < b.key_end) page = pgs_page(p, b, key);
  s_page[tid] = page;
  __syncthreads();
#pragma unroll 1
  for (int r = 0; r < b.nrows; ++r) {
    float share = 0.f;
    if (page >= 0 && s_lse[r] != INFINITY) {
      int s, hq;
      b.row(p, G, r, s, hq);
      const float x = reinterpret_cast<const float *>(p.ws + L.logit_off)[((size_t)s * p.c.Hq + hq) * L.Lp + key];
      const float bid = exp2f(x - s_lse[r]);
      const int dpg = checked_page(p.c.demand_table + (size_t)s * p.c.max_pages + key / p.c.page_size,
                                   p.c.num_demand_pages, p.status);
      if (dpg >= 0) {
        float *dp = p.c.demand_pages + ((size_t)dpg * p.c.Hq + hq) * p.c.page_size + key % p.c.page_size;
        const float dm = *dp;
        share = bid / ((p.earlier ? dm : dm + bid) + p.eps);
        *dp = dm + bid;
      }
    }
    s_share[r][tid] = share;
    float t = share;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) s_sum[warp][r] = t;
  }
  __syncthreads();
  const int sub = tid % LPR, grp = tid / LPR;
  const int nkeys = b.key_end - b.key0;
  for (int r0 = 0; r0 < b.nrows; r0 += RB) {
    float num[RB][NV];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int e = 0; e < NV; ++e) num[r][e] = 0.f;
    for (int kk = grp; kk < nkeys; kk += KPR) {
      const int pg = s_page[kk];
      if (pg < 0) continue;
      float vf[NV];
      PgsVec<E>::to_float(
          __ldg(reinterpret_cast<const uint4 *>(
                    static_cast<const E *>(p.c.v_pages) +
                    (((size_t)pg * p.c.Hkv + b.hkv) * p.c.page_size + (b.key0 + kk) % p.c.page_size) * D) +
                sub),
          vf);
#pragma unroll
      for (int r = 0; r < RB; ++r) {
        const float sh = r0 + r < b.nrows ? s_share[r0 + r][kk] : 0.f;
#pragma unroll
        for (int e = 0; e < NV; ++e) num[r][e] = fmaf(sh, vf[e], num[r][e]);
      }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int e = 0; e < NV; ++e) s_red[r][grp][sub * NV + e] = num[r][e];
    __syncthreads();
    for (int i = tid; i < RB * (D + 1); i += kPgsThreads) {
      const int r = i / (D + 1), e = i % (D + 1);
      if (r0 + r >= b.nrows) break;
      float a = 0.f;
      if (e < D)
        for (int gi = 0; gi < KPR; ++gi) a += s_red[r][gi][e];
      else
        for (int w = 0; w < kPgsThreads / 32; ++w) a += s_sum[w][r0 + r];
      int s, hq;
      b.row(p, G, r0 + r, s, hq);
      reinterpret_cast<float *>(p.ws +
                                L.acc_off)[(((size_t)s * p.c.Hq + hq) * L.nchunk + b.chunk) * acc_stride(D) + e] = a;
    }
    __syncthreads();
  }
}

// out = sum of the chunks' numerators / sum of their row sums, in chunk order.
template <typename E, int D>
__global__ void pgs_combine(PagedDecode p, PgsLayout L) {
  const int row = blockIdx.x, t = threadIdx.x;
  const int len = paged_len(p, row / p.c.Hq, nullptr);
  float a = 0.f, rs = 0.f;
  if (len > 0) {
    const int own = (len - p.prefix_len + kPgsChunk - 1) / kPgsChunk;
    const float *pa = reinterpret_cast<const float *>(p.ws + L.acc_off) + (size_t)row * L.nchunk * acc_stride(D);
    for (int c = 0; c < L.prefix_chunks + own; ++c) {
      a += pa[c * acc_stride(D) + t];
      rs += pa[c * acc_stride(D) + D];
    }
    a /= rs;
  }
  if constexpr (sizeof(E) == 4)
    static_cast<float *>(p.out)[(size_t)row * D + t] = a;
  else
    static_cast<__nv_bfloat16 *>(p.out)[(size_t)row * D + t] = __float2bfloat16_rn(a);
}

template <typename E, int D>
static cudaError_t launch_pgs_t(const PagedDecode &p, cudaStream_t stream) {
  const int G = p.c.Hq / p.c.Hkv;
  const PgsLayout L = pgs_layout((int64_t)p.c.S * p.c.Hq, p.max_len, p.prefix_len, D);
  const int own_groups = L.own_chunks > 0 ? (G + kPgsRows - 1) / kPgsRows : 0;
  const int prefix_groups = L.prefix_chunks > 0 ? (p.c.S * G + kPgsRows - 1) / kPgsRows : 0;
  const int nx = L.own_chunks > L.prefix_chunks ? L.own_chunks : L.prefix_chunks;
  if (nx > 0) {
    const dim3 grid(nx, p.c.Hkv, own_groups * p.c.S + prefix_groups);
    pgs_logits<E, D><<<grid, kPgsThreads, 0, stream>>>(p, L, own_groups);
    pgs_update<E, D><<<grid, kPgsThreads, 0, stream>>>(p, L, own_groups);
  }
  pgs_combine<E, D><<<p.c.S * p.c.Hq, D, 0, stream>>>(p, L);
  return cudaGetLastError();
}

cudaError_t launch_paged_decode_simt(const PagedDecode &p, cudaStream_t stream) {
  return p.c.d == 128 ? launch_pgs_t<float, 128>(p, stream) : launch_pgs_t<float, 64>(p, stream);
}

}  // namespace da
