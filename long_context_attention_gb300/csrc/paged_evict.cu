// Eviction from the paged cache by accumulated demand.
//
// Definition: the score of token t for a key head is the sum of its query heads'
// totals, added in fp32 in the heads' order; the first `sinks` and the last
// `recent` tokens and those whose score is NaN score +infinity.  Of each key head
// the m = min(length, keep) tokens with the highest scores stay, equal scores by
// the lower place.  They keep their order and become tokens 0 .. m - 1.
//
// evict_select: a cluster per (sequence, key head), its scores in the CTAs' shared
// memory as integers of the same order.  The m-th highest is found by three counts
// of 11, 11 and 10 bits, the CTAs' counts summed through distributed shared
// memory; then each CTA writes the places of its tokens that stay.
//
// evict_move: rows to their new places.  In place, token list[r] >= r goes to r, so
// a block that takes rows in order, has read a batch before it writes it, and is
// alone on its bytes, never overwrites what is still to be read.  Blocks are
// therefore alone on a slice of a key head's rows (down to 32 bytes, a sector)
// instead of a part of the rows; to other pages the rows are split.
//
// What bounds it: HBM (4 bytes a total, then the rows that stay, once each way).
#include "da_evict.h"
#include "da_ptx.cuh"

namespace da {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kCopies = 4;   // of the counts: neighbouring lanes' scores fall into few bins

EvictWorkspace evict_workspace(int S, int Hkv, int max_keep, int max_len) {
  EvictWorkspace w;
  const int64_t items = (int64_t)S * Hkv;
  // CTAs of a cluster: up to 8 while the GPU has room and each still has 1024 keys
  int c = 1;
  while (c < kEvictCtas && ((items * c < 152 && max_len > c * 1024) || max_len > c * kEvictKeys / 3)) c *= 2;
  w.cluster = c;
  w.slice = (int)round_up((max_len + c - 1) / c, 32);
  w.shared = w.slice <= kEvictKeys;
  auto next = [](size_t off, int64_t bytes) { return (size_t)round_up((int64_t)off + bytes, 256); };
  w.info_off = kStatusBytes;
  w.list_off = next(w.info_off, (int64_t)S * 8);
  w.key_off = next(w.list_off, items * max_keep * 4);
  w.total = next(w.key_off, w.shared ? 0 : items * c * w.slice * 4);
  return w;
}

__device__ __forceinline__ uint32_t ev_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void ev_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t ev_peer(const void *local, uint32_t rank) {   // a word of a peer's shared memory
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Scores as integers of the same order; NaN as +infinity, -0 as 0.
__device__ __forceinline__ uint32_t ev_key(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xff800000u;
  if (u == 0x80000000u) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select(EvictArgs a, EvictWorkspace w, int page_shift) {
  extern __shared__ uint32_t sel_keys[];
  __shared__ uint32_t s_hist[kCopies + 1][kBins];   // the first pass's (the third's in its first copy); the second's
  __shared__ uint32_t s_above[kSelWarps], s_equal[kSelWarps], s_count[2], s_pick[2];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t rank = ev_rank(), C = (uint32_t)w.cluster;
  pdl_wait();
  pdl_launch_dependents();
  const int item = blockIdx.x / w.cluster, s = item / a.c.Hkv, h = item % a.c.Hkv, G = a.c.Hq / a.c.Hkv;
  const int len = __ldcg(a.c.seq_lens + s), keep = __ldcg(a.keep + s);
  const bool good = len >= 0 && len <= a.max_len && keep >= 0 && min(len, keep) <= a.max_keep;
  const int m = good ? min(len, keep) : 0;
  if (h == 0 && rank == 0 && tid == 0) {
    if (!good) atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
    reinterpret_cast<int2 *>(a.ws + w.info_off)[s] = make_int2(m, good ? m : len);
  }
  int32_t *list = (a.kept != nullptr ? a.kept : reinterpret_cast<int32_t *>(a.ws + w.list_off)) + (size_t)item * a.max_keep;
  if (a.kept != nullptr)
    for (int i = m + (int)rank * kSelThreads + tid; i < a.max_keep; i += (int)C * kSelThreads) list[i] = -1;
  if (m == 0) return;   // (the same in every CTA of the cluster)
  const int per = (int)round_up((len + w.cluster - 1) / w.cluster, 32);
  const int t0 = min((int)rank * per, len), cnt = min(len - t0, per);
  if (m == len) {
    for (int i = tid; i < cnt; i += kSelThreads) list[t0 + i] = t0 + i;
    return;
  }
  uint32_t *keys = w.shared ? sel_keys
                            : reinterpret_cast<uint32_t *>(a.ws + w.key_off) + ((size_t)item * w.cluster + rank) * w.slice;
  const int32_t *dtab = a.c.demand_table + (size_t)s * a.c.max_pages;
  const int ps = 1 << page_shift;
  for (int i = tid; i < (kCopies + 1) * kBins; i += kSelThreads) s_hist[0][i] = 0;
  __syncthreads();
  // four tokens a thread: they lie in one page
#pragma unroll 2
  for (int i = 4 * tid; i < cnt; i += 4 * kSelThreads) {
    const int t = t0 + i, page = __ldcg(dtab + (t >> page_shift));
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((unsigned)page < (unsigned)a.c.num_demand_pages) {
      const float *at = a.c.demand_pages + ((((size_t)page * a.c.Hq + (size_t)h * G) << page_shift) + (t & (ps - 1)));
      f = __ldcg(reinterpret_cast<const float4 *>(at));
#pragma unroll 2
      for (int g = 1; g < G; ++g) {
        const float4 o = __ldcg(reinterpret_cast<const float4 *>(at + ((size_t)g << page_shift)));
        f.x = __fadd_rn(f.x, o.x), f.y = __fadd_rn(f.y, o.y), f.z = __fadd_rn(f.z, o.z), f.w = __fadd_rn(f.w, o.w);
      }
    } else {
      atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
    }
    const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e >= cnt) break;
      const uint32_t key = ev_key(t + e < a.sinks || t + e >= len - a.recent ? INFINITY : v[e]);
      keys[i + e] = key;
      atomicAdd(&s_hist[lane % kCopies][key >> 21], 1u);
    }
  }
  __syncthreads();
  // three counts: the digits of the m-th highest key, and how many keys equal to it stay
  uint32_t prefix = 0, need = (uint32_t)m;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    uint32_t *hist = s_hist[pass == 1 ? kCopies : 0];
    if (pass > 0) {
      const int above = pass == 1 ? 21 : 10;
      for (int i = tid; i < cnt; i += kSelThreads) {
        const uint32_t key = keys[i];
        if (key >> above == prefix) atomicAdd(&hist[(key >> shift) & (uint32_t)(bins - 1)], 1u);
      }
    } else {
      for (int i = tid; i < kBins; i += kSelThreads)
#pragma unroll
        for (int k = 1; k < kCopies; ++k) hist[i] += hist[k * kBins + i];
    }
    if (C > 1)
      ev_sync();
    else
      __syncthreads();
    // thread i: 4 bins (2 in the last pass) from the top
    const int own = bins / kSelThreads;
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = 0;
      if (j < own) {
        const int bin = bins - 1 - (tid * own + j);
        if (C > 1)
          for (uint32_t r = 0; r < C; ++r) c[j] += ev_peer(hist + bin, r);
        else
          c[j] = hist[bin];
      }
      sum += c[j];
    }
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_above[warp] = inc;
    __syncthreads();
    uint32_t before = inc - sum;
    for (int i = 0; i < warp; ++i) before += s_above[i];
    if (before < need && need <= before + sum) {   // one thread
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < own && before < need && need <= before + c[j]) {
          s_pick[0] = (uint32_t)(bins - 1 - (tid * own + j));
          s_pick[1] = need - before;
          break;
        }
        before += c[j];
      }
    }
    __syncthreads();
    prefix = prefix << (pass == 2 ? 10 : 11) | s_pick[0];
    need = s_pick[1];
    // the first pass's counts are not read any more once every CTA has passed the second's barrier
    if (pass == 1) {
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[0][i] = 0;
      __syncthreads();
    }
  }
  // tokens above the key, and equal ones, before each warp's run of the CTA's keys
  const int run = (int)round_up((cnt + kSelWarps - 1) / kSelWarps, 32);
  const int r0 = min(warp * run, cnt), r1 = min(r0 + run, cnt);
  uint32_t above = 0, equal = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    const uint32_t key = keys[i];
    above += key > prefix;
    equal += key == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) s_above[warp] = above, s_equal[warp] = equal;
  __syncthreads();
  if (tid == 0) {
    uint32_t x = 0, y = 0;
    for (int i = 0; i < kSelWarps; ++i) {
      const uint32_t xa = s_above[i], ya = s_equal[i];
      s_above[i] = x, s_equal[i] = y;
      x += xa, y += ya;
    }
    s_count[0] = x, s_count[1] = y;
  }
  if (C > 1)
    ev_sync();
  else
    __syncthreads();
  uint32_t na = s_above[warp], ne = s_equal[warp];
  for (uint32_t r = 0; r < rank; ++r) na += ev_peer(&s_count[0], r), ne += ev_peer(&s_count[1], r);
  for (int i = r0; i < r1; i += 32) {
    const bool in = i + lane < r1;
    const uint32_t key = in ? keys[i + lane] : 0u;
    const uint32_t ba = __ballot_sync(0xffffffffu, in && key > prefix), be = __ballot_sync(0xffffffffu, in && key == prefix);
    const uint32_t lt = (1u << lane) - 1u;
    const uint32_t xa = na + __popc(ba & lt), xe = ne + __popc(be & lt);
    if (in && (key > prefix || (key == prefix && xe < need))) list[xa + min(xe, need)] = t0 + i + lane;
    na += __popc(ba);
    ne += __popc(be);
  }
  if (C > 1) ev_sync();   // no CTA leaves while a peer may read it
}

// ------------------------------------------------------------------------- the rows
constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 8;   // of a thread in flight

// One block: rows of a slice of one key head's keys or values (part < 2 slices), or
// the totals of one of its query heads.
struct MoveRows {
  const uint8_t *in;     // of page 0, first row of the head
  uint8_t *out;
  size_t page_bytes;     // from page to page
  int row_bytes, num_pages;
  const int32_t *src, *dst;
};

template <typename V>
__device__ __forceinline__ V ev_load(const uint8_t *p);
template <>
__device__ __forceinline__ uint4 ev_load<uint4>(const uint8_t *p) { return __ldcg(reinterpret_cast<const uint4 *>(p)); }
template <>
__device__ __forceinline__ float ev_load<float>(const uint8_t *p) { return __ldcg(reinterpret_cast<const float *>(p)); }

// Rows from .. to - 1 of the list, a batch of kMoveLoads steps at a time.  The places
// of a batch are found while the one before it is on its way: one read after the
// other (list, tables, rows) took 4.5 us a batch.
template <typename V>
__device__ __forceinline__ void move_rows(const EvictArgs &a, const MoveRows &x, const int32_t *list, int from, int to, int lane_row,
                                          int lane_byte, int rows_per_step, int sh, int *status) {
  const int ps = 1 << sh;
  int t[kMoveLoads], ip[kMoveLoads], op[kMoveLoads];
  auto entries = [&](int r0) {   // of the list
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) {
      const int r = r0 + lane_row + u * rows_per_step;
      t[u] = r < to ? __ldcg(list + r) : -1;
    }
  };
  auto pages = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) {
      const int r = r0 + lane_row + u * rows_per_step;
      ip[u] = t[u] >= 0 ? __ldg(x.src + (t[u] >> sh)) : 0;
      op[u] = t[u] >= 0 ? __ldg(x.dst + (r >> sh)) : 0;
    }
  };
  const int batch = kMoveLoads * rows_per_step;
  entries(from);
  pages(from);
  for (int r0 = from; r0 < to; r0 += batch) {
    V v[kMoveLoads];
    uint8_t *at[kMoveLoads];
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u) {
      const int r = r0 + lane_row + u * rows_per_step;
      at[u] = nullptr;
      if (t[u] >= 0) {
        if ((unsigned)ip[u] < (unsigned)x.num_pages && (unsigned)op[u] < (unsigned)x.num_pages) {
          const uint8_t *p = x.in + (size_t)ip[u] * x.page_bytes + (size_t)((t[u] & (ps - 1)) * x.row_bytes + lane_byte);
          uint8_t *q = x.out + (size_t)op[u] * x.page_bytes + (size_t)((r & (ps - 1)) * x.row_bytes + lane_byte);
          if (p != q) {
            at[u] = q;
            v[u] = ev_load<V>(p);
          }
        } else {
          atomicCAS(status, DA_OK, DA_ERR_INVALID);
        }
      }
    }
    entries(r0 + batch);
    pages(r0 + batch);
    __syncthreads();   // the batch has been read
#pragma unroll
    for (int u = 0; u < kMoveLoads; ++u)
      if (at[u] != nullptr) *reinterpret_cast<V *>(at[u]) = v[u];
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move(EvictArgs a, EvictWorkspace w, int sh, int slices) {
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, G = a.c.Hq / a.c.Hkv, parts = 2 * slices + G;
  const int item = blockIdx.x / parts, part = blockIdx.x % parts, s = item / a.c.Hkv, h = item % a.c.Hkv;
  const int2 info = __ldcg(reinterpret_cast<const int2 *>(a.ws + w.info_off) + s);
  const int m = info.x;
  if (h == 0 && part == 0 && blockIdx.y == 0 && tid == 0) a.new_lens[s] = info.y;
  const int32_t *list = (a.kept != nullptr ? a.kept : reinterpret_cast<const int32_t *>(a.ws + w.list_off)) +
                        (size_t)item * a.max_keep;
  const bool place = a.dst_page_table == nullptr;
  int from = 0, to = m;
  if (place) {   // the first row that moves: list[r] - r does not decrease
    int n = m;
    while (n > 0) {
      const int step = (n + kMoveThreads - 1) / kMoveThreads, r = from + tid * step;
      const int k = __syncthreads_count(tid * step < n && __ldcg(list + r) == r);
      if (k == 0) break;
      const int skip = (k - 1) * step + 1;
      from += skip;
      n = min(step - 1, n - skip);
    }
  } else {
    const int per = (m + gridDim.y - 1) / gridDim.y;
    from = min((int)blockIdx.y * per, m);
    to = min(from + per, m);
  }
  if (from >= to) return;
  const size_t smax = (size_t)s * a.c.max_pages, dmax = (size_t)s * (place ? a.c.max_pages : a.dst_max_pages);
  MoveRows x;
  if (part < 2 * slices) {
    const int eb = a.c.dtype == DA_BF16 ? 2 : 4;
    x.row_bytes = a.c.d * eb;
    x.page_bytes = ((size_t)a.c.Hkv * x.row_bytes) << sh;
    uint8_t *pool = reinterpret_cast<uint8_t *>(part < slices ? a.c.k_pages : a.c.v_pages) + (((size_t)h * x.row_bytes) << sh);
    x.in = x.out = pool;
    x.num_pages = a.c.num_pages;
    x.src = a.c.page_table + smax;
    x.dst = (place ? a.c.page_table : a.dst_page_table) + dmax;
    const int bytes = x.row_bytes / slices, lanes = bytes / 16;   // of a row: powers of two
    move_rows<uint4>(a, x, list, from, to, tid / lanes, part % slices * bytes + tid % lanes * 16, kMoveThreads / lanes, sh,
                     a.status);
  } else {
    const int hq = h * G + part - 2 * slices;
    x.row_bytes = 4;
    x.page_bytes = ((size_t)a.c.Hq * 4) << sh;
    x.in = x.out = reinterpret_cast<uint8_t *>(a.c.demand_pages) + (((size_t)hq * 4) << sh);
    x.num_pages = a.c.num_demand_pages;
    x.src = a.c.demand_table + smax;
    x.dst = (place ? a.c.demand_table : a.dst_demand_table) + dmax;
    move_rows<float>(a, x, list, from, to, tid, 0, kMoveThreads, sh, a.status);
  }
}

int launch_evict(const EvictArgs &a, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int prep = once.run([] {
    return cudaFuncSetAttribute(evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictKeys * 4) != cudaSuccess
               ? DA_ERR_CUDA
               : DA_OK;
  });
  if (prep != DA_OK) return prep;
  const EvictWorkspace w = evict_workspace(a.c.S, a.c.Hkv, a.max_keep < a.max_len ? a.max_keep : a.max_len, a.max_len);
  int sh = 0;
  while ((1 << sh) < a.c.page_size) ++sh;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.c.S * a.c.Hkv * w.cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = w.shared ? (size_t)w.slice * 4 : 0;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)w.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // (see launch_after)
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, evict_select, a, w, sh) != cudaSuccess) return DA_ERR_CUDA;
  // in place, blocks come from slices of the rows; to other pages, from parts of the list
  const int64_t rows = (int64_t)a.c.S * a.c.Hkv * 2;
  const int row_bytes = a.c.d * (a.c.dtype == DA_BF16 ? 2 : 4);
  int slices = 1, chunks = 1;
  if (a.dst_page_table == nullptr)
    while (rows * slices < 608 && row_bytes / slices > 32) slices *= 2;
  else
    while (rows * chunks < 1216 && chunks * 512 < a.max_keep) chunks *= 2;
  const int64_t blocks = (int64_t)a.c.S * a.c.Hkv * (2 * slices + a.c.Hq / a.c.Hkv);
  return launch_after(evict_move, dim3((unsigned)blocks, (unsigned)chunks), kMoveThreads, 0, stream, a, w, sh, slices) ==
                 cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

}  // namespace da
