// C ABI of the rotary positions and the paged cache (append, decode step, chunks,
// eviction): argument validation and dispatch to the kernels.
#include <cmath>

#include "da_chunk.cuh"
#include "da_evict.h"
#include "da_paged.h"
#include "da_rope.h"

namespace da {
size_t pgt_workspace(int S, int Hq, int Hkv, int d, int max_len, int prefix_len, int dtype);
bool pgt_fits(int S, int Hq, int Hkv, int d, int max_len, int prefix_len, int dtype);
int launch_paged_decode(const PagedDecode &p, cudaStream_t stream);
inline int chunk_most(int N, int max_new, int max_len) {   // new tokens of a sequence, at most
  const int n = max_new < N ? max_new : N;
  return n < max_len ? n : max_len;
}
size_t chunk_workspace(int S, int Hq, int Hkv, int d, long long N, int max_new, int max_len, int dtype);
int launch_paged_chunk(const PagedChunk &p, cudaStream_t stream);
}  // namespace da

using namespace da;

namespace {

constexpr int kMaxHeads = 1 << 14;   // a launch grid's second dimension counts rows of q, k and v
constexpr int kMaxTokens = 1 << 30;
constexpr unsigned long long kWaitLimitNsHost = 1000ull * 1000ull * 1000ull;

int elem_bytes(int dtype) { return dtype == DA_BF16 ? 2 : 4; }
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A rotation spec (nullable: no rotation) as kernel parameters.
int check_spec(const dilution_attn_rope_spec *spec, int d, RopeParams &rp) {
  rp = RopeParams{};
  rp.sign = 1.f;
  rp.n_axes = 1;
  if (spec == nullptr) return DA_OK;
  if (spec->n_pairs < 0 || 2 * spec->n_pairs > d) return DA_ERR_INVALID;
  if (spec->n_axes < 1 || spec->n_axes > DA_MAX_ROPE_AXES) return DA_ERR_INVALID;
  if (spec->adjacent != 0 && spec->adjacent != 1) return DA_ERR_INVALID;
  if (spec->n_pairs > 0 && (spec->inv_freq == nullptr || !aligned(spec->inv_freq, 4))) return DA_ERR_INVALID;
  for (int j = 0; j < spec->n_pairs; ++j) {
    if (spec->pair_axis[j] >= spec->n_axes) return DA_ERR_INVALID;
    rp.axis_bits[j / 16] |= (uint32_t)spec->pair_axis[j] << (2 * (j % 16));
  }
  rp.inv_freq = spec->inv_freq;
  rp.n_pairs = spec->n_pairs;
  rp.n_axes = spec->n_axes;
  return DA_OK;
}

// Whether rows of d elements at these strides can be moved in 16-byte pieces
// and the rotated part is made of whole pieces.
bool pieces_ok(const void *p, const long long *strides, const long long *extents, int n, int dtype) {
  const int nv = 16 / elem_bytes(dtype);
  if (!aligned(p, 16)) return false;
  for (int i = 0; i < n; ++i)
    if (extents[i] > 1 && strides[i] % nv != 0) return false;
  return true;
}
bool pairs_ok(int n_pairs, int adjacent, int dtype) { return adjacent || n_pairs % (16 / elem_bytes(dtype)) == 0; }

// An output must not address an element twice: its strides, sorted, each step
// over the extent below (rows of d elements at the bottom).
bool distinct(const long long *strides, const long long *extents, int n, int d) {
  long long span = d, below = -1;
  for (int taken = 0; taken < n; ++taken) {   // the smallest stride not yet taken (ties by index)
    int at = -1;
    for (int i = 0; i < n; ++i) {
      const long long key = strides[i] * 4 + i;
      if (key > below && (at < 0 || key < strides[at] * 4 + at)) at = i;
    }
    below = strides[at] * 4 + at;
    if (extents[at] <= 1) continue;
    if (strides[at] < span) return false;
    span += strides[at] * (extents[at] - 1);
  }
  return true;
}

bool strides_sane(const long long *strides, int n) {
  for (int i = 0; i < n; ++i)
    if (strides[i] < 0 || strides[i] > (1ll << 40)) return false;
  return true;
}

// Whether one of n x h rows of row_bytes bytes, at byte strides step (n) and
// head (h), meets the bytes [lo, hi).
bool rows_meet(const void *p, long long n, long long step, int h, long long head, long long row_bytes, const void *lo_,
               long long len) {
  const long long at = (long long)reinterpret_cast<uintptr_t>(p), lo = (long long)reinterpret_cast<uintptr_t>(lo_);
  if (at >= lo + len || at + (n - 1) * step + (h - 1) * head + row_bytes <= lo) return false;
  for (int i = 0; i < h; ++i) {
    const long long row = at + i * head, gap = lo - (row + row_bytes);   // the first row that ends behind lo
    const long long t = gap < 0 ? 0 : step > 0 ? gap / step + 1 : n;
    if (t < n && row + t * step < lo + len) return true;
  }
  return false;
}

int rope_call(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, void *q_out,
              const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides, const int32_t *positions,
              int pos_batch, const dilution_attn_rope_spec *spec, int B, int Hq, int Hk, int T, int d, int dtype,
              float sign, void *stream) {
  if (B < 0 || Hq < 0 || Hk < 0 || T < 0) return DA_ERR_INVALID;
  if (dtype != DA_F32 && dtype != DA_BF16) return DA_ERR_INVALID;
  if (!head_dim_supported(d)) return DA_ERR_UNSUPPORTED;
  if (T > DA_MAX_T || Hq > kMaxHeads || Hk > kMaxHeads || (int64_t)B * T > kMaxTokens) return DA_ERR_UNSUPPORTED;
  if (spec == nullptr || (pos_batch != 1 && pos_batch != B)) return DA_ERR_INVALID;
  RopeParams rp;
  const int st = check_spec(spec, d, rp);
  if (st != DA_OK) return st;
  if (B == 0 || T == 0 || Hq + Hk == 0) return DA_OK;
  if (positions == nullptr || !aligned(positions, 4)) return DA_ERR_INVALID;
  rp.positions = positions;
  rp.pos_stride_axis = (long long)pos_batch * T;
  rp.pos_stride_b = pos_batch == 1 ? 0 : T;
  rp.sign = sign;
  bool vec = true;
  RopeTensor t[2] = {};
  const void *in[2] = {q, k};
  void *out[2] = {q_out, k_out};
  const int64_t *is[2] = {q_strides, k_strides}, *os[2] = {q_out_strides, k_out_strides};
  const int H[2] = {Hq, Hk};
  for (int i = 0; i < 2; ++i) {
    if (H[i] == 0) continue;
    if (in[i] == nullptr || out[i] == nullptr) return DA_ERR_INVALID;
    if (!aligned(in[i], elem_bytes(dtype)) || !aligned(out[i], elem_bytes(dtype))) return DA_ERR_INVALID;
    const long long ext[3] = {B, H[i], T}, dense[3] = {(long long)H[i] * T * d, (long long)T * d, d};
    long long si[3], so[3];
    for (int j = 0; j < 3; ++j) {
      si[j] = is[i] != nullptr ? is[i][j] : dense[j];
      so[j] = os[i] != nullptr ? os[i][j] : dense[j];
    }
    if (!strides_sane(si, 3) || !strides_sane(so, 3) || !distinct(so, ext, 3, d)) return DA_ERR_INVALID;
    if (out[i] == in[i])   // in place: every row where it was
      for (int j = 0; j < 3; ++j)
        if (ext[j] > 1 && si[j] != so[j]) return DA_ERR_INVALID;
    vec = vec && pieces_ok(in[i], si, ext, 3, dtype) && pieces_ok(out[i], so, ext, 3, dtype);
    t[i] = RopeTensor{in[i], out[i], si[0], si[1], si[2], so[0], so[1], so[2]};
  }
  if (Hq > 0 && Hk > 0 && (q_out == k_out || q_out == k || k_out == q)) return DA_ERR_INVALID;
  const RopePath path = !vec ? kRopeScalar : pairs_ok(rp.n_pairs, spec->adjacent, dtype) ? kRopeUnits : kRopeAny;
  return launch_rope(t[0], t[1], rp, spec->adjacent != 0, path, B, Hq, Hk, T, d, dtype,
                     reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

// Sizes, type and pointers of a paged cache.
int check_cache(const dilution_attn_paged_cache *c) {
  if (c == nullptr) return DA_ERR_INVALID;
  if (c->S < 0 || c->Hq < 1 || c->Hkv < 1 || c->Hq % c->Hkv != 0 || c->num_pages < 0 || c->num_demand_pages < 0 ||
      c->max_pages < 0)
    return DA_ERR_INVALID;
  if (c->dtype != DA_F32 && c->dtype != DA_BF16) return DA_ERR_INVALID;
  const int ps = c->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return ps < 1 ? DA_ERR_INVALID : DA_ERR_UNSUPPORTED;
  if (!head_dim_supported(c->d)) return DA_ERR_UNSUPPORTED;
  if (c->Hq > kMaxHeads || (int64_t)c->S * c->Hq > (1 << 24) || (int64_t)c->max_pages * ps > DA_MAX_T)
    return DA_ERR_UNSUPPORTED;
  if (c->S == 0) return DA_OK;
  const void *tables[] = {c->page_table, c->demand_table, c->seq_lens};
  for (const void *p : tables)
    if (p == nullptr || !aligned(p, 4)) return DA_ERR_INVALID;
  const void *pools[] = {c->k_pages, c->v_pages, c->demand_pages};
  for (const void *p : pools)
    if (p == nullptr || !aligned(p, 16)) return DA_ERR_INVALID;
  return DA_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need) return DA_ERR_WORKSPACE;
  return aligned(ws, 256) ? DA_OK : DA_ERR_INVALID;
}

bool options_valid(float tau, const float *tau_bh, float eps, int flags) {
  return std::isfinite(tau) && tau >= 0.f && std::isfinite(eps) && eps > 0.f &&
         (flags & ~DA_FLAG_EARLIER_DEMAND_ONLY) == 0 && aligned(tau_bh, 4);
}
int check_options(float tau, const float *tau_bh, float eps, int flags, int dtype) {
  if (!options_valid(tau, tau_bh, eps, flags)) return DA_ERR_INVALID;
  return dtype == DA_BF16 && eps < 1e-18f ? DA_ERR_UNSUPPORTED : DA_OK;
}
HeadScale head_scale(float tau, const float *tau_bh, int d) {
  const double per_tau = 1.4426950408889634 / std::sqrt((double)d);
  return HeadScale{tau_bh, (float)((double)tau * per_tau), per_tau};
}

PagedDebug no_stall() {
  PagedDebug d;
  for (int k = 0; k < kPagedKernels; ++k) d.limit_ns[k] = kWaitLimitNsHost, d.stall_block[k] = -1;
  return d;
}

int decode_call(const void *q, const dilution_attn_paged_cache *cache, const int32_t *prefix_table, int n_prefix_pages,
                int max_len, void *out, float tau, const float *tau_bh, float eps, int flags, void *workspace,
                size_t workspace_bytes, void *status, void *stream, const PagedDebug &dbg) {
  int st = check_cache(cache);
  if (st != DA_OK) return st;
  const dilution_attn_paged_cache &c = *cache;
  if (!options_valid(tau, tau_bh, eps, flags)) return DA_ERR_INVALID;
  if (max_len < 0 || (int64_t)max_len > (int64_t)c.max_pages * c.page_size) return DA_ERR_INVALID;
  if (n_prefix_pages < 0 || (int64_t)n_prefix_pages * c.page_size > max_len) return DA_ERR_INVALID;
  if (n_prefix_pages > 0 && (prefix_table == nullptr || !aligned(prefix_table, 4))) return DA_ERR_INVALID;
  if (c.dtype == DA_BF16 && eps < 1e-18f) return DA_ERR_UNSUPPORTED;
  if (c.S == 0) return DA_OK;
  if (q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 16)) return DA_ERR_INVALID;
  const int prefix_len = n_prefix_pages * c.page_size;
  st = check_workspace(workspace, workspace_bytes, pgt_workspace(c.S, c.Hq, c.Hkv, c.d, max_len, prefix_len, c.dtype));
  if (st != DA_OK) return st;
  if (status == nullptr || !aligned(status, 256)) return DA_ERR_INVALID;
  if ((int64_t)c.num_pages * c.Hkv > 0x7FFFFFFF) return DA_ERR_UNSUPPORTED;   // a copy's coordinate
  // what the kernels count in 32 bits: places in the demand pool (16 floats each), work units
  if ((int64_t)c.num_demand_pages * c.Hq * (c.page_size / 16) >= 0xFFFFFFFFll) return DA_ERR_UNSUPPORTED;
  if (!pgt_fits(c.S, c.Hq, c.Hkv, c.d, max_len, prefix_len, c.dtype)) return DA_ERR_UNSUPPORTED;
  PagedDecode p{};
  p.c = c;
  p.q = q;
  p.out = out;
  p.prefix_table = n_prefix_pages > 0 ? prefix_table : nullptr;
  p.prefix_len = prefix_len;
  p.max_len = max_len;
  p.hs = head_scale(tau, tau_bh, c.d);
  p.eps = eps;
  p.earlier = (flags & DA_FLAG_EARLIER_DEMAND_ONLY) != 0;
  p.status = reinterpret_cast<int *>(status);
  p.ws = reinterpret_cast<uint8_t *>(workspace);
  p.dbg = dbg;
  return launch_paged_decode(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int dilution_attn_rope(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, void *q_out,
                       const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides,
                       const int32_t *positions, int pos_batch, const dilution_attn_rope_spec *spec, int B, int Hq,
                       int Hk, int T, int d, int dtype, void *stream) {
  return rope_call(q, q_strides, k, k_strides, q_out, q_out_strides, k_out, k_out_strides, positions, pos_batch, spec,
                   B, Hq, Hk, T, d, dtype, 1.f, stream);
}

int dilution_attn_rope_bwd(const void *dq_out, const int64_t *dq_out_strides, const void *dk_out,
                           const int64_t *dk_out_strides, void *dq, const int64_t *dq_strides, void *dk,
                           const int64_t *dk_strides, const int32_t *positions, int pos_batch,
                           const dilution_attn_rope_spec *spec, int B, int Hq, int Hk, int T, int d, int dtype,
                           void *stream) {
  return rope_call(dq_out, dq_out_strides, dk_out, dk_out_strides, dq, dq_strides, dk, dk_strides, positions,
                   pos_batch, spec, B, Hq, Hk, T, d, dtype, -1.f, stream);
}

size_t dilution_attn_paged_append_workspace_size(void) { return kStatusBytes; }

int dilution_attn_paged_append(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                               const void *v, const int64_t *v_strides, const float *demand,
                               const int64_t *demand_strides, void *q_out, const int32_t *cu_tokens, int N,
                               const dilution_attn_paged_cache *cache, const dilution_attn_rope_spec *spec,
                               const int32_t *positions, void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_cache(cache);
  if (st != DA_OK) return st;
  const dilution_attn_paged_cache &c = *cache;
  RopeParams rp;
  st = check_spec(spec, c.d, rp);
  if (st != DA_OK) return st;
  if (N < 0) return DA_ERR_INVALID;
  if (N > kMaxTokens) return DA_ERR_UNSUPPORTED;
  if (N == 0 || c.S == 0) return DA_OK;
  if (k == nullptr || v == nullptr || cu_tokens == nullptr || !aligned(cu_tokens, 4)) return DA_ERR_INVALID;
  if ((q == nullptr) != (q_out == nullptr)) return DA_ERR_INVALID;
  if (!aligned(positions, 4) || !aligned(demand, 4)) return DA_ERR_INVALID;
  st = check_workspace(workspace, workspace_bytes, kStatusBytes);
  if (st != DA_OK) return st;
  rp.positions = positions;
  rp.pos_stride_axis = N;
  AppendArgs a{};
  const int eb = elem_bytes(c.dtype);
  const int adjacent = spec != nullptr ? spec->adjacent : 0;
  bool vec = pairs_ok(rp.n_pairs, adjacent, c.dtype) && (q_out == nullptr || aligned(q_out, 16));
  const void *in[3] = {q, k, v};
  const int64_t *is[3] = {q_strides, k_strides, v_strides};
  const int H[3] = {c.Hq, c.Hkv, c.Hkv};
  long long s[3][2];
  for (int i = 0; i < 3; ++i) {
    s[i][0] = is[i] != nullptr ? is[i][0] : (long long)H[i] * c.d;
    s[i][1] = is[i] != nullptr ? is[i][1] : c.d;
    if (in[i] == nullptr) continue;
    const long long ext[2] = {N, H[i]};
    if (!aligned(in[i], eb) || !strides_sane(s[i], 2)) return DA_ERR_INVALID;
    vec = vec && pieces_ok(in[i], s[i], ext, 2, c.dtype);
  }
  if (q_out != nullptr && !aligned(q_out, eb)) return DA_ERR_INVALID;
  const long long ds[2] = {demand_strides != nullptr ? demand_strides[0] : c.Hq,
                           demand_strides != nullptr ? demand_strides[1] : 1};
  if (!strides_sane(ds, 2)) return DA_ERR_INVALID;
  if (q_out != nullptr) {   // what is still to be read: q_out may be a contiguous q, and lies over nothing else
    const long long len = (long long)N * c.Hq * c.d * eb;
    const bool dense = (N == 1 || s[0][0] == (long long)c.Hq * c.d) && (c.Hq == 1 || s[0][1] == c.d);
    for (int i = q_out == q && dense ? 1 : 0; i < 3; ++i)
      if (rows_meet(in[i], N, s[i][0] * eb, H[i], s[i][1] * eb, (long long)c.d * eb, q_out, len)) return DA_ERR_INVALID;
    if (demand != nullptr && rows_meet(demand, N, ds[0] * 4, c.Hq, ds[1] * 4, 4, q_out, len)) return DA_ERR_INVALID;
  }
  a.q = q, a.k = k, a.v = v, a.demand = demand, a.q_out = q_out, a.cu_tokens = cu_tokens;
  a.q_t = s[0][0], a.q_h = s[0][1], a.k_t = s[1][0], a.k_h = s[1][1], a.v_t = s[2][0], a.v_h = s[2][1];
  a.dem_t = ds[0], a.dem_h = ds[1];
  a.N = N, a.adjacent = adjacent;
  a.status = reinterpret_cast<int *>(workspace);
  return launch_append(a, c, rp, vec, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

size_t dilution_attn_paged_decode_workspace_size(int S, int Hq, int Hkv, int d, int max_len, int n_prefix_pages,
                                                 int page_size, int dtype) {
  if (dtype != DA_F32 && dtype != DA_BF16) return 0;
  if (S < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_len < 0 || n_prefix_pages < 0 || page_size < 1 || !head_dim_supported(d))
    return 0;
  if ((int64_t)n_prefix_pages * page_size > max_len) return 0;
  return pgt_workspace(S, Hq, Hkv, d, max_len, n_prefix_pages * page_size, dtype);
}

int dilution_attn_paged_decode(const void *q, const dilution_attn_paged_cache *cache, const int32_t *prefix_table,
                               int n_prefix_pages, int max_len, void *out, float tau, const float *tau_bh, float eps,
                               int flags, void *workspace, size_t workspace_bytes, void *stream) {
  return decode_call(q, cache, prefix_table, n_prefix_pages, max_len, out, tau, tau_bh, eps, flags, workspace,
                     workspace_bytes, workspace, stream, no_stall());
}

int dilution_attn_paged_decode_ex(const void *q, const dilution_attn_paged_cache *cache, const int32_t *prefix_table,
                                  int n_prefix_pages, int max_len, void *out, float tau, const float *tau_bh, float eps,
                                  int flags, void *workspace, size_t workspace_bytes, void *status, void *stream) {
  return decode_call(q, cache, prefix_table, n_prefix_pages, max_len, out, tau, tau_bh, eps, flags, workspace,
                     workspace_bytes, status, stream, no_stall());
}

size_t dilution_attn_paged_chunk_workspace_size(int S, int Hq, int Hkv, int d, int N, int max_new, int max_len, int dtype) {
  if (dtype != DA_F32 && dtype != DA_BF16) return 0;
  if (S < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || N < 0 || max_new < 0 || max_len < 0 || max_len > kMaxTokens ||
      !head_dim_supported(d))
    return 0;
  return chunk_workspace(S, Hq, Hkv, d, N, chunk_most(N, max_new, max_len), max_len, dtype);
}

int dilution_attn_paged_chunk(const void *q, const dilution_attn_paged_cache *cache, const int32_t *cu_tokens, int N,
                              int max_new, int max_len, void *out, float tau, const float *tau_bh, float eps, int flags,
                              void *workspace, size_t workspace_bytes, void *status, void *stream) {
  int st = check_cache(cache);
  if (st != DA_OK) return st;
  const dilution_attn_paged_cache &c = *cache;
  st = check_options(tau, tau_bh, eps, flags, c.dtype);
  if (st != DA_OK) return st;
  if (N < 0 || max_new < 0 || max_len < 0 || (int64_t)max_len > (int64_t)c.max_pages * c.page_size) return DA_ERR_INVALID;
  if (N > kMaxTokens || max_len > kMaxTokens || (int64_t)c.num_pages * c.Hkv > 0x7FFFFFFF)   // (a copy's coordinate)
    return DA_ERR_UNSUPPORTED;
  if (N == 0 || c.S == 0) return DA_OK;
  if (q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 16)) return DA_ERR_INVALID;
  if (cu_tokens == nullptr || !aligned(cu_tokens, 4)) return DA_ERR_INVALID;
  max_new = chunk_most(N, max_new, max_len);
  st = check_workspace(workspace, workspace_bytes, chunk_workspace(c.S, c.Hq, c.Hkv, c.d, N, max_new, max_len, c.dtype));
  if (st != DA_OK) return st;
  if (status != nullptr && !aligned(status, 256)) return DA_ERR_INVALID;
  PagedChunk p{};
  p.c = c;
  p.q = q;
  p.out = out;
  p.cu = cu_tokens;
  p.N = N;
  p.max_new = p.all_new = max_new;
  p.max_len = max_len;
  p.hs = head_scale(tau, tau_bh, c.d);
  p.eps = eps;
  p.earlier = (flags & DA_FLAG_EARLIER_DEMAND_ONLY) != 0;
  p.status = reinterpret_cast<int *>(status != nullptr ? status : workspace);
  p.ws = reinterpret_cast<uint8_t *>(workspace);
  return launch_paged_chunk(p, reinterpret_cast<cudaStream_t>(stream));
}

size_t dilution_attn_paged_evict_workspace_size(int S, int Hkv, int max_keep, int max_len) {
  if (S < 0 || Hkv < 1 || max_keep < 0 || max_len < 0 || max_len > kMaxTokens) return 0;
  return evict_workspace(S, Hkv, max_keep < max_len ? max_keep : max_len, max_len).total;
}

int dilution_attn_paged_evict(const dilution_attn_paged_cache *cache, const int32_t *dst_page_table,
                              const int32_t *dst_demand_table, int dst_max_pages, const int32_t *keep, int max_keep,
                              int max_len, int sinks, int recent, int32_t *new_lens, int32_t *kept, void *workspace,
                              size_t workspace_bytes, void *status, void *stream) {
  int st = check_cache(cache);
  if (st != DA_OK) return st;
  const dilution_attn_paged_cache &c = *cache;
  if (max_keep < 0 || max_len < 0 || sinks < 0 || recent < 0 ||
      (int64_t)max_len > (int64_t)c.max_pages * c.page_size)
    return DA_ERR_INVALID;
  if ((dst_page_table == nullptr) != (dst_demand_table == nullptr) || !aligned(dst_page_table, 4) ||
      !aligned(dst_demand_table, 4))
    return DA_ERR_INVALID;
  if (max_len > kMaxTokens) return DA_ERR_UNSUPPORTED;
  if (kept == nullptr && max_keep > max_len) max_keep = max_len;   // (kept's rows hold max_keep)
  const int most = max_keep < max_len ? max_keep : max_len;
  if (dst_page_table != nullptr && (dst_max_pages < 0 || (int64_t)dst_max_pages * c.page_size < most)) return DA_ERR_INVALID;
  if (c.S == 0) return DA_OK;
  if (keep == nullptr || new_lens == nullptr || !aligned(keep, 4) || !aligned(new_lens, 4) || !aligned(kept, 4))
    return DA_ERR_INVALID;
  st = check_workspace(workspace, workspace_bytes, evict_workspace(c.S, c.Hkv, most, max_len).total);
  if (st != DA_OK) return st;
  if (status != nullptr && !aligned(status, 256)) return DA_ERR_INVALID;
  EvictArgs a{};
  a.c = c;
  a.dst_page_table = dst_page_table, a.dst_demand_table = dst_demand_table;
  a.dst_max_pages = dst_max_pages;
  a.keep = keep;
  a.max_keep = max_keep, a.max_len = max_len, a.sinks = sinks, a.recent = recent;
  a.new_lens = new_lens, a.kept = kept;
  a.status = reinterpret_cast<int *>(status != nullptr ? status : workspace);
  a.ws = reinterpret_cast<uint8_t *>(workspace);
  return launch_evict(a, reinterpret_cast<cudaStream_t>(stream));
}

int dilution_attn_debug_paged_decode_stall(const void *q, const dilution_attn_paged_cache *cache,
                                           const int32_t *prefix_table, int n_prefix_pages, int max_len, void *out,
                                           float tau, float eps, void *workspace, size_t workspace_bytes, void *stream,
                                           int stall_kernel, int stall_block, long long wait_limit_ns) {
  if (stall_kernel < 0 || stall_kernel >= kPagedKernels || stall_block < 0 || wait_limit_ns < 1000 ||
      wait_limit_ns > (long long)kWaitLimitNsHost)
    return DA_ERR_INVALID;
  PagedDebug dbg = no_stall();
  dbg.limit_ns[stall_kernel] = (unsigned long long)wait_limit_ns;
  dbg.stall_block[stall_kernel] = stall_block;
  return decode_call(q, cache, prefix_table, n_prefix_pages, max_len, out, tau, nullptr, eps, 0, workspace,
                     workspace_bytes, workspace, stream, dbg);
}

}  // extern "C"
