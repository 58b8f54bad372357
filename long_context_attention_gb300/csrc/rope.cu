// Rotary positions: the rotation of queries and keys on their way into
// attention (and of their gradients on the way back), and the append to a
// paged cache, which rotates on the way.
//
// Mathematics.  Pair j of a head at position n (of the pair's axis) turns by
// theta = n * inv_freq_j radians.  Only theta modulo one turn matters, so the
// frequency is held in turns per position as a 64-bit fixed-point fraction
//     F = inv_freq_j / (2 pi) * 2^64  mod 2^64:
// the 24-bit mantissa of inv_freq_j times the first 96 bits of 1 / (2 pi),
// shifted by the exponent, within 1.01 units for every |inv_freq_j| < 2^24 (with the
// first 64 bits alone within inv_freq_j / 2 units: 2^24 - 1 at position 2^31 was off by
// 6e-3 radians).  n * F mod 2^64 is then the angle to n 2^-64 turns, of which the upper
// 32 bits (to 2^-32 turns, 1.5e-9 radians, below fp32's rounding of the cosine) go to
// sine and cosine, formed from their series.
// No fp64 (GB300 has few fp64 units), no long fp32 products; 32-bit multiplies and
// funnel shifts (a version in 64-bit operations cost 140 instructions a pair and
// bounded the append).  The products x cos - y sin run in fp32 and round once to the output's
// type.
//
// What bounds it: bytes.  Each element is read once and written once; sin and
// cos are computed in registers for one token and 16 bytes of a head's row and
// serve `hpt` heads in turn, so they are a small part of the instructions (of two
// heads they are most of them: 4 x 36238 tokens of 2 x 128 bf16 take 37.2 us, the
// bytes 22).  The loads of several heads are issued together before the first
// store: an output may be its input, so the compiler cannot move a load over a
// store by itself (one head at a time kept 32 bytes a thread in flight: 4.9 TB/s at
// 4 x 24 x 16384 x 64 bf16; now 6.3, and 6.8 at 24 x 131072 x 128 fp32).
#include "da_rope.h"
#include "da_ptx.cuh"

#include <cuda_bf16.h>

namespace da {

// inv_freq in turns per position, times 2^64 modulo 2^64 (hi, lo).  Frequencies
// of magnitude 2^24 and above, infinities and NaN give ok = false.
__device__ __forceinline__ uint2 turns_fixed(float f, bool &ok) {
  constexpr uint32_t kHi = 0x28BE60DBu, kMid = 0x9391054Au, kLo = 0x7F09D5F4u;   // floor(2^96 / (2 pi))
  const uint32_t u = __float_as_uint(f);
  int e = (int)((u >> 23) & 0xffu);
  uint32_t m = u & 0x7fffffu;
  if (e == 0)
    e = 1;
  else
    m |= 0x800000u;
  const int shift = 150 - e;   // |f| = m 2^-shift
  ok = shift >= 0;
  // the 118-bit product without its lowest word, least word first
  const unsigned long long p0 = (unsigned long long)m * kMid + (((unsigned long long)m * kLo) >> 32);
  const unsigned long long p1 = (unsigned long long)m * kHi + (p0 >> 32);
  const uint32_t w0 = (uint32_t)p0, w1 = (uint32_t)p1, w2 = (uint32_t)(p1 >> 32);
  // bits shift .. shift + 63 of it
  const int words = shift >> 5;
  const uint32_t a = words == 0 ? w0 : words == 1 ? w1 : words == 2 ? w2 : 0u;
  const uint32_t b = words == 0 ? w1 : words == 1 ? w2 : 0u;
  const uint32_t c = words == 0 ? w2 : 0u;
  uint32_t lo = __funnelshift_r(a, b, shift), hi = __funnelshift_r(b, c, shift);   // (by shift mod 32)
  if (u >> 31) {
    lo = 0u - lo;
    hi = ~hi + (lo == 0u);
  }
  return make_uint2(hi, lo);
}

// cos and sin of the angle pos F, F in turns per position.  The angle's top bits
// give the nearest quarter turn, the rest an angle of at most pi / 4, whose Taylor
// series to the 9th and 8th power are within 2e-9 and 3e-8 (half an fp32 step of 1);
// a quarter turn swaps the two and sets the signs.  unit: radians of the angle's
// last bit (NaN: the frequency is not valid).
__device__ __forceinline__ void rope_sincos(uint2 F, float unit, int pos, float &c, float &s) {
  // the upper word of pos F mod 2^64: the angle as a signed 0.32 turn
  uint32_t a = F.x * (uint32_t)pos + __umulhi(F.y, (uint32_t)pos);
  if (pos < 0) a -= F.y;
  const uint32_t q = a + 0x20000000u;   // its top two bits: the quarter
  const float x = (float)(int)(a - (q & 0xC0000000u)) * unit;
  const float x2 = x * x;
  float sn = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);                           // 1 / 9!, -1 / 7!
  sn = fmaf(x2, sn, 8.3333333e-3f);
  sn = fmaf(x2, sn, -1.6666667e-1f);
  sn = fmaf(x2 * x, sn, x);
  float cs = fmaf(x2, 2.4801587e-5f, -1.3888889e-3f);                           // 1 / 8!, -1 / 6!
  cs = fmaf(x2, cs, 4.1666667e-2f);
  cs = fmaf(x2, cs, -0.5f);
  cs = fmaf(x2, cs, 1.f);
  const bool swap = (q & 0x40000000u) != 0u;
  // the cosine is negative in quarters 1 and 2, the sine in 2 and 3
  c = __uint_as_float(__float_as_uint(swap ? sn : cs) ^ ((q + 0x40000000u) & 0x80000000u));
  s = __uint_as_float(__float_as_uint(swap ? cs : sn) ^ (q & 0x80000000u));
}

template <typename E>
struct RopeVec;   // 16 bytes of a row
template <>
struct RopeVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct RopeVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float &y) { y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16 &y) { y = __float2bfloat16_rn(x); }

// The two 16-byte vectors of a row that unit u of a token handles, and the
// angles of the N pairs they hold.  Units cover a row of d elements in d / 2N
// steps.  Half-split pairs: a rotated unit holds elements [N u, N u + N) and
// their partners n_pairs further on.  Adjacent pairs: vectors 2u and 2u + 1.
template <typename E, bool ADJ>
struct RopeUnit {
  static constexpr int N = RopeVec<E>::N;
  int va, vb;                 // element offsets of the two vectors
  bool rot;                   // whether any of their pairs rotate (half-split: all or none)
  int pairs;
  float c[N], s[N];           // half-split: N pairs; adjacent: N / 2 of each vector

  __device__ __forceinline__ void place(int u, int n_pairs) {
    pairs = n_pairs;
    if constexpr (ADJ) {
      va = 2 * u * N;
      vb = va + N;
      rot = va < 2 * n_pairs;
    } else {
      const int rot_units = n_pairs / N;
      rot = u < rot_units;
      va = rot ? u * N : 2 * n_pairs + 2 * (u - rot_units) * N;
      vb = rot ? va + n_pairs : va + N;
    }
  }
  // `angle(j, c, s)` gives the cosine and sine of pair j.
  template <typename F>
  __device__ __forceinline__ void turn(F &&angle) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      c[i] = 1.f, s[i] = 0.f;
      if constexpr (ADJ) {
        if (va / 2 + i < pairs) angle(va / 2 + i, c[i], s[i]);
      } else {
        if (rot) angle(va + i, c[i], s[i]);
      }
    }
  }
  // Pairs from n on of a piece as they were.
  static __device__ __forceinline__ void keep(uint4 &a, const uint4 &was, int n) {
    constexpr int W = N == 8 ? 1 : 2;   // 32-bit words of a pair
    if (n <= 0) a.x = was.x;
    if (n <= 1 / W) a.y = was.y;
    if (n <= 2 / W) a.z = was.z;
    if (n <= 3 / W) a.w = was.w;
  }
  __device__ __forceinline__ void apply(uint4 &a, uint4 &b) const {
    using V = RopeVec<E>;
    if (!rot) return;         // passes bit for bit
    float x[N], y[N];
    V::unpack(a, x);
    V::unpack(b, y);
    if constexpr (ADJ) {
      const uint4 a0 = a, b0 = b;
      float ra[N], rb[N];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        ra[2 * i] = fmaf(x[2 * i], c[i], -x[2 * i + 1] * s[i]);
        ra[2 * i + 1] = fmaf(x[2 * i + 1], c[i], x[2 * i] * s[i]);
        rb[2 * i] = fmaf(y[2 * i], c[N / 2 + i], -y[2 * i + 1] * s[N / 2 + i]);
        rb[2 * i + 1] = fmaf(y[2 * i + 1], c[N / 2 + i], y[2 * i] * s[N / 2 + i]);
      }
      a = V::pack(ra);
      b = V::pack(rb);
      if (va / 2 + N > pairs) {   // pairs past the rotated part pass bit for bit
        keep(a, a0, pairs - va / 2);
        keep(b, b0, pairs - vb / 2);
      }
    } else {
      float ra[N], rb[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ra[i] = fmaf(x[i], c[i], -y[i] * s[i]);
        rb[i] = fmaf(y[i], c[i], x[i] * s[i]);
      }
      a = V::pack(ra);
      b = V::pack(rb);
    }
  }
};

// A token's positions on every axis, read once.
struct RopePlace {
  int v[DA_MAX_ROPE_AXES];
  __device__ __forceinline__ RopePlace(const RopeParams &rp, long long b, long long t, int fallback) {
#pragma unroll
    for (int a = 0; a < DA_MAX_ROPE_AXES; ++a) {
      v[a] = fallback;
      if (rp.positions != nullptr && a < rp.n_axes)
        v[a] = rp.positions[a * rp.pos_stride_axis + b * rp.pos_stride_b + t];
    }
  }
  __device__ __forceinline__ int on(int axis) const {
    return axis == 0 ? v[0] : axis == 1 ? v[1] : axis == 2 ? v[2] : v[3];
  }
};

constexpr int kRopeThreads = 128;
// Heads loaded together: 4 in the rotation of more than 2 heads a thread (131072 x
// 24 x 128 fp32: 480 us, 497 with 2), 2 of fewer (4 x 36238 tokens of 2 heads of 128:
// 39.4 us, 42.7 with 4), where rows exchange their parts (6 heads of the same tokens, bf16:
// 115 us, 135 with 4) and in the append (16 prompts: 24 us, 28 with 4).
constexpr int kRopeBatch = 4, kFewBatch = 2;

// The pairs' frequencies in turns and their axes, formed once a warp (every
// thread for its own pairs cost half the instructions of a rotation of few heads,
// and reads of the axes by lanes of different pairs one after another).  The
// pairs N u + i of neighbouring pieces u lie next to each other.
template <int N>
struct RopeTable {
  uint4 e[DA_MAX_ROPE_PAIRS];   // frequency (hi, lo; turned back: negated), axis, unit (see rope_sincos)
  static __device__ __forceinline__ int slot(int j) { return j % N * (DA_MAX_ROPE_PAIRS / N) + j / N; }
  __device__ __forceinline__ void fill(const RopeParams &rp) {   // all lanes of the warp
#pragma unroll
    for (int i = 0; i < DA_MAX_ROPE_PAIRS / 32; ++i) {
      const int j = 32 * i + threadIdx.x % 32;
      if (j < rp.n_pairs) {
        bool ok;
        const uint2 F = turns_fixed(rp.inv_freq[j] * rp.sign, ok);
        const uint32_t w = j % 32 < 16 ? rp.axis_bits[2 * i] : rp.axis_bits[2 * i + 1];
        const float unit = ok ? 1.4629180792671596e-9f : __int_as_float(0x7fc00000);   // 2 pi 2^-32
        e[slot(j)] = make_uint4(F.x, F.y, (w >> (2 * (j % 16))) & 3u, __float_as_uint(unit));
      }
    }
    __syncwarp();
  }
  template <bool ONE>   // of one axis
  __device__ __forceinline__ void angle(int j, const RopePlace &at, float &c, float &s) const {
    const uint4 v = e[slot(j)];
    rope_sincos(make_uint2(v.x, v.y), __uint_as_float(v.w), ONE ? at.v[0] : at.on((int)v.z), c, s);
  }
};

// 16 bytes that are read once or written once: kept out of L1.
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// The tokens of the rotation kernels: a thread takes piece (or pair) u of one.
struct RopeWalk {
  int tokens, T, shift;   // shift: log2 of a row's pieces (or pairs)
  __device__ __forceinline__ int piece() const { return threadIdx.x & ((1 << shift) - 1); }
  __device__ __forceinline__ int token() const { return blockIdx.x * (kRopeThreads >> shift) + (threadIdx.x >> shift); }
};
// Its rows of every head.
template <typename E>
struct RopeRows {
  int b, t, Hq;
  const E *qi, *ki;
  E *qo, *ko;
  long long qih, kih, qoh, koh;
  __device__ __forceinline__ RopeRows(const RopeTensor &q, const RopeTensor &k, int heads_q, int tok, int T)
      : b((unsigned)tok / (unsigned)T), t(tok - b * T), Hq(heads_q), qih(q.in_h), kih(k.in_h), qoh(q.out_h), koh(k.out_h) {
    qi = static_cast<const E *>(q.in) + (b * q.in_b + t * q.in_t);
    ki = static_cast<const E *>(k.in) + (b * k.in_b + t * k.in_t);
    qo = static_cast<E *>(q.out) + (b * q.out_b + t * q.out_t);
    ko = static_cast<E *>(k.out) + (b * k.out_b + t * k.out_t);
  }
  __device__ __forceinline__ const E *in(int h) const { return h < Hq ? qi + h * qih : ki + (h - Hq) * kih; }
  __device__ __forceinline__ E *out(int h) const { return h < Hq ? qo + h * qoh : ko + (h - Hq) * koh; }
};

// grid.x: runs of tokens, grid.y: groups of hpt heads of q followed by k.
template <typename E, bool ADJ, int BATCH>
__global__ void __launch_bounds__(kRopeThreads, BATCH <= 2 ? 8 : sizeof(E) == 2 ? 7 : 6)
    rope_kernel(RopeTensor q, RopeTensor k, const __grid_constant__ RopeParams rp, RopeWalk w, int Hq, int Hk, int hpt) {
  __shared__ RopeTable<RopeVec<E>::N> tables[kRopeThreads / 32];
  const int h0 = blockIdx.y * hpt, h1 = min(h0 + hpt, Hq + Hk);
  RopeUnit<E, ADJ> ru;
  ru.place(w.piece(), rp.n_pairs);
  const bool live = w.token() < w.tokens;
  const RopeRows<E> at(q, k, Hq, live ? w.token() : 0, w.T);
  uint4 va[BATCH], vb[BATCH];
  auto load = [&](int hb) {
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (hb + j < h1) {
        const E *src = at.in(hb + j);
        va[j] = ld_once(src + ru.va);
        vb[j] = ld_once(src + ru.vb);
      }
  };
  // the angles while the first loads are on their way
  pdl_wait();
  if (live) load(h0);
  RopeTable<RopeVec<E>::N> &table = tables[threadIdx.x / 32];
  const RopePlace place(rp, at.b, at.t, 0);
  table.fill(rp);
  if (!live) return;
  if (rp.n_axes == 1)
    ru.turn([&](int j, float &c, float &s) { table.template angle<true>(j, place, c, s); });
  else
    ru.turn([&](int j, float &c, float &s) { table.template angle<false>(j, place, c, s); });
  for (int hb = h0; hb < h1; hb += BATCH) {
    if (hb > h0) load(hb);
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (hb + j < h1) {
        E *dst = at.out(hb + j);
        ru.apply(va[j], vb[j]);
        __stcs(reinterpret_cast<uint4 *>(dst + ru.va), va[j]);
        __stcs(reinterpret_cast<uint4 *>(dst + ru.vb), vb[j]);
      }
  }
}

// The same for rows in 16-byte pieces whose rotated part is not made of whole
// pieces (half-split pairs, n_pairs of any size: the partner of an element lies
// anywhere in the row).  The lanes of a row exchange it through shared memory.
// (One thread per pair with 2-byte accesses took 539 us for 2 x 48 x 51971 x 64
// bf16 with 3 pairs, whose copies take 188.)  4 x 36238 tokens of 6 heads with 5 pairs
// less than whole rows: bf16 of 64 / 128 61.6 / 115 us (the bytes 33 / 66), fp32 82.6 / 159
// (66 / 131): every lane forms the angles of its own elements, so each pair's twice.
template <typename E>
__global__ void __launch_bounds__(kRopeThreads)
    rope_any_kernel(RopeTensor q, RopeTensor k, const __grid_constant__ RopeParams rp, RopeWalk w, int Hq, int Hk, int hpt) {
  constexpr int N = RopeVec<E>::N, B = kFewBatch;
  __shared__ __align__(16) E s_rows[B][kRopeThreads * N];   // the block's rows, one after another
  __shared__ RopeTable<N> tables[kRopeThreads / 32];
  const int u = w.piece(), base = (threadIdx.x - u) * N, n = rp.n_pairs;   // lanes of a row: 8 to 32, so a row is one warp's
  const int h0 = blockIdx.y * hpt, h1 = min(h0 + hpt, Hq + Hk);
  RopeTable<N> &table = tables[threadIdx.x / 32];
  const bool live = w.token() < w.tokens;
  const RopeRows<E> at(q, k, Hq, live ? w.token() : 0, w.T);
  // the turn of each element: x cos + partner sin (the sine negative for the first of a pair)
  float c[N], s[N];
  int other[N];
  pdl_wait();
  {
    const RopePlace place(rp, at.b, at.t, 0);
    table.fill(rp);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int x = u * N + e;
      other[e] = -1;
      if (x < 2 * n) {
        const int j = x < n ? x : x - n;
        table.template angle<false>(j, place, c[e], s[e]);
        other[e] = base + (x < n ? x + n : x - n);
        if (x < n) s[e] = -s[e];
      }
    }
  }
  for (int hb = h0; hb < h1; hb += B) {
    uint4 v[B];
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (live && hb + j < h1) v[j] = ld_once(at.in(hb + j) + u * N);
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (live && hb + j < h1) *reinterpret_cast<uint4 *>(&s_rows[j][threadIdx.x * N]) = v[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (!live || hb + j >= h1) continue;
      if (u * N < 2 * n) {   // pieces past the rotated part pass bit for bit
        float x[N];
        RopeVec<E>::unpack(v[j], x);
        alignas(16) E y[N];
        *reinterpret_cast<uint4 *>(y) = v[j];
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (other[e] >= 0) from_f32(fmaf(x[e], c[e], to_f32(s_rows[j][other[e]]) * s[e]), y[e]);
        v[j] = *reinterpret_cast<uint4 *>(y);
      }
      __stcs(reinterpret_cast<uint4 *>(at.out(hb + j) + u * N), v[j]);
    }
    __syncwarp();
  }
}

// Two elements of a row, of any alignment: pair j < n_pairs, or two elements
// past the rotated part.
template <typename E, typename F>
__device__ __forceinline__ void rope_pair(const E *src, E *dst, int j, int n_pairs, bool adjacent, F &&angle) {
  const bool rot = j < n_pairs;
  const int a = rot ? (adjacent ? 2 * j : j) : 2 * j;
  const int b = rot && !adjacent ? j + n_pairs : a + 1;
  const E ea = src[a], eb = src[b];
  if (!rot) {
    dst[a] = ea;
    dst[b] = eb;
    return;
  }
  float c, s;
  angle(j, c, s);
  const float x = to_f32(ea), y = to_f32(eb);
  from_f32(fmaf(x, c, -y * s), dst[a]);
  from_f32(fmaf(y, c, x * s), dst[b]);
}

// Any alignment: one thread per pair of elements (d / 2 of them a row).  Bound by the
// accesses of one element: 4 x 36238 tokens of 6 heads, half-split or adjacent pairs
// alike, bf16 of 64 / 128 92 / 188 us (the bytes 33 / 66), fp32 98 / 193 (66 / 131).
template <typename E>
__global__ void __launch_bounds__(kRopeThreads)
    rope_scalar_kernel(RopeTensor q, RopeTensor k, const __grid_constant__ RopeParams rp, int adjacent, RopeWalk w, int Hq,
                       int Hk, int hpt) {
  __shared__ RopeTable<1> tables[kRopeThreads / 32];
  const int j = w.piece();
  const int h0 = blockIdx.y * hpt, h1 = min(h0 + hpt, Hq + Hk);
  RopeTable<1> &table = tables[threadIdx.x / 32];
  pdl_wait();
  table.fill(rp);
  if (w.token() >= w.tokens) return;
  const RopeRows<E> at(q, k, Hq, w.token(), w.T);
  float c = 1.f, s = 0.f;
  if (j < rp.n_pairs) table.angle<false>(j, RopePlace(rp, at.b, at.t, 0), c, s);
  for (int h = h0; h < h1; ++h)
    rope_pair(at.in(h), at.out(h), j, rp.n_pairs, adjacent != 0, [&](int, float &cc, float &ss) { cc = c, ss = s; });
}

// Heads per thread: sin and cos are shared by the heads a thread visits, but a
// short input needs the heads spread over threads to fill the GPU.
static int heads_per_thread(long long n_units, int heads, int most) {
  const long long threads = n_units * heads, want = 152ll * 1024;
  const long long h = threads / want, cap = heads < most ? heads : most;
  return (int)(h < 1 ? 1 : h > cap ? cap : h);
}

cudaError_t launch_rope(const RopeTensor &q, const RopeTensor &k, const RopeParams &rp, bool adjacent, RopePath path,
                        int B, int Hq, int Hk, int T, int d, int dtype, cudaStream_t stream) {
  const int n = dtype == DA_BF16 ? 8 : 4;
  const int units = path == kRopeUnits ? d / (2 * n) : path == kRopeAny ? d / n : d / 2;   // a power of two
  RopeWalk w;
  w.tokens = B * T;
  w.T = T;
  w.shift = 0;
  while ((1 << w.shift) < units) ++w.shift;
  // 2 x 32 heads x 51971 x 128 bf16: 272 us with 16 heads at most, 296 with 8, 276 with 24
  const int hpt = heads_per_thread((long long)w.tokens * units, Hq + Hk, 16);
  const int run = kRopeThreads >> w.shift;
  const dim3 grid((unsigned)(((int64_t)w.tokens + run - 1) / run), (unsigned)((Hq + Hk + hpt - 1) / hpt));
#define DA_ROPE_UNITS(E, BATCH)                                                                                 \
  adjacent ? launch_after(rope_kernel<E, true, BATCH>, grid, kRopeThreads, 0, stream, q, k, rp, w, Hq, Hk, hpt) \
           : launch_after(rope_kernel<E, false, BATCH>, grid, kRopeThreads, 0, stream, q, k, rp, w, Hq, Hk, hpt)
#define DA_ROPE(E)                                                                                              \
  if (path == kRopeAny)                                                                                         \
    return launch_after(rope_any_kernel<E>, grid, kRopeThreads, 0, stream, q, k, rp, w, Hq, Hk, hpt);           \
  if (path == kRopeScalar)                                                                                      \
    return launch_after(rope_scalar_kernel<E>, grid, kRopeThreads, 0, stream, q, k, rp, (int)adjacent, w, Hq,   \
                        Hk, hpt);                                                                               \
  return hpt > 2 ? DA_ROPE_UNITS(E, kRopeBatch) : DA_ROPE_UNITS(E, kFewBatch);
  if (dtype == DA_BF16) {
    DA_ROPE(__nv_bfloat16)
  } else {
    DA_ROPE(float)
  }
#undef DA_ROPE
#undef DA_ROPE_UNITS
}

// ---------------------------------------------------------------------------
// Append to the paged cache.
//
// A block takes a run of up to 128 tokens and up to kAppendHeads heads.  Every
// thread first issues the loads of its first 16-byte pieces (they do not depend
// on where the token goes); meanwhile the block's threads place all the tokens,
// one each: the sequence by a binary search of cu_tokens (held in shared memory
// with the lengths up to kAppendSearch sequences, so one global read serves
// both), the pages from the tables.  Then it walks the run.  Placing takes three
// dependent reads (~3 us), on which blocks of 16 tokens spent most of their time.
// The demand goes out with neighbouring threads on neighbouring tokens.
// ---------------------------------------------------------------------------
constexpr int kAppendSearch = 1024;
// Heads that share a thread's sines and cosines (48 rows of 64: 228 us, 8 heads 259, 4 heads 323).
constexpr int kAppendHeads = 16;

struct TokenPlace {
  int pos;            // place in its sequence; -1: skip this token
  int page, dpage;
};

__device__ __forceinline__ TokenPlace place_token(int n, const int32_t *cu, const int32_t *lens, const AppendArgs &a,
                                                  const dilution_attn_paged_cache &c) {
  TokenPlace p{-1, 0, 0};
  if (n >= a.N || n >= cu[c.S]) return p;   // padding
  int lo = 0, hi = c.S - 1;                 // the last sequence that starts at or before n
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (cu[mid] <= n)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int first = cu[lo], end = cu[lo + 1];
  const int len = lens[lo];
  const long long pos = (long long)len - end + n;
  const long long pg = pos / c.page_size;
  bool ok = first >= 0 && first <= n && n < end && end <= a.N && pos >= 0 && end - first <= len && pg < c.max_pages;
  if (ok) {
    p.page = __ldcg(c.page_table + (size_t)lo * c.max_pages + pg);
    p.dpage = __ldcg(c.demand_table + (size_t)lo * c.max_pages + pg);
    ok = p.page >= 0 && p.page < c.num_pages && p.dpage >= 0 && p.dpage < c.num_demand_pages;
  }
  if (ok)
    p.pos = (int)pos;
  else
    atomicCAS(a.status, DA_OK, DA_ERR_INVALID);
  return p;
}

// grid.x: runs of tokens; grid.y: groups of heads of [q | k | v], then the
// demand.  VEC: 16-byte pieces (units of RopeUnit); else pairs of elements.
template <typename E, bool ADJ, bool VEC>
__global__ void __launch_bounds__(kRopeThreads)
    append_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ dilution_attn_paged_cache c,
                  const __grid_constant__ RopeParams rp) {
  __shared__ int32_t s_cu[kAppendSearch], s_len[kAppendSearch];
  __shared__ TokenPlace s_place[kRopeThreads];
  __shared__ RopeTable<VEC ? RopeVec<E>::N : 1> tables[kRopeThreads / 32];
  RopeTable<VEC ? RopeVec<E>::N : 1> &table = tables[threadIdx.x / 32];
  const int Hq = a.q != nullptr ? c.Hq : 0;
  const int rows = Hq + 2 * c.Hkv;
  const int groups = (rows + a.hpt - 1) / a.hpt;
  const bool is_demand = (int)blockIdx.y == groups;
  const int n0 = blockIdx.x * a.tokens;
  const int h0 = blockIdx.y * a.hpt, h1 = min(h0 + a.hpt, rows);
  const int h_turn = Hq + c.Hkv;                 // heads below turn, the values pass
  // this thread's piece, and its first token of the block's run
  const int tt0 = threadIdx.x / a.units, u = threadIdx.x - tt0 * a.units, step = kRopeThreads / a.units;
  const bool mine = !is_demand && tt0 < step;
  const int last = min(a.tokens, a.N - n0);
  auto source = [&](long long n, int h) -> const E * {
    if (h < Hq) return static_cast<const E *>(a.q) + n * a.q_t + h * a.q_h;
    if (h < h_turn) return static_cast<const E *>(a.k) + n * a.k_t + (h - Hq) * a.k_h;
    return static_cast<const E *>(a.v) + n * a.v_t + (h - h_turn) * a.v_h;
  };
  RopeUnit<E, ADJ> ru;
  uint4 va[kFewBatch], vb[kFewBatch];
  auto load = [&](int tt, int hb) {
#pragma unroll
    for (int j = 0; j < kFewBatch; ++j)
      if (hb + j < h1) {
        const E *src = source(n0 + tt, hb + j);
        va[j] = ld_once(src + ru.va);
        vb[j] = ld_once(src + ru.vb);
      }
  };
  pdl_wait();
  if constexpr (VEC) {
    ru.place(u, h0 < h_turn ? rp.n_pairs : 0);
    if (mine && tt0 < last) load(tt0, h0);
  }
  if (!is_demand) table.fill(rp);
  const int32_t *cu = a.cu_tokens, *lens = c.seq_lens;
  if (c.S + 1 <= kAppendSearch) {
    for (int i = threadIdx.x; i <= c.S; i += kRopeThreads) {
      s_cu[i] = __ldcg(a.cu_tokens + i);
      if (i < c.S) s_len[i] = __ldcg(c.seq_lens + i);
    }
    cu = s_cu;
    lens = s_len;
    __syncthreads();
  }
  if (threadIdx.x < a.tokens) s_place[threadIdx.x] = place_token(n0 + threadIdx.x, cu, lens, a, c);
  __syncthreads();
  if (is_demand) {   // [page][head][row]
    for (int i = threadIdx.x; i < a.tokens * c.Hq; i += kRopeThreads) {
      const int t = i % a.tokens, h = i / a.tokens;
      const TokenPlace p = s_place[t];
      if (p.pos < 0) continue;
      const float x = a.demand != nullptr ? a.demand[(long long)(n0 + t) * a.dem_t + (long long)h * a.dem_h] : 0.f;
      c.demand_pages[((size_t)p.dpage * c.Hq + h) * c.page_size + p.pos % c.page_size] = x;
    }
    return;
  }
  if (!mine) return;
  for (int tt = tt0; tt < last; tt += step) {
    if constexpr (VEC) {
      if (tt > tt0) load(tt, h0);
    }
    const TokenPlace p = s_place[tt];
    const long long n = n0 + tt;
    if (p.pos >= 0) {
      const RopePlace where(rp, 0, n, p.pos);
      auto angle = [&](int j, float &cc, float &ss) { table.template angle<false>(j, where, cc, ss); };
      auto target = [&](int h) -> E * {
        if (h < Hq) return static_cast<E *>(a.q_out) + ((size_t)n * c.Hq + h) * c.d;
        const bool is_k = h < h_turn;
        const size_t row = ((size_t)p.page * c.Hkv + (h - (is_k ? Hq : h_turn))) * c.page_size + p.pos % c.page_size;
        return static_cast<E *>(is_k ? c.k_pages : c.v_pages) + row * c.d;
      };
      if constexpr (VEC) {
        if (h0 < h_turn) ru.turn(angle);
        for (int hb = h0; hb < h1; hb += kFewBatch) {
          if (hb > h0) load(tt, hb);
#pragma unroll
          for (int j = 0; j < kFewBatch; ++j)
            if (hb + j < h1) {
              E *dst = target(hb + j);
              if (hb + j < h_turn) ru.apply(va[j], vb[j]);
              *reinterpret_cast<uint4 *>(dst + ru.va) = va[j];
              *reinterpret_cast<uint4 *>(dst + ru.vb) = vb[j];
            }
        }
      } else {
        float c1 = 1.f, s1 = 0.f;
        if (u < rp.n_pairs && h0 < h_turn) angle(u, c1, s1);
        for (int h = h0; h < h1; ++h)
          rope_pair(source(n, h), target(h), u, h < h_turn ? rp.n_pairs : 0, ADJ,
                    [&](int, float &cc, float &ss) { cc = c1, ss = s1; });
      }
    }
  }
}

cudaError_t launch_append(const AppendArgs &args, const dilution_attn_paged_cache &c, const RopeParams &rp, bool vec,
                          cudaStream_t stream) {
  AppendArgs a = args;
  const int nv = c.dtype == DA_BF16 ? 8 : 4;
  a.units = vec ? c.d / (2 * nv) : c.d / 2;
  const int rows = (a.q != nullptr ? c.Hq : 0) + 2 * c.Hkv;
  a.hpt = heads_per_thread((long long)a.N * a.units, rows, kAppendHeads);
  // a block's run: longer ones share the placing, as long as there are 10 blocks
  // for each SM, more than are resident (27100 tokens of 4 heads, d = 128: 27 us
  // with 10, 33 with 7, 44 with 4, 29 with 20)
  const int step = kRopeThreads / a.units, heads = (rows + a.hpt - 1) / a.hpt + 1;
  int64_t turns = ((int64_t)a.N + step - 1) / step * heads / (10 * 152);
  if (turns > kRopeThreads / step) turns = kRopeThreads / step;
  a.tokens = step * (int)(turns < 1 ? 1 : turns);
  const dim3 grid((unsigned)((a.N + a.tokens - 1) / a.tokens), (unsigned)heads);
#define DA_APPEND(E, ADJ, VEC) launch_after(append_kernel<E, ADJ, VEC>, grid, kRopeThreads, 0, stream, a, c, rp)
  if (c.dtype == DA_BF16) {
    if (vec) return a.adjacent ? DA_APPEND(__nv_bfloat16, true, true) : DA_APPEND(__nv_bfloat16, false, true);
    return a.adjacent ? DA_APPEND(__nv_bfloat16, true, false) : DA_APPEND(__nv_bfloat16, false, false);
  }
  if (vec) return a.adjacent ? DA_APPEND(float, true, true) : DA_APPEND(float, false, true);
  return a.adjacent ? DA_APPEND(float, true, false) : DA_APPEND(float, false, false);
#undef DA_APPEND
}

}  // namespace da
