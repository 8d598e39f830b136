// Rows of a matrix to 8-bit codes with one scale each: a merged weight's
// output channels, or activations per token; optionally behind the RMS norm
// with the residual's addition, which is how a decoder layer produces them.
//
//   v_j   = x_j                                       (dora_quantize_rows)
//   v_j   = h_j w_j / sqrt(mean(h^2) + eps),  h = x (+ residual), rounded to
//           the dtype                                 (dora_rmsnorm_quant)
//   scale = max_j |v_j| / 127,   q_j = rint(v_j / scale)
//
// The codes do not need the rms (but where it decides whether there is a step at
// all): it is a common factor of the row, so with u_j = h_j w_j and a = max |u_j|,
// q_j = rint(u_j (127 / a))  and  scale = (a / 127) / rms.  The row's sum of
// squares and its maximum are therefore reduced together, in one pass and with
// one block barrier, and the row stays in registers in between: x (and the
// residual) are read once, h and the codes written once.
//
// Sums, maxima and products are fp32; h is rounded to the dtype because it is
// stored and read again by the next layer, and the norm is of that stored
// value.  A row whose sum of squares, or whose scale, is beyond fp32's range
// counts as not finite.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "compose.cuh"
#include "sm100.cuh"

namespace dora {

constexpr float kCodeMax = 127.f;
constexpr float kMinNormal = 1.17549435e-38f;  // 2^-126
constexpr uint32_t kInfBits = 0x7f800000u;

// Pairs of fp32 values in one instruction (each rounded as alone).
__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split_f32(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// max(a, |b|, |c|), NaN if any is.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

enum RowMode : int {
  kRowQuant = 0,    // x -> codes
  kRowNorm = 1,     // rms norm of x -> codes
  kRowNormAdd = 2,  // x + residual -> h; rms norm of h -> codes
};

struct RowArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* h_out;
  int8_t* q;
  float* scale;
  long long rows;  // at most 2^30, as d
  int d;
  float eps;
};

// VEC elements of a row as raw registers (VEC = 16 bytes' worth, or 1 where
// a row may start at any element).  Plain loads: the buffers may have been
// written by the kernel this one was launched behind, and h may be written
// over x or the residual.
template <typename E, int VEC>
struct RowVec;

template <>
struct RowVec<__nv_bfloat16, 8> {
  using raw = uint4;
  static __device__ __forceinline__ raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ void unpack(const raw& u, float (&v)[8]) {
    v[0] = bf16lo_to_f32(u.x); v[1] = bf16hi_to_f32(u.x);
    v[2] = bf16lo_to_f32(u.y); v[3] = bf16hi_to_f32(u.y);
    v[4] = bf16lo_to_f32(u.z); v[5] = bf16hi_to_f32(u.z);
    v[6] = bf16lo_to_f32(u.w); v[7] = bf16hi_to_f32(u.w);
  }
  static __device__ __forceinline__ raw pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                      pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
  }
};

template <>
struct RowVec<__nv_bfloat16, 1> {
  using raw = uint16_t;
  static __device__ __forceinline__ raw zero() { return 0; }
  static __device__ __forceinline__ void unpack(const raw& u, float (&v)[1]) {
    v[0] = __uint_as_float(static_cast<uint32_t>(u) << 16);
  }
  static __device__ __forceinline__ raw pack(const float (&v)[1]) { return f32_to_bf16_rn(v[0]); }
};

template <>
struct RowVec<float, 4> {
  using raw = float4;
  static __device__ __forceinline__ raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void unpack(const raw& u, float (&v)[4]) {
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
  static __device__ __forceinline__ raw pack(const float (&v)[4]) {
    return make_float4(v[0], v[1], v[2], v[3]);
  }
};

template <>
struct RowVec<float, 1> {
  using raw = float;
  static __device__ __forceinline__ raw zero() { return 0.f; }
  static __device__ __forceinline__ void unpack(const raw& u, float (&v)[1]) { v[0] = u; }
  static __device__ __forceinline__ raw pack(const float (&v)[1]) { return v[0]; }
};

template <typename E, int VEC>
__device__ __forceinline__ typename RowVec<E, VEC>::raw load_vec(const void* m, size_t at) {
  return *reinterpret_cast<const typename RowVec<E, VEC>::raw*>(static_cast<const E*>(m) + at);
}
template <typename E, int VEC>
__device__ __forceinline__ void store_vec(void* m, size_t at,
                                          const typename RowVec<E, VEC>::raw& v) {
  *reinterpret_cast<typename RowVec<E, VEC>::raw*>(static_cast<E*>(m) + at) = v;
}

// The first n of VEC elements, the others zero.
template <typename E, int VEC>
__device__ __forceinline__ typename RowVec<E, VEC>::raw load_first(const E* p, int n) {
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = e < n ? static_cast<float>(p[e]) : 0.f;
  return RowVec<E, VEC>::pack(v);  // exact: the values are E's
}

// The codes of VEC values: u inv rounded to an integer, half to even, by the
// addition of 1.5 2^23 in the product's rounding, which leaves the code in the
// low byte (a conversion instruction has a quarter of the rate, and was the
// longest part of the kernel's arithmetic).  |u inv| is at most 127 up to a
// rounding of inv, so the nearest integer is at most 127.
constexpr float kRoundMagic = 12582912.f;

template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* p, const float (&u)[VEC], float inv) {
  uint32_t q[VEC], w[(VEC + 3) / 4];
  if constexpr (VEC > 1) {
    const uint64_t inv2 = pair_f32(inv, inv), magic2 = pair_f32(kRoundMagic, kRoundMagic);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      float a, b;
      split_f32(fma_f32x2(pair_f32(u[e], u[e + 1]), inv2, magic2), a, b);
      q[e] = __float_as_uint(a);
      q[e + 1] = __float_as_uint(b);
    }
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040),
                         __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
  } else {
    w[0] = __float_as_uint(__fmaf_rn(u[0], inv, kRoundMagic));
  }
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
    *p = static_cast<int8_t>(w[0]);
  }
}

// Elements [VEC - n, 2 VEC - n) of the two vectors a, b, n in 0 .. VEC - 1:
// shifts by one, two and four elements under the bits of n.
template <typename E, int VEC>
__device__ __forceinline__ typename RowVec<E, VEC>::raw shift_in(
    const typename RowVec<E, VEC>::raw& a, const typename RowVec<E, VEC>::raw& b, int n) {
  static_assert(sizeof(a) == 16, "vectors of four words");
  uint32_t w[8];
  *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(&a);
  *reinterpret_cast<uint4*>(w + 4) = *reinterpret_cast<const uint4*>(&b);
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 7; i >= 1; --i) w[i] = n & 1 ? __funnelshift_l(w[i - 1], w[i], 16) : w[i];
    n >>= 1;
  }
#pragma unroll
  for (int i = 7; i >= 2; --i) w[i] = n & 1 ? w[i - 1] : w[i];
#pragma unroll
  for (int i = 7; i >= 4; --i) w[i] = n & 2 ? w[i - 2] : w[i];
  typename RowVec<E, VEC>::raw out;
  *reinterpret_cast<uint4*>(&out) = *reinterpret_cast<const uint4*>(w + 4);
  return out;
}

// A row in vectors.  RAGGED false: it is a whole number of them.  RAGGED: they
// are taken at multiples of VEC elements of the whole matrix, so that x, the
// residual, h and the codes share one alignment whatever the row length; of a
// row these are its `vecs` whole ones from column `head`, and the `loose`
// elements before and behind them (fewer than 2 VEC) go one to a lane of its
// last warp.  No vector reaches into another row, and there are never more
// than d / VEC, so that a row of 2^n - 1 columns takes no more threads than one
// of 2^n.  (With first and last vectors that were masked and stored by element:
// 122 against 78 us at [8192, 8191] bf16 with a residual, 93 against 41 without.)
template <int VEC, bool RAGGED>
struct RowSpan {
  int d, lead, head, vecs, loose;
  __host__ __device__ __forceinline__ RowSpan(long long row, int cols) : d(cols) {
    lead = RAGGED ? static_cast<int>(static_cast<size_t>(row) * cols % VEC) : 0;
    head = RAGGED ? ((VEC - lead) % VEC < cols ? (VEC - lead) % VEC : cols) : 0;
    vecs = (cols - head) / VEC;
    loose = RAGGED ? cols - vecs * VEC : 0;
  }
  __host__ __device__ __forceinline__ size_t column(int c) const {
    return static_cast<size_t>(c) * VEC + head;
  }
  __host__ __device__ __forceinline__ int loose_column(int e) const {
    return e < head ? e : vecs * VEC + e;
  }
  // Vector c takes the last `lead` elements of the weight's vector before this
  // one, and the first of this one: column(c) = weight_vec(c) VEC - lead.
  __host__ __device__ __forceinline__ int weight_vec(int c) const { return lead ? c + 1 : c; }
  // How many elements of the weight's vector v there are.
  __host__ __device__ __forceinline__ int weight_count(int v) const {
    if (v < 0 || v * VEC >= d) return 0;
    return v * VEC + VEC > d ? d - v * VEC : VEC;
  }
  // The weight at the columns of vector c: where rows are ragged, put together
  // from two vectors of the weight (element by element, each load of a warp
  // touched four times the lines: 27 against 17 us at [2047, 4099] fp32).
  template <typename E>
  __device__ __forceinline__ typename RowVec<E, VEC>::raw weight(const void* w, int c) const {
    using RV = RowVec<E, VEC>;
    const E* p = static_cast<const E*>(w);
    if constexpr (!RAGGED) {
      return *reinterpret_cast<const typename RV::raw*>(p + c * VEC);
    } else {
      auto whole = [&](int v) -> typename RV::raw {
        const int n = weight_count(v);
        if (n == 0) return RV::zero();
        if (n < VEC) return load_first<E, VEC>(p + v * VEC, n);
        return *reinterpret_cast<const typename RV::raw*>(p + v * VEC);
      };
      const int k = weight_vec(c);
      return shift_in<E, VEC>(whole(k - 1), whole(k), lead);
    }
  }
};

// h of one vector: x, or x + residual rounded to the dtype.
template <typename E, int VEC, int MODE>
__device__ __forceinline__ typename RowVec<E, VEC>::raw row_h(
    const typename RowVec<E, VEC>::raw& x, const typename RowVec<E, VEC>::raw& r) {
  using RV = RowVec<E, VEC>;
  if constexpr (MODE != kRowNormAdd) return x;
  float a[VEC], b[VEC];
  RV::unpack(x, a);
  RV::unpack(r, b);
#pragma unroll
  for (int e = 0; e < VEC; ++e) a[e] += b[e];
  return RV::pack(a);
}

// u of one vector: what the codes are proportional to.
template <typename E, int VEC, int MODE>
__device__ __forceinline__ void row_u(const typename RowVec<E, VEC>::raw& h,
                                      const typename RowVec<E, VEC>::raw& w, float (&u)[VEC]) {
  using RV = RowVec<E, VEC>;
  RV::unpack(h, u);
  if constexpr (MODE != kRowQuant) {
    float g[VEC];
    RV::unpack(w, g);
    if constexpr (VEC > 1) {
#pragma unroll
      for (int e = 0; e < VEC; e += 2)
        split_f32(mul_f32x2(pair_f32(u[e], u[e + 1]), pair_f32(g[e], g[e + 1])), u[e], u[e + 1]);
    } else {
      u[0] *= g[0];
    }
  }
}

// The codes of one vector.
template <typename E, int VEC, int MODE>
__device__ __forceinline__ void row_codes(const typename RowVec<E, VEC>::raw& h,
                                          const typename RowVec<E, VEC>::raw& w, float inv,
                                          int8_t* q) {
  float u[VEC];
  row_u<E, VEC, MODE>(h, w, u);
  if (inv == 0.f) {  // also where u is not finite
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = 0.f;
  }
  store_codes<VEC>(q, u, inv);
}

// One vector's share of the row's sum of squares (two partial sums) and
// maximum, which is NaN if a value is.
template <typename E, int VEC, int MODE>
__device__ __forceinline__ void row_stats(const typename RowVec<E, VEC>::raw& h,
                                          const typename RowVec<E, VEC>::raw& w, uint64_t& sq,
                                          float& top) {
  float u[VEC];
  row_u<E, VEC, MODE>(h, w, u);
#pragma unroll
  for (int e = 0; e < VEC; e += 2) top = max_abs_nan(top, u[e], u[VEC > 1 ? e + 1 : e]);
  if constexpr (MODE != kRowQuant) {
    RowVec<E, VEC>::unpack(h, u);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const uint64_t v = pair_f32(u[e], VEC > 1 ? u[VEC > 1 ? e + 1 : e] : 0.f);
      sq = fma_f32x2(v, v, sq);
    }
  }
}

// Sum and maximum over the `warps` warps of a row's group, in a fixed order;
// the same value in every thread.  `red`: the group's slots (two per warp).
__device__ __forceinline__ void row_reduce(uint64_t sq2, float top1, int warps, int warp, int lane,
                                           uint2* red, float& sq, uint32_t& top) {
  float a, b;
  split_f32(sq2, a, b);
  sq = a + b;
  // As bit patterns, which order like the values (they are not negative) with
  // infinity and NaN on top.
  top = __float_as_uint(top1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  top = __reduce_max_sync(0xffffffffu, top);
  if (warps == 1) return;
  if (lane == 0) red[warp] = make_uint2(__float_as_uint(sq), top);
  __syncthreads();
  const uint2 v = lane < warps ? red[lane] : make_uint2(0u, 0u);
  sq = __uint_as_float(v.x);
  top = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  top = __reduce_max_sync(0xffffffffu, top);
}

// Factor of the codes from the row's maximum: 127 / max rounded up, so that a
// value of half the maximum, code 63.5 exactly, never falls short of the half
// that goes to the even 64 (rounded to nearest, it did for 66 of the 128
// mantissas of a bf16 maximum).  Every other code of a row of 8-bit mantissas is
// at least 1/510 of its power of two from a half, against 2^-23 that the factor
// is off, or its 127 / max is exact: such rows get the codes of the definition.
// (The nearest quotient, or the next where the sign of the exact residual says
// that it is below; the rounded-up division is a call, whose registers cost the
// norm at [8192, 8192] bf16 47 instead of 38 us.)
__device__ __forceinline__ float code_factor(float top) {
  const float inv = __fdiv_rn(kCodeMax, top);
  const uint32_t up = __fmaf_rn(top, inv, -kCodeMax) < 0.f ? 1u : 0u;
  return __uint_as_float(__float_as_uint(inv) + up);
}

// What a row that is only quantised is held with, from its maximum: factor 0 for
// one that is not finite and for one whose step max / 127 would not be a normal
// number, scale NaN and 0 there.
__device__ __forceinline__ float quant_inv(uint32_t top) {
  const bool live = top < kInfBits && __uint_as_float(top) >= kCodeMax * kMinNormal;
  return live ? code_factor(__uint_as_float(top)) : 0.f;
}
__device__ __forceinline__ float quant_scale(uint32_t top, float inv) {
  if (top >= kInfBits) return __uint_as_float(0x7fc00000u);
  return inv == 0.f ? 0.f : __fdiv_rn(__uint_as_float(top), kCodeMax);
}

// Behind the norm the step is max|h w| / 127 / rms.  For an ordinary row
// (sq + eps < 2^100 keeps 1 / rms in 2^-50 .. 2^75) it is a normal number whatever
// the rms, which therefore only the thread that stores the scale forms.
__device__ __forceinline__ bool norm_row_ordinary(float sq, uint32_t top, float eps) {
  return __fadd_rn(sq, eps) < 0x1p100f && __uint_as_float(top) >= 0x1p-50f &&
         __uint_as_float(top) <= 0x1p40f;
}
// Of the others, one that is not finite is held as codes 0 with scale NaN and one
// of zeros as codes 0 with scale 0, which are all there are in practice.  The rest
// need their rms: their scale is kRowAgain until they are taken again, behind the
// block's last row.  (Products up to 2^-150 are 0 too, but only a 1 / rms above
// 2^30 gives those a step.)
constexpr float kRowAgain = -1.f;
__device__ __forceinline__ bool norm_row_finite(float sq, uint32_t top) {
  return top < kInfBits && __float_as_uint(sq) < kInfBits;
}
__device__ __forceinline__ bool norm_row_again(float sq, uint32_t top, float eps) {
  return norm_row_finite(sq, top) && (top != 0u || eps < 0x1p-60f);
}
__device__ __forceinline__ float norm_rstd(float sq, int d, float eps) {
  const float mean = __fdiv_rn(sq, static_cast<float>(d));
  return __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(mean, eps)));
}
__device__ __forceinline__ float norm_scale(float sq, uint32_t top, int d, float eps) {
  return __fmul_rn(__fdiv_rn(__uint_as_float(top), kCodeMax), norm_rstd(sq, d, eps));
}

// max|h w| may be too small for its quotient by 127, or h w for fp32, where
// 1 / rms (up to 2^75 for the smallest eps) brings the step back into range: such
// a row is computed with h lifted by 2^96.  That is exact, since 1 / rms is then
// above 1/2 and |h| at most 2 sqrt(d), and the row's maximum becomes at most
// 2^-23.
constexpr float kRowLift = 0x1p96f;
__device__ __forceinline__ bool norm_row_lifts(float sq, uint32_t top, int d, float eps) {
  const float a = __uint_as_float(top);
  if (a >= kCodeMax * kMinNormal) return false;
  // (products below 2^-150 are 0; a little beyond the bound costs only time)
  return __fmul_rn(__fadd_rn(a, 0x1p-149f), norm_rstd(sq, d, eps)) >= 126.f * kMinNormal;
}

// Indices of the thread and the block, read here and not kept from an earlier use.
struct FreshIndex {
  int tid_x, tid_y, cta, ctas, threads, groups;
  __device__ __forceinline__ FreshIndex() {
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid_x));
    asm volatile("mov.u32 %0, %%tid.y;" : "=r"(tid_y));
    asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(cta));
    asm volatile("mov.u32 %0, %%nctaid.x;" : "=r"(ctas));
    asm volatile("mov.u32 %0, %%ntid.x;" : "=r"(threads));
    asm volatile("mov.u32 %0, %%ntid.y;" : "=r"(groups));
  }
};

// A row that needs its rms, again from memory, element by element; the same way in
// all its threads, which have met at a barrier since h was stored.  Behind the
// loop over the rows, small, and with nothing kept for it there: in the loop, by
// vectors, its registers cost the ragged norm with a residual ([8192, 8191] bf16)
// 94 instead of 76 us; so 78, and the norm of [4096, 14336] fp32 133 instead of 131.
template <typename E, int MODE>
__device__ __forceinline__ void norm_row_from_memory(const RowArgs& P, int row, int tid,
                                                     int threads, uint2 (&red)[2][32],
                                                     int& buf) {
  const int d = P.d;
  const E* h = static_cast<const E*>(MODE == kRowNormAdd ? P.h_out : P.x) +
               static_cast<size_t>(row) * d;
  const E* w = static_cast<const E*>(P.weight);
  float lift = 1.f;
  auto stats = [&](float& sq, uint32_t& top) {
    float s = 0.f, m = 0.f;
#pragma unroll 1
    for (int c = tid; c < d; c += threads) {
      const float v = static_cast<float>(h[c]);
      s = __fmaf_rn(v, v, s);
      m = fmaxf(m, fabsf(__fmul_rn(__fmul_rn(v, lift), static_cast<float>(w[c]))));
    }
    row_reduce(pair_f32(s, 0.f), m, threads >> 5, tid >> 5, tid & 31, red[buf], sq, top);
    buf ^= 1;
  };
  float sq;
  uint32_t top;
  stats(sq, top);
  if (norm_row_lifts(sq, top, d, P.eps)) {
    float unused;
    lift = kRowLift;
    stats(unused, top);
  }
  float inv = 0.f, scale = 0.f;
  if (__uint_as_float(top) >= kCodeMax * kMinNormal) {
    scale = __fmul_rn(norm_scale(sq, top, d, P.eps), lift == 1.f ? 1.f : 1.f / kRowLift);
    if (__float_as_uint(scale) >= kInfBits || norm_rstd(sq, d, P.eps) == 0.f)
      scale = __uint_as_float(0x7fc00000u);  // the scale, or mean + eps, is beyond fp32
    else if (scale >= kMinNormal)
      inv = code_factor(__uint_as_float(top));
    else
      scale = 0.f;
  }
  if (tid == 0) P.scale[row] = scale;
#pragma unroll 1
  for (int c = tid; c < d; c += threads) {
    const float u[1] = {
        __fmul_rn(__fmul_rn(static_cast<float>(h[c]), lift), static_cast<float>(w[c]))};
    if (DORA_BOUNDS_OK(row < P.rows))
      store_codes<1>(P.q + static_cast<size_t>(row) * d + c, u, inv);
  }
}

// The factor of a row: 0 where its codes are 0 or are to be taken again.
template <int MODE>
__device__ __forceinline__ float row_inv(float sq, uint32_t top, float eps) {
  if constexpr (MODE == kRowQuant) return quant_inv(top);
  return norm_row_ordinary(sq, top, eps) ? code_factor(__uint_as_float(top)) : 0.f;
}
// The row's scale, which no thread but the one that stores it waits for.  `again`
// (shared by the row's threads) is set where the row is to be taken again.
template <int MODE>
__device__ __forceinline__ float row_scale(float sq, uint32_t top, float inv, int d, float eps,
                                           int& again) {
  if constexpr (MODE == kRowQuant) return quant_scale(top, inv);
  if (inv != 0.f) return norm_scale(sq, top, d, eps);
  if (!norm_row_finite(sq, top)) return __uint_as_float(0x7fc00000u);
  if (!norm_row_again(sq, top, eps)) return 0.f;
  again = 1;
  return kRowAgain;
}

// Behind the loop over a block's rows: those that were left, if any was (`again`:
// one flag per block, at a fixed address; by row group its address had to live
// through the loop, with the registers and the time named above).
template <typename E, int MODE>
__device__ __forceinline__ void norm_rows_again(const RowArgs& P, const int& again,
                                                uint2 (&red)[2][32]) {
  const FreshIndex at;
  auto sync_row = [&] {
    if (at.threads > 32)
      __syncthreads();
    else
      __syncwarp();
  };
  sync_row();  // what the row's threads stored
  if (again == 0) return;
  int buf = 0;
  const int rows = static_cast<int>(P.rows);
  for (int row = at.cta * at.groups + at.tid_y; row < rows; row += at.ctas * at.groups)
    if (static_cast<const volatile float*>(P.scale)[row] == kRowAgain) {
      sync_row();  // all have read it
      norm_row_from_memory<E, MODE>(P, row, at.tid_x, at.threads, red, buf);
    }
}

// Rows of up to NV vectors per thread.  A group of blockDim.x threads (a
// multiple of 32) takes a row; blockDim.y groups share a block only where a
// group is one warp.  Blocks walk the rows with the grid's stride, which has
// to be the blocks that are resident at once (one more per SM runs as a second
// wave: 81 instead of 62 us at [25600, 5120]); the register bound keeps the
// two in step.
// AHEAD: the next row's loads are on their way while a row is reduced and
// stored, which the norm needs (93 instead of 88 % of the HBM rate at [8192,
// 8192]) and rows of which an SM holds one block (24 instead of 30 us for
// [2048, 14336] fp32); several blocks of rows that are only quantised overlap by
// themselves, and the registers cost them more (62 against 67 us at [25600,
// 5120]).
// NV: 16-byte vectors per thread, 4, or 1 for rows that a warp holds so (short
// rows need many of them in flight); or elements, where the matrix itself is
// not aligned.
constexpr int kRowVecs = 4;
constexpr int kRowScalars = 16;
constexpr int kRowGroups = 8;     // rows of one warp that share a block
constexpr int kRowThreads = 512;  // of a block that walks a row in two passes
// Registers per thread, and the threads per SM they leave room for, 1024 or 512:
// 64 KiB of loads in flight, or 32 and the next row's (the norms hold the
// weight too, and one of them has two streams; 112 registers leave room for no
// more threads, and cost the one without a residual 3 %).
__host__ __device__ constexpr int row_regs(int mode, int nv) {
  return nv == 1 ? 40 : mode == kRowQuant ? 64 : 128;
}
// That one does with fewer in fp32, which leave room for 640 threads, where one
// more block of them fits: [8192, 5120] in 37 instead of 51 us.  (Elsewhere 11.9
// against 10.8 at [2047, 4099]; in bf16 they spill.)
constexpr int kRowFewRegs = 96;
// (a quarter of the SM's registers serves a quarter of its warps)
__host__ __device__ constexpr int row_threads_per_sm(int regs) {
  return 16384 / (32 * regs) * 4 * 32;
}
// The largest block that its registers allow, in whole 512 threads.
__host__ __device__ constexpr int row_max_threads(int mode) {
  return row_threads_per_sm(row_regs(mode, kRowVecs)) >= 1024 ? 1024 : 512;
}

template <typename E, int VEC, int NV, int MODE, bool RAGGED, bool AHEAD,
          int REGS = row_regs(MODE, NV)>
__global__ void __maxnreg__(REGS) row_quant_kernel(const RowArgs P) {
  using RV = RowVec<E, VEC>;
  using RV1 = RowVec<E, 1>;
  using raw = typename RV::raw;
  using raw1 = typename RV1::raw;
  // The weight stays in registers over a block's rows: these start alike, since
  // the grid's stride is a multiple of VEC rows where rows are ragged.
  // Element by element there is no room for it, and it is read for each row.
  constexpr bool kHoldWeight = MODE != kRowQuant && VEC > 1;
  __shared__ uint2 red[2][32];
  __shared__ int again;
  if constexpr (MODE != kRowQuant) {
    if (threadIdx.x + threadIdx.y == 0) again = 0;
    if (blockDim.y > 1) __syncthreads();  // its other writers: thread 0 of each group
  }
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // (the norm's rows as ints: with two registers more the ragged one with a residual
  // spills; those that are only quantised took 75 instead of 62 us so at [25600, 5120])
  using Row = std::conditional_t<MODE == kRowQuant, long long, int>;
  const Row first = static_cast<Row>(blockIdx.x) * blockDim.y + threadIdx.y;
  const Row stride = static_cast<Row>(gridDim.x) * blockDim.y, rows = static_cast<Row>(P.rows);
  // (where they start alike, they have the same vectors and loose elements)
  const RowSpan<VEC, RAGGED> span(first, P.d);
  const bool last_warp = RAGGED && warp == warps - 1;
  const int loose = last_warp && lane < span.loose ? span.loose_column(lane) : -1;
  raw w[MODE != kRowQuant ? NV : 1];
  raw1 wl = RV1::zero();
  auto load_weight = [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      w[i] = c < span.vecs ? span.template weight<E>(P.weight, c) : RV::zero();
    }
    if constexpr (RAGGED)
      if (loose >= 0) wl = load_vec<E, 1>(P.weight, loose);
  };
  int buf = 0;
  raw x[NV], t[MODE == kRowNormAdd ? NV : 1];
  raw1 xl = RV1::zero(), tl = RV1::zero();
  auto load_row = [&](Row row) {
    const size_t at = static_cast<size_t>(row) * P.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      x[i] = c < span.vecs ? load_vec<E, VEC>(P.x, at + span.column(c)) : RV::zero();
      if constexpr (MODE == kRowNormAdd)
        t[i] = c < span.vecs ? load_vec<E, VEC>(P.residual, at + span.column(c)) : RV::zero();
    }
    if constexpr (RAGGED)
      if (loose >= 0) {
        xl = load_vec<E, 1>(P.x, at + loose);
        if constexpr (MODE == kRowNormAdd) tl = load_vec<E, 1>(P.residual, at + loose);
      }
  };
  if (AHEAD && first < rows) load_row(first);  // before the weight's are waited for
  if constexpr (kHoldWeight) load_weight();
  for (Row row = first; row < rows; row += stride) {
    const size_t at = static_cast<size_t>(row) * P.d;
    if (!AHEAD) load_row(row);
    raw h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      h[i] = row_h<E, VEC, MODE>(x[i], t[MODE == kRowNormAdd ? i : 0]);
      if constexpr (MODE == kRowNormAdd)
        if (c < span.vecs) store_vec<E, VEC>(P.h_out, at + span.column(c), h[i]);
    }
    const raw1 hl = row_h<E, 1, MODE>(xl, tl);
    if constexpr (RAGGED && MODE == kRowNormAdd)
      if (loose >= 0) store_vec<E, 1>(P.h_out, at + loose, hl);
    if (AHEAD && row + stride < rows) load_row(row + stride);
    if constexpr (MODE != kRowQuant && !kHoldWeight) load_weight();
    uint64_t sq2 = 0;
    float top1 = 0.f, sq;
    uint32_t top;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      row_stats<E, VEC, MODE>(h[i], w[MODE != kRowQuant ? i : 0], sq2, top1);
    if (last_warp) row_stats<E, 1, MODE>(hl, wl, sq2, top1);
    row_reduce(sq2, top1, warps, warp, lane, red[buf], sq, top);
    buf ^= 1;  // the slots are written again two rows on, past a barrier
    const float inv = row_inv<MODE>(sq, top, P.eps);
    if (threadIdx.x == 0)
      P.scale[row] = row_scale<MODE>(sq, top, inv, P.d, P.eps, again);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < span.vecs && DORA_BOUNDS_OK(span.column(c) + VEC <= static_cast<size_t>(P.d)))
        row_codes<E, VEC, MODE>(h[i], w[MODE != kRowQuant ? i : 0], inv,
                                P.q + at + span.column(c));
    }
    if constexpr (RAGGED)
      if (loose >= 0 && DORA_BOUNDS_OK(loose < P.d))
        row_codes<E, 1, MODE>(hl, wl, inv, P.q + at + loose);
  }
  if constexpr (MODE != kRowQuant)
    norm_rows_again<E, MODE>(P, again, red);
}

// Rows longer than the registers hold: two passes over the row, the second
// from L2 (of h, as this thread stored it, where there is a residual), with a
// few vectors on their way at a time (one by one [4096, 14336] fp32 took 80 us, 147
// with a residual, against 65 and 133; with the weight's as well they spill, 129
// and 274).
constexpr int kRowLongVecs = 4;  // half that of two streams
template <typename E, int VEC, int MODE, bool RAGGED>
__global__ void __launch_bounds__(kRowThreads, 2) row_quant_long_kernel(const RowArgs P) {
  using RV = RowVec<E, VEC>;
  using RV1 = RowVec<E, 1>;
  using raw = typename RV::raw;
  using raw1 = typename RV1::raw;
  constexpr int U = MODE == kRowNormAdd ? kRowLongVecs / 2 : kRowLongVecs;
  __shared__ uint2 red[2][32];
  __shared__ int again;
  if (threadIdx.x == 0) again = 0;
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int buf = 0;
  using Row = std::conditional_t<MODE == kRowQuant, long long, int>;
  const Row rows = static_cast<Row>(P.rows);
  for (Row row = blockIdx.x; row < rows; row += gridDim.x) {
    const RowSpan<VEC, RAGGED> span(row, P.d);
    const size_t at = static_cast<size_t>(row) * P.d;
    const bool last_warp = RAGGED && warp == warps - 1;
    const int loose = last_warp && lane < span.loose ? span.loose_column(lane) : -1;
    auto weight = [&](int c) {
      if constexpr (MODE == kRowQuant)
        return RV::zero();
      else
        return span.template weight<E>(P.weight, c);
    };
    uint64_t sq2 = 0;
    float top1 = 0.f, sq;
    uint32_t top;
    for (int c0 = threadIdx.x; c0 < span.vecs; c0 += U * blockDim.x) {
      raw h[U], t[MODE == kRowNormAdd ? U : 1];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + i * blockDim.x;
        h[i] = c < span.vecs ? load_vec<E, VEC>(P.x, at + span.column(c)) : RV::zero();
        if constexpr (MODE == kRowNormAdd)
          t[i] = c < span.vecs ? load_vec<E, VEC>(P.residual, at + span.column(c)) : RV::zero();
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + i * blockDim.x;
        if (c < span.vecs) {
          if constexpr (MODE == kRowNormAdd) {
            h[i] = row_h<E, VEC, MODE>(h[i], t[i]);
            store_vec<E, VEC>(P.h_out, at + span.column(c), h[i]);
          }
          row_stats<E, VEC, MODE>(h[i], weight(c), sq2, top1);
        }
      }
    }
    raw1 hl = RV1::zero(), wl = RV1::zero();
    if constexpr (RAGGED)
      if (loose >= 0) {
        hl = load_vec<E, 1>(P.x, at + loose);
        if constexpr (MODE == kRowNormAdd) {
          hl = row_h<E, 1, MODE>(hl, load_vec<E, 1>(P.residual, at + loose));
          store_vec<E, 1>(P.h_out, at + loose, hl);
        }
        if constexpr (MODE != kRowQuant) wl = load_vec<E, 1>(P.weight, loose);
      }
    if (last_warp) row_stats<E, 1, MODE>(hl, wl, sq2, top1);
    row_reduce(sq2, top1, warps, warp, lane, red[buf], sq, top);
    buf ^= 1;
    const float inv = row_inv<MODE>(sq, top, P.eps);
    if (threadIdx.x == 0)
      P.scale[row] = row_scale<MODE>(sq, top, inv, P.d, P.eps, again);
    for (int c0 = threadIdx.x; c0 < span.vecs; c0 += U * blockDim.x) {
      raw h[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + i * blockDim.x;
        h[i] = c < span.vecs ? load_vec<E, VEC>(MODE == kRowNormAdd ? P.h_out : P.x,
                                                at + span.column(c))
                             : RV::zero();
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = c0 + i * blockDim.x;
        if (c < span.vecs && DORA_BOUNDS_OK(span.column(c) + VEC <= static_cast<size_t>(P.d)))
          row_codes<E, VEC, MODE>(h[i], weight(c), inv, P.q + at + span.column(c));
      }
    }
    if constexpr (RAGGED)
      if (loose >= 0 && DORA_BOUNDS_OK(loose < P.d))
        row_codes<E, 1, MODE>(hl, wl, inv, P.q + at + loose);
  }
  if constexpr (MODE != kRowQuant)
    norm_rows_again<E, MODE>(P, again, red);
}

// The values that codes stand for: x = q scale in fp32, then rounded to the
// dtype.  A stream in the shape of the compose kernels: a thread keeps its
// columns and walks rows, several rows' codes in flight.
constexpr int kDequantRowUnroll = 8;

template <typename E, int VEC>
struct CodeVec;
template <typename E>
struct CodeVec<E, 8> { using raw = uint2; };
template <typename E>
struct CodeVec<E, 4> { using raw = uint32_t; };
template <typename E>
struct CodeVec<E, 1> { using raw = uint8_t; };

__device__ __forceinline__ uint32_t code_word(const uint2& r, int i) { return i ? r.y : r.x; }
__device__ __forceinline__ uint32_t code_word(uint32_t r, int) { return r; }
__device__ __forceinline__ uint32_t code_word(uint8_t r, int) { return r; }

// The VEC codes of r times s.  A code plus 128, in the low byte of 2^23, is the
// number 2^23 + 128 + code: two exact additions away from a conversion
// instruction's result, at four times its rate.
template <int VEC, typename R>
__device__ __forceinline__ void code_values(const R& r, float s, float (&o)[VEC]) {
  if constexpr (VEC == 1) {
    o[0] = static_cast<float>(static_cast<int8_t>(code_word(r, 0))) * s;
  } else {
    const uint64_t s2 = pair_f32(s, s), off2 = pair_f32(-8388736.f, -8388736.f);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const uint32_t w = code_word(r, e / 4) ^ 0x80808080u;
      const float a = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 + e % 4));
      const float b = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 + (e + 1) % 4));
      split_f32(mul_f32x2(add_f32x2(pair_f32(a, b), off2), s2), o[e], o[e + 1]);
    }
  }
}

template <typename E, int VEC>
__global__ void __launch_bounds__(kStreamThreads)
    dequant_rows_kernel(const int8_t* q, const float* scale, long long rows, int cols, E* x,
                        int bx) {
  using raw = typename CodeVec<E, VEC>::raw;
  const int by = kStreamThreads / bx;
  const int c = (static_cast<int>(blockIdx.x) * bx + static_cast<int>(threadIdx.x) % bx) * VEC;
  grid_dependency_wait();
  grid_dependency_trigger();
  if (c >= cols) return;
  const long long step = static_cast<long long>(gridDim.y) * by;
  for (long long r0 = static_cast<long long>(blockIdx.y) * by + threadIdx.x / bx; r0 < rows;
       r0 += step * kDequantRowUnroll) {
    raw v[kDequantRowUnroll];
    float s[kDequantRowUnroll];
#pragma unroll
    for (int u = 0; u < kDequantRowUnroll; ++u) {
      const long long r = r0 + u * step;
      if (r < rows) {
        v[u] = *reinterpret_cast<const raw*>(q + static_cast<size_t>(r) * cols + c);
        s[u] = scale[r];
      }
    }
#pragma unroll
    for (int u = 0; u < kDequantRowUnroll; ++u) {
      const long long r = r0 + u * step;
      if (r >= rows || !DORA_BOUNDS_OK(c + VEC <= cols)) continue;
      float o[VEC];
      code_values<VEC>(v[u], s[u], o);
      *reinterpret_cast<typename RowVec<E, VEC>::raw*>(x + static_cast<size_t>(r) * cols + c) =
          RowVec<E, VEC>::pack(o);
    }
  }
}

// The same for any number of columns, where the matrix is aligned as a whole:
// vectors of the flat matrix, whose elements may belong to several rows.  A
// thread's vectors are a fixed number of elements apart, so that the rows they
// lie in follow by addition; one of two rows is computed with both scales.
// (With a division for each vector, and element by element where it is of two
// rows: 45 against 36 us at [8192, 8191], 8.4 against 4.4 at [30000, 129].)
template <typename E, int VEC>
__global__ void __launch_bounds__(kStreamThreads)
    dequant_flat_kernel(const int8_t* q, const float* scale, long long rows, int cols, E* x) {
  using raw = typename CodeVec<E, VEC>::raw;
  constexpr int U = 4;
  grid_dependency_wait();
  grid_dependency_trigger();
  const size_t total = static_cast<size_t>(rows) * cols;
  const uint32_t step = gridDim.x * kStreamThreads * VEC;  // elements
  const uint32_t step_rows = step / static_cast<uint32_t>(cols);
  const int step_cols = static_cast<int>(step - step_rows * cols);
  size_t i = (static_cast<size_t>(blockIdx.x) * kStreamThreads + threadIdx.x) * VEC;
  size_t r = i / cols;
  int col = static_cast<int>(i - r * cols);
  while (i < total) {
    raw v[U];
    float s[U];
    size_t row[U];
    int first[U];  // elements of that row from the vector's start
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const size_t at = i + static_cast<size_t>(k) * step;
      if (at < total) s[k] = scale[r];
      if (at + VEC <= total) v[k] = *reinterpret_cast<const raw*>(q + at);
      row[k] = r;
      first[k] = cols - col;
      r += step_rows;
      col += step_cols;
      if (col >= cols) {
        col -= cols;
        ++r;
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k, i += step) {
      if (i >= total) continue;
      float o[VEC];
      if (i + VEC <= total && (first[k] >= VEC || cols >= VEC)) {
        code_values<VEC>(v[k], s[k], o);
        if (first[k] < VEC) {
          float t[VEC];
          code_values<VEC>(v[k], scale[row[k] + 1], t);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[e] = e < first[k] ? o[e] : t[e];
        }
        *reinterpret_cast<typename RowVec<E, VEC>::raw*>(x + i) = RowVec<E, VEC>::pack(o);
      } else {  // the matrix's end, or rows shorter than a vector
        for (int e = 0; e < VEC && i + e < total; ++e) {
          const size_t j = e < first[k] ? row[k] : row[k] + 1 + (e - first[k]) / cols;
          x[i + e] = static_cast<E>(static_cast<float>(q[i + e]) * scale[j]);
        }
      }
    }
  }
}

}  // namespace dora
