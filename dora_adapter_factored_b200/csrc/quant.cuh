// Rows of a matrix to 8-bit codes with one scale each: a merged weight's
// output channels, or activations per token; optionally behind the RMS norm
// with the residual's addition, which is how a decoder layer produces them.
//
//   v_j   = x_j                                       (dora_quantize_rows)
//   v_j   = h_j w_j / sqrt(mean(h^2) + eps),  h = x (+ residual), rounded to
//           the dtype                                 (dora_rmsnorm_quant)
//   scale = max_j |v_j| / 127,   q_j = rint(v_j / scale)
//
// The codes do not need the rms: it is a common factor of the row, so with
// u_j = h_j w_j and a = max |u_j|,  q_j = rint(u_j (127 / a))  and
// scale = (a / 127) / rms.  The row's sum of squares and its maximum are
// therefore reduced together, in one pass and with one block barrier, and the
// row stays in registers in between: x (and the residual) are read once, h
// and the codes written once.
//
// Sums, maxima and products are fp32; h is rounded to the dtype because it is
// stored and read again by the next layer, and the norm is of that stored
// value.  A sum of squares beyond fp32's range counts as not finite.
#pragma once

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
  long long rows;
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
// 122 against 77 us at [8192, 8191] bf16 with a residual, 93 against 42 without.)
template <int VEC, bool RAGGED>
struct RowSpan {
  int d, lead, head, vecs, loose;
  __device__ __forceinline__ RowSpan(long long row, int cols) : d(cols) {
    lead = RAGGED ? static_cast<int>(static_cast<size_t>(row) * cols % VEC) : 0;
    head = RAGGED ? min((VEC - lead) % VEC, cols) : 0;
    vecs = (cols - head) / VEC;
    loose = RAGGED ? cols - vecs * VEC : 0;
  }
  __device__ __forceinline__ size_t column(int c) const {
    return static_cast<size_t>(c) * VEC + head;
  }
  __device__ __forceinline__ int loose_column(int e) const {
    return e < head ? e : vecs * VEC + e;
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
        if (v < 0 || v * VEC >= d) return RV::zero();
        if (v * VEC + VEC > d) return load_first<E, VEC>(p + v * VEC, d - v * VEC);
        return *reinterpret_cast<const typename RV::raw*>(p + v * VEC);
      };
      const int k = lead ? c + 1 : c;  // column(c) = k VEC - lead
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

// Factor of the codes from the row's maximum (and, where it is a norm, its sum
// of squares, which has to be finite): 0 for a row that is not finite and for
// one whose step max / 127 would not be a normal number.  127 / max is rounded
// up: a value of half the maximum, code 63.5 exactly, then never falls short of
// the half that goes to the even 64 (rounded to nearest, it did for 66 of the 128
// mantissas of a bf16 maximum).  Every other code of a row of 8-bit mantissas is
// at least 1/510 of its power of two from a half, against 2^-23 that the factor
// is off, or its 127 / max is exact: such rows get the codes of the definition.
template <int MODE>
__device__ __forceinline__ float row_inv(float sq, uint32_t top) {
  bool live = top < kInfBits && __uint_as_float(top) >= kCodeMax * kMinNormal;
  if constexpr (MODE != kRowQuant) live = live && __float_as_uint(sq) < kInfBits;
  // (the nearest, or the next where the sign of the exact residual says that it
  // is below; the rounded-up division is a call, whose registers cost the norm at
  // [8192, 8192] bf16 47 instead of 38 us)
  const float a = __uint_as_float(top), inv = __fdiv_rn(kCodeMax, a);
  const uint32_t up = __fmaf_rn(a, inv, -kCodeMax) < 0.f ? 1u : 0u;
  return live ? __uint_as_float(__float_as_uint(inv) + up) : 0.f;
}

// The row's scale, which no thread but the one that stores it waits for: NaN
// for a row that is not finite, 0 where there is no step.
template <int MODE>
__device__ __forceinline__ float row_scale(float sq, uint32_t top, float inv, int d, float eps) {
  const bool finite =
      top < kInfBits && (MODE == kRowQuant || __float_as_uint(sq) < kInfBits);
  if (!finite) return __uint_as_float(0x7fc00000u);
  if (inv == 0.f) return 0.f;
  const float step = __fdiv_rn(__uint_as_float(top), kCodeMax);
  if constexpr (MODE == kRowQuant) return step;
  const float mean = __fdiv_rn(sq, static_cast<float>(d));
  return __fmul_rn(step, __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(mean, eps))));
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
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const long long first = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.y;
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
  auto load_row = [&](long long row) {
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
  if (AHEAD && first < P.rows) load_row(first);  // before the weight's are waited for
  if constexpr (kHoldWeight) load_weight();
  for (long long row = first; row < P.rows; row += stride) {
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
    if (AHEAD && row + stride < P.rows) load_row(row + stride);
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
    const float inv = row_inv<MODE>(sq, top);
    if (threadIdx.x == 0) P.scale[row] = row_scale<MODE>(sq, top, inv, P.d, P.eps);
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
}

// Rows longer than the registers hold: two passes over the row, the second
// from L2 (of h, as this thread stored it, where there is a residual), with a
// few vectors on their way at a time (one by one [4096, 14336] fp32 took 80 us, 147
// with a residual, against 65 and 131; with the weight's as well they spill, 129
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
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int buf = 0;
  for (long long row = blockIdx.x; row < P.rows; row += gridDim.x) {
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
    const float inv = row_inv<MODE>(sq, top);
    if (threadIdx.x == 0) P.scale[row] = row_scale<MODE>(sq, top, inv, P.d, P.eps);
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
}

// The values that codes stand for: x = q scale, one rounding.  A stream in the
// shape of the compose kernels: a thread keeps its columns and walks rows,
// several rows' codes in flight.
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
