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

// The codes of VEC values: rint(u inv), half to even.  |u inv| <= 127 up to
// two roundings, so the nearest integer is at most 127.
template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* p, const float (&u)[VEC], float inv) {
  uint32_t w[(VEC + 3) / 4];
#pragma unroll
  for (int i = 0; i < (VEC + 3) / 4; ++i) w[i] = 0;
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    w[e / 4] |= (static_cast<uint32_t>(__float2int_rn(u[e] * inv)) & 0xffu) << (8 * (e % 4));
  if constexpr (VEC == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else if constexpr (VEC == 4)
    *reinterpret_cast<uint32_t*>(p) = w[0];
  else
    *p = static_cast<int8_t>(w[0]);
}

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
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] *= g[e];
  }
}

// One vector's share of the row's sum of squares and maximum.  The maximum is
// taken over the bit patterns of |u|, which order like the values and put
// infinities and NaN on top.
template <typename E, int VEC, int MODE>
__device__ __forceinline__ void row_stats(const typename RowVec<E, VEC>::raw& h,
                                          const typename RowVec<E, VEC>::raw& w, float& sq,
                                          uint32_t& top) {
  float u[VEC];
  row_u<E, VEC, MODE>(h, w, u);
#pragma unroll
  for (int e = 0; e < VEC; ++e) top = max(top, __float_as_uint(u[e]) & 0x7fffffffu);
  if constexpr (MODE != kRowQuant) {
    RowVec<E, VEC>::unpack(h, u);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sq = fmaf(u[e], u[e], sq);
  }
}

// Sum and maximum over the `warps` warps of a row's group, in a fixed order;
// the same value in every thread.  `red`: the group's slots (two per warp).
__device__ __forceinline__ void row_reduce(float& sq, uint32_t& top, int warps, int warp, int lane,
                                           uint2* red) {
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

// Factor of the codes and the row's scale from its sum of squares and
// maximum.  A row that is not finite gets codes 0 and scale NaN; one whose
// step would not be a normal number gets codes 0 and scale 0.
template <int MODE>
__device__ __forceinline__ void row_scale(float sq, uint32_t top, int d, float eps, float& inv,
                                          float& scale) {
  const float a = __uint_as_float(top);
  const float step = __fdiv_rn(a, kCodeMax);
  float rstd = 1.f;
  bool finite = top < kInfBits;
  if constexpr (MODE != kRowQuant) {
    finite = finite && __float_as_uint(sq) < kInfBits;
    rstd = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sq, static_cast<float>(d)), eps)));
  }
  inv = 0.f;
  scale = 0.f;
  if (!finite) {
    scale = __uint_as_float(0x7fc00000u);
  } else if (step >= kMinNormal) {
    inv = __fdiv_rn(kCodeMax, a);
    scale = MODE == kRowQuant ? step : __fmul_rn(step, rstd);
  }
}

// Rows of up to kRowNV vectors per thread.  A group of blockDim.x threads (a
// multiple of 32) takes a row; blockDim.y groups share a block only where a
// group is one warp.  Blocks walk the rows with the grid's stride.
constexpr int kRowVecs = 4;     // 16-byte vectors per thread
constexpr int kRowScalars = 16; // elements per thread where rows are not aligned
constexpr int kRowThreads = 512;
__host__ __device__ constexpr int row_nv(int vec) { return vec > 1 ? kRowVecs : kRowScalars; }

template <typename E, int VEC, int MODE>
__global__ void __launch_bounds__(kRowThreads) row_quant_kernel(const RowArgs P) {
  using RV = RowVec<E, VEC>;
  using raw = typename RV::raw;
  constexpr int NV = row_nv(VEC);
  __shared__ uint2 red[2][32];
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int nvec = P.d / VEC;
  const raw* w_in = reinterpret_cast<const raw*>(P.weight);
  raw w[NV];
  if constexpr (MODE != kRowQuant) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      w[i] = c < nvec ? w_in[c] : RV::zero();
    }
  }
  const long long first = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.y;
  int buf = 0;
  for (long long row = first; row < P.rows; row += stride) {
    const size_t at = static_cast<size_t>(row) * P.d;
    const raw* x = reinterpret_cast<const raw*>(static_cast<const E*>(P.x) + at);
    const raw* r = MODE == kRowNormAdd
                       ? reinterpret_cast<const raw*>(static_cast<const E*>(P.residual) + at)
                       : nullptr;
    raw h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      h[i] = c < nvec ? x[c] : RV::zero();
    }
    if constexpr (MODE == kRowNormAdd) {
      raw t[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        t[i] = c < nvec ? r[c] : RV::zero();
      }
      raw* ho = reinterpret_cast<raw*>(static_cast<E*>(P.h_out) + at);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        h[i] = row_h<E, VEC, MODE>(h[i], t[i]);
        if (c < nvec) ho[c] = h[i];
      }
    }
    float sq = 0.f, inv, scale;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) row_stats<E, VEC, MODE>(h[i], w[i], sq, top);
    row_reduce(sq, top, warps, warp, lane, red[buf]);
    buf ^= 1;  // the slots are written again two rows on, past a barrier
    row_scale<MODE>(sq, top, P.d, P.eps, inv, scale);
    if (threadIdx.x == 0) P.scale[row] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nvec && DORA_BOUNDS_OK((c + 1) * VEC <= P.d && row < P.rows)) {
        float u[VEC];
        row_u<E, VEC, MODE>(h[i], w[i], u);
        if (inv == 0.f) {  // also where u is not finite
#pragma unroll
          for (int e = 0; e < VEC; ++e) u[e] = 0.f;
        }
        store_codes<VEC>(P.q + at + static_cast<size_t>(c) * VEC, u, inv);
      }
    }
  }
}

// Rows longer than the registers hold: two passes over the row, the second
// from L2 (of h, as this thread stored it, where there is a residual).
template <typename E, int VEC, int MODE>
__global__ void __launch_bounds__(kRowThreads) row_quant_long_kernel(const RowArgs P) {
  using RV = RowVec<E, VEC>;
  using raw = typename RV::raw;
  __shared__ uint2 red[2][32];
  grid_dependency_wait();
  grid_dependency_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int nvec = P.d / VEC;
  const raw* w_in = reinterpret_cast<const raw*>(P.weight);
  int buf = 0;
  for (long long row = blockIdx.x; row < P.rows; row += gridDim.x) {
    const size_t at = static_cast<size_t>(row) * P.d;
    const raw* x = reinterpret_cast<const raw*>(static_cast<const E*>(P.x) + at);
    raw* ho = reinterpret_cast<raw*>(static_cast<E*>(P.h_out) + at);
    float sq = 0.f, inv, scale;
    uint32_t top = 0;
    for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
      raw h = x[c];
      if constexpr (MODE == kRowNormAdd) {
        h = row_h<E, VEC, MODE>(
            h, reinterpret_cast<const raw*>(static_cast<const E*>(P.residual) + at)[c]);
        ho[c] = h;
      }
      row_stats<E, VEC, MODE>(h, MODE != kRowQuant ? w_in[c] : RV::zero(), sq, top);
    }
    row_reduce(sq, top, warps, warp, lane, red[buf]);
    buf ^= 1;
    row_scale<MODE>(sq, top, P.d, P.eps, inv, scale);
    if (threadIdx.x == 0) P.scale[row] = scale;
    for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
      const raw h = MODE == kRowNormAdd ? ho[c] : x[c];
      float u[VEC];
      row_u<E, VEC, MODE>(h, MODE != kRowQuant ? w_in[c] : RV::zero(), u);
      if (inv == 0.f) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) u[e] = 0.f;
      }
      store_codes<VEC>(P.q + at + static_cast<size_t>(c) * VEC, u, inv);
    }
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
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        o[e] = static_cast<float>(static_cast<int8_t>(code_word(v[u], e / 4) >> (8 * (e % 4)))) *
               s[u];
      *reinterpret_cast<typename RowVec<E, VEC>::raw*>(x + static_cast<size_t>(r) * cols + c) =
          RowVec<E, VEC>::pack(o);
    }
  }
}

}  // namespace dora
