// Linear layer on 8-bit codes with a scale per token and per output channel:
//
//   y[t, j] = (sum_k xq[t, k] wq[j, k]) x_scale[t] w_scale[j] (+ bias[j])
//
// The sum is an exact int32 (d_in <= 131071 keeps 128^2 d_in below 2^31), so
// neither the kernel that a shape selects nor how it splits k changes a bit
// of y: a token's row is the same alone and in any batch.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace dora {

struct LinearArgs {
  const int8_t* xq;      // [T, d_in]
  const float* x_scale;  // [T]
  const int8_t* wq;      // [d_out, d_in]
  const float* w_scale;  // [d_out]
  const float* bias;     // [d_out] or NULL
  void* y;               // [T, d_out]
  int T, d_out, d_in;
};

// fp32 value of one accumulated sum, the same operations in every kernel: the
// conversion, one product with each scale, the bias in the second one's
// rounding.
__device__ __forceinline__ float linear_value(int acc, float sx, float sw, float bias,
                                              bool has_bias) {
  const float v = __fmul_rn(static_cast<float>(acc), sx);
  return has_bias ? __fmaf_rn(v, sw, bias) : __fmul_rn(v, sw);
}

__device__ __forceinline__ void linear_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void linear_store(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------ few tokens
// The weight's stream: CUDA-core dot products (4 products per instruction)
// of kDotRows output channels by TT tokens per warp, lanes along k.  Each
// weight byte is read once per token tile, by 16-byte loads that bypass L1,
// where x stays; kDotRows rows share every load of x.  `splits` warps share
// a row's k where the rows alone would not occupy the SMs.
constexpr int kDotRows = 4;
constexpr int kDotTokens = 8;  // most tokens per tile
constexpr int kDotWarps = 8;

__device__ __forceinline__ uint4 load_stream16(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
  c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
  c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

// VEC16: rows of both operands start at 16-byte boundaries and d_in is a
// multiple of 16; otherwise bytes.
template <typename O, int TT, bool VEC16>
__global__ void __launch_bounds__(kDotWarps * 32) dot_i8_kernel(const LinearArgs P, int splits) {
  static_assert(kDotRows * TT <= 32, "one lane per result");
  __shared__ int part[kDotWarps][kDotRows * TT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = kDotWarps / splits;  // row groups per block
  const int slice = warp % splits;
  const int row0 = (static_cast<int>(blockIdx.x) * groups + warp / splits) * kDotRows;
  grid_dependency_wait();
  grid_dependency_trigger();
  // Rows past d_out and tokens past T repeat the last one; not stored.
  const int8_t* wp[kDotRows];
  const int8_t* xp[TT];
#pragma unroll
  for (int r = 0; r < kDotRows; ++r)
    wp[r] = P.wq + static_cast<size_t>(min(row0 + r, P.d_out - 1)) * P.d_in;
  const bool has_bias = P.bias != nullptr;
  for (int t0 = static_cast<int>(blockIdx.y) * TT; t0 < P.T;
       t0 += static_cast<int>(gridDim.y) * TT) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
      xp[t] = P.xq + static_cast<size_t>(min(t0 + t, P.T - 1)) * P.d_in;
    int acc[kDotRows][TT];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[r][t] = 0;
    if constexpr (VEC16) {
#pragma unroll 2
      for (int k = (slice * 32 + lane) * 16; k < P.d_in; k += splits * 512) {
        uint4 w[kDotRows];
#pragma unroll
        for (int r = 0; r < kDotRows; ++r) w[r] = load_stream16(wp[r] + k);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint4 x = *reinterpret_cast<const uint4*>(xp[t] + k);
#pragma unroll
          for (int r = 0; r < kDotRows; ++r) acc[r][t] = dot16(w[r], x, acc[r][t]);
        }
      }
    } else {
#pragma unroll 4
      for (int k = slice * 32 + lane; k < P.d_in; k += splits * 32) {
        int w[kDotRows];
#pragma unroll
        for (int r = 0; r < kDotRows; ++r) w[r] = wp[r][k];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const int x = xp[t][k];
#pragma unroll
          for (int r = 0; r < kDotRows; ++r) acc[r][t] += w[r] * x;
        }
      }
    }
    // Lane r * TT + t keeps result (r, t).
    int mine = 0;
#pragma unroll
    for (int r = 0; r < kDotRows; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int s = __reduce_add_sync(0xffffffffu, acc[r][t]);
        if (lane == r * TT + t) mine = s;
      }
    if (splits > 1) {
      if (lane < kDotRows * TT) part[warp][lane] = mine;
      __syncthreads();
      if (slice == 0 && lane < kDotRows * TT)
        for (int s = 1; s < splits; ++s) mine += part[warp + s][lane];
    }
    const int row = row0 + lane / TT, tok = t0 + lane % TT;
    if (slice == 0 && lane < kDotRows * TT && row < P.d_out && tok < P.T &&
        DORA_BOUNDS_OK(row >= 0 && tok >= 0)) {
      linear_store(static_cast<O*>(P.y) + static_cast<size_t>(tok) * P.d_out + row,
                   linear_value(mine, P.x_scale[tok], P.w_scale[row],
                                has_bias ? P.bias[row] : 0.f, has_bias));
    }
    if (splits > 1) __syncthreads();  // before `part` is written again
  }
}

}  // namespace dora
