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

// ---------------------------------------------------------- tensor cores
// One tile of 128 output channels by up to 256 tokens per CTA: the weight's
// rows are the MMA's M, the tokens its N (so that a small batch wastes no
// rows, and the epilogue's lanes are consecutive channels of y).  TMA brings
// k-blocks of 128 codes of both operands into a ring of 128-byte-swizzled
// stages; one thread issues the MMAs into an int32 accumulator in TMEM.
// `splits` CTAs of a cluster share a tile's k where the tiles alone would
// leave SMs idle: each leaves its partial in shared memory and takes a share
// of the columns, summed over the cluster's shared memory (int32, exact in any
// order).  Not persistent: with up to 113 KiB and 256 TMEM columns per CTA two
// CTAs share an SM, so one's epilogue runs beside the other's stream.
constexpr int kTileI8M = 128;
constexpr int kTileI8K = 128;  // codes per k-block: one 128-byte swizzle row
constexpr int kTileI8MaxN = 256;
constexpr int kTileI8Threads = 128;
constexpr int kTileI8MaxStages = 12;
constexpr uint32_t kTileI8WBytes = kTileI8M * kTileI8K;  // 16 KiB of weight per stage

struct alignas(64) TileI8Dev {
  CUtensorMap tm_w;  // wq [d_out, ld], box 128 x 128
  CUtensorMap tm_x;  // xq [T, ld],     box 128 x n
  LinearArgs a;
  int n;             // tokens per tile, a multiple of 16
  int kb;            // k-blocks
  int splits;
  int stages;
  uint32_t tmem_cols, idesc;
};

struct TileI8Tail {
  uint64_t full[kTileI8MaxStages];
  uint64_t empty[kTileI8MaxStages];
  uint64_t acc;
  float sx[kTileI8MaxN];
  uint32_t tmem_slot;
  int abort_flag;
};

// Dynamic shared memory a CTA may ask for beside the static TileI8Tail.
constexpr int kTileI8MaxDynSmem = 232448 - static_cast<int>(sizeof(TileI8Tail) + 127) / 128 * 128;

__device__ __forceinline__ void tile_give_up(volatile int* abort_flag) {
  *abort_flag = 1;
  record_error(DORA_ERR_TIMEOUT);
}

template <typename O>
__global__ void __launch_bounds__(kTileI8Threads)
    tile_i8_kernel(const __grid_constant__ TileI8Dev P, unsigned long long timeout_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ TileI8Tail tail;
  volatile int* abort_flag = &tail.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = static_cast<int>(blockIdx.x) % P.splits;  // = rank in the cluster
  const int row0 = static_cast<int>(blockIdx.x) / P.splits * kTileI8M;
  const int t0 = static_cast<int>(blockIdx.y) * P.n;
  const int kb0 = static_cast<int>(static_cast<long long>(slice) * P.kb / P.splits);
  const int kb1 = static_cast<int>(static_cast<long long>(slice + 1) * P.kb / P.splits);
  const uint32_t stage_bytes = kTileI8WBytes + static_cast<uint32_t>(P.n) * kTileI8K;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(&tail.full[s], 1);
      mbar_init(&tail.empty[s], 1);
    }
    mbar_init(&tail.acc, 1);
    tail.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&P.tm_w);
    prefetch_tmap(&P.tm_x);
  }
  if (warp == 0) {
    tmem_alloc(&tail.tmem_slot, P.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tail.tmem_slot;
  grid_dependency_wait();
  grid_dependency_trigger();  // not before TMEM is held: the next grid may want it too

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int k = kb0; k < kb1; ++k) {
        if (!mbar_wait(&tail.empty[stage], phase ^ 1u, timeout_ns, abort_flag)) {
          tile_give_up(abort_flag);
          break;
        }
        uint8_t* st = ring + stage * stage_bytes;
        mbar_arrive_expect_tx(&tail.full[stage], stage_bytes);
        tma_load_2d(st, &P.tm_w, &tail.full[stage], k * kTileI8K, row0, pol_w);
        tma_load_2d(st + kTileI8WBytes, &P.tm_x, &tail.full[stage], k * kTileI8K, t0, pol_x);
        ++issued;
        if (++stage == P.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // Every copy lands before the CTA can exit, also after a give-up.
      for (int j = max(0, issued - P.stages); j < issued; ++j)
        mbar_wait(&tail.full[j % P.stages], static_cast<uint32_t>((j / P.stages) & 1),
                  kDrainTimeoutNs, nullptr);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int k = kb0; k < kb1; ++k) {
        if (!mbar_wait(&tail.full[stage], phase, timeout_ns, abort_flag)) {
          tile_give_up(abort_flag);
          break;
        }
        tc_fence_after_sync();
        const uint32_t w = smem_addr(ring + stage * stage_bytes), x = w + kTileI8WBytes;
#pragma unroll
        for (int kk = 0; kk < kTileI8K / 32; ++kk)
          umma_i8(tmem, sw128_kmajor_desc(w + kk * 32), sw128_kmajor_desc(x + kk * 32), P.idesc,
                  (k > kb0 || kk > 0) ? 1u : 0u);
        umma_commit(&tail.empty[stage]);
        if (++stage == P.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      umma_commit(&tail.acc);  // also after a give-up: completes once the issued MMAs have
      mbar_wait(&tail.acc, 0, kDrainTimeoutNs, nullptr);
    }
  } else {
    for (int c = static_cast<int>(threadIdx.x) - 64; c < P.n; c += 64)
      tail.sx[c] = t0 + c < P.a.T ? P.a.x_scale[t0 + c] : 0.f;
  }
  __syncwarp();
  const int row = row0 + static_cast<int>(threadIdx.x);  // TMEM lane = channel of the tile
  const bool has_bias = P.a.bias != nullptr;
  const bool row_ok = row < P.a.d_out;
  const float sw = row_ok ? P.a.w_scale[row] : 0.f;
  const float bias = row_ok && has_bias ? P.a.bias[row] : 0.f;
  if (!mbar_wait(&tail.acc, 0, timeout_ns, abort_flag)) tile_give_up(abort_flag);
  __syncthreads();  // every wait is over, sx is written
  tc_fence_after_sync();
  const bool ok = *abort_flag == 0;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  O* y = static_cast<O*>(P.a.y);
  if (P.splits == 1) {
    for (int c0 = 0; c0 < P.n; c0 += 16) {
      int v[16];
      tmem_load_16cols(lane_base + c0, v);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const int t = t0 + c0 + c;
        if (ok && row_ok && t < P.a.T && DORA_BOUNDS_OK(row >= 0 && t >= 0))
          linear_store(y + static_cast<size_t>(t) * P.a.d_out + row,
                       linear_value(v[c], tail.sx[c0 + c], sw, bias, has_bias));
      }
      __syncwarp();
    }
  } else {
    // The ring is free: its copies have landed and its MMAs have completed.
    int* part = reinterpret_cast<int*>(ring);  // [n][128]
    for (int c0 = 0; c0 < P.n; c0 += 16) {
      int v[16];
      tmem_load_16cols(lane_base + c0, v);
#pragma unroll
      for (int c = 0; c < 16; ++c) part[(c0 + c) * kTileI8M + threadIdx.x] = v[c];
    }
    __syncwarp();
    cluster_sync();
    const uint32_t mine = smem_addr(part) + threadIdx.x * 4;
    for (int c = slice; c < P.n && t0 + c < P.a.T; c += P.splits) {
      int sum = 0;
      for (int s = 0; s < P.splits; ++s)
        sum += ld_cluster_s32(
            mapa_shared(mine + static_cast<uint32_t>(c * kTileI8M * 4), static_cast<uint32_t>(s)));
      const int t = t0 + c;
      if (ok && row_ok && DORA_BOUNDS_OK(row >= 0 && t < P.a.T))
        linear_store(y + static_cast<size_t>(t) * P.a.d_out + row,
                     linear_value(sum, tail.sx[c], sw, bias, has_bias));
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its partial
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, P.tmem_cols);
  }
}

// Rows of `cols` codes at any address to rows of `ld` (a multiple of 16 that
// holds them), the rest zero: what TMA can read.  A thread writes 16 codes,
// gathered from aligned words where those lie inside the source.
constexpr int kPadThreads = 256;

struct PadArgs {
  const int8_t* src;
  int8_t* dst;
  long long rows;
  int cols, ld;
};

__global__ void __launch_bounds__(kPadThreads) pad_rows_kernel(const PadArgs A, const PadArgs B) {
  grid_dependency_wait();
  grid_dependency_trigger();
  const PadArgs& P = blockIdx.y == 0 ? A : B;
  const int chunks = P.ld / 16;
  const long long total = P.rows * chunks;
  const uintptr_t begin = reinterpret_cast<uintptr_t>(P.src);
  const uintptr_t end = begin + static_cast<uintptr_t>(P.rows) * P.cols;
  for (long long i = static_cast<long long>(blockIdx.x) * kPadThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kPadThreads) {
    const long long r = i / chunks;
    const int c = static_cast<int>(i % chunks) * 16;
    const uintptr_t at = begin + static_cast<uintptr_t>(r) * P.cols + c;
    const uintptr_t lo = at & ~static_cast<uintptr_t>(3);
    uint32_t out[4];
    if (c + 16 <= P.cols && lo >= begin && lo + 20 <= end) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(lo);
      const uint32_t sh = static_cast<uint32_t>(at & 3) * 8;
      uint32_t w[5];
#pragma unroll
      for (int k = 0; k < 5; ++k) w[k] = p[k];
#pragma unroll
      for (int k = 0; k < 4; ++k) out[k] = __funnelshift_r(w[k], w[k + 1], sh);
    } else {
      const uint8_t* p = reinterpret_cast<const uint8_t*>(at);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        out[k] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (c + 4 * k + b < P.cols) out[k] |= static_cast<uint32_t>(p[4 * k + b]) << (8 * b);
      }
    }
    if (DORA_BOUNDS_OK(r < P.rows && c + 16 <= P.ld))
      *reinterpret_cast<uint4*>(P.dst + static_cast<size_t>(r) * P.ld + c) =
          make_uint4(out[0], out[1], out[2], out[3]);
  }
}

}  // namespace dora
