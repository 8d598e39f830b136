// Linear layer on 8-bit codes with a scale per token and per output channel:
//
//   y[t, j] = (sum_k xq[t, k] wq[j, k]) x_scale[t] w_scale[j] (+ bias[j])
//
// The sum is an exact int32 (d_in <= 131071 keeps 128^2 d_in below 2^31), so
// neither the kernel that a shape selects nor how it splits k changes a bit
// of y: a token's row is the same alone and in any batch.
#pragma once

#include <type_traits>

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
// conversion, the product with the token's scale, and the product with the
// channel's and the bias (+0 where there is none) in one rounding.
__device__ __forceinline__ float linear_value(int acc, float sx, float sw, float bias) {
  return __fmaf_rn(__fmul_rn(static_cast<float>(acc), sx), sw, bias);
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

// Four codes from any address as a word: put together from the two aligned
// words they lie in where both are inside [begin, end), else byte by byte, of
// which the first `n` are read and the others zero.
__device__ __forceinline__ uint32_t load4_any(const int8_t* p, int n, uintptr_t begin,
                                              uintptr_t end) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p), lo = at & ~static_cast<uintptr_t>(3);
  if (n >= 4 && lo >= begin && lo + 8 <= end) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(lo);
    return __funnelshift_r(w[0], w[1], static_cast<uint32_t>(at & 3) * 8);
  }
  uint32_t v = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (b < n) v |= (static_cast<uint32_t>(p[b]) & 0xffu) << (8 * b);
  return v;
}

// VEC16: rows of both operands start at 16-byte boundaries and d_in is a
// multiple of 16; otherwise rows start at any byte.
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
      const uintptr_t w0 = reinterpret_cast<uintptr_t>(P.wq);
      const uintptr_t w1 = w0 + static_cast<uintptr_t>(P.d_out) * P.d_in;
      const uintptr_t x0 = reinterpret_cast<uintptr_t>(P.xq);
      const uintptr_t x1 = x0 + static_cast<uintptr_t>(P.T) * P.d_in;
#pragma unroll 2
      for (int k = (slice * 32 + lane) * 4; k < P.d_in; k += splits * 128) {
        const int n = P.d_in - k;
        uint32_t w[kDotRows];
#pragma unroll
        for (int r = 0; r < kDotRows; ++r) w[r] = load4_any(wp[r] + k, n, w0, w1);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint32_t x = load4_any(xp[t] + k, n, x0, x1);
#pragma unroll
          for (int r = 0; r < kDotRows; ++r)
            acc[r][t] = __dp4a(static_cast<int>(w[r]), static_cast<int>(x), acc[r][t]);
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
                                P.bias != nullptr ? P.bias[row] : 0.f));
    }
    if (splits > 1) __syncthreads();  // before `part` is written again
  }
}

// ---------------------------------------------------------- tensor cores
// The weight's rows are the MMA's M and the tokens its N, so that a small
// batch wastes no rows and the lanes of an epilogue warp are consecutive
// channels of y.  TMA brings k-blocks of 128 codes of both operands into a
// ring of 128-byte-swizzled stages; one thread issues the MMAs into an int32
// accumulator in TMEM (lane = channel, column = token).
//
// Where the tiles alone would leave SMs idle, S CTAs (or pairs) of a cluster
// share a tile's k.  Each finishes n / S of the tile's columns from its own
// accumulator and from what the others push into its shared memory.
constexpr int kI8M = 128;  // channels per CTA (TMEM lanes)
constexpr int kI8K = 128;  // codes per k-block: one 128-byte swizzle row
constexpr int kI8MaxN = 256;  // tokens per tile of a pair
constexpr int kI8MaxStages = 12;
constexpr uint32_t kI8WBytes = kI8M * kI8K;  // 16 KiB of weight per stage and CTA

// A wait of a whole (converged) warp: the same answer in every lane.
__device__ __forceinline__ bool i8_wait(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                        const volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait_fast(bar, parity, timeout_ns, abort));
}

__device__ __forceinline__ void linear_give_up(volatile int* abort_flag) {
  *abort_flag = 1;
  record_error(DORA_ERR_TIMEOUT);
}

// The MMA issuer's k loop, shared by both kernels: a converged warp walks the
// stages and an elected lane issues a k-block's MMAs and the commit that frees
// the stage.  The loop has to turn around faster than a k-block's MMAs run
// (256 cycles at N = 128), so the next stage's barrier is tried before this
// one's MMAs are issued, and the descriptors are 32-bit sums (the low words;
// a stage or a K step only moves the start address).  Returns false after a
// give-up.
struct I8Stage {
  int stage;
  uint32_t phase;
};

template <typename Mma, typename Commit, typename GiveUp>
__device__ __forceinline__ bool i8_mma_loop(int kblocks, int stages, uint32_t ring,
                                            uint32_t stage_bytes, uint64_t* full, I8Stage& at,
                                            unsigned long long timeout_ns,
                                            const volatile int* abort_flag, Mma&& mma,
                                            Commit&& commit, GiveUp&& give_up) {
  const uint64_t d0 = sw128_kmajor_desc(ring);
  const uint32_t base = static_cast<uint32_t>(d0);
  const uint64_t high = d0 & 0xFFFFFFFF00000000ull;
  bool ready = mbar_try_wait(&full[at.stage], at.phase);
  for (int k = 0; k < kblocks; ++k) {
    if (!__all_sync(0xffffffffu, ready) &&
        !i8_wait(&full[at.stage], at.phase, timeout_ns, abort_flag)) {
      give_up();
      return false;
    }
    const int stage = at.stage;
    if (++at.stage == stages) {
      at.stage = 0;
      at.phase ^= 1u;
    }
    if (k + 1 < kblocks) ready = mbar_try_wait(&full[at.stage], at.phase);
    if (elect_one()) {
      const uint32_t w = base + static_cast<uint32_t>(stage) * (stage_bytes >> 4);
      const uint32_t x = w + (kI8WBytes >> 4);
#pragma unroll
      for (int kk = 0; kk < kI8K / 32; ++kk)
        mma(high | (w + kk * 2), high | (x + kk * 2), (k > 0 || kk > 0) ? 1u : 0u);
      commit(stage);
    }
    __syncwarp();
  }
  return true;
}

// This thread's channel of y: what its columns are scaled and stored with.
// All lanes of a warp call put together (its pairs of lanes exchange values).
template <typename O>
struct ChannelOut {
  O* y;  // the channel's column 0; where `pairs`, of the even channel of its pair
  float sw, bias;
  bool ok;
  bool pairs;  // bf16: channels 2i and 2i + 1 are stored together, 4 bytes aligned
  int T;
  long long d_out;
  // (made before the accumulator is waited for: the scale comes from memory)
  __device__ __forceinline__ ChannelOut(const LinearArgs& a, int row) {
    ok = row < a.d_out && DORA_BOUNDS_OK(row >= 0);
    pairs = sizeof(O) == 2 && a.d_out % 2 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 3) == 0;
    y = static_cast<O*>(a.y) + (pairs ? row & ~1 : row);
    sw = ok ? a.w_scale[row] : 0.f;
    bias = ok && a.bias != nullptr ? a.bias[row] : 0.f;
    T = a.T;
    d_out = a.d_out;
  }
  // N columns from token t.  Their scales (16-byte aligned in shared memory)
  // are read before any is stored: a load between the stores would have to
  // wait for them, since y might alias it.  bf16 values are rounded two to an
  // instruction and stored by pairs of channels: the even lane of a pair
  // stores both channels of one column, the odd lane those of the next.  The
  // instructions per column set the epilogue's time, so the cases of a full
  // and a cut tile, of pairs and single channels, are apart.
  template <int N>
  __device__ __forceinline__ void put(int t, const int (&acc)[N], const float* sx) const {
    float s[N];
#pragma unroll
    for (int c = 0; c < N; c += 4)
      *reinterpret_cast<float4*>(s + c) = *reinterpret_cast<const float4*>(sx + c);
    const int left = ok ? T - t : 0;
    if (sizeof(O) == 2 && pairs) {
      if (__all_sync(0xffffffffu, left >= N))
        put_pairs<N, true>(t, acc, s, left);
      else
        put_pairs<N, false>(t, acc, s, left);
    } else {
      O* p = y + t * d_out;
#pragma unroll
      for (int c = 0; c < N; ++c, p += d_out)
        if (c < left) linear_store(p, linear_value(acc[c], s[c], sw, bias));
    }
  }
  template <int N, bool FULL>
  __device__ __forceinline__ void put_pairs(int t, const int (&acc)[N], const float (&s)[N],
                                            int left) const {
    const int odd = threadIdx.x & 1;
    const uint32_t pick = odd ? 0x3276u : 0x5410u;
    O* p = y + (t + odd) * d_out;
    left -= odd;
#pragma unroll
    for (int c = 0; c < N; c += 2, p += 2 * d_out) {
      const uint32_t v = pack_bf16x2_rn(linear_value(acc[c], s[c], sw, bias),
                                        linear_value(acc[c + 1], s[c + 1], sw, bias));
      const uint32_t u = __shfl_xor_sync(0xffffffffu, v, 1);
      if (FULL || c < left) *reinterpret_cast<uint32_t*>(p) = __byte_perm(v, u, pick);
    }
  }
};

// Epilogue warps of a CTA: two per quarter of the TMEM lanes (a warp reads the
// quarter of its index modulo 4), which take the 16-column groups in turn.
constexpr int kI8EpiWarps = 8;
constexpr int kI8ColStep = 16 * (kI8EpiWarps / 4);  // from a warp's group of 16 to its next

// Calls f(c, v) with this warp's groups of 16 among the n accumulator columns
// (a multiple of 16) from `tmem`, the next group on its way meanwhile.
template <typename F>
__device__ __forceinline__ void for_columns(uint32_t tmem, int n, int warp, F&& f) {
  int c = (warp >> 2) * 16;
  if (c >= n) return;
  int a[16], b[16];
  tmem_load_16cols(tmem + c, a);
  for (; c < n; c += 2 * kI8ColStep) {
    tmem_wait_16cols(a);
    if (c + kI8ColStep < n) tmem_load_16cols(tmem + c + kI8ColStep, b);
    f(c, a);
    __syncwarp();
    if (c + kI8ColStep < n) {
      tmem_wait_16cols(b);
      if (c + 2 * kI8ColStep < n) tmem_load_16cols(tmem + c + 2 * kI8ColStep, a);
      f(c + kI8ColStep, b);
      __syncwarp();
    }
  }
}

// Partials of a split k in the CTA that sums them: [S - 1 other slices][n / S
// columns][128 channels] int32, so that a warp's store of one column is 128
// consecutive bytes.
__host__ __device__ constexpr uint32_t i8_partial_bytes(int n, int S) {
  return static_cast<uint32_t>(S - 1) * static_cast<uint32_t>(n / S) * kI8M * 4u;
}

// Epilogue warps: pushes the columns that other CTAs finish to them.  `slice`:
// this CTA's share of k; the CTA of slice s has cluster rank s * rank_step +
// rank_off.  n is a multiple of 16 and n / S of 4.
template <int S>
__device__ __forceinline__ void i8_push_partials(uint32_t lane_base, int n, int warp, int lane,
                                                 int slice, int rank_step, int rank_off,
                                                 const int* part) {
  const int cols = n / S;
  const uint32_t mine = smem_addr(part) + static_cast<uint32_t>((warp & 3) * 32 + lane) * 4u;
  for_columns(lane_base, n, warp, [&](int c0, const int(&v)[16]) {
    int owner = c0 / cols, in = c0 - owner * cols;  // of the next four columns
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
      if (owner != slice) {
        const int from = slice < owner ? slice : slice - 1;
        const uint32_t to = mapa_shared(
            mine + static_cast<uint32_t>((from * cols + in) * kI8M) * 4u,
            static_cast<uint32_t>(owner * rank_step + rank_off));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st_cluster_u32(to + static_cast<uint32_t>(e * kI8M * 4), static_cast<uint32_t>(v[q + e]));
      }
      in += 4;
      if (in == cols) {
        in = 0;
        ++owner;
      }
    }
  });
}

// Epilogue warps: adds the others' partials to this CTA's own columns of the
// tile at token t0 and stores them.
template <int S, typename O>
__device__ __forceinline__ void i8_finish_columns(const ChannelOut<O>& out, const float* sx,
                                                  uint32_t lane_base, int n, int warp, int lane,
                                                  int slice, int t0, const int* part) {
  const int cols = n / S;
  const int* p = part + (warp & 3) * 32 + lane;
  auto group = [&](auto& sum, int c) {
    constexpr int N = sizeof(sum) / sizeof(int);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
#pragma unroll
      for (int e = 0; e < N; ++e) sum[e] += p[(s * cols + c + e) * kI8M];
    out.put(t0 + slice * cols + c, sum, sx + slice * cols + c);
    __syncwarp();
  };
  const uint32_t own = lane_base + static_cast<uint32_t>(slice * cols);
  const int whole = cols & ~15;
  for (int c = (warp >> 2) * 16; c < whole; c += kI8ColStep) {
    int sum[16];
    tmem_load_16cols(own + c, sum);
    tmem_wait_16cols(sum);
    group(sum, c);
  }
  for (int c = whole + (warp >> 2) * 4; c < cols; c += kI8EpiWarps) {
    int sum[4];
    tmem_load_4cols_wait(own + c, sum);
    group(sum, c);
  }
}

// ------------------------------------------------ single CTAs: small batches
// One tile of 128 channels by up to 128 tokens per CTA.  Not persistent: with
// up to 113 KiB and 128 TMEM columns per CTA two CTAs share an SM, so one's
// epilogue runs beside the other's stream.
constexpr int kTileI8MaxN = 128;  // tokens
constexpr int kTileI8Threads = kI8EpiWarps * 32;

struct alignas(64) TileI8Dev {
  CUtensorMap tm_w;  // wq [d_out, ld], box 128 x 128
  CUtensorMap tm_x;  // xq [T, ld],     box 128 x n
  LinearArgs a;
  int n;             // tokens per tile
  int kb;            // k-blocks
  int stages;
  int ahead;         // k-blocks of the weight to bring into L2 early
  uint32_t part_off; // of the partials, from the ring's start
  int part_over_ring;
  uint32_t tmem_cols, idesc;
};

struct TileI8Tail {
  uint64_t full[kI8MaxStages];
  uint64_t empty[kI8MaxStages];
  uint64_t acc;
  alignas(16) float sx[kTileI8MaxN];
  uint32_t tmem_slot;
  int abort_flag;
};

// Dynamic shared memory a CTA may ask for beside the static TileI8Tail.
constexpr int kTileI8MaxDynSmem = 232448 - static_cast<int>(sizeof(TileI8Tail) + 127) / 128 * 128;

template <typename O, int S>
__global__ void __launch_bounds__(kTileI8Threads)
    tile_i8_kernel(const __grid_constant__ TileI8Dev P, unsigned long long timeout_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ TileI8Tail tail;
  volatile int* abort_flag = &tail.abort_flag;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int slice = static_cast<int>(blockIdx.x) % S;  // = rank in the cluster
  const int row0 = static_cast<int>(blockIdx.x) / S * kI8M;
  const int t0 = static_cast<int>(blockIdx.y) * P.n;
  const int kb0 = static_cast<int>(static_cast<long long>(slice) * P.kb / S);
  const int kb1 = static_cast<int>(static_cast<long long>(slice + 1) * P.kb / S);
  const uint32_t stage_bytes = kI8WBytes + static_cast<uint32_t>(P.n) * kI8K;

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
  if constexpr (S > 1)
    cluster_sync();  // the other CTAs run: their shared memory may be written
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tail.tmem_slot;
  // The weight's first k-blocks come into L2 while the kernel before this one
  // still runs (a prefetch reads nothing, so the weight may even be its
  // output): 12.8 instead of 13.9 us per call for 24 tokens at 8192 x 8192, 14.7
  // instead of 16.8 with the norm before each.
  if (warp == 0 && elect_one())
    for (int k = kb0; k < min(kb1, kb0 + P.ahead); ++k)
      tma_prefetch_2d(&P.tm_w, k * kI8K, row0);
  __syncwarp();
  grid_dependency_wait();
  grid_dependency_trigger();  // not before TMEM is held: the next grid may want it too

  if (warp == 0) {
    const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (int k = kb0; k < kb1; ++k) {
      if (!i8_wait(&tail.empty[stage], phase ^ 1u, timeout_ns, abort_flag)) {
        linear_give_up(abort_flag);
        break;
      }
      if (elect_one()) {
        uint8_t* st = ring + stage * stage_bytes;
        mbar_arrive_expect_tx(&tail.full[stage], stage_bytes);
        tma_load_2d(st, &P.tm_w, &tail.full[stage], k * kI8K, row0, pol_w);
        tma_load_2d(st + kI8WBytes, &P.tm_x, &tail.full[stage], k * kI8K, t0, pol_x);
      }
      __syncwarp();
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
  } else if (warp == 1) {
    I8Stage at{0, 0};
    i8_mma_loop(
        kb1 - kb0, P.stages, smem_addr(ring), stage_bytes, tail.full, at, timeout_ns, abort_flag,
        [&](uint64_t w, uint64_t x, uint32_t accumulate) {
          umma_i8(tmem, w, x, P.idesc, accumulate);
        },
        [&](int stage) { umma_commit(&tail.empty[stage]); },
        [&] { linear_give_up(abort_flag); });
    // Also after a give-up: completes once the issued MMAs have.
    if (elect_one()) umma_commit(&tail.acc);
    __syncwarp();
    mbar_wait(&tail.acc, 0, kDrainTimeoutNs, nullptr);
  } else {
    for (int c = static_cast<int>(threadIdx.x) - 64; c < P.n; c += kTileI8Threads - 64)
      tail.sx[c] = t0 + c < P.a.T ? P.a.x_scale[t0 + c] : 0.f;
  }
  __syncwarp();
  ChannelOut<O> out(P.a, row0 + (warp & 3) * 32 + lane);
  if (!mbar_wait_fast(&tail.acc, 0, timeout_ns, abort_flag)) linear_give_up(abort_flag);
  __syncthreads();  // every wait is over, sx is written
  tc_fence_after_sync();
  if (*abort_flag != 0) out.ok = false;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  if constexpr (S == 1) {
    for_columns(lane_base, P.n, warp,
                [&](int c, const int(&v)[16]) { out.put(t0 + c, v, tail.sx + c); });
  } else {
    // Behind the ring, or over it once every CTA's copies have landed and its
    // MMAs have completed.
    if (P.part_over_ring) {
      __syncwarp();
      cluster_sync();
    }
    const int* part = reinterpret_cast<const int*>(ring + P.part_off);
    i8_push_partials<S>(lane_base, P.n, warp, lane, slice, 1, 0, part);
    // A slice that gave up leaves every sum of the tile incomplete.
    if (*abort_flag != 0 && threadIdx.x < S)
      st_cluster_u32(mapa_shared(smem_addr(&tail.abort_flag), threadIdx.x), 1u);
    __syncwarp();
    cluster_sync();
    if (*abort_flag != 0) out.ok = false;
    i8_finish_columns<S>(out, tail.sx, lane_base, P.n, warp, lane, slice, t0, part);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, P.tmem_cols);
  }
}

// ------------------------------------------------------- CTA pairs: the rest
// Tiles of 256 channels by n tokens on CTA pairs (one MMA of M = 256 for both,
// issued by rank 0 of the pair): each CTA stages its 128 rows of the weight
// and half of the tokens, 32 KiB per k-block at n = 256 where a CTA alone
// stages 48 for half the work.  At the 8-bit rate a k-block lasts 512 cycles,
// in which its bytes cross shared memory twice (copied in, read by the MMA):
// 128 bytes a cycle, what shared memory moves, against 192 on single CTAs.
// S == 1: persistent, over all tiles, with two accumulators of 256 columns so
// that a tile's epilogue runs beside the next one's MMAs.  S > 1: one tile per
// cluster of S pairs, which share its k.
constexpr int kPairI8Threads = (kI8EpiWarps + 2) * 32;  // + copies, + MMA

struct alignas(64) PairI8Dev {
  CUtensorMap tm_w;  // wq [d_out, ld], box 128 x 128
  CUtensorMap tm_x;  // xq [T, ld],     box 128 x n / 2
  LinearArgs a;
  int n;             // tokens per tile, a multiple of 32
  int kb;            // k-blocks
  int stages;
  int tiles_m, tiles_n, group;  // `group` token tiles go together, channels outside
  uint32_t part_off;            // of the partials, from the ring's start
  int part_over_ring;
  uint32_t idesc;
};

// Barriers (per CTA, same offsets in both CTAs of a pair):
//   full[s]       rank 0: its producer's expected bytes plus both CTAs' copies.
//   empty[s]      both: rank 0's commit after the MMAs reading stage s.
//   acc_full[b]   both: rank 0's commit after a tile's MMAs into accumulator b.
//   acc_empty[b]  rank 0: one arrival per epilogue warp of both CTAs.
//   drain         rank 0: the last MMAs have completed.
struct PairI8Tail {
  uint64_t full[kI8MaxStages];
  uint64_t empty[kI8MaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  alignas(16) float sx[2][kI8MaxN];  // a tile's token scales, one copy per accumulator
  uint32_t tmem_slot;
  int abort_flag;
};

constexpr int kPairI8MaxDynSmem = 232448 - static_cast<int>(sizeof(PairI8Tail) + 127) / 128 * 128;

// Token tile and channel tile of the i-th tile: groups of token tiles, inside
// a group all its token tiles of one channel tile before the next, so that the
// weight is streamed once per group and the group's tokens stay in L2.
__device__ __forceinline__ void pair_tile(const PairI8Dev& P, int i, int& tm, int& tn) {
  const int per_group = P.group * P.tiles_m;
  const int g = i / per_group, j = i - g * per_group;
  const int width = min(P.group, P.tiles_n - g * P.group);
  tm = j / width;
  tn = g * P.group + j - tm * width;
}

template <typename O, int S>
__global__ void __launch_bounds__(kPairI8Threads)
    pair_i8_kernel(const __grid_constant__ PairI8Dev P, unsigned long long timeout_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ PairI8Tail tail;
  volatile int* abort_flag = &tail.abort_flag;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), half = rank & 1u, lead = rank & ~1u;
  const int slice = static_cast<int>(rank >> 1);
  const int kb0 = static_cast<int>(static_cast<long long>(slice) * P.kb / S);
  const int kb1 = static_cast<int>(static_cast<long long>(slice + 1) * P.kb / S);
  const uint32_t stage_bytes = kI8WBytes + static_cast<uint32_t>(P.n / 2) * kI8K;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << lead);
  const int chan = static_cast<int>(half) * kI8M + (warp & 3) * 32 + lane;  // in the tile
  const int tiles = P.tiles_m * P.tiles_n;
  const int first = static_cast<int>(blockIdx.x) / (2 * S);
  const int step = static_cast<int>(gridDim.x) / (2 * S);
  // Reaches every CTA of the cluster: a slice that gave up leaves every sum of the
  // tile incomplete.
  auto give_up = [&] {
    for (uint32_t r = 0; r < 2 * S; ++r)
      if (r != rank) st_cluster_u32(mapa_shared(smem_addr(&tail.abort_flag), r), 1u);
    fence_cluster();  // there before this thread's part in the last barrier
    linear_give_up(abort_flag);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(&tail.full[s], 1);
      mbar_init(&tail.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail.acc_full[b], 1);
      mbar_init(&tail.acc_empty[b], 2 * kI8EpiWarps);
    }
    mbar_init(&tail.drain, 1);
    tail.abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&P.tm_w);
    prefetch_tmap(&P.tm_x);
  }
  if (warp == 0) {
    tmem_alloc_pair(&tail.tmem_slot, 512);
    tmem_relinquish_pair();
  }
  // Both CTAs' barriers are initialised before either signals the other.
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = tail.tmem_slot;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  grid_dependency_wait();
  grid_dependency_trigger();  // not before TMEM is held: the next grid may want it too

  if (warp == kI8EpiWarps) {
    // ---------------------------------------------------------- copy producer
    const uint64_t pol = policy_evict_last();
    const uint32_t full0 = mapa_shared(smem_addr(&tail.full[0]), lead);
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    for (int i = first; ok && i < tiles; i += step) {
      int tm, tn;
      pair_tile(P, i, tm, tn);
      const int row = tm * 2 * kI8M + static_cast<int>(half) * kI8M;
      const int tok = tn * P.n + static_cast<int>(half) * (P.n / 2);
      for (int k = kb0; k < kb1; ++k) {
        if (!i8_wait(&tail.empty[stage], phase ^ 1u, timeout_ns, abort_flag)) {
          give_up();
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* st = ring + stage * stage_bytes;
          const uint32_t bar = full0 + stage * static_cast<uint32_t>(sizeof(uint64_t));
          if (half == 0) mbar_arrive_expect_tx(&tail.full[stage], 2 * stage_bytes);
          tma_load_2d_pair(st, &P.tm_w, bar, k * kI8K, row, pol);
          tma_load_2d_pair(st + kI8WBytes, &P.tm_x, bar, k * kI8K, tok, pol);
        }
        __syncwarp();
        ++issued;
        if (++stage == P.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // Every copy lands before the CTA can exit: rank 0 sees its full barriers
    // complete; rank 1's copies complete on those, so it waits for its stages
    // to be consumed.
    for (long long j = issued > P.stages ? issued - P.stages : 0; j < issued; ++j) {
      const uint32_t par = static_cast<uint32_t>((j / P.stages) & 1);
      // (after a give-up a stage may never be filled by the peer or consumed: once
      // this limit has passed, the copies issued before it have landed)
      if (!mbar_wait(half == 0 ? &tail.full[j % P.stages] : &tail.empty[j % P.stages], par,
                     kDrainTimeoutNs, nullptr))
        break;
    }
  } else if (warp == kI8EpiWarps + 1) {
    // ------------------------------------------------------------- MMA issuer
    if (half == 0) {
      I8Stage at{0, 0};
      int it = 0;
      bool ok = true;
      for (int i = first; ok && i < tiles; i += step, ++it) {
        const int b = it & 1;
        if (!i8_wait(&tail.acc_empty[b], static_cast<uint32_t>(((it >> 1) & 1) ^ 1), timeout_ns,
                     abort_flag)) {
          give_up();
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem + static_cast<uint32_t>(b * kI8MaxN);
        ok = i8_mma_loop(
            kb1 - kb0, P.stages, smem_addr(ring), stage_bytes, tail.full, at, timeout_ns,
            abort_flag,
            [&](uint64_t w, uint64_t x, uint32_t accumulate) {
              umma_i8_pair(d, w, x, P.idesc, accumulate);
            },
            [&](int stage) { umma_commit_pair(&tail.empty[stage], pair_mask); }, give_up);
        if (elect_one()) umma_commit_pair(&tail.acc_full[b], pair_mask);
        __syncwarp();
      }
      // Also after a give-up: no MMA is in flight when the CTAs leave.
      if (elect_one()) umma_commit_pair(&tail.drain, static_cast<uint16_t>(1u << lead));
      __syncwarp();
      mbar_wait(&tail.drain, 0, kDrainTimeoutNs, nullptr);
    }
  } else {
    // ---------------------------------------------------- epilogue (warps 0-7)
    const uint32_t empty0 = mapa_shared(smem_addr(&tail.acc_empty[0]), lead);
    int it = 0;
    for (int i = first; i < tiles; i += step, ++it) {
      int tm, tn;
      pair_tile(P, i, tm, tn);
      const int b = it & 1, t0 = tn * P.n;
      // The scales' copy of this accumulator: a warp is back here with the same
      // one two tiles on, past a barrier that every warp reached after reading
      // it.  No warp leaves the loop early, so each barrier completes.
      float* sx = tail.sx[b];
      ChannelOut<O> out(P.a, tm * 2 * kI8M + chan);
      for (int c = static_cast<int>(threadIdx.x); c < P.n; c += kI8EpiWarps * 32)
        sx[c] = t0 + c < P.a.T ? P.a.x_scale[t0 + c] : 0.f;
      named_barrier_sync(1, kI8EpiWarps * 32);
      if (!i8_wait(&tail.acc_full[b], static_cast<uint32_t>((it >> 1) & 1), timeout_ns,
                   abort_flag)) {
        give_up();
        continue;
      }
      tc_fence_after_sync();
      if constexpr (S == 1) {
        if (*abort_flag != 0) out.ok = false;
        const uint32_t acc = lane_base + static_cast<uint32_t>(b * kI8MaxN);
        for_columns(acc, P.n, warp, [&](int c, const int(&v)[16]) {
          // This warp's last columns are in registers: hand it back (to the tile
          // after the next; where there is none, nobody waits for it, and no
          // arrival is on its way to a CTA that has left).
          if (c + kI8ColStep >= P.n && i + 2 * step < tiles) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
              mbar_arrive_cluster_relaxed(empty0 + b * static_cast<uint32_t>(sizeof(uint64_t)));
          }
          out.put(t0 + c, v, sx + c);
        });
      }
    }
  }
  if constexpr (S > 1) {
    // The one tile's partials: behind the ring, or over it once no copy or MMA
    // of any CTA of the cluster is in flight.
    int tm, tn;
    pair_tile(P, first, tm, tn);
    const int* part = reinterpret_cast<const int*>(ring + P.part_off);
    ChannelOut<O> out(P.a, tm * 2 * kI8M + chan);
    __syncwarp();
    tc_fence_before_sync();
    if (P.part_over_ring) cluster_sync();
    tc_fence_after_sync();
    if (warp < kI8EpiWarps)
      i8_push_partials<S>(lane_base, P.n, warp, lane, slice, 2, static_cast<int>(half), part);
    __syncwarp();
    cluster_sync();
    if (warp < kI8EpiWarps) {
      if (*abort_flag != 0) out.ok = false;
      i8_finish_columns<S>(out, tail.sx[0], lane_base, P.n, warp, lane, slice, tn * P.n, part);
    }
  }
  // Neither CTA leaves (or frees TMEM) while the other may still signal it or
  // read its shared memory through the MMAs.
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync_relaxed();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 512);
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
