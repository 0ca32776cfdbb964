// gemm_norm.hip -- gemm_rmsnorm_run: the root-mean-square norm with the
// residual's addition; its output is 16-bit, or E4M3 with one scale a row, the
// A operand of gemm_scaled_run.
//
//   h[m][n] = x[m][n] + r[m][n]                         (fp32; H = h rounded)
//   y[m][n] = h[m][n] * w[n] / sqrt(mean_n h[m][n]^2 + eps)
//   S[m]    = max(max_n |y[m][n]|, 2^-100) / 448,  Q[m][n] = e4m3(y[m][n] / S[m])
//
// Every input is read once and every output written once, so with many rows
// the HBM rate is the bound, and with one row the latency of a load, a
// reduction and a store.  A row stays in the registers of the threads that
// own it: max |y| is max |h w| over the root, so the sum of squares and the
// maximum come out of one reduction and nothing is read again.  Where max |h w|
// leaves fp32's normal range, which max |y| need not do, the maximum is taken
// again over y itself.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_common.h"
#include "gemm_launch.h"

namespace lsm {

constexpr float kE4M3Max = 448.f;
constexpr float kAmaxMin = 0x1p-100f;    // keeps 448 / max |y| finite and S normal

struct NormArgs {
  const uint16_t *X, *R, *W;   // R may be NULL
  uint16_t *H;                 // may be NULL
  void *Y;
  float *S;
  int64_t M;
  int N;
  int64_t ldx, ldr, ldh, ldy;
  float eps;
};

template <int IN>
__device__ __forceinline__ float norm_f32(uint32_t bits) {
  if constexpr (IN == IN_BF16)
    return __builtin_bit_cast(float, bits << 16);
  else
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

template <int IN>
__device__ __forceinline__ uint16_t norm_16(float v) {     // round to nearest even
  if constexpr (IN == IN_BF16)
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// The sum and the maximum (as bits, so that a NaN outranks every number) over
// the 64 lanes, in every lane.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ void wave_sum_max(float &sum, uint32_t &top) {
  auto step = [&](uint32_t s, uint32_t t) {
    sum += __builtin_bit_cast(float, s);
    top = t > top ? t : top;
  };
  auto pair = [&](uint32_t s0, uint32_t s1, uint32_t t0, uint32_t t1) {
    sum = __builtin_bit_cast(float, s0) + __builtin_bit_cast(float, s1);
    top = t0 > t1 ? t0 : t1;
  };
  auto bits = [&] { return __builtin_bit_cast(uint32_t, sum); };
  step(dpp<0xB1>(bits()), dpp<0xB1>(top));      // lanes 1 apart
  step(dpp<0x4E>(bits()), dpp<0x4E>(top));      // 2 apart
  step(dpp<0x141>(bits()), dpp<0x141>(top));    // mirrored in 8: the other four
  step(dpp<0x140>(bits()), dpp<0x140>(top));    // mirrored in 16: the other eight
  // each swap leaves the lanes' own 16 (32) and the other 16 (32) in the two results
  const auto s16 = __builtin_amdgcn_permlane16_swap(bits(), bits(), false, false);
  const auto t16 = __builtin_amdgcn_permlane16_swap(top, top, false, false);
  pair(s16[0], s16[1], t16[0], t16[1]);
  const auto s32 = __builtin_amdgcn_permlane32_swap(bits(), bits(), false, false);
  const auto t32 = __builtin_amdgcn_permlane32_swap(top, top, false, false);
  pair(s32[0], s32[1], t32[0], t32[1]);
}

// The same over the `waves` waves of a workgroup, in every thread.
__device__ __forceinline__ void row_sum_max(float &sum, uint32_t &top, int waves) {
  wave_sum_max(sum, top);
  __shared__ float s_sum[16];
  __shared__ uint32_t s_top[16];
  if constexpr (LSM_LDS_POISON) {   // poison build: before the writes
    if (threadIdx.x < 16) s_sum[threadIdx.x] = __builtin_nanf(""), s_top[threadIdx.x] = ~0u;
    __syncthreads();
  }
  if ((threadIdx.x & 63) == 0) {
    s_sum[threadIdx.x >> 6] = sum;
    s_top[threadIdx.x >> 6] = top;
  }
  __syncthreads();
  sum = 0.f;
  top = 0;
  for (int w = 0; w < waves; w++) {
    sum += s_sum[w];
    top = s_top[w] > top ? s_top[w] : top;
  }
}

// Eight consecutive elements, at any alignment (one 16- or 8-byte access each:
// gfx950 takes global accesses at any byte).
constexpr int kChunk = 8;

template <int IN>
__device__ __forceinline__ void load_chunk(float (&v)[kChunk], const uint16_t *at) {
  u32x4 d;
  __builtin_memcpy(&d, at, sizeof(d));
#pragma unroll
  for (int i = 0; i < kChunk; i++) v[i] = norm_f32<IN>((d[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
}

template <int IN>
__device__ __forceinline__ void store_chunk16(uint16_t *at, const float (&v)[kChunk]) {
  u32x4 d;
#pragma unroll
  for (int i = 0; i < 4; i++)
    d[i] = (uint32_t)norm_16<IN>(v[2 * i]) | ((uint32_t)norm_16<IN>(v[2 * i + 1]) << 16);
  __builtin_memcpy(at, &d, sizeof(d));
}

// y / S as E4M3, round to nearest even.  |y / S| is at most 448 but for fp32
// rounding, which the conversion's own rounding absorbs; a NaN stays one.
__device__ __forceinline__ void store_chunk8(uint8_t *at, const float (&v)[kChunk]) {
  v2i32 d = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; i++) {
    d[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], d[i], false);
    d[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], d[i], true);
  }
  __builtin_memcpy(at, &d, sizeof(d));
}

// The scale of an E4M3 row (stored by the row's first thread) and its
// reciprocal, 448 / max |y|.
__device__ __forceinline__ float row_scale(const NormArgs &p, int64_t m, int t, float amax) {
  amax = amax < kAmaxMin ? kAmaxMin : amax;                // a NaN stays
  if (t == 0) p.S[m] = amax / kE4M3Max;
  return kE4M3Max / amax;
}

// Whether max |h w| lies in fp32's normal range and max |y| is its product with
// the root.  Otherwise (zero, subnormal, infinite or NaN; alike in all of a
// row's threads) `top` is to be max |y|: y is h times the root, which is at most
// sqrt(N), times w, and overflows only where the formula does.
__device__ __forceinline__ bool in_normal_range(uint32_t top) { return top - 0x00800000u < 0x7F000000u; }

// A row's chunk c of eight elements starts at 8 c; the last one, if the row is
// no multiple of eight, is moved back to end with the row, and its first `skip`
// elements are the previous chunk's: both threads compute the same values for
// them and store the same bytes, but only one adds them to the sum.
struct Chunk {
  int at, skip;          // first element; how many of the eight another chunk has (8 or more: all)
  __device__ __forceinline__ Chunk(int c, int N) : at(min(kChunk * c, N - kChunk)), skip(kChunk * c - at) {}
  __device__ __forceinline__ bool mine() const { return skip < kChunk; }
};

// A chunk's h and w, and its share of the row's sum and maximum.
template <int IN>
__device__ __forceinline__ void take_chunk(const NormArgs &p, int64_t m, const Chunk &c, float (&h)[kChunk],
                                           float (&w)[kChunk], float &sum, uint32_t &top) {
  load_chunk<IN>(h, p.X + m * p.ldx + c.at);
  if (p.R) {
    float r[kChunk];
    load_chunk<IN>(r, p.R + m * p.ldr + c.at);
#pragma unroll
    for (int i = 0; i < kChunk; i++) h[i] += r[i];
  }
  load_chunk<IN>(w, p.W + c.at);
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < kChunk; i++) {
    all += h[i] * h[i];
    const uint32_t b = __builtin_bit_cast(uint32_t, h[i] * w[i]) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
  if (c.skip != 0) {
    all = 0.f;
#pragma unroll
    for (int i = 1; i < kChunk; i++)
      if (i >= c.skip) all += h[i] * h[i];
  }
  sum += all;
}

// max |y| of a chunk, as bits.
__device__ __forceinline__ uint32_t top_of_y(const float (&h)[kChunk], const float (&w)[kChunk], float root) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kChunk; i++) {
    const uint32_t b = __builtin_bit_cast(uint32_t, h[i] * root * w[i]) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
  return top;
}

template <int IN, bool Q8>
__device__ __forceinline__ void finish_chunk(const NormArgs &p, int64_t m, const Chunk &c, const float (&h)[kChunk],
                                             const float (&w)[kChunk], float root, float inv) {
  if (!c.mine()) return;
  if (p.H) store_chunk16<IN>(p.H + m * p.ldh + c.at, h);
  float y[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; i++) y[i] = h[i] * root * w[i];
  if constexpr (Q8) {
#pragma unroll
    for (int i = 0; i < kChunk; i++) y[i] *= inv;
    store_chunk8((uint8_t *)p.Y + m * p.ldy + c.at, y);
  } else {
    store_chunk16<IN>((uint16_t *)p.Y + m * p.ldy + c.at, y);
  }
}

// The workgroup's number in a grid of two dimensions: one of them holds fewer
// than 2^32 threads.
__device__ __forceinline__ int64_t workgroup() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// One row to a workgroup, V chunks to a thread (8 <= N <= 8 V threads), or,
// with ROWS > 1, one row to each of ROWS waves (N <= 512).  Every element is
// read before the reduction and written after it, so an output may stand in
// an input's place.
template <int IN, bool Q8, int V, int ROWS>
__global__ __launch_bounds__(ROWS > 1 ? 64 * ROWS : 1024) void rmsnorm_kernel(const NormArgs p) {
  const int threads = ROWS > 1 ? 64 : blockDim.x;
  const int t = ROWS > 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t m = ROWS > 1 ? workgroup() * ROWS + (threadIdx.x >> 6) : workgroup();
  if (m >= p.M) return;                  // whole waves of rows that meet no barrier, or whole workgroups
  float h[V][kChunk], w[V][kChunk];
  float sum = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < V; v++) take_chunk<IN>(p, m, Chunk(t + v * threads, p.N), h[v], w[v], sum, top);
  if constexpr (ROWS > 1)
    wave_sum_max(sum, top);
  else
    row_sum_max(sum, top, threads >> 6);
  const float root = rsqrtf(sum / (float)p.N + p.eps);
  float inv = 1.f;
  if constexpr (Q8) {
    float amax = root * __builtin_bit_cast(float, top);
    if (!in_normal_range(top)) {
      top = 0;
#pragma unroll
      for (int v = 0; v < V; v++) top = max(top, top_of_y(h[v], w[v], root));
      if constexpr (ROWS > 1) {
        wave_sum_max(sum, top);
      } else {
        __syncthreads();                 // every wave has read the first reduction
        row_sum_max(sum, top, threads >> 6);
      }
      amax = __builtin_bit_cast(float, top);
    }
    inv = row_scale(p, m, t, amax);
  }
#pragma unroll
  for (int v = 0; v < V; v++) finish_chunk<IN, Q8>(p, m, Chunk(t + v * threads, p.N), h[v], w[v], root, inv);
}

// Rows of fewer than 8 elements, or more than the registers of 1024 threads
// hold: read twice, in chunks and then the elements behind the last whole
// chunk.  A thread reads and writes the same elements, so here too an output
// may stand in an input's place.
template <int IN, bool Q8>
__global__ __launch_bounds__(1024) void rmsnorm_any_kernel(const NormArgs p) {
  const int64_t m = workgroup();
  if (m >= p.M) return;
  const int chunks = p.N / kChunk, tail = kChunk * chunks + threadIdx.x;
  const uint16_t *x = p.X + m * p.ldx, *r = p.R + m * p.ldr;
  float sum = 0.f, ht = 0.f, wt = 0.f;
  uint32_t top = 0;
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    float h[kChunk], w[kChunk];
    take_chunk<IN>(p, m, Chunk(c, p.N), h, w, sum, top);
  }
  if (tail < p.N) {
    ht = norm_f32<IN>(x[tail]) + (p.R ? norm_f32<IN>(r[tail]) : 0.f);
    wt = norm_f32<IN>(p.W[tail]);
    sum += ht * ht;
    const uint32_t b = __builtin_bit_cast(uint32_t, ht * wt) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
  row_sum_max(sum, top, blockDim.x >> 6);
  const float root = rsqrtf(sum / (float)p.N + p.eps);
  float inv = 1.f;
  if constexpr (Q8) {
    float amax = root * __builtin_bit_cast(float, top);
    if (!in_normal_range(top)) {
      float none = 0.f;
      top = tail < p.N ? __builtin_bit_cast(uint32_t, ht * root * wt) & 0x7FFFFFFFu : 0;
      for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        float h[kChunk], w[kChunk];
        uint32_t unused = 0;
        take_chunk<IN>(p, m, Chunk(c, p.N), h, w, none, unused);
        top = max(top, top_of_y(h, w, root));
      }
      __syncthreads();                   // every wave has read the first reduction
      row_sum_max(none, top, blockDim.x >> 6);
      amax = __builtin_bit_cast(float, top);
    }
    inv = row_scale(p, m, threadIdx.x, amax);
  }
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    float h[kChunk], w[kChunk];
    take_chunk<IN>(p, m, Chunk(c, p.N), h, w, sum, top);
    finish_chunk<IN, Q8>(p, m, Chunk(c, p.N), h, w, root, inv);
  }
  if (tail < p.N) {
    const float y = ht * root * wt;
    if (p.H) p.H[m * p.ldh + tail] = norm_16<IN>(ht);
    if constexpr (Q8)
      ((uint8_t *)p.Y)[m * p.ldy + tail] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(y * inv, y * inv, 0, false);
    else
      ((uint16_t *)p.Y)[m * p.ldy + tail] = norm_16<IN>(y);
  }
}

static hipError_t launch_norm(const void *kernel, const NormArgs &p, int64_t blocks, int threads, hipStream_t s) {
  NormArgs a = p;
  void *params[] = {&a};
  const int64_t x = blocks < (1 << 21) ? blocks : 1 << 21;
  return hipLaunchKernel(kernel, dim3((unsigned)x, (unsigned)ceil_div(blocks, x)), dim3((unsigned)threads), params, 0, s);
}

template <int IN, bool Q8>
static hipError_t dispatch_norm(const NormArgs &p, hipStream_t s) {
  if (p.N < kChunk || p.N > 32768)
    return launch_norm((const void *)rmsnorm_any_kernel<IN, Q8>, p, p.M, p.N < kChunk ? 64 : 1024, s);
  if (p.N <= 512) return launch_norm((const void *)rmsnorm_kernel<IN, Q8, 1, 4>, p, ceil_div(p.M, 4), 256, s);
  // As few chunks a thread as 1024 threads allow: measured at 2^25 elements
  // (bf16 with residual to E4M3), rows of 4096 take 42.2, 48.7 and 54.2 us with
  // 1, 2 and 4 chunks a thread (fewer registers, more waves, more loads in
  // flight), rows of 8192 45.4, 49.3 and 53.3 us, one row of 4096 2.4 and 2.6 us.
  const int v = p.N <= 8192 ? 1 : p.N <= 16384 ? 2 : 4;
  const int threads = (int)ceil_div(p.N, 512 * v) * 64;
  if (v == 1) return launch_norm((const void *)rmsnorm_kernel<IN, Q8, 1, 1>, p, p.M, threads, s);
  if (v == 2) return launch_norm((const void *)rmsnorm_kernel<IN, Q8, 2, 1>, p, p.M, threads, s);
  return launch_norm((const void *)rmsnorm_kernel<IN, Q8, 4, 1>, p, p.M, threads, s);
}

}  // namespace lsm

extern "C" int gemm_rmsnorm_run(gemm_handle_t h, const void *X, const void *R, const void *W, void *H, void *Y,
                                float *S, int64_t M, int64_t N, int64_t ldx, int64_t ldr, int64_t ldh, int64_t ldy,
                                float eps, int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h || M < 0 || N < 0 || !(eps >= 0.f)) return GEMM_ERR_INVALID_ARG;
  if (dtype < GEMM_NORM_BF16_BF16 || dtype > GEMM_NORM_F16_E4M3) return GEMM_ERR_INVALID_ARG;
  const bool q8 = dtype == GEMM_NORM_BF16_E4M3 || dtype == GEMM_NORM_F16_E4M3;
  const bool bf16 = dtype == GEMM_NORM_BF16_BF16 || dtype == GEMM_NORM_BF16_E4M3;
  if (M == 0 || N == 0) return GEMM_OK;
  if (!X || !W || !Y || (q8 && !S)) return GEMM_ERR_INVALID_ARG;
  if (ldx < N || ldy < N || (R && ldr < N) || (H && ldh < N)) return GEMM_ERR_INVALID_ARG;

  const int64_t kMaxDim = (int64_t)1 << 30, kMaxLd = (int64_t)1 << 40;
  if (M >= kMaxDim || N >= kMaxDim || ldx >= kMaxLd || ldy >= kMaxLd || (R && ldr >= kMaxLd) ||
      (H && ldh >= kMaxLd))
    return GEMM_ERR_UNSUPPORTED;
  if (((uintptr_t)X | (uintptr_t)R | (uintptr_t)W | (uintptr_t)H | (q8 ? 0 : (uintptr_t)Y)) & 1)
    return GEMM_ERR_UNSUPPORTED;
  if (q8 && ((uintptr_t)S & 3)) return GEMM_ERR_UNSUPPORTED;

  const int64_t x_bytes = footprint_bytes(M, ldx, N, 2), y_bytes = footprint_bytes(M, ldy, N, q8 ? 1 : 2);
  const int64_t r_bytes = R ? footprint_bytes(M, ldr, N, 2) : 0, h_bytes = H ? footprint_bytes(M, ldh, N, 2) : 0;
  if (x_bytes < 0 || y_bytes < 0 || r_bytes < 0 || h_bytes < 0) return GEMM_ERR_UNSUPPORTED;
  // An output may take X's or R's place (same address, pitch and type); any
  // other overlap of an output is refused.
  struct Range {
    const void *p;
    int64_t bytes, ld;
    bool out, in16;
  } r[6] = {{X, x_bytes, ldx, false, true}, {R, r_bytes, ldr, false, true}, {W, 2 * N, 0, false, false},
            {H, h_bytes, ldh, true, true},  {Y, y_bytes, ldy, true, !q8},   {q8 ? S : nullptr, 4 * M, 0, true, false}};
  for (int i = 0; i < 6; i++)
    for (int j = i + 1; j < 6; j++) {
      if (!r[i].p || !r[j].p || !(r[i].out || r[j].out) || !ranges_overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes))
        continue;
      const bool in_place = r[i].out != r[j].out && r[i].in16 && r[j].in16 && r[i].p == r[j].p &&
                            (r[i].ld == r[j].ld || M == 1);
      if (!in_place) return GEMM_ERR_INVALID_ARG;
    }

  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  const NormArgs p{(const uint16_t *)X, (const uint16_t *)R, (const uint16_t *)W, (uint16_t *)H, Y, S,
                   M, (int)N, ldx, ldr, ldh, ldy, eps};
  const hipError_t e = bf16 ? (q8 ? dispatch_norm<IN_BF16, true>(p, stream) : dispatch_norm<IN_BF16, false>(p, stream))
                            : (q8 ? dispatch_norm<IN_F16, true>(p, stream) : dispatch_norm<IN_F16, false>(p, stream));
  return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
