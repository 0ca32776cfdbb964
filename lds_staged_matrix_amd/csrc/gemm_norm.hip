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
// reduction and a store.  A row stays in the registers of the T threads that
// own it: max |y| is max |h w| over the root, so the sum of squares and the
// maximum come out of one reduction and nothing is read again.
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

// The same over the T threads of a row, in every thread.
template <int T>
__device__ __forceinline__ void row_sum_max(float &sum, uint32_t &top) {
  wave_sum_max(sum, top);
  if constexpr (T > 64) {
    __shared__ float s_sum[T / 64];
    __shared__ uint32_t s_top[T / 64];
    if ((threadIdx.x & 63) == 0) {
      s_sum[threadIdx.x >> 6] = sum;
      s_top[threadIdx.x >> 6] = top;
    }
    __syncthreads();
    sum = 0.f;
    top = 0;
#pragma unroll
    for (int w = 0; w < T / 64; w++) {
      sum += s_sum[w];
      top = s_top[w] > top ? s_top[w] : top;
    }
  }
}

// E consecutive elements (8: one 16-byte access; 1: rows or row starts that
// are not 16-byte aligned) at element e of a row.  A chunk of 8 that crosses
// the row's end is taken element by element: nothing outside the row is read
// or written.
template <int E>
__device__ __forceinline__ void load_chunk(uint32_t (&v)[E], const uint16_t *row, int e, int N) {
  if constexpr (E == 1) {
    v[0] = e < N ? row[e] : 0;
  } else if (e + E <= N) {
    const u32x4 d = *(const u32x4 *)(row + e);
#pragma unroll
    for (int i = 0; i < E; i++) v[i] = (d[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
  } else {
#pragma unroll
    for (int i = 0; i < E; i++) v[i] = e + i < N ? row[e + i] : 0;
  }
}

template <int E>
__device__ __forceinline__ void store_chunk16(uint16_t *row, int e, int N, const uint16_t (&v)[E]) {
  if constexpr (E == 1) {
    if (e < N) row[e] = v[0];
  } else if (e + E <= N) {
    u32x4 d;
#pragma unroll
    for (int i = 0; i < 4; i++) d[i] = (uint32_t)v[2 * i] | ((uint32_t)v[2 * i + 1] << 16);
    *(u32x4 *)(row + e) = d;
  } else {
#pragma unroll
    for (int i = 0; i < E; i++)
      if (e + i < N) row[e + i] = v[i];
  }
}

// y / S as E4M3, round to nearest even.  |y / S| is at most 448 but for fp32
// rounding, which the conversion's own rounding absorbs; a NaN stays one.
template <int E>
__device__ __forceinline__ void store_chunk8(uint8_t *row, int e, int N, const float (&v)[E]) {
  if constexpr (E == 1) {
    if (e < N) row[e] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[0], 0, false);
  } else {
    v2i32 d = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; i++) {
      d[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], d[i], false);
      d[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], d[i], true);
    }
    if (e + E <= N) {
      *(v2i32 *)(row + e) = d;
    } else {
#pragma unroll
      for (int i = 0; i < E; i++)
        if (e + i < N) row[e + i] = (uint8_t)(d[i / 4] >> (8 * (i & 3)));
    }
  }
}

// The root's reciprocal and, for E4M3 output, 448 / max |y| (and the scale,
// stored by the row's first thread).
template <bool Q8>
__device__ __forceinline__ void row_factors(const NormArgs &p, int64_t m, int t, float sum, uint32_t top,
                                            float &root, float &inv) {
  root = rsqrtf(sum / (float)p.N + p.eps);
  inv = 1.f;
  if constexpr (Q8) {
    float amax = root * __builtin_bit_cast(float, top);
    amax = amax < kAmaxMin ? kAmaxMin : amax;              // a NaN stays
    inv = kE4M3Max / amax;
    if (t == 0) p.S[m] = amax / kE4M3Max;
  }
}

template <int IN, bool Q8, int E>
__device__ __forceinline__ void finish_chunk(const NormArgs &p, int64_t m, int e, const float (&h)[E],
                                             const uint32_t (&w)[E], float root, float inv) {
  if constexpr (Q8) {
    float q[E];
#pragma unroll
    for (int i = 0; i < E; i++) q[i] = h[i] * root * norm_f32<IN>(w[i]) * inv;
    store_chunk8<E>((uint8_t *)p.Y + m * p.ldy, e, p.N, q);
  } else {
    uint16_t y[E];
#pragma unroll
    for (int i = 0; i < E; i++) y[i] = norm_16<IN>(h[i] * root * norm_f32<IN>(w[i]));
    store_chunk16<E>((uint16_t *)p.Y + m * p.ldy, e, p.N, y);
  }
}

// One chunk's h and w, and their share of the row's sum and maximum.
template <int IN, int E>
__device__ __forceinline__ void take_chunk(const NormArgs &p, int64_t m, int e, float (&h)[E], uint32_t (&w)[E],
                                           float &sum, uint32_t &top) {
  uint32_t x[E], r[E];
  load_chunk<E>(x, p.X + m * p.ldx, e, p.N);
  if (p.R) load_chunk<E>(r, p.R + m * p.ldr, e, p.N);
  load_chunk<E>(w, p.W, e, p.N);
#pragma unroll
  for (int i = 0; i < E; i++) {
    h[i] = norm_f32<IN>(x[i]);
    if (p.R) h[i] += norm_f32<IN>(r[i]);
    sum += h[i] * h[i];
    const uint32_t b = __builtin_bit_cast(uint32_t, h[i] * norm_f32<IN>(w[i])) & 0x7FFFFFFFu;
    top = b > top ? b : top;
  }
}

template <int IN, int E>
__device__ __forceinline__ void store_h(const NormArgs &p, int64_t m, int e, const float (&h)[E]) {
  if (!p.H) return;
  uint16_t v[E];
#pragma unroll
  for (int i = 0; i < E; i++) v[i] = norm_16<IN>(h[i]);
  store_chunk16<E>(p.H + m * p.ldh, e, p.N, v);
}

// T threads a row (a whole number of waves), V chunks a thread: N <= T V E.
template <int IN, bool Q8, int E, int V, int T>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rmsnorm_kernel(const NormArgs p) {
  const int t = T < 256 ? threadIdx.x % T : threadIdx.x;
  const int64_t m = T < 256 ? (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T : blockIdx.x;
  if (m >= p.M) return;                  // whole waves, and only where a row needs no barrier
  float h[V][E];
  uint32_t w[V][E];
  float sum = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int v = 0; v < V; v++) take_chunk<IN, E>(p, m, (t + v * T) * E, h[v], w[v], sum, top);
#pragma unroll
  for (int v = 0; v < V; v++) store_h<IN, E>(p, m, (t + v * T) * E, h[v]);
  row_sum_max<T>(sum, top);
  float root, inv;
  row_factors<Q8>(p, m, t, sum, top, root, inv);
#pragma unroll
  for (int v = 0; v < V; v++) finish_chunk<IN, Q8, E>(p, m, (t + v * T) * E, h[v], w[v], root, inv);
}

// Rows longer than the registers of 1024 threads hold: the row is read twice.
// H is written with the second reading, so it may stand in X's or R's place.
template <int IN, bool Q8, int E>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(const NormArgs p) {
  constexpr int T = 1024;
  const int t = threadIdx.x;
  const int64_t m = blockIdx.x;
  float sum = 0.f;
  uint32_t top = 0;
  float h[E];
  uint32_t w[E];
  for (int e = t * E; e < p.N; e += T * E) take_chunk<IN, E>(p, m, e, h, w, sum, top);
  row_sum_max<T>(sum, top);
  float root, inv;
  row_factors<Q8>(p, m, t, sum, top, root, inv);
  for (int e = t * E; e < p.N; e += T * E) {
    take_chunk<IN, E>(p, m, e, h, w, sum, top);
    store_h<IN, E>(p, m, e, h);
    finish_chunk<IN, Q8, E>(p, m, e, h, w, root, inv);
  }
}

template <int IN, bool Q8, int E, int V, int T>
static hipError_t launch_norm(const NormArgs &p, hipStream_t s) {
  NormArgs a = p;
  void *params[] = {&a};
  const int64_t blocks = T < 256 ? ceil_div(p.M, 256 / T) : p.M;
  return hipLaunchKernel((const void *)rmsnorm_kernel<IN, Q8, E, V, T>, dim3((unsigned)blocks),
                         dim3(T < 256 ? 256 : T), params, 0, s);
}

template <int IN, bool Q8, int E>
static hipError_t launch_norm_rows(const NormArgs &p, hipStream_t s) {
  // chunks of 8, or single elements with 8 times as many to a thread
  constexpr int V1 = 8 / E, V2 = 16 / E, V4 = 32 / E;
  if (p.N <= 512) return launch_norm<IN, Q8, E, V1, 64>(p, s);
  if (p.N <= 1024) return launch_norm<IN, Q8, E, V2, 64>(p, s);
  if (p.N <= 2048) return launch_norm<IN, Q8, E, V1, 256>(p, s);
  if (p.N <= 4096) return launch_norm<IN, Q8, E, V2, 256>(p, s);
  if (p.N <= 8192) return launch_norm<IN, Q8, E, V4, 256>(p, s);
  if (p.N <= 16384) return launch_norm<IN, Q8, E, V2, 1024>(p, s);
  if constexpr (E == 8)                  // single elements: 32 a thread do not fit 128 registers
    if (p.N <= 32768) return launch_norm<IN, Q8, E, V4, 1024>(p, s);
  NormArgs a = p;
  void *params[] = {&a};
  return hipLaunchKernel((const void *)rmsnorm_long_kernel<IN, Q8, E>, dim3((unsigned)p.M), dim3(1024), params, 0,
                         s);
}

template <int IN, bool Q8>
static hipError_t dispatch_norm(const NormArgs &p, hipStream_t s) {
  // 16-byte accesses (8-byte ones of E4M3 output) need every row to start on one
  const uintptr_t in = (uintptr_t)p.X | (uintptr_t)p.R | (uintptr_t)p.W | (uintptr_t)p.H;
  const int64_t pitch = p.ldx | (p.R ? p.ldr : 0) | (p.H ? p.ldh : 0) | p.ldy;
  const bool wide = (in & 15) == 0 && ((uintptr_t)p.Y & (Q8 ? 7 : 15)) == 0 && pitch % 8 == 0;
  return wide ? launch_norm_rows<IN, Q8, 8>(p, s) : launch_norm_rows<IN, Q8, 1>(p, s);
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
