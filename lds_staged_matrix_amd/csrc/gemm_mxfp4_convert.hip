// gemm_mxfp4_convert.hip -- gemm_mxfp4_quantize_run and gemm_mxfp4_dequantize_run:
// matrices to MXFP4 (gemm_mxfp4.h) and back.
//
//   e = floor(log2 max |x|) - 2 over a block of 32 k, from -127 up
//   S = e + 127,   q = x / 2^e rounded to E2M1, to nearest even, at most 6
//   y = q * 2^(S - 127)
//
// 6 = 1.5 * 2^2 is the largest E2M1 number, so a block's largest size lands in
// [4, 8) and what rounds beyond 6 stops there.  Every element is read once and
// written once: the HBM rate is the bound, and with one row the latency of a
// load, a reduction over four lanes and a store.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_launch.h"
#include "gemm_mxfp4.h"

namespace lsm {

struct MxArgs {
  const void *X;      // the 16- or 32-bit matrix of the quantisation, the elements of the other way
  uint8_t *S;
  void *Y;
  int64_t M;
  int K;
  int64_t ldx, ldy, lds;   // ldx, ldy: elements; rows of 4-bit elements: bytes
  int k_parts;
};

template <int T>
struct MxElem {
  static constexpr int SIZE = T == OUT_F32 ? 4 : 2;
};

// Eight consecutive elements, at any alignment of an element.
template <int T>
__device__ __forceinline__ void mx_load8(float (&v)[8], const char *at) {
  if constexpr (T == OUT_F32) {
    __builtin_memcpy(v, at, 32);
  } else {
    u32x4 d;
    __builtin_memcpy(&d, at, 16);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t b = (d[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
      if constexpr (T == OUT_BF16)
        v[i] = __builtin_bit_cast(float, b << 16);
      else
        v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)b);
    }
  }
}

template <int T>
__device__ __forceinline__ float mx_load1(const char *at) {
  if constexpr (T == OUT_F32) {
    float v;
    __builtin_memcpy(&v, at, 4);
    return v;
  } else {
    uint16_t b;
    __builtin_memcpy(&b, at, 2);
    if constexpr (T == OUT_BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
    return (float)__builtin_bit_cast(_Float16, b);
  }
}

// A block's scale from the largest |x| as fp32 bits (which order as the numbers
// do, with infinities and NaNs above all): the exponent field less 2, which is
// S, since e + 127 = (field - 127 - 2) + 127; fields of 2 and less, the subnormal
// numbers among them, stop at e = -127.
__device__ __forceinline__ int mx_scale(uint32_t top) {
  const int field = (int)(top >> 23);
  return field == 255 ? kMxNaN : field > 2 ? field - 2 : 0;
}
// The scale as the conversions take it: an fp32 number of which they use the
// exponent, 2^(S - 127); for S = 0 that is 2^-127, a subnormal.
__device__ __forceinline__ float mx_scale_f32(int s) {
  return __builtin_bit_cast(float, s == 0 ? 0x00400000u : (uint32_t)s << 23);
}

// Eight elements as a dword, element 0 in the lowest four bits
// (v_cvt_scalef32_pk_fp4_f32 divides by the scale, rounds to nearest even and
// stops at 6).  A block with an infinity or a NaN keeps zeros under its NaN.
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8], int s) {
  const float scale = mx_scale_f32(s);
  uint32_t d = 0;
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[0], v[1], scale, 0);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2], v[3], scale, 1);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4], v[5], scale, 2);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6], v[7], scale, 3);
  return s == kMxNaN ? 0u : d;
}

// Rows and k of a workgroup's tile: 16 rows make whole 16-byte pieces of the
// scales' rows, 512 k a row's load of 8 elements a lane.
constexpr int kMxRows = 16, kMxK = 512, kMxBlocks = kMxK / kMxBlock;

struct MxTile {
  int64_t m0;
  int k0;
};
__device__ __forceinline__ MxTile mx_tile(const MxArgs &p) {
  const uint32_t row = blockIdx.x / (uint32_t)p.k_parts, part = blockIdx.x % (uint32_t)p.k_parts;
  return {(int64_t)row * kMxRows, (int)part * kMxK};
}

// K-contiguous X: four lanes hold a block, a wave a row's 512 k at a time, four
// rows in all.  The scales meet in LDS and leave as 16-byte pieces.
template <int T>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const MxArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t scales[kMxBlocks][kMxRows];
  if constexpr (LSM_LDS_POISON) {   // poison build: all of LDS, before any write
    lds_poison((char *)scales, sizeof scales, threadIdx.x, 256);
    __syncthreads();
  }
  const MxTile t = mx_tile(p);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int k = t.k0 + 8 * lane;
  const int rows = (int)min((int64_t)kMxRows, p.M - t.m0);
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * i + wave;
#pragma unroll
    for (int e = 0; e < 8; e++) v[i][e] = 0.f;
    if (r < rows && k < p.K)
      mx_load8<T>(v[i], (const char *)p.X + ((t.m0 + r) * p.ldx + k) * MxElem<T>::SIZE);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * i + wave;
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) top = max(top, __builtin_bit_cast(uint32_t, v[i][e]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));   // lanes 1 apart
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));   // 2 apart
    const int s = mx_scale(top);
    if ((lane & 3) == 0) scales[lane >> 2][r] = (uint8_t)s;
    if (r < rows && k < p.K)
      *(uint32_t *)((uint8_t *)p.Y + (t.m0 + r) * p.ldy + k / 2) = mx_pack8(v[i], s);
  }
  __syncthreads();
  const int kb = t.k0 / kMxBlock + threadIdx.x;
  if (threadIdx.x < kMxBlocks && kb < p.K / kMxBlock) {
    uint8_t *out = p.S + (int64_t)kb * p.lds + t.m0;
    if (rows == kMxRows) {
      *(u32x4 *)out = *(const u32x4 *)scales[threadIdx.x];
    } else {
      for (int r = 0; r < rows; r++) out[r] = scales[threadIdx.x][r];
    }
  }
}

// Consecutive elements of a row of an MN-contiguous X, as fp32 bits.
template <int T, int V>
__device__ __forceinline__ void mx_load_across(float (&v)[V], const char *at) {
  if constexpr (V == 1) {
    v[0] = mx_load1<T>(at);
  } else if constexpr (T == OUT_F32) {
    __builtin_memcpy(v, at, 4 * V);
  } else {
    uint16_t d[V];
    __builtin_memcpy(d, at, 2 * V);
#pragma unroll
    for (int i = 0; i < V; i++) {
      if constexpr (T == OUT_BF16)
        v[i] = __builtin_bit_cast(float, (uint32_t)d[i] << 16);
      else
        v[i] = (float)__builtin_bit_cast(_Float16, d[i]);
    }
  }
}

// MN-contiguous X: a lane holds a block of each of V neighbouring rows and
// reads V elements of every k at once; 16 lanes stand side by side, so that a
// wave reads 128 bytes (16-bit elements) of four blocks' rows and writes 64
// bytes of each of Q's.  V = 4, or 1 where there are fewer than four rows (8192 x
// 8192 bf16: 40.8 us with 4, 70 with 1).  The last lane of rows that are no
// multiple of V is moved back to end with them, and writes what its neighbour
// writes too.
template <int T, int V>
__global__ __launch_bounds__(256) void mxfp4_quantize_mn_kernel(const MxArgs p) {
  const uint32_t row = blockIdx.x / (uint32_t)p.k_parts, part = blockIdx.x % (uint32_t)p.k_parts;
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)row * (16 * V) + V * (lane & 15), m = at + V <= p.M ? at : p.M - V;
  const int kb = (int)part * kMxBlocks + 4 * (threadIdx.x >> 6) + (lane >> 4);
  if (at >= p.M || kb >= p.K / kMxBlock) return;
  const char *x = (const char *)p.X + ((int64_t)kb * kMxBlock * p.ldx + m) * MxElem<T>::SIZE;
  float v[kMxBlock][V];
#pragma unroll
  for (int e = 0; e < kMxBlock; e++) mx_load_across<T, V>(v[e], x + e * p.ldx * MxElem<T>::SIZE);
  uint8_t scale[V];
#pragma unroll
  for (int r = 0; r < V; r++) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kMxBlock; e++) top = max(top, __builtin_bit_cast(uint32_t, v[e][r]) & 0x7FFFFFFFu);
    const int s = mx_scale(top);
    scale[r] = (uint8_t)s;
    u32x4 d;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; e++) w[e] = v[8 * i + e][r];
      d[i] = mx_pack8(w, s);
    }
    *(u32x4 *)((uint8_t *)p.Y + (m + r) * p.ldy + kb * (kMxBlock / 2)) = d;
  }
  __builtin_memcpy(p.S + (int64_t)kb * p.lds + m, scale, V);
}

// Eight values of a dword of elements.
template <int T>
__device__ __forceinline__ void mx_store8(char *at, uint32_t q, int s) {
  const float scale = mx_scale_f32(s);
  float v[8];
  typedef float v2f32 __attribute__((ext_vector_type(2)));
  auto pair = [&](int i, v2f32 x) { v[2 * i] = x[0], v[2 * i + 1] = x[1]; };
  pair(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 0));
  pair(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 1));
  pair(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 2));
  pair(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 3));
  if (s == kMxNaN)
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __builtin_nanf("");
  if constexpr (T == OUT_F32) {
    __builtin_memcpy(at, v, 32);
  } else {
    u32x4 d;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (T == OUT_BF16)
        d[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v[2 * i + 1]) << 16;
      else
        d[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i + 1]) << 16;
    }
    __builtin_memcpy(at, &d, 16);
  }
}

template <int T>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const MxArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t scales[kMxBlocks][kMxRows];
  if constexpr (LSM_LDS_POISON) {   // poison build: all of LDS, before any write
    lds_poison((char *)scales, sizeof scales, threadIdx.x, 256);
    __syncthreads();
  }
  const MxTile t = mx_tile(p);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int k = t.k0 + 8 * lane;
  const int rows = (int)min((int64_t)kMxRows, p.M - t.m0);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * i + wave;
    q[i] = 0;
    if (r < rows && k < p.K) q[i] = *(const uint32_t *)((const uint8_t *)p.X + (t.m0 + r) * p.ldx + k / 2);
  }
  const int kb = t.k0 / kMxBlock + threadIdx.x;
  if (threadIdx.x < kMxBlocks && kb < p.K / kMxBlock) {
    const uint8_t *in = p.S + (int64_t)kb * p.lds + t.m0;
    if (rows == kMxRows) {
      *(u32x4 *)scales[threadIdx.x] = *(const u32x4 *)in;
    } else {
      for (int r = 0; r < rows; r++) scales[threadIdx.x][r] = in[r];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int r = 4 * i + wave;
    if (r < rows && k < p.K)
      mx_store8<T>((char *)p.Y + ((t.m0 + r) * p.ldy + k) * MxElem<T>::SIZE, q[i], scales[lane >> 2][r]);
  }
}

// Workgroups of a launch whose tiles hold `rows` rows and 512 k.
static int64_t mx_workgroups(int64_t M, int64_t K, int rows) { return ceil_div(M, rows) * ceil_div(K, kMxK); }

static hipError_t launch_mx(const void *kernel, MxArgs a, int rows, hipStream_t s) {
  a.k_parts = (int)ceil_div(a.K, kMxK);
  void *params[] = {&a};
  return hipLaunchKernel(kernel, dim3((unsigned)mx_workgroups(a.M, a.K, rows)), dim3(256), params, 0, s);
}

template <template <int> class K>
static const void *mx_kernel(int dtype) {
  return mxfp4_out(dtype) == OUT_BF16 ? K<OUT_BF16>::get() : mxfp4_out(dtype) == OUT_F16 ? K<OUT_F16>::get() : K<OUT_F32>::get();
}
template <int T>
struct Quantize {
  static const void *get() { return (const void *)mxfp4_quantize_kernel<T>; }
};
template <int T>
struct QuantizeMN {
  static const void *get() { return (const void *)mxfp4_quantize_mn_kernel<T, 4>; }
};
template <int T>
struct QuantizeFewMN {
  static const void *get() { return (const void *)mxfp4_quantize_mn_kernel<T, 1>; }
};
template <int T>
struct Dequantize {
  static const void *get() { return (const void *)mxfp4_dequantize_kernel<T>; }
};

// What the two directions check alike: an MXFP4 matrix at (Q, S) and one of the
// input's or output's type at P, of `outer` rows of `inner` elements.
static int check_convert(const void *P, const void *Q, const void *S, int64_t M, int64_t K, int64_t ldp, int64_t ldq,
                         int64_t lds, int64_t outer, int64_t inner, int dtype, bool quantize, int tile_rows) {
  if (!P || !Q || !S || ldp < inner || ldq < K || lds < M) return GEMM_ERR_INVALID_ARG;
  const int64_t kMaxDim = (int64_t)1 << 30, kMaxLd = (int64_t)1 << 40;
  if (M >= kMaxDim || K >= kMaxDim || ldp >= kMaxLd || ldq >= kMaxLd || lds >= kMaxLd) return GEMM_ERR_UNSUPPORTED;
  if (K % kMxBlock || ldq % kMxBlock || lds % 16) return GEMM_ERR_UNSUPPORTED;
  const int64_t size = mxfp4_out(dtype) == OUT_F32 ? 4 : 2;
  if (((uintptr_t)P & (uintptr_t)(size - 1)) || ((uintptr_t)Q & 15) || ((uintptr_t)S & 15)) return GEMM_ERR_UNSUPPORTED;
  if (mx_workgroups(M, K, tile_rows) * 256 >= (int64_t)1 << 32) return GEMM_ERR_UNSUPPORTED;
  const int64_t p_bytes = footprint_bytes(outer, ldp, inner, size), q_bytes = footprint_bytes(M, ldq / 2, K / 2, 1);
  const int64_t s_bytes = footprint_bytes(K / kMxBlock, lds, M, 1);
  if (p_bytes < 0 || q_bytes < 0 || s_bytes < 0) return GEMM_ERR_UNSUPPORTED;
  if (ranges_overlap(P, p_bytes, Q, q_bytes) || ranges_overlap(P, p_bytes, S, s_bytes)) return GEMM_ERR_INVALID_ARG;
  if (quantize && ranges_overlap(Q, q_bytes, S, s_bytes)) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

}  // namespace lsm

extern "C" int gemm_mxfp4_quantize_run(gemm_handle_t h, const void *X, void *Q, void *S, int64_t M, int64_t K,
                                       int64_t ldx, int64_t ldq, int64_t lds, int layoutX, int dtype,
                                       hipStream_t stream) {
  using namespace lsm;
  if (!h || M < 0 || K < 0 || dtype < GEMM_MXFP4_BF16 || dtype > GEMM_MXFP4_F32) return GEMM_ERR_INVALID_ARG;
  if (layoutX != GEMM_K_CONTIG && layoutX != GEMM_MN_CONTIG) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || K == 0) return GEMM_OK;
  const bool kc = layoutX == GEMM_K_CONTIG;
  const int rows = kc ? kMxRows : M < 4 ? 16 : 64;
  const int st = check_convert(X, Q, S, M, K, ldx, ldq, lds, kc ? M : K, kc ? K : M, dtype, true, rows);
  if (st != GEMM_OK) return st;

  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  const MxArgs a{X, (uint8_t *)S, Q, M, (int)K, ldx, ldq / 2, lds, 0};
  const void *kernel = kc      ? mx_kernel<Quantize>(dtype)
                       : M < 4 ? mx_kernel<QuantizeFewMN>(dtype)
                               : mx_kernel<QuantizeMN>(dtype);
  return launch_mx(kernel, a, rows, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

extern "C" int gemm_mxfp4_dequantize_run(gemm_handle_t h, const void *Q, const void *S, void *Y, int64_t M, int64_t K,
                                         int64_t ldq, int64_t lds, int64_t ldy, int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h || M < 0 || K < 0 || dtype < GEMM_MXFP4_BF16 || dtype > GEMM_MXFP4_F32) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || K == 0) return GEMM_OK;
  const int st = check_convert(Y, Q, S, M, K, ldy, ldq, lds, M, K, dtype, false, kMxRows);
  if (st != GEMM_OK) return st;

  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  const MxArgs a{Q, (uint8_t *)S, Y, M, (int)K, ldq / 2, ldy, lds, 0};
  return launch_mx(mx_kernel<Dequantize>(dtype), a, kMxRows, stream) == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
