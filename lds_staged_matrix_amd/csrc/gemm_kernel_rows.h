// gemm_kernel_rows.h -- products of a few rows with a K-contiguous weight
// matrix, for gfx950: E4M3 weights (scaled product) and 4-bit weights.
//
// With a few rows the product reads every weight once and does little with
// it, so the time is the weights' bytes over the HBM rate, as long as enough
// loads are in flight on every CU and nothing else takes longer.
//  * A workgroup owns 16 * NT columns and 16 * RB rows of C; its waves split K
//    among them in blocks of 128, interleaved, so that the waves of a workgroup
//    together read whole lines of each weight row.  Splitting K inside the
//    workgroup is what fills every CU when N is a few thousand; the
//    partial sums meet in LDS and are added in wave order, so a result does not
//    depend on timing.
//  * Loads take a block row by row: the lanes of a quarter wave read 256 (64,
//    128) consecutive bytes.  In the order of the MFMA operands, 16 lanes would
//    each read 16 bytes of another row, and the address path, one line at a
//    time, would feed a CU no more than 16 bytes a clock, which the
//    activations alone exceed (measured: 64 rows x 8192 x 8192 took 39.7 us).
//    The registers go through a slice of LDS of the wave's own, in the
//    swizzled layout of lds_layout.h, and come back as operands; a wave's LDS
//    instructions run in order, so no barrier is needed.
//  * A wave's next block is loaded while it multiplies the present one.
// The activations come from the L2: RB * 16 rows for 16 * NT columns.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_common.h"
#include "gemm_kernel_dma.h"

namespace lsm {

constexpr int kRowsBlockK = 128;         // k of one load block

constexpr int kRowsMaxWaves = 8;         // of a workgroup

// Orders a wave's own LDS writes and reads, lane against lane, in the compiler
// (the hardware runs them in order).
__device__ __forceinline__ void wave_lds_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// Poison build: a wave's slice, before the writes of each block.
template <int BYTES>
__device__ __forceinline__ void poison_slice(char *slice, int lane) {
  if constexpr (LSM_LDS_POISON) {
    lds_poison(slice, BYTES, lane, 64);
    wave_lds_order();
  }
}

// 16 bytes at base + voff + soff: voff one register a lane, constant over the K
// loop, soff uniform.  (As a flat address the compiler keeps base + voff in two
// registers and adds to them in every round.)  The record count is no bound
// here: the callers' offsets stay inside the operand.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void *base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, ~0u, kBufferWord3);
}
__device__ __forceinline__ u32x4 rows_load(__amdgpu_buffer_rsrc_t rs, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, voff, soff, 0));
}

// Where in K a workgroup starts, in blocks of `full`: each XCD at an eighth of
// its own.  Workgroups that start together everywhere ask for the same
// kilobyte of rows that lie a power of two apart, which a part of the HBM
// channels holds: 1 x 16384 x 8192 E4M3 took 30.0 us, with the eighths 23.2
// (5.8 TB/s), 32 rows of it 35.2 and 27.2; 4 bits, 1 x 28672 x 8192, 30.0 and 26.9
// (but 48 x 8192 x 8192 19.7 and 20.3).  Inside an XCD all start together, so that the activations they share stay in its L2 (a start of
// each tile's own took 16.4 instead of 11.8 us for 1 x 8192 x 8192 E4M3).
__device__ __forceinline__ int rows_start(int full) {
  return (int)((uint32_t)(blockIdx.x & 7) * (uint32_t)full >> 3);
}

// LDS bytes of one wave's slice: `arows` rows of A and `bcols` columns of B, one block of each.
constexpr int rows_slice_bytes(int arows, int a_es, int bcols, int b_bits) {
  return arows * kRowsBlockK * a_es + bcols * kRowsBlockK * b_bits / 8;
}

// LDS bytes of a workgroup: the waves' slices, whose place the partial sums take.
constexpr int rows_lds_bytes(int waves, int slice, int blocks) {
  return waves * (slice > 1024 * blocks ? slice : 1024 * blocks);
}

// The workgroup's partial sums, added in wave order through `red` (waves * RB
// * NT KiB of LDS); `store(m, n, v)` takes each entry of the 16 RB x 16 NT
// tile, rows and columns counted from the tile's.
template <int RB, int NT, class Store>
__device__ __forceinline__ void reduce_rows(const v4f32 (&acc)[RB][NT], float *red, int waves, int wave,
                                            int lane, Store store) {
  constexpr int TILE = RB * NT * 256;
  if constexpr (LSM_LDS_POISON) {   // poison build: the sums' region, before its writes
    lds_poison((char *)red, waves * TILE * 4, threadIdx.x, blockDim.x);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int r = 0; r < 4; r++) red[wave * TILE + ((i * NT + t) * 4 + r) * 64 + lane] = acc[i][t][r];
  __syncthreads();
  for (int e = wave * 64 + lane; e < TILE; e += waves * 64) {
    float v = red[e];
    for (int w = 1; w < waves; w++) v += red[w * TILE + e];
    // accumulator layout of the 16 x 16 MFMAs (AccLayout<16>)
    const int l = e & 63, r = (e >> 6) & 3, b = e >> 8;
    store(16 * (b / NT) + 4 * (l >> 4) + r, 16 * (b % NT) + (l & 15), v);
  }
}

template <int OUT>
__device__ __forceinline__ void store_rows(void *C, int64_t idx, float v) {
  ((typename OutElem<OUT>::type *)C)[idx] = (typename OutElem<OUT>::type)v;
}

// ------------------------------------------------------------------- E4M3
//
// C[m][n] = sum_k a(m,k) b(k,n) * sc.a[m] * sc.b[n], both operands
// K-contiguous, K a multiple of 16.  AR (8, 16, 32, 48 or 64): rows of A that
// are loaded.  IN: IN_E4M3 (fp8 MFMAs) or IN_E4M3_AS_BF16 (exact products, fp32
// sums).
template <int AR, int NT>
struct RowsE4M3 {
  static constexpr int RB = AR <= 16 ? 1 : AR / 16;
  static constexpr int SLICE = rows_slice_bytes(AR, 1, 16 * NT, 8);
  static constexpr int WAVES_PER_SIMD = RB <= 2 ? 4 : 2;   // 128 registers a lane, or 256
};

template <int AR, int NT, int IN, int OUT>
__global__ __launch_bounds__((64 * kRowsMaxWaves), (RowsE4M3<AR, NT>::WAVES_PER_SIMD)) void lds_gemm_rows_e4m3_kernel(
    const char *__restrict__ A, const char *__restrict__ B, void *__restrict__ C, int M, int N, int K,
    uint32_t lda, uint32_t ldb, int64_t ldc, int tiles_m, RowColScale sc) {
  using T = RowsE4M3<AR, NT>;
  constexpr int RB = T::RB, LA = AR / 8, LB = 2 * NT;   // loads of 8 rows x 128 bytes
  constexpr int ROW = kRowsBlockK;                      // bytes of a row's block
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int id = xcd_logical_id(blockIdx.x, gridDim.x);
  const int m0 = (id % tiles_m) * 16 * RB, n0 = (id / tiles_m) * 16 * NT;

  // Rows and columns past the end read the last one; their sums are not stored.
  const auto rsa = rows_rsrc(A + (int64_t)m0 * lda), rsb = rows_rsrc(B + (int64_t)n0 * ldb);
  const int lrow = lane >> 3, lchunk = lane & 7;        // of a load
  uint32_t aoff[LA], boff[LB];
#pragma unroll
  for (int i = 0; i < LA; i++) aoff[i] = (uint32_t)min(8 * i + lrow, M - 1 - m0) * lda + 16u * lchunk;
#pragma unroll
  for (int i = 0; i < LB; i++) boff[i] = (uint32_t)min(8 * i + lrow, N - 1 - n0) * ldb + 16u * lchunk;
  char *slice = smem + wave * T::SLICE, *sa = slice + LB * 1024;

  u32x4 a[LA], b[LB];
  // PART: the block is cut short by K, and what lies behind K counts as zero.
  auto load = [&](int kb, auto part) {
    constexpr bool PART = decltype(part)::value;
    const uint32_t k0 = kb * kRowsBlockK;
    const bool past = PART && (int)(k0 + 16 * lchunk) >= K;
    // past K: the row's start, whatever it holds, and then zeros
    const uint32_t add = PART ? past ? 0u - 16u * lchunk : k0 : 0u;
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < LB; i++) {
      b[i] = rows_load(rsb, boff[i] + add, PART ? 0 : k0);
      if (past) b[i] = zero;
    }
#pragma unroll
    for (int i = 0; i < LA; i++) {
      a[i] = rows_load(rsa, aoff[i] + add, PART ? 0 : k0);
      if (past) a[i] = zero;
    }
  };
  // operand of row r (of a slice part): the 16 bytes at k = 16 g and at 64 + 16 g
  // (32 in a row would meet in banks two by two: lds_layout.h, frag16_kc8_offset)
  auto frag = [&](const char *part, int r) {
    const u32x4 lo = *(const u32x4 *)(part + kc_chunk_offset(r, g, ROW));
    const u32x4 hi = *(const u32x4 *)(part + kc_chunk_offset(r, g + 4, ROW));
    return __builtin_bit_cast(v8i32, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  v4f32 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[i][t] = v4f32{0.f, 0.f, 0.f, 0.f};

  // The products of the loaded block; next() issues the next one's loads.
  auto block = [&](auto next) {
    wave_lds_order();
    poison_slice<T::SLICE>(slice, lane);
#pragma unroll
    for (int i = 0; i < LB; i++) *(u32x4 *)(slice + kc_chunk_offset(8 * i + lrow, lchunk, ROW)) = b[i];
#pragma unroll
    for (int i = 0; i < LA; i++) *(u32x4 *)(sa + kc_chunk_offset(8 * i + lrow, lchunk, ROW)) = a[i];
    wave_lds_order();
    next();
    v8i32 fa[RB], fb[NT];
#pragma unroll
    for (int i = 0; i < RB; i++) fa[i] = frag(sa, AR >= 16 ? 16 * i + c : c & (AR - 1));
#pragma unroll
    for (int t = 0; t < NT; t++) fb[t] = frag(slice, 16 * t + c);
    if constexpr (IN == IN_E4M3) {
#pragma unroll
      for (int i = 0; i < RB; i++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[i][t] = mfma16_step<IN_E4M3>(fa[i], fb[t], acc[i][t]);
    } else {
      mfma_e4m3_as_bf16<16>(acc, fa, fb);
    }
  };
  // Whole blocks go round the waves; the last wave takes the cut one first.
  const int full = K / kRowsBlockK, start = rows_start(full);
  auto at = [&](int kb) { return kb + start < full ? kb + start : kb + start - full; };
  const std::false_type whole{};
  if (K % kRowsBlockK != 0 && wave == waves - 1) {
    load(full, std::true_type{});
    block([] {});
  }
  int kb = wave;
  if (kb < full) {
    load(at(kb), whole);
    for (; kb + waves < full; kb += waves) block([&] { load(at(kb + waves), whole); });
    block([] {});
  }

  __syncthreads();                                      // the partial sums take the slices' place
  reduce_rows<RB, NT>(acc, (float *)smem, waves, wave, lane, [&](int dm, int dn, float v) {
    const int m = m0 + dm, n = n0 + dn;
    if (m < M && n < N) store_rows<OUT>(C, (int64_t)m * ldc + n, scale_entry(v, m, n, M, N, sc));
  });
}

// ------------------------------------------------------------------ 4 bits
//
// C[m][n] = sum_k a(m,k) * S[k / group][n] * (q(k,n) - z[k / group][n]).
//
// Weight n's row holds two 4-bit values a byte, even k in the low half, so the
// 16 bytes that a lane reads of its column are 32 consecutive k.
//  * k across lanes.  A lane's 32 k would put the four 16-lane groups of one
//    MFMA into four different scale groups when a group is 32 long.  Four
//    permlane swaps transpose the 4 x 4 dwords of the lane groups (row i of
//    lanes, dword j -> row j, dword i), after which dword j of every lane
//    belongs to k = 32 j .. 32 j + 31 of the block: one MFMA never spans two
//    groups, for every group length.
//  * From 4 to 16 bits.  16 + q, q < 16, is exactly 2^4 * 1.qqqq in bf16 and
//    in fp16: the 4 bits go to the top of the fraction under a constant
//    exponent, one shift and one and-or for two weights.  A 16-bit pair holds
//    nibbles i and i + 4 of its dword, and the activations' pairs are permuted
//    to match.
//  * Zero point and scale.  sum a (q - z) = sum a (16 + q) - (16 + z) sum a,
//    where sum a over the group comes from one more MFMA against ones, shared
//    by the NT column blocks; both MFMA sums are of exact products, and
//    |16 + q| <= 31 keeps what cancels within a few times the result's own
//    rounding errors.  In fp16 a packed subtraction makes q - z, exact for every
//    byte z; it replaces the MFMAs against ones from 17 rows on (48 x 8192 x 8192,
//    groups of 64: 19.7 and 17.7 us; but 16 x 8192 x 8192 9.5 and 10.2, where one
//    such MFMA costs less).  Then the group's sum is scaled in fp32.
//  * An infinite activation would turn a (16 + q) - (16 + z) a into a NaN, and
//    a very large one might overflow there or before it meets a small scale,
//    where the definition has a finite or infinite value: an entry that is not
//    finite is therefore summed again term by term, in fp64, whose range holds
//    every product of three factors and every sum of them.
typedef _Float16 v2f16 __attribute__((ext_vector_type(2)));

template <int IN>
struct W4 {
  // where 4 bits stand in 16 + q, its exponent and the constant 1
  static constexpr int POS = IN == IN_BF16 ? 3 : 6;
  static constexpr uint32_t MASK = IN == IN_BF16 ? 0x00780078u : 0x03C003C0u;
  static constexpr uint32_t BASE = IN == IN_BF16 ? 0x41804180u : 0x4C004C00u;
  static constexpr uint32_t ONES = IN == IN_BF16 ? 0x3F803F80u : 0x3C003C00u;
};

template <int IN>
__device__ __forceinline__ float to_f32(uint16_t x) {
  if constexpr (IN == IN_BF16)
    return __builtin_bit_cast(float, (uint32_t)x << 16);
  else
    return (float)__builtin_bit_cast(_Float16, x);
}

// Eight weights (one dword) as the pairs (16 + q_i, 16 + q_{i+4}): a shift and
// one v_and_or_b32 a pair, with its two constants in registers (`mask`,
// `base`: W4<IN>::MASK and BASE behind w4_constant).
template <int IN>
__device__ __forceinline__ v8i16 w4_unpack(uint32_t w, uint32_t mask, uint32_t base) {
  u32x4 f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int sh = 4 * i - W4<IN>::POS;
    f[i] = ((sh < 0 ? w << -sh : w >> sh) & mask) | base;
  }
  return __builtin_bit_cast(v8i16, f);
}

// The pair (16 + z, 16 + z) in fp16, z < 256.
__device__ __forceinline__ v2f16 w4_zero_f16(uint32_t z) {
  const _Float16 v = (_Float16)(float)(16u + z);
  return v2f16{v, v};
}
__device__ __forceinline__ v8i16 w4_minus_f16(v8i16 w, v2f16 z) {
  u32x4 f = __builtin_bit_cast(u32x4, w);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t pair = f[i];
    f[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2f16, pair) - z);
  }
  return __builtin_bit_cast(v8i16, f);
}

__device__ __forceinline__ uint32_t w4_constant(uint32_t v) {
  asm("" : "+v"(v));         // not folded into an and and an or with literals
  return v;
}

// Eight activations in the same order of pairs.
__device__ __forceinline__ u32x4 w4_pairs(u32x4 a) {
  u32x4 f;
  f[0] = __builtin_amdgcn_perm(a[2], a[0], 0x05040100u);
  f[1] = __builtin_amdgcn_perm(a[2], a[0], 0x07060302u);
  f[2] = __builtin_amdgcn_perm(a[3], a[1], 0x05040100u);
  f[3] = __builtin_amdgcn_perm(a[3], a[1], 0x07060302u);
  return f;
}

// Transposes the dwords of the four 16-lane groups: dword j of group i <->
// dword i of group j.
__device__ __forceinline__ u32x4 lane_group_transpose(u32x4 w) {
  const auto p = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto q = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto x = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
  const auto y = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
  return u32x4{x[0], x[1], y[0], y[1]};
}

struct W4Args {
  const uint16_t *A;
  const uint8_t *B;
  const uint16_t *S;
  const uint8_t *Z;      // any readable row of N bytes where zmask is 0
  void *C;
  int M, N, K, G, gshift;             // K groups of 2^gshift
  int64_t lda, ldb, lds, ldz, ldc;    // ldb in bytes
  int tiles_m, out_f32;
  uint32_t zmask, zadd;               // zero point = (byte & zmask) + zadd
};

// One entry, summed term by term in the order of k, in fp64; 32 of them, which
// share a scale, are loaded at once.  A NaN ends it: the sum stays one.
template <int IN>
__device__ __forceinline__ float w4_entry(const W4Args &p, int m, int n) {
  const uint16_t *a = p.A + (int64_t)m * p.lda;
  const uint8_t *b = p.B + (int64_t)n * p.ldb;
  double v = 0.;
  for (int k = 0; k < p.K && !__builtin_isnan(v); k += 32) {
    const int64_t gi = k >> p.gshift;
    const int z = (int)((p.Z[gi * p.ldz + n] & p.zmask) + p.zadd);
    const double s = to_f32<IN>(p.S[gi * p.lds + n]);
    const u32x4 q = *(const u32x4 *)(b + k / 2);
    u32x4 x[4];
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = *(const u32x4 *)(a + k + 8 * j);
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const uint32_t pair = x[j][i / 2];
        v += to_f32<IN>((uint16_t)(pair >> (16 * (i & 1)))) * ((double)((int)((q[j] >> (4 * i)) & 15) - z) * s);
      }
  }
  return (float)v;
}

// The dword of lane 16 t + c, for every t, in every lane (c = lane & 15): rows
// of 16 lanes copied over the others by permlane swaps.
template <int NT>
__device__ __forceinline__ void spread_rows(uint32_t (&out)[NT], uint32_t v) {
  if constexpr (NT == 1) {
    out[0] = v;
  } else {
    const auto x = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // rows 0 0 2 2 and 1 1 3 3
    if constexpr (NT == 2) {
      out[0] = x[0];
      out[1] = x[1];
    } else {
      const auto y = __builtin_amdgcn_permlane32_swap(x[0], x[0], false, false);
      const auto z = __builtin_amdgcn_permlane32_swap(x[1], x[1], false, false);
      out[0] = y[0];
      out[1] = z[0];
      out[2] = y[1];
      out[3] = z[1];
    }
  }
}

// AR (4, 16, 32 or 48): rows of A that are loaded; GS: k steps of 32 in a scale
// group (4 stands for every group of 128 or more).
template <int AR, int NT>
struct RowsW4 {
  static constexpr int RB = AR <= 16 ? 1 : AR / 16;
  static constexpr int SLICE = rows_slice_bytes(AR, 2, 16 * NT, 4);
  static constexpr int WAVES_PER_SIMD = RB == 1 ? 4 : 2;   // 128 registers a lane, or 256
};

template <int IN, int AR, int NT, int GS>
__global__ __launch_bounds__((64 * kRowsMaxWaves), (RowsW4<AR, NT>::WAVES_PER_SIMD)) void lds_gemm_w4_kernel(const W4Args p) {
  using T = RowsW4<AR, NT>;
  constexpr int RB = T::RB, LA = AR / 4;                // loads of A: 4 rows x 256 bytes, of B: 16 rows x 64
  constexpr int AROW = 2 * kRowsBlockK, BROW = kRowsBlockK / 2;
  constexpr int NG = 4 / GS;                            // scale groups in a block
  constexpr bool SUB = IN == IN_F16 && RB > 1;          // q - z by subtraction
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int M = p.M, N = p.N, K = p.K;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int id = xcd_logical_id(blockIdx.x, gridDim.x);
  const int m0 = (id % p.tiles_m) * 16 * RB, n0 = (id / p.tiles_m) * 16 * NT;

  // Rows and columns past the end read the last one; their sums are not stored.
  // 32-bit offsets from the tile's first row and column (the host bounds lda and ldb).
  const auto rsa = rows_rsrc(p.A + (int64_t)m0 * p.lda), rsb = rows_rsrc(p.B + (int64_t)n0 * p.ldb);
  uint32_t aoff[LA], boff[NT];
#pragma unroll
  for (int i = 0; i < LA; i++) aoff[i] = (uint32_t)min(4 * i + g, M - 1 - m0) * (uint32_t)(2 * p.lda) + 16u * c;
#pragma unroll
  for (int t = 0; t < NT; t++)
    boff[t] = (uint32_t)min(16 * t + (lane >> 2), N - 1 - n0) * (uint32_t)p.ldb + 16u * (lane & 3);
  const uint32_t scol = (uint32_t)min(n0 + (lane & (16 * NT - 1)), N - 1);   // whose scale this lane loads
  char *slice = smem + wave * T::SLICE, *sa = slice + NT * 1024;

  u32x4 a[LA], b[NT];
  uint16_t s16[NG];                      // scales and zero points of column scol
  uint8_t z8[NG];
  // Quarter `at` of the loads of block kb: the weights, scales and zero points
  // come with the first, and a quarter of A with each.  PART: the block is cut
  // short by K, and what lies behind K reads the row's start instead; the k
  // steps of that are skipped.
  auto load = [&](int kb, int at, auto part) {
    constexpr bool PART = decltype(part)::value;
    const int k0 = kb * kRowsBlockK;
    if (at == 0) {
#pragma unroll
      for (int t = 0; t < NT; t++)
        b[t] = rows_load(rsb, PART && k0 + 32 * (lane & 3) >= K ? boff[t] - 16 * (lane & 3) : boff[t] + (PART ? k0 / 2 : 0),
                         PART ? 0 : k0 / 2);
#pragma unroll
      for (int i = 0; i < NG; i++) {
        const int64_t gi = min((k0 + 32 * GS * i) >> p.gshift, p.G - 1);
        s16[i] = (p.S + gi * p.lds)[scol];
        z8[i] = (p.Z + gi * p.ldz)[scol];
      }
    }
#pragma unroll
    for (int i = at * LA / 4; i < (at + 1) * LA / 4; i++)
      a[i] = rows_load(rsa, PART && k0 + 8 * c >= K ? aoff[i] - 16 * c : aoff[i] + (PART ? 2 * k0 : 0), PART ? 0 : 2 * k0);
    // Loads stay where they are, a quarter before each k step: all of them at
    // once would hold the wave at the address queue, and left to itself the
    // compiler moves them behind the products.
    if constexpr (NT == 4)
      __builtin_amdgcn_sched_barrier(0x006);   // VALU and SALU instructions may cross: more would not fit the registers
    else
      __builtin_amdgcn_sched_barrier(0x386);   // and LDS instructions
  };

  v4f32 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[i][t] = v4f32{0.f, 0.f, 0.f, 0.f};

  const v8i16 ones = __builtin_bit_cast(v8i16, u32x4{W4<IN>::ONES, W4<IN>::ONES, W4<IN>::ONES, W4<IN>::ONES});
  const uint32_t mask = w4_constant(W4<IN>::MASK), base = w4_constant(W4<IN>::BASE);
  // The products of the loaded block, of which the first `left` k exist; next(j)
  // issues quarter j of the next block's loads.  The wave that multiplies goes
  // before the one that fills its slice (16 rows and more: 48 x 8192 x 8192 bf16
  // took 17.3 us without the priorities and 15.9 with them, 32 rows 13.3 and
  // 12.4; 4 x 28672 x 8192 33.7 and 35.0).
  auto block = [&](int left, auto next) {
    if constexpr (AR >= 16) __builtin_amdgcn_s_setprio(0);
    wave_lds_order();
    poison_slice<T::SLICE>(slice, lane);
#pragma unroll
    for (int t = 0; t < NT; t++)
      *(u32x4 *)(slice + kc_chunk_offset(16 * t + (lane >> 2), lane & 3, BROW)) = b[t];
#pragma unroll
    for (int i = 0; i < LA; i++) *(u32x4 *)(sa + kc_chunk_offset(4 * i + g, c, AROW)) = w4_pairs(a[i]);
    wave_lds_order();
    if constexpr (AR >= 16) __builtin_amdgcn_s_setprio(1);
    uint32_t sz[NG];                     // scale | zero point << 16
#pragma unroll
    for (int i = 0; i < NG; i++) sz[i] = s16[i] | ((z8[i] & p.zmask) + p.zadd) << 16;
    u32x4 w[NT];
#pragma unroll
    for (int t = 0; t < NT; t++)
      w[t] = lane_group_transpose(*(const u32x4 *)(slice + kc_chunk_offset(16 * t + c, g, BROW)));
#pragma unroll
    for (int gi = 0; gi < NG; gi++) {
      v4f32 sum[RB], part[RB][NT];       // sum: unless SUB
#pragma unroll
      for (int i = 0; i < RB; i++) {
        sum[i] = v4f32{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; t++) part[i][t] = v4f32{0.f, 0.f, 0.f, 0.f};
      }
      uint32_t v[NT];
      spread_rows<NT>(v, sz[gi]);
#pragma unroll
      for (int j = gi * GS; j < (gi + 1) * GS; j++) {
        next(j);
        if (32 * j < left) {
          v8i16 fa[RB];
#pragma unroll
          for (int i = 0; i < RB; i++) {
            const int row = AR >= 16 ? 16 * i + c : c & (AR - 1);
            fa[i] = *(const v8i16 *)(sa + kc_chunk_offset(row, 4 * j + g, AROW));
            if constexpr (!SUB) sum[i] = mfma_16x16x32<IN>(fa[i], ones, sum[i]);
          }
#pragma unroll
          for (int t = 0; t < NT; t++) {
            v8i16 fb = w4_unpack<IN>(w[t][j], mask, base);
            if constexpr (SUB) fb = w4_minus_f16(fb, w4_zero_f16(v[t] >> 16));
#pragma unroll
            for (int i = 0; i < RB; i++) part[i][t] = mfma_16x16x32<IN>(fa[i], fb, part[i][t]);
          }
        }
      }
      if (32 * gi * GS < left) {
#pragma unroll
        for (int t = 0; t < NT; t++) {
          const float s = to_f32<IN>((uint16_t)v[t]), z = 16.f + (float)(v[t] >> 16);
#pragma unroll
          for (int i = 0; i < RB; i++)
#pragma unroll
            for (int r = 0; r < 4; r++)
              acc[i][t][r] += SUB ? s * part[i][t][r] : s * (part[i][t][r] - z * sum[i][r]);
        }
      }
    }
  };
  // Whole blocks go round the waves; the last wave takes the cut one first.
  const int full = K / kRowsBlockK, left = K % kRowsBlockK;
  int kb = wave;
  const std::false_type whole{};
  const auto load_all = [&](int at, auto part) {
#pragma unroll
    for (int j = 0; j < 4; j++) load(at, j, part);
  };
  if (left != 0 && wave == waves - 1) {
    load_all(full, std::true_type{});
    block(left, [](int) {});
  }
  if (kb < full) {
    const int start = rows_start(full);
    auto at = [&](int b) { return b + start < full ? b + start : b + start - full; };
    load_all(at(kb), whole);
    for (; kb + waves < full; kb += waves) block(kRowsBlockK, [&](int j) { load(at(kb + waves), j, whole); });
    block(kRowsBlockK, [](int) {});
  }

  __syncthreads();                       // the partial sums take the slices' place
  reduce_rows<RB, NT>(acc, (float *)smem, waves, wave, lane, [&](int dm, int dn, float v) {
    const int m = m0 + dm, n = n0 + dn;
    if (m >= M || n >= N) return;
    if (!__builtin_isfinite(v)) v = w4_entry<IN>(p, m, n);
    if (p.out_f32)
      store_rows<OUT_F32>(p.C, (int64_t)m * p.ldc + n, v);
    else
      store_rows<IN == IN_BF16 ? OUT_BF16 : OUT_F16>(p.C, (int64_t)m * p.ldc + n, v);
  });
}

}  // namespace lsm
