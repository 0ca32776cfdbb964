// gemm_kernel_rows.h -- products of a few rows with a K-contiguous weight
// matrix, for gfx950: E4M3 weights (scaled product) and 4-bit weights.
//
// With M <= 64 rows the product reads every weight once and does little with
// it, so the time is the weights' bytes over the HBM rate, as long as enough
// loads are in flight on every CU and nothing else takes longer.
//  * No LDS staging: a weight is used by one wave only, so it goes straight
//    from memory into that wave's MFMA operand registers, 16 bytes a lane and
//    load.  The order of k inside a product is free as long as both operands
//    agree, so the loads need no transposition.
//  * A workgroup owns 16 * NT columns and 16 * RB rows of C; its waves split K
//    among them in blocks of 128, interleaved, so that the waves of a workgroup
//    together read whole lines of each weight row.  Splitting K inside the
//    workgroup is what puts 16 waves on every CU when N is a few thousand; the
//    partial sums meet in LDS and are added in wave order, so a result does not
//    depend on timing.
//  * Each wave loads its next block before it multiplies the present one.
// The activations come from the L2 in fragment form: 16 * RB rows of 128 k
// for 16 * NT columns of weights.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"

namespace lsm {

constexpr int kRowsBlockK = 128;         // k of one load block

// The workgroup's partial sums, added in wave order through `red` (waves * RB
// * NT KiB of LDS); `store(m, n, v)` takes each entry of the 16 RB x 16 NT
// tile, rows and columns counted from the tile's.
template <int RB, int NT, class Store>
__device__ __forceinline__ void reduce_rows(const v4f32 (&acc)[RB][NT], float *red, int waves, int wave,
                                            int lane, Store store) {
  constexpr int TILE = RB * NT * 256;
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
// K-contiguous, K a multiple of 16.  Lane (c = lane & 15, g = lane >> 4) holds
// the 32 bytes at k = 32 g of its block for row c of A and column c of B.
template <int RB, int NT, int OUT>
__global__ __launch_bounds__(64 / (RB * NT) >= 16 ? 1024 : 64 * (64 / (RB * NT))) void lds_gemm_rows_e4m3_kernel(
    const char *__restrict__ A, const char *__restrict__ B, void *__restrict__ C, int M, int N, int K,
    int64_t lda, int64_t ldb, int64_t ldc, int tiles_m, RowColScale sc) {
  extern __shared__ float red[];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int id = xcd_logical_id(blockIdx.x, gridDim.x);
  const int m0 = (id % tiles_m) * 16 * RB, n0 = (id / tiles_m) * 16 * NT;

  // Rows and columns past the end read the last one; their sums are not stored.
  const char *arow[RB], *brow[NT];
#pragma unroll
  for (int i = 0; i < RB; i++) arow[i] = A + (int64_t)min(m0 + 16 * i + c, M - 1) * lda;
#pragma unroll
  for (int t = 0; t < NT; t++) brow[t] = B + (int64_t)min(n0 + 16 * t + c, N - 1) * ldb;

  v4f32 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[i][t] = v4f32{0.f, 0.f, 0.f, 0.f};

  struct Block {
    u32x4 a[RB][2], b[NT][2];
  };
  auto load = [&](Block &f, int kb) {
    const int k = kb * kRowsBlockK + 32 * g;
    // a chunk at k >= K reads the row's start and counts as zero below
    const int o0 = k < K ? k : 0, o1 = k + 16 < K ? k + 16 : 0;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      f.b[t][0] = *(const u32x4 *)(brow[t] + o0);
      f.b[t][1] = *(const u32x4 *)(brow[t] + o1);
    }
#pragma unroll
    for (int i = 0; i < RB; i++) {
      f.a[i][0] = *(const u32x4 *)(arow[i] + o0);
      f.a[i][1] = *(const u32x4 *)(arow[i] + o1);
    }
  };
  auto frag = [&](const u32x4 (&p)[2]) {
    return __builtin_bit_cast(v8i32, __builtin_shufflevector(p[0], p[1], 0, 1, 2, 3, 4, 5, 6, 7));
  };

  const int blocks = (K + kRowsBlockK - 1) / kRowsBlockK;
  Block cur;
  if (wave < blocks) load(cur, wave);
  for (int kb = wave; kb < blocks; kb += waves) {
    Block nxt;
    if (kb + waves < blocks) load(nxt, kb + waves);
    if ((kb + 1) * kRowsBlockK > K) {      // zeros on both sides: a NaN may stand at the row's start
      const int k = kb * kRowsBlockK + 32 * g;
      const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; h++)
        if (k + 16 * h >= K) {
#pragma unroll
          for (int t = 0; t < NT; t++) cur.b[t][h] = zero;
#pragma unroll
          for (int i = 0; i < RB; i++) cur.a[i][h] = zero;
        }
    }
    v8i32 fa[RB], fb[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) fb[t] = frag(cur.b[t]);
#pragma unroll
    for (int i = 0; i < RB; i++) fa[i] = frag(cur.a[i]);
    mfma_e4m3_as_bf16<16>(acc, fa, fb);   // HBM-bound: the exact form costs nothing
    cur = nxt;
  }

  reduce_rows<RB, NT>(acc, red, waves, wave, lane, [&](int dm, int dn, float v) {
    const int m = m0 + dm, n = n0 + dn;
    if (m < M && n < N) store_rows<OUT>(C, (int64_t)m * ldc + n, scale_entry(v, m, n, M, N, sc));
  });
}

// ------------------------------------------------------------------ 4 bits
//
// C[m][n] = sum_k a(m,k) * S[k / group][n] * (q(k,n) - z[k / group][n]).
//
// Weight n's row holds two 4-bit values a byte, even k in the low half, so a
// lane's 16 bytes are 32 consecutive k.
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
//    by the NT column blocks; then the group's sum is scaled in fp32.  Both
//    MFMA sums are of exact products, and |16 + q| <= 31 keeps what cancels
//    within a few times the result's own rounding errors.
//  * An infinite activation would turn a (16 + q) - (16 + z) a into a NaN, and
//    a very large one might overflow there, where the definition has a finite
//    or infinite value: an entry that is not finite is therefore summed again
//    term by term.
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

// Eight weights (one dword) as the pairs (16 + q_i, 16 + q_{i+4}).
template <int IN>
__device__ __forceinline__ v8i16 w4_unpack(uint32_t w) {
  u32x4 f;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int sh = 4 * i - W4<IN>::POS;
    f[i] = ((sh < 0 ? w << -sh : w >> sh) & W4<IN>::MASK) | W4<IN>::BASE;
  }
  return __builtin_bit_cast(v8i16, f);
}

// Eight activations in the same order of pairs.
__device__ __forceinline__ v8i16 w4_pairs(u32x4 a) {
  u32x4 f;
  f[0] = __builtin_amdgcn_perm(a[2], a[0], 0x05040100u);
  f[1] = __builtin_amdgcn_perm(a[2], a[0], 0x07060302u);
  f[2] = __builtin_amdgcn_perm(a[3], a[1], 0x05040100u);
  f[3] = __builtin_amdgcn_perm(a[3], a[1], 0x07060302u);
  return __builtin_bit_cast(v8i16, f);
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
  const uint8_t *Z;      // NULL: every zero point is 8
  void *C;
  int M, N, K, G, gshift;             // K groups of 2^gshift
  int64_t lda, ldb, lds, ldz, ldc;    // ldb in bytes
  int tiles_m, out_f32;
};

// One entry, summed term by term in the order of k.
template <int IN>
__device__ __forceinline__ float w4_entry(const W4Args &p, int m, int n) {
  const uint16_t *a = p.A + (int64_t)m * p.lda;
  const uint8_t *b = p.B + (int64_t)n * p.ldb;
  float v = 0.f;
  for (int k = 0; k < p.K; k++) {
    const int64_t gi = k >> p.gshift;
    const int q = (b[k >> 1] >> (4 * (k & 1))) & 15;
    const int z = p.Z ? p.Z[gi * p.ldz + n] : 8;
    v += to_f32<IN>(a[k]) * ((float)(q - z) * to_f32<IN>(p.S[gi * p.lds + n]));
  }
  return v;
}

// GS: k steps of 32 in a scale group (4 stands for every group of 128 or more).
template <int IN, int RB, int NT, int GS>
__global__ __launch_bounds__(64 / (RB * NT) >= 16 ? 1024 : 64 * (64 / (RB * NT))) void lds_gemm_w4_kernel(
    const W4Args p) {
  constexpr int NG = 4 / GS;             // scale groups in a block
  extern __shared__ float red[];
  const int M = p.M, N = p.N, K = p.K;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int id = xcd_logical_id(blockIdx.x, gridDim.x);
  const int m0 = (id % p.tiles_m) * 16 * RB, n0 = (id / p.tiles_m) * 16 * NT;

  // Rows and columns past the end read the last one; their sums are not stored.
  const uint16_t *arow[RB];
  const uint8_t *brow[NT];
  int col[NT];
#pragma unroll
  for (int i = 0; i < RB; i++) arow[i] = p.A + (int64_t)min(m0 + 16 * i + c, M - 1) * p.lda + 8 * g;
#pragma unroll
  for (int t = 0; t < NT; t++) {
    col[t] = min(n0 + 16 * t + c, N - 1);
    brow[t] = p.B + (int64_t)col[t] * p.ldb;
  }

  v4f32 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; i++)
#pragma unroll
    for (int t = 0; t < NT; t++) acc[i][t] = v4f32{0.f, 0.f, 0.f, 0.f};

  struct Block {
    u32x4 b[NT];
    u32x4 a[RB][4];
    uint16_t s[NT][NG];
    uint8_t z[NT][NG];
  };
  auto load = [&](Block &f, int kb) {
    const int k0 = kb * kRowsBlockK;
    const int kl = k0 + 32 * g;
    const int ob = kl < K ? kl / 2 : 0;  // past K: any weights, their k steps are skipped
#pragma unroll
    for (int t = 0; t < NT; t++) f.b[t] = *(const u32x4 *)(brow[t] + ob);
#pragma unroll
    for (int i = 0; i < NG; i++) {
      const int64_t gi = min((k0 + 32 * GS * i) >> p.gshift, p.G - 1);
#pragma unroll
      for (int t = 0; t < NT; t++) {
        f.s[t][i] = p.S[gi * p.lds + col[t]];
        f.z[t][i] = p.Z ? p.Z[gi * p.ldz + col[t]] : (uint8_t)8;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int k = k0 + 32 * j < K ? k0 + 32 * j : 0;
#pragma unroll
      for (int i = 0; i < RB; i++) f.a[i][j] = *(const u32x4 *)(arow[i] + k);
    }
  };

  const v8i16 ones = __builtin_bit_cast(v8i16, u32x4{W4<IN>::ONES, W4<IN>::ONES, W4<IN>::ONES, W4<IN>::ONES});
  const int blocks = (K + kRowsBlockK - 1) / kRowsBlockK;
  Block cur;
  if (wave < blocks) load(cur, wave);
  for (int kb = wave; kb < blocks; kb += waves) {
    Block nxt;
    if (kb + waves < blocks) load(nxt, kb + waves);
    const int left = K - kb * kRowsBlockK;          // k of this block that exist
    u32x4 w[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) w[t] = lane_group_transpose(cur.b[t]);
#pragma unroll
    for (int gi = 0; gi < NG; gi++) {
      v4f32 sum[RB], part[RB][NT];
#pragma unroll
      for (int i = 0; i < RB; i++) {
        sum[i] = v4f32{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NT; t++) part[i][t] = v4f32{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int j = gi * GS; j < (gi + 1) * GS; j++) {
        if (32 * j < left) {
          v8i16 fa[RB];
#pragma unroll
          for (int i = 0; i < RB; i++) {
            fa[i] = w4_pairs(cur.a[i][j]);
            sum[i] = mfma_16x16x32<IN>(fa[i], ones, sum[i]);
          }
#pragma unroll
          for (int t = 0; t < NT; t++) {
            const v8i16 fb = w4_unpack<IN>(w[t][j]);
#pragma unroll
            for (int i = 0; i < RB; i++) part[i][t] = mfma_16x16x32<IN>(fa[i], fb, part[i][t]);
          }
        }
      }
      if (32 * gi * GS < left) {
#pragma unroll
        for (int t = 0; t < NT; t++) {
          const float s = to_f32<IN>(cur.s[t][gi]);
          const float z = 16.f + (float)cur.z[t][gi];
#pragma unroll
          for (int i = 0; i < RB; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) acc[i][t][r] += s * (part[i][t][r] - z * sum[i][r]);
        }
      }
    }
    cur = nxt;
  }

  reduce_rows<RB, NT>(acc, red, waves, wave, lane, [&](int dm, int dn, float v) {
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
