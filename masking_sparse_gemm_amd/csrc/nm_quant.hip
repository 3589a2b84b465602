// nm_quant.hip -- weights in 4 bits with one 16-bit scale for each group of stored columns
// (nm_quantize, nm_dequantize) and their product with one or a few columns (nm_matvec).
//
// A group of `group` consecutive stored values of a row has scale s = round16(max |w| / 7) and
// codes q = clamp(rint(w / s), -8, 7); the group stands for s q.  Codes are stored as q + 8 in
// the order the product reads them: blocks of 16 rows x 128 stored columns, 1 KB each, so that
// one 16-byte load of every lane of a wave takes a whole block, and lane 16 j + r gets, in
// word w, the eight columns 32 w + 8 j .. + 7 of row r -- its share of the A operand of the
// 16 x 16 matrix-core instruction for columns 32 w .. 32 w + 31.  Inside a word the even
// columns lie in the low half and the odd ones in the high half, column pair p at bits 4 p and
// 4 p + 16: one shift and one and-or turn a word into a pair of 16-bit floats.
#include <algorithm>

#include "nm_grid.h"
#include "nm_launch.h"
#include "nm_mfma.h"

namespace nm {
namespace {

constexpr int kBlockCols = 128;       // stored columns of a block of codes

// ---------------------------------------------------------------------------------------
// nm_quantize: one wave per block of 16 rows x 128 columns; lane 16 j + r reads its 32
// elements, the four lanes of a row share the group maxima by lane exchange.
// ---------------------------------------------------------------------------------------

template <int DT>
struct WeightElem;
template <>
struct WeightElem<kF32> { typedef uint32_t type; };
template <>
struct WeightElem<kF16> { typedef uint16_t type; };
template <>
struct WeightElem<kBF16> { typedef uint16_t type; };

template <int DT>
__device__ __forceinline__ float to_f32(typename WeightElem<DT>::type v) {
  if constexpr (DT == kF32) return __uint_as_float(v);
  else if constexpr (DT == kF16) return f16_to_f32(v);
  else return bf16_to_f32(v);
}

template <bool BF16>
__device__ __forceinline__ float scale_to_f32(uint32_t s) {
  if constexpr (BF16) return bf16_to_f32(s);
  else return f16_to_f32(s);
}
template <bool BF16>
__device__ __forceinline__ uint32_t f32_to_scale(float s) {
  if constexpr (BF16) return f32_to_bf16(s);
  else return f32_to_f16(s);
}

// Eight elements of a row from column c; zeros past column C.  kWhole: C % 8 == 0, so the
// eight are wholly inside or outside and their address is 16-byte aligned.
template <int DT, bool kWhole>
__device__ __forceinline__ void load8(const typename WeightElem<DT>::type* row, int64_t c,
                                      int64_t C, float (&v)[8]) {
  if constexpr (kWhole) {
    if (c >= C) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    } else if constexpr (DT == kF32) {
      const u32x4_t a = *reinterpret_cast<const u32x4_t*>(row + c);
      const u32x4_t b = *reinterpret_cast<const u32x4_t*>(row + c + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
      const u32x4_t a = *reinterpret_cast<const u32x4_t*>(row + c);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = to_f32<DT>((uint16_t)(a[i / 2] >> (16 * (i & 1))));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < C ? to_f32<DT>(row[c + i]) : 0.f;
  }
}

// Bits of |x|: as unsigned numbers they order like |x|, with NaN above infinity, so a group
// that holds a NaN gets a NaN scale.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <int DT, bool BF16S, bool kBlocked, bool kWhole>
__global__ void __launch_bounds__(256)
    quantize_kernel(const typename WeightElem<DT>::type* __restrict__ W, int64_t R, int64_t C,
                    int64_t S, int64_t blocks, int log_group, u32x4_t* __restrict__ codes,
                    uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
  const int64_t groups = (C + (1 << log_group) - 1) >> log_group;
  for (int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); b < blocks;
       b += (int64_t)gridDim.x * 4) {
    const int64_t g = b / S, s = b % S, row = 16 * g + r;
    float v[4][8];
    uint32_t top[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int64_t c = kBlockCols * s + 32 * w + 8 * j;
      if constexpr (kBlocked) {  // (g, step, 16, 32): a step is one instruction's columns
        const int64_t steps = C / 32, step = 4 * s + w;
        load8<DT, true>(W + ((g * steps + step) * 16 + r) * 32 - 32 * step,
                        step < steps ? c : C, C, v[w]);
      } else {
        load8<DT, kWhole>(W + (row < R ? row : 0) * C, row < R ? c : C, C, v[w]);
      }
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = max(t, abs_bits(v[w][i]));
      t = max(t, (uint32_t)__shfl_xor((int)t, 16));
      top[w] = max(t, (uint32_t)__shfl_xor((int)t, 32));
    }
    if (log_group >= 6) {
      top[0] = top[1] = max(top[0], top[1]);
      top[2] = top[3] = max(top[2], top[3]);
    }
    if (log_group == 7) top[0] = top[1] = top[2] = top[3] = max(top[0], top[2]);
    u32x4_t out;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t s16 = f32_to_scale<BF16S>(__uint_as_float(top[w]) / 7.f);
      const float sc = scale_to_f32<BF16S>(s16);
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = rintf(v[w][i] / sc);
        // a scale of zero, and elements that are no number, take code 0
        const int code = sc != 0.f && q == q ? (int)fminf(fmaxf(q, -8.f), 7.f) + 8 : 8;
        word |= (uint32_t)code << (4 * (i >> 1) + 16 * (i & 1));
      }
      out[w] = word;
      const int64_t gi = (kBlockCols * s + 32 * w) >> log_group;
      if (((32 * w) & ((1 << log_group) - 1)) == 0 && j == 0 && gi < groups)
        scales[(g * groups + gi) * 16 + r] = (uint16_t)s16;
    }
    codes[b * 64 + lane] = out;
  }
}

// ---------------------------------------------------------------------------------------
// nm_dequantize: the same assignment of columns to lanes, s q rounded once to the scales' type.
// ---------------------------------------------------------------------------------------
template <bool BF16S, bool kBlocked, bool kWhole>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const u32x4_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                      int64_t R, int64_t C, int64_t S, int64_t blocks, int log_group,
                      uint16_t* __restrict__ W) {
  const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
  const int64_t groups = (C + (1 << log_group) - 1) >> log_group;
  for (int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); b < blocks;
       b += (int64_t)gridDim.x * 4) {
    const int64_t g = b / S, s = b % S, row = 16 * g + r;
    const u32x4_t in = codes[b * 64 + lane];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int64_t c = kBlockCols * s + 32 * w + 8 * j;
      if (c >= C || (!kBlocked && row >= R)) continue;
      const float sc =
          scale_to_f32<BF16S>(scales[(g * groups + ((kBlockCols * s + 32 * w) >> log_group)) * 16 + r]);
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int code = (int)((in[w] >> (4 * (i >> 1) + 16 * (i & 1))) & 15u) - 8;
        h[i] = f32_to_scale<BF16S>(sc * (float)code);
      }
      if constexpr (kBlocked || kWhole) {
        const int64_t at = kBlocked ? ((g * (C / 32) + 4 * s + w) * 16 + r) * 32 + 8 * j : row * C + c;
        *reinterpret_cast<u32x4_t*>(W + at) =
            u32x4_t{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < C) W[row * C + c + i] = (uint16_t)h[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// nm_matvec.  y[r, t] = sum over groups of s[r, g] * (sum over the group of q x).
//
// A code becomes a 16-bit float by bit patterns alone: 16 + u for the stored u = q + 8 (for
// bf16 u goes to mantissa bits 3 .. 6 under the exponent of 16, for fp16 to bits 6 .. 9), and
// the matrix cores take off the 24 again with a second instruction whose A operand is the
// constant -24 at every stored place (for 2:4, under the same positions).  Products are exact,
// sums fp32; the group's sum is scaled in fp32.
// ---------------------------------------------------------------------------------------

// Four pairs of eight codes as 16-bit floats 16 + u.
template <bool BF16>
__device__ __forceinline__ u32x4_t codes_to_float(uint32_t w) {
  if constexpr (BF16)
    return u32x4_t{((w << 3) & 0x00780078u) | 0x41804180u, ((w >> 1) & 0x00780078u) | 0x41804180u,
                   ((w >> 5) & 0x00780078u) | 0x41804180u, ((w >> 9) & 0x00780078u) | 0x41804180u};
  else
    return u32x4_t{((w << 6) & 0x03C003C0u) | 0x4C004C00u, ((w << 2) & 0x03C003C0u) | 0x4C004C00u,
                   ((w >> 2) & 0x03C003C0u) | 0x4C004C00u, ((w >> 6) & 0x03C003C0u) | 0x4C004C00u};
}

template <bool BF16>
__device__ __forceinline__ float4_t mfma_dense(const u32x4_t& a, const u32x4_t& b,
                                               const float4_t& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

struct B16 {
  u32x4_t lo, hi;
};
template <bool BF16>
__device__ __forceinline__ float4_t mfma_sparse(const u32x4_t& a, const u32x4_t& b0,
                                                const u32x4_t& b1, const float4_t& c,
                                                uint32_t idx) {
  const B16 b{b0, b1};
  if constexpr (BF16)
    return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                     __builtin_bit_cast(bf16x16_t, b), c, (int)idx,
                                                     0, 0);
  else
    return __builtin_amdgcn_smfmac_f32_16x16x64_f16(__builtin_bit_cast(f16x8_t, a),
                                                    __builtin_bit_cast(f16x16_t, b), c, (int)idx,
                                                    0, 0);
}

// X (K x T) in the order of the B operand: for each tile of 16 columns and each eight rows of
// K, 16 columns of eight values (256 bytes); zeros past K and T.
__global__ void __launch_bounds__(256)
    columns_kernel(const uint16_t* __restrict__ X, int64_t K, int64_t T, int64_t K8, int64_t total,
                   u32x4_t* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t n = i & 15, k8 = (i >> 4) % K8, t = (i >> 4) / K8 * 16 + n;
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      h[e] = t < T && 8 * k8 + e < K ? X[(8 * k8 + e) * T + t] : 0u;
    out[i] = u32x4_t{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
  }
}

struct MatvecArgs {
  const u32x4_t* codes;
  const uint16_t* scales;
  const uint8_t* meta;  // 2:4: the blocked metadata, else null
  const u32x4_t* x;     // columns_kernel's order, or for one column X itself
  void* y;
  int64_t R, T;
  int64_t K;       // rows of X
  int64_t K8;      // eights of rows in columns_kernel's order
  int S;           // blocks of 128 stored columns in a row
  int steps;       // instructions along a row: 32 stored columns each
  int groups;      // groups in a row
};

// Eight values of the single column from row k; zeros past K.  kWhole: K % 8 == 0.
__device__ __forceinline__ u32x4_t one_column(const MatvecArgs& a, int64_t k) {
  if (k + 8 <= a.K) return *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(a.x) + k);
  uint32_t h[8];
  const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x);
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = k + e < a.K ? x[k + e] : 0u;
  return u32x4_t{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
}

// One workgroup: 16 rows x 16 NT columns of Y; its waves take the blocks of 128 stored columns
// in turn and add their sums in wave order at the end.
template <bool BF16, bool SPARSE, int LOG_GROUP, bool ONE, int NT, int WAVES, int YT>
__global__ void __launch_bounds__(64 * WAVES) matvec_kernel(MatvecArgs a) {
  __shared__ float4_t part[WAVES][NT][64];
  const int lane = threadIdx.x & 63, n = lane & 15, j = lane >> 4;
  const int wave = threadIdx.x >> 6;
  const int64_t g = blockIdx.x, t0 = (int64_t)blockIdx.y * (16 * NT);
  const uint32_t off = BF16 ? 0xC1C0C1C0u : 0xCE00CE00u;  // -24, -24
  const u32x4_t offs{off, off, off, off};
  float4_t total[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) total[t] = float4_t{0.f, 0.f, 0.f, 0.f};

  for (int s = wave; s < a.S; s += WAVES) {
    const u32x4_t c = a.codes[(g * a.S + s) * 64 + lane];
    float4_t acc[NT];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int step = 4 * s + w;
      if (step >= a.steps) break;
      if (((32 * w) & ((1 << LOG_GROUP) - 1)) == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
      }
      uint32_t idx = 0;
      if constexpr (SPARSE)
        idx = *reinterpret_cast<const uint16_t*>(a.meta + ((g * a.steps + step) * 16 + n) * 8 + 2 * j);
      const u32x4_t wf = codes_to_float<BF16>(c[w]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (SPARSE) {
          u32x4_t b0, b1;
          if constexpr (ONE) {
            b0 = one_column(a, 64 * (int64_t)step + 8 * j);
            b1 = one_column(a, 64 * (int64_t)step + 32 + 8 * j);
          } else {
            const int64_t at = ((t0 / 16 + t) * a.K8 + 8 * (int64_t)step) * 16 + n;
            b0 = a.x[at + 16 * j];
            b1 = a.x[at + 16 * (4 + j)];
          }
          acc[t] = mfma_sparse<BF16>(wf, b0, b1, acc[t], idx);
          acc[t] = mfma_sparse<BF16>(offs, b0, b1, acc[t], idx);
        } else {
          u32x4_t b;
          if constexpr (ONE) b = one_column(a, 32 * (int64_t)step + 8 * j);
          else b = a.x[((t0 / 16 + t) * a.K8 + 4 * (int64_t)step + j) * 16 + n];
          acc[t] = mfma_dense<BF16>(wf, b, acc[t]);
          acc[t] = mfma_dense<BF16>(offs, b, acc[t]);
        }
      }
      if (((32 * (w + 1)) & ((1 << LOG_GROUP) - 1)) == 0 || step + 1 == a.steps) {
        const int gi = (kBlockCols * s + 32 * w) >> LOG_GROUP;
        const u32x2_t sv = *reinterpret_cast<const u32x2_t*>(a.scales + (g * a.groups + gi) * 16 + 4 * j);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            total[t][i] += scale_to_f32<BF16>((sv[i / 2] >> (16 * (i & 1))) & 0xFFFFu) * acc[t][i];
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) part[wave][t][lane] = total[t];
  __syncthreads();
  // rows 4 j + i of column n: one output per thread of the first waves
  for (int e = threadIdx.x; e < NT * 256; e += 64 * WAVES) {
    const int t = e >> 8, i = (e >> 6) & 3, l = e & 63;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) y += part[w][t][l][i];
    const int64_t row = 16 * g + 4 * (l >> 4) + i, col = t0 + 16 * t + (l & 15);
    if (row < a.R && col < a.T) store_from_f32<YT>(a.y, row * a.T + col, y);
  }
}

template <bool BF16, bool SPARSE, int LOG_GROUP, bool ONE, int YT>
hipError_t launch_matvec_cols(const MatvecArgs& a, hipStream_t s) {
  constexpr int kWaves = 8;
  const unsigned rows = (unsigned)((a.R + 15) / 16);
  if constexpr (ONE) {
    matvec_kernel<BF16, SPARSE, LOG_GROUP, true, 1, kWaves, YT><<<rows, 64 * kWaves, 0, s>>>(a);
  } else if (a.T <= 16) {
    matvec_kernel<BF16, SPARSE, LOG_GROUP, false, 1, kWaves, YT><<<rows, 64 * kWaves, 0, s>>>(a);
  } else {
    matvec_kernel<BF16, SPARSE, LOG_GROUP, false, 2, kWaves, YT>
        <<<dim3(rows, (unsigned)((a.T + 31) / 32)), 64 * kWaves, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <bool BF16, bool SPARSE, int LOG_GROUP>
hipError_t launch_matvec_y(const MatvecArgs& a, int y_dt, hipStream_t s) {
  constexpr int kSame = BF16 ? kBF16 : kF16;
  if (a.T == 1)
    return y_dt == kF32 ? launch_matvec_cols<BF16, SPARSE, LOG_GROUP, true, kF32>(a, s)
                        : launch_matvec_cols<BF16, SPARSE, LOG_GROUP, true, kSame>(a, s);
  return y_dt == kF32 ? launch_matvec_cols<BF16, SPARSE, LOG_GROUP, false, kF32>(a, s)
                      : launch_matvec_cols<BF16, SPARSE, LOG_GROUP, false, kSame>(a, s);
}

template <bool BF16, bool SPARSE>
hipError_t launch_matvec_group(const MatvecArgs& a, int log_group, int y_dt, hipStream_t s) {
  if (log_group == 5) return launch_matvec_y<BF16, SPARSE, 5>(a, y_dt, s);
  if (log_group == 6) return launch_matvec_y<BF16, SPARSE, 6>(a, y_dt, s);
  return launch_matvec_y<BF16, SPARSE, 7>(a, y_dt, s);
}

int log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

template <int DT, bool BF16S>
hipError_t launch_quantize_as(const void* W, int64_t R, int64_t C, bool blocked, int group,
                              void* codes, void* scales, hipStream_t s) {
  typedef typename WeightElem<DT>::type E;
  const int64_t S = (C + kBlockCols - 1) / kBlockCols, blocks = (R + 15) / 16 * S;
  const unsigned grid = stride_grid(blocks, 4);
  const E* w = static_cast<const E*>(W);
  u32x4_t* c = static_cast<u32x4_t*>(codes);
  uint16_t* sc = static_cast<uint16_t*>(scales);
  const int lg = log2_of(group);
  if (blocked)
    quantize_kernel<DT, BF16S, true, true><<<grid, 256, 0, s>>>(w, R, C, S, blocks, lg, c, sc);
  else if (C % 8 == 0)
    quantize_kernel<DT, BF16S, false, true><<<grid, 256, 0, s>>>(w, R, C, S, blocks, lg, c, sc);
  else
    quantize_kernel<DT, BF16S, false, false><<<grid, 256, 0, s>>>(w, R, C, S, blocks, lg, c, sc);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const void* W, int dt, int64_t R, int64_t C, bool blocked, int group,
                           void* codes, void* scales, int scale_dt, hipStream_t s) {
  const bool b = scale_dt == kBF16;
  if (dt == kF32)
    return b ? launch_quantize_as<kF32, true>(W, R, C, blocked, group, codes, scales, s)
             : launch_quantize_as<kF32, false>(W, R, C, blocked, group, codes, scales, s);
  if (dt == kF16)
    return b ? launch_quantize_as<kF16, true>(W, R, C, blocked, group, codes, scales, s)
             : launch_quantize_as<kF16, false>(W, R, C, blocked, group, codes, scales, s);
  return b ? launch_quantize_as<kBF16, true>(W, R, C, blocked, group, codes, scales, s)
           : launch_quantize_as<kBF16, false>(W, R, C, blocked, group, codes, scales, s);
}

hipError_t launch_dequantize(const void* codes, const void* scales, int scale_dt, int64_t R,
                             int64_t C, bool blocked, int group, void* W, hipStream_t s) {
  const int64_t S = (C + kBlockCols - 1) / kBlockCols, blocks = (R + 15) / 16 * S;
  const unsigned grid = stride_grid(blocks, 4);
  const u32x4_t* c = static_cast<const u32x4_t*>(codes);
  const uint16_t* sc = static_cast<const uint16_t*>(scales);
  uint16_t* w = static_cast<uint16_t*>(W);
  const int lg = log2_of(group);
  const bool b = scale_dt == kBF16;
#define NM_DEQ(BL, WH)                                                                     \
  (b ? dequantize_kernel<true, BL, WH><<<grid, 256, 0, s>>>(c, sc, R, C, S, blocks, lg, w)  \
     : dequantize_kernel<false, BL, WH><<<grid, 256, 0, s>>>(c, sc, R, C, S, blocks, lg, w))
  if (blocked) NM_DEQ(true, true);
  else if (C % 8 == 0) NM_DEQ(false, true);
  else NM_DEQ(false, false);
#undef NM_DEQ
  return hipGetLastError();
}

size_t matvec_workspace_bytes(int64_t K, int64_t T) {
  if (T <= 1) return 0;
  return (size_t)((K + kBlockCols - 1) / kBlockCols * 16) * (size_t)((T + 31) / 32 * 2) * 256;
}

hipError_t launch_matvec(const void* codes, const void* scales, const void* meta, int64_t R,
                         int64_t K, int group, const void* X, int64_t T, int dt, void* Y, int y_dt,
                         void* workspace, hipStream_t s) {
  const int64_t C = meta ? K / 2 : K;
  MatvecArgs a;
  a.codes = static_cast<const u32x4_t*>(codes);
  a.scales = static_cast<const uint16_t*>(scales);
  a.meta = static_cast<const uint8_t*>(meta);
  a.y = Y;
  a.R = R;
  a.T = T;
  a.K = K;
  a.K8 = (K + kBlockCols - 1) / kBlockCols * 16;
  a.S = (int)((C + kBlockCols - 1) / kBlockCols);
  a.steps = (int)((C + 31) / 32);
  a.groups = (int)((C + group - 1) / group);
  if (T == 1) {
    a.x = static_cast<const u32x4_t*>(X);
  } else {
    u32x4_t* x = static_cast<u32x4_t*>(workspace);
    const int64_t total = a.K8 * ((T + 31) / 32 * 2) * 16;
    columns_kernel<<<stride_grid(total, 256), 256, 0, s>>>(static_cast<const uint16_t*>(X), K, T,
                                                           a.K8, total, x);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.x = x;
  }
  const int lg = log2_of(group);
  if (dt == kBF16)
    return meta ? launch_matvec_group<true, true>(a, lg, y_dt, s)
                : launch_matvec_group<true, false>(a, lg, y_dt, s);
  return meta ? launch_matvec_group<false, true>(a, lg, y_dt, s)
              : launch_matvec_group<false, false>(a, lg, y_dt, s);
}

}  // namespace nm
