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
// 4 p + 16: a mask takes a pair out of a word, a code in each half.
#include <algorithm>
#include <type_traits>

#include "nm_grid.h"
#include "nm_launch.h"
#include "nm_mfma.h"
#include "nm_tiles.h"

namespace nm {
namespace {

constexpr int kBlockCols = 128;       // stored columns of a block of codes

// ---------------------------------------------------------------------------------------
// nm_quantize: one wave per block of 16 rows x 128 columns; lane 16 j + r reads its 32
// elements, the four lanes of a row share the group maxima by lane exchange.  One pass, bound by
// memory: 11008 x 2048 kept values of bf16 take 10.8 us (57 MB, 5.3 TB/s; a large copy reaches
// 5.2), 768 x 768 4.0 us, which is a launch.
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

typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));

// Eight elements of a row from column c, as they are stored; zeros past column C.  kWhole: C % 8
// == 0, so the eight are wholly inside or outside and their address is 16-byte aligned; else eight
// that lie inside are read as they stand and only a row's last ones one by one (quantize and
// dequantize of 4096 x 4100 bf16: 11.6 and 13.0 us, 27.1 and 40.3 with all one by one).
template <int DT>
struct Eight {
  static constexpr int kWords = DT == kF32 ? 8 : 4;
  uint32_t w[kWords];

  template <bool kWhole>
  __device__ __forceinline__ void load(const typename WeightElem<DT>::type* row, int64_t c,
                                       int64_t C) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
    if constexpr (kWhole) {
      if (c >= C) return;
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(row + c + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * h + i] = v[i];
      }
    } else if (c + 8 <= C) {
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const u32x4_any_t v = *reinterpret_cast<const u32x4_any_t*>(row + c + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * h + i] = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < C) {
          if constexpr (DT == kF32) w[i] = row[c + i];
          else w[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
        }
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (DT == kF32) return __uint_as_float(w[i]);
    else if constexpr (DT == kBF16) return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else return f16_to_f32(w[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
  }
  // The largest |x| as sign-cleared bits, which order like |x| with NaN above infinity, so that a
  // group that holds a NaN gets a NaN scale; 16-bit types: one of the even and one of the odd
  // elements in the halves of the word.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) t = larger(t, w[i] & (DT == kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu));
    return t;
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (DT == kF32) return max(a, b);
    else
      return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2_t, a),
                                                                    __builtin_bit_cast(ushort2_t, b)));
  }
  static __device__ __forceinline__ float to_float(uint32_t top) {
    if constexpr (DT == kF32) return __uint_as_float(top);
    else return to_f32<DT>((uint16_t)max(top >> 16, top & 0xFFFFu));
  }
};

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <int DT, bool BF16S, bool kBlocked, bool kWhole, int LOG_GROUP>
__global__ void __launch_bounds__(256)
    quantize_kernel(const typename WeightElem<DT>::type* __restrict__ W, int64_t R, int64_t C,
                    int64_t S, int64_t blocks, u32x4_t* __restrict__ codes,
                    uint16_t* __restrict__ scales) {
  constexpr int kWords = 1 << (LOG_GROUP - 5);  // code words of a lane that share a scale
  const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
  const int64_t groups = (C + (1 << LOG_GROUP) - 1) >> LOG_GROUP;
  for (int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); b < blocks;
       b += (int64_t)gridDim.x * 4) {
    const int64_t g = b / S, s = b % S, row = 16 * g + r;
    Eight<DT> v[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int64_t c = kBlockCols * s + 32 * w + 8 * j;
      if constexpr (kBlocked) {  // (g, step, 16, 32): a step is one instruction's columns
        const int64_t steps = C / 32, step = 4 * s + w;
        v[w].template load<true>(W + ((g * steps + step) * 16 + r) * 32 - 32 * step,
                                 step < steps ? c : C, C);
      } else {
        v[w].template load<kWhole>(W + (row < R ? row : 0) * C, row < R ? c : C, C);
      }
    }
    u32x4_t out;
#pragma unroll
    for (int w0 = 0; w0 < 4; w0 += kWords) {
      uint32_t top = 0;
#pragma unroll
      for (int w = w0; w < w0 + kWords; ++w) top = Eight<DT>::larger(top, v[w].top());
      top = Eight<DT>::larger(top, (uint32_t)__shfl_xor((int)top, 16));
      top = Eight<DT>::larger(top, (uint32_t)__shfl_xor((int)top, 32));
      const uint32_t s16 = f32_to_scale<BF16S>(Eight<DT>::to_float(top) / 7.f);
      const float sc = scale_to_f32<BF16S>(s16);
      if (DT != kF32 && __all(abs_bits(sc) >= 0x0D800000u)) {  // 2^-100: 1 / sc is finite
        // Both numbers have at most 11 significant bits, so a quotient of this size is a half
        // integer or at least 2^-13 away from one, and w * (1 / sc) is within 2^-18 of it:
        // brought to a multiple of 2^-15 by the addition of 384 (|quotient| is below 11), it rounds
        // as the quotient.  The four codes of a half word add up as the digits of a float.
        const float inv = 1.f / sc;
#pragma unroll
        for (int w = w0; w < w0 + kWords; ++w) {
          uint32_t half[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float digits = 0.f;
#pragma unroll
            for (int p = 3; p >= 0; --p) {
              const float q = rintf(__builtin_fmaf(v[w].value(2 * p + h), inv, 384.f));
              digits = __builtin_fmaf(digits, 16.f, __builtin_amdgcn_fmed3f(q, 376.f, 391.f));
            }
            half[h] = (uint32_t)(digits - 376.f * 4369.f);  // 4369 = 0x1111
          }
          out[w] = half[0] | half[1] << 16;
          if (abs_bits(sc) >= 0x7F800000u) out[w] = 0x88888888u;  // no numbers: codes 0
        }
      } else {
#pragma unroll
        for (int w = w0; w < w0 + kWords; ++w) {
          uint32_t word = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float q = rintf(v[w].value(i) / sc);
            // a scale of zero, and elements that are no number, take code 0
            const int code = sc != 0.f && q == q ? (int)fminf(fmaxf(q, -8.f), 7.f) + 8 : 8;
            word |= (uint32_t)code << (4 * (i >> 1) + 16 * (i & 1));
          }
          out[w] = word;
        }
      }
      const int64_t gi = (kBlockCols * s + 32 * w0) >> LOG_GROUP;
      if (j == 0 && gi < groups) scales[(g * groups + gi) * 16 + r] = (uint16_t)s16;
    }
    codes[b * 64 + lane] = out;
  }
}

// ---------------------------------------------------------------------------------------
// nm_dequantize: the same assignment of columns to lanes, s q rounded once to the scales' type.
// Bound by memory: 11008 x 2048 values of bf16 in 11.2 us (57 MB, 5.1 TB/s).
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
      } else if (c + 8 <= C) {
        *reinterpret_cast<u32x4_any_t*>(W + row * C + c) =
            u32x4_any_t{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
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
// A code becomes the 16-bit float that it is, exactly, so the matrix cores' products are exact and
// an infinite x gives what it gives in q x; sums are fp32; the group's sum is scaled in fp32.
// ---------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t in_register(uint32_t c) {
  asm volatile("" : "+v"(c));
  return c;
}

// Eight codes as four pairs of 16-bit floats.
template <bool BF16>
struct Codes;

// bf16: the stored u = q + 8 of a pair, masked where they stand, are subnormal fp16 numbers, u
// 2^-24 or u 2^-20; one mixed-precision multiply-add each makes them q in fp32, whose upper halves
// are bf16.  17 instructions a word.
template <>
struct Codes<true> {
  uint32_t low = in_register(0x000F000Fu), high = in_register(0x00F000F0u);
  float low_scale = __uint_as_float(in_register(0x4B800000u));   // 2^24
  float high_scale = __uint_as_float(in_register(0x49800000u));  // 2^20
  float minus8 = __uint_as_float(in_register(0xC1000000u));

  __device__ __forceinline__ uint32_t pair(uint32_t u, float scale) const {
    float even, odd;
    asm("v_fma_mix_f32 %0, %1, %2, %3 op_sel_hi:[1,0,0]" : "=v"(even) : "v"(u), "v"(scale), "v"(minus8));
    asm("v_fma_mix_f32 %0, %1, %2, %3 op_sel:[1,0,0] op_sel_hi:[1,0,0]"
        : "=v"(odd) : "v"(u), "v"(scale), "v"(minus8));
    return __builtin_amdgcn_perm(__float_as_uint(odd), __float_as_uint(even), 0x07060302u);
  }
  __device__ __forceinline__ u32x4_t floats(uint32_t w) const {
    const uint32_t v = w >> 8;
    return u32x4_t{pair(w & low, low_scale), pair(w & high, high_scale), pair(v & low, low_scale),
                   pair(v & high, high_scale)};
  }
};

// fp16: u goes to the mantissa's upper bits under the exponent of 16, and 24 is taken off again.
// 12 instructions a word.
template <>
struct Codes<false> {
  uint32_t mask = in_register(0x03C003C0u), sixteen = in_register(0x4C004C00u);
  uint32_t minus24 = in_register(0xCE00CE00u);

  __device__ __forceinline__ uint32_t pair(uint32_t u) const {
    typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, (u & mask) | sixteen) +
                                            __builtin_bit_cast(half2_t, minus24));
  }
  __device__ __forceinline__ u32x4_t floats(uint32_t w) const {
    return u32x4_t{pair(w << 6), pair(w << 2), pair(w >> 2), pair(w >> 6)};
  }
};

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

struct MatvecArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const uint8_t* meta;  // 2:4: the blocked metadata, else null
  const uint16_t* x;
  void* y;
  int64_t R, T, K;
  int S;       // blocks of 128 stored columns in a row
  int steps;   // instructions along a row: 32 stored columns each
  int groups;  // groups in a row
  // several columns:
  int slice;       // blocks of a slice of the stored columns
  int log_along;   // log2 of the waves that share 16 rows
  float4_t* part;  // slices x blocks of 16 rows x tiles of 16 columns x 64 lanes
};

// One block of 128 stored columns of 16 rows, as one lane holds it, and where the lane finds it:
// with the wave's own scalar bases the loads need no vector address arithmetic.
template <bool SPARSE, int LOG_GROUP>
struct CodeBlock {
  static constexpr int kGroups = kBlockCols >> LOG_GROUP;
  u32x4_t codes;
  u32x2_t scales[kGroups];
  uint16_t meta[4];

  // Rows of block g, columns of block s.
  __device__ __forceinline__ void load(const MatvecArgs& a, int64_t g, int s, int lane) {
    const uint32_t n = lane & 15, j = lane >> 4;
    codes = *reinterpret_cast<const u32x4_t*>(a.codes + (g * a.S + s) * 1024 + (uint32_t)lane * 16);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int gi = min(s * kGroups + i, a.groups - 1);
      scales[i] = *reinterpret_cast<const u32x2_t*>(a.scales + (g * a.groups + gi) * 32 + j * 8);
    }
    if constexpr (SPARSE) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int step = min(4 * s + w, a.steps - 1);
        meta[w] = *reinterpret_cast<const uint16_t*>(a.meta + (g * a.steps + step) * 128 + n * 8 + j * 2);
      }
    }
  }

  // total[t] += this block times the B operands operand(w, half, t): for step w 32 rows of X (of
  // the two halves of 64, for 2:4), 16 columns.
  template <bool BF16, int NT, typename F>
  __device__ __forceinline__ void multiply(float4_t (&total)[NT], const Codes<BF16>& convert,
                                           F&& operand) const {
    float4_t acc[NT];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (((32 * w) & ((1 << LOG_GROUP) - 1)) == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = float4_t{0.f, 0.f, 0.f, 0.f};
      }
      const u32x4_t wf = convert.floats(codes[w]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const u32x4_t b0 = operand(w, 0, t);
        if constexpr (SPARSE) {
          const u32x4_t b1 = operand(w, 1, t);
          acc[t] = mfma_sparse<BF16>(wf, b0, b1, acc[t], meta[w]);
        } else {
          acc[t] = mfma_dense<BF16>(wf, b0, acc[t]);
        }
      }
      if (((32 * (w + 1)) & ((1 << LOG_GROUP) - 1)) == 0) {
        const u32x2_t sv = scales[(32 * w) >> LOG_GROUP];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            total[t][i] += scale_to_f32<BF16>((sv[i / 2] >> (16 * (i & 1))) & 0xFFFFu) * acc[t][i];
      }
    }
  }
};

// Few columns, with X whole in LDS, a run of its rows for each column; FEW: more than one.  A
// workgroup has 16 rows; its waves take the blocks of 128 stored columns in turn, each with the next
// one's loads in flight, and add their sums in wave order at the end.  The instruction's columns
// past the last hold the last again and are dropped.  Blocks past the matrix's last columns hold
// code 0 against zeros of X, so there are no ends to treat.
// Bound by the first loads' latency on small matrices, from there by the few loads that a unit keeps
// in flight: one column 4096 x 4096 4.7 us (1.9 TB/s), 4096 x 11008 8.0 (3.0), 16384 x 12288
// 23.2 (4.6); two columns of 4096 x 4096 5.4; the smaller ones' codes are in cache.
template <bool BF16, bool SPARSE, int LOG_GROUP, int WAVES, bool FEW, int YT>
__global__ void __launch_bounds__(64 * WAVES) matvec_kernel(MatvecArgs a) {
  constexpr int kEights = SPARSE ? 8 : 4;  // eights of X's rows to a step
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, j = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Codes<BF16> convert;
  const int64_t g = blockIdx.x;
  const int T = FEW ? (int)a.T : 1;
  CodeBlock<SPARSE, LOG_GROUP> next;
  if (wave < a.S) next.load(a, g, wave, lane);
  const int chunks = a.S * 4 * kEights;  // X and the zeros after it, to whole blocks
  const int pitch = 16 * chunks + kColumnPad;
  const int64_t have = a.K * T;
  for (int c = threadIdx.x; c < chunks * T; c += 64 * WAVES) {
    const int64_t at = 8 * (int64_t)c;
    u32x4_t v;
    if (at + 8 <= have) {
      v = *reinterpret_cast<const u32x4_t*>(a.x + at);
    } else {
      uint32_t h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = at + e < have ? a.x[at + e] : 0u;
      v = u32x4_t{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
    }
    if constexpr (FEW) {
      int k = 8 * c / T, t = 8 * c - k * T;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        *reinterpret_cast<uint16_t*>(smem + t * pitch + 2 * k) = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
        if (++t == T) {
          t = 0;
          ++k;
        }
      }
    } else {
      reinterpret_cast<u32x4_t*>(smem)[c] = v;
    }
  }
  __syncthreads();
  float4_t total[1] = {float4_t{0.f, 0.f, 0.f, 0.f}};
  const int col = (lane & 15) < T ? lane & 15 : T - 1;
  for (int s = wave; s < a.S; s += WAVES) {
    const CodeBlock<SPARSE, LOG_GROUP> cur = next;
    if (s + WAVES < a.S) next.load(a, g, s + WAVES, lane);
    const u32x4_t* x =
        reinterpret_cast<const u32x4_t*>(smem + (FEW ? col * pitch : 0)) + 4 * s * kEights + j;
    cur.template multiply<BF16, 1>(total, convert, [&](int w, int half, int) {
      return x[w * kEights + 4 * half];
    });
  }
  __syncthreads();  // X's place in LDS takes the waves' sums
  float4_t* part = reinterpret_cast<float4_t*>(smem);
  part[wave * 64 + lane] = total[0];
  __syncthreads();
  if ((int)threadIdx.x < 16 * T) {  // lane 16 j + t holds rows 4 j + i of column t
    const int row = threadIdx.x / T, t = threadIdx.x - row * T;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) y += part[w * 64 + 16 * (row / 4) + t][row % 4];
    if (16 * g + row < a.R) store_from_f32<YT>(a.y, (16 * g + row) * T + t, y);
  }
}

// Several columns.  A workgroup of eight waves has 16 rows for every 2^log_along of them, 16 NT
// columns and a slice of the stored columns.  X's rows for the slice are laid out in LDS once: 16
// columns (32 bytes) a row first, then, by one transposing read and one write in place, each 32
// rows x 16 columns as the B operand that the products read (16 bytes a lane, no bank conflicts).
// The waves that share rows take the slice's blocks in turn and add their sums in wave order.
// With more than one slice the sums go to the workspace, where join_slices_kernel adds them in
// slice order.
// Bound by laying out X, which every workgroup does for its slice, and by the launch of the second
// kernel (4 us): 2:4 4096 x 11008 with 32 columns 13.0 us and the join, 5003 x 11007 with 5 columns
// 13.8 us and the join, 16384 x 8192 with 32 columns 26.1 us and the join (2.4 TB/s in all).
constexpr int kSliceWaves = 8;

template <bool BF16, bool SPARSE, int LOG_GROUP, int NT, int YT>
__global__ void __launch_bounds__(64 * kSliceWaves) matvec_slice_kernel(MatvecArgs a) {
  typedef CodeBlock<SPARSE, LOG_GROUP> Block;
  constexpr int kBlockRows = SPARSE ? 256 : 128;  // rows of X to a block
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, n = lane & 15, j = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int along = 1 << a.log_along, first = wave & (along - 1);
  const Codes<BF16> convert;
  const int64_t last = (a.R + 15) / 16 - 1;
  const int64_t mine = (int64_t)blockIdx.x * (kSliceWaves >> a.log_along) + (wave >> a.log_along);
  const int64_t g = mine < last ? mine : last;  // rows past the matrix: dropped below
  const int t0 = blockIdx.z * (16 * NT), T = (int)a.T, cols = min(T - t0, 16 * NT);
  const int s0 = blockIdx.y * a.slice, blocks = min(a.slice, a.S - s0);

  Block next;  // loads of the wave's next block; past the last one, of that again
  if (blocks > 0) next.load(a, g, s0 + min(first, blocks - 1), lane);

  // ---- X ----
  const int64_t k0 = (int64_t)s0 * kBlockRows;
  const int rows = blocks * kBlockRows;
  const int tile_bytes = rows * 32;
  const int have = (int)(a.K - k0 < rows ? a.K - k0 : rows);  // rows of X in the slice
  if (T % 8 == 0) {  // rows of X are whole 16-byte pieces
    constexpr int kBatch = 8;  // loads in flight: a loop of single ones would wait for each
    for (int c0 = threadIdx.x; c0 < rows * 2 * NT; c0 += kBatch * 64 * kSliceWaves) {
      u32x4_t v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * 64 * kSliceWaves, row = c / (2 * NT), p = c % (2 * NT);
        v[i] = row < have && 8 * p < cols
                   ? *reinterpret_cast<const u32x4_t*>(a.x + (k0 + row) * T + t0 + 8 * p)
                   : u32x4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * 64 * kSliceWaves, row = c / (2 * NT), p = c % (2 * NT);
        if (row < rows)
          *reinterpret_cast<u32x4_t*>(smem + (p >> 1) * tile_bytes + row * 32 +
                                      16 * (p & 1)) = v[i];
      }
    }
  } else {
    for (int c = threadIdx.x; c < rows * 2 * NT; c += 64 * kSliceWaves)
      reinterpret_cast<u32x4_t*>(smem)[c] = u32x4_t{0, 0, 0, 0};
    __syncthreads();
    auto put = [&](int row, int col, uint16_t v) {
      *reinterpret_cast<uint16_t*>(smem + (col >> 4) * tile_bytes + row * 32 +
                                   2 * (col & 15)) = v;
    };
    if (T <= 16 * NT) {  // X as one run of numbers, eight at a time (k0 T is a multiple of 8)
      const int numbers = have * T;
      const uint16_t* x = a.x + k0 * T;
      for (int e = threadIdx.x * 8; e < numbers; e += 64 * kSliceWaves * 8) {
        uint32_t h[8];
        if (e + 8 <= numbers) {
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + e);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = (v[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = e + i < numbers ? x[e + i] : 0u;
        }
        int row = e / T, col = e % T;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (e + i < numbers) put(row, col, (uint16_t)h[i]);
          if (++col == T) {
            col = 0;
            ++row;
          }
        }
      }
    } else {  // columns of a wider X, one number at a time
      for (int c = threadIdx.x; c < have * 16 * NT; c += 64 * kSliceWaves) {
        const int row = c / (16 * NT), col = c % (16 * NT);
        if (col < cols) put(row, col, a.x[(k0 + row) * T + t0 + col]);
      }
    }
  }
  __syncthreads();

  // ---- the slice ----
  float4_t total[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) total[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#if defined(__HIP_DEVICE_COMPILE__)
  for (int c = wave; c < rows / 32 * NT; c += kSliceWaves) {
    uint8_t* p = smem + c * 1024;
    const uint32_t off = (8 * j + (n >> 2)) * 32 + 8 * (n & 3);
    const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(p + off));
    const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(p + off + 128));
    *reinterpret_cast<short8_t*>(p + lane * 16) = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
#endif
  __syncthreads();
#pragma unroll 1  // the loop is entered a few times: unrolled, its code would come from memory anew
  for (int s = first; s < blocks; s += along) {
    const Block cur = next;
    next.load(a, g, s0 + min(s + along, blocks - 1), lane);
    const uint8_t* x = smem + s * kBlockRows * 32;
    cur.template multiply<BF16, NT>(total, convert, [&](int w, int half, int t) {
      return *reinterpret_cast<const u32x4_t*>(x + t * tile_bytes +
                                               (w * (kBlockRows / 128) + half) * 1024 + lane * 16);
    });
  }

  if (along > 1) {  // X's place in LDS takes the waves' sums
    float4_t* part = reinterpret_cast<float4_t*>(smem);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) part[(wave * NT + t) * 64 + lane] = total[t];
    __syncthreads();
    if (first != 0) return;
    for (int w = 1; w < along; ++w)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float4_t v = part[((wave + w) * NT + t) * 64 + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) total[t][i] += v[i];
      }
  }
  if (mine > last) return;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (gridDim.y > 1) {
      const int64_t tiles = (int64_t)gridDim.z * NT;
      a.part[((blockIdx.y * (last + 1) + mine) * tiles + blockIdx.z * NT + t) * 64 + lane] = total[t];
      continue;
    }
    const int64_t col = t0 + 16 * t + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = 16 * mine + 4 * j + i;
      if (row < a.R && col < a.T) store_from_f32<YT>(a.y, row * a.T + col, total[t][i]);
    }
  }
}

// One thread for each four rows of a column; `pieces` of them to a slice.
template <int YT>
__global__ void __launch_bounds__(256)
    join_slices_kernel(const float4_t* __restrict__ part, int slices, int64_t pieces, int64_t tiles,
                       int64_t R, int64_t T, void* __restrict__ y) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= pieces) return;
  const int lane = e & 63;
  const int64_t col = (e >> 6) % tiles * 16 + (lane & 15);
  const int64_t row = (e >> 6) / tiles * 16 + (lane >> 4) * 4;
  if (col >= T) return;
  float4_t total{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < slices; ++s) {
    const float4_t v = part[s * pieces + e];
#pragma unroll
    for (int i = 0; i < 4; ++i) total[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row + i < R) store_from_f32<YT>(y, (row + i) * T + col, total[i]);
}

// How several columns are cut.  Each workgroup reads X's rows of its slice, so rows are shared by
// few waves where that leaves workgroups for all 256 units, and one slice is taken where X fits the
// LDS; a slice of 64 KB leaves room for a second workgroup on the unit.
struct MatvecPlan {
  int nt, log_along, slice, slices;
  int64_t groups, tiles;  // workgroups along rows, along columns of X
  int64_t pieces;         // work-items that join the slices: one for four rows of a column
  int64_t bytes;          // of workspace
  MatvecPlan(int64_t R, int64_t K, int64_t T, bool sparse) {
    const int64_t block_rows = sparse ? 256 : 128, S = (K + block_rows - 1) / block_rows;
    nt = T > 16 ? 2 : 1;
    tiles = (T + 16 * nt - 1) / (16 * nt);
    const int64_t block_bytes = block_rows * 32 * nt;
    const auto groups_of = [&](int log) {
      const int64_t rows = 16 * (kSliceWaves >> log);
      return (R + rows - 1) / rows;
    };
    if (S * block_bytes <= 128 << 10) {
      const int64_t most = S * block_bytes <= 64 << 10 ? 512 : 256;
      slices = 1;
      log_along = 3;
      while (log_along > 0 && groups_of(log_along) * tiles > most) --log_along;
    } else {
      const int64_t per = (64 << 10) / block_bytes;
      slices = (int)((S + per - 1) / per);
      log_along = 0;
      while (log_along < 3 && groups_of(log_along) * tiles * slices < 256) ++log_along;
    }
    slice = (int)std::max<int64_t>(1, (S + slices - 1) / slices);
    slices = (int)std::max<int64_t>(1, (S + slice - 1) / slice);
    groups = groups_of(log_along);
    pieces = slices > 1 ? (R + 15) / 16 * tiles * nt * 64 : 0;
    bytes = slices * pieces * 16;
  }
};

template <bool BF16, bool SPARSE, int LOG_GROUP, int NT, int YT>
hipError_t launch_matvec_slices(const MatvecArgs& a, const MatvecPlan& p, hipStream_t s) {
  auto kernel = matvec_slice_kernel<BF16, SPARSE, LOG_GROUP, NT, YT>;
  static const hipError_t attr = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, 128 << 10);
  if (attr != hipSuccess) return attr;
  const size_t lds = std::max((size_t)p.slice * (SPARSE ? 8192 : 4096) * NT,
                              (size_t)kSliceWaves * NT * 1024);
  kernel<<<dim3((unsigned)p.groups, (unsigned)p.slices, (unsigned)p.tiles), 64 * kSliceWaves, lds,
           s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.slices == 1) return e;
  join_slices_kernel<YT><<<(unsigned)((p.pieces + 255) / 256), 256, 0, s>>>(
      a.part, p.slices, p.pieces, p.tiles * NT, a.R, a.T, a.y);
  return hipGetLastError();
}

// Eight waves to 16 rows fill the device where rows are many, sixteen where they are few.
template <bool BF16, bool SPARSE, int LOG_GROUP, bool FEW, int YT>
hipError_t launch_matvec_whole(const MatvecArgs& a, size_t lds, hipStream_t s) {
  const unsigned groups = (unsigned)((a.R + 15) / 16);
  const int waves = groups > 256 ? 8 : 16;
  const auto kernel = waves == 8 ? matvec_kernel<BF16, SPARSE, LOG_GROUP, 8, FEW, YT>
                                 : matvec_kernel<BF16, SPARSE, LOG_GROUP, 16, FEW, YT>;
  if constexpr (FEW) {
    static const hipError_t attr8 = hipFuncSetAttribute(
        reinterpret_cast<const void*>(matvec_kernel<BF16, SPARSE, LOG_GROUP, 8, true, YT>),
        hipFuncAttributeMaxDynamicSharedMemorySize, (int)kFewLds);
    static const hipError_t attr16 = hipFuncSetAttribute(
        reinterpret_cast<const void*>(matvec_kernel<BF16, SPARSE, LOG_GROUP, 16, true, YT>),
        hipFuncAttributeMaxDynamicSharedMemorySize, (int)kFewLds);
    if (attr8 != hipSuccess) return attr8;
    if (attr16 != hipSuccess) return attr16;
  }
  kernel<<<groups, 64 * waves, lds, s>>>(a);
  return hipGetLastError();
}

template <bool BF16, bool SPARSE, int LOG_GROUP, int YT>
hipError_t launch_matvec_cols(const MatvecArgs& a, const MatvecPlan& p, hipStream_t s) {
  const int64_t whole = column_lds(a.R, a.K, a.T);
  if (whole) {
    const size_t lds = std::max((size_t)whole, (size_t)16 * 1024);
    return a.T == 1 ? launch_matvec_whole<BF16, SPARSE, LOG_GROUP, false, YT>(a, lds, s)
                    : launch_matvec_whole<BF16, SPARSE, LOG_GROUP, true, YT>(a, lds, s);
  }
  return p.nt == 1 ? launch_matvec_slices<BF16, SPARSE, LOG_GROUP, 1, YT>(a, p, s)
                   : launch_matvec_slices<BF16, SPARSE, LOG_GROUP, 2, YT>(a, p, s);
}

template <bool BF16, bool SPARSE, int LOG_GROUP>
hipError_t launch_matvec_y(const MatvecArgs& a, const MatvecPlan& p, int y_dt, hipStream_t s) {
  constexpr int kSame = BF16 ? kBF16 : kF16;
  return y_dt == kF32 ? launch_matvec_cols<BF16, SPARSE, LOG_GROUP, kF32>(a, p, s)
                      : launch_matvec_cols<BF16, SPARSE, LOG_GROUP, kSame>(a, p, s);
}

template <bool BF16, bool SPARSE>
hipError_t launch_matvec_group(const MatvecArgs& a, const MatvecPlan& p, int log_group, int y_dt,
                               hipStream_t s) {
  if (log_group == 5) return launch_matvec_y<BF16, SPARSE, 5>(a, p, y_dt, s);
  if (log_group == 6) return launch_matvec_y<BF16, SPARSE, 6>(a, p, y_dt, s);
  return launch_matvec_y<BF16, SPARSE, 7>(a, p, y_dt, s);
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
  const auto launch = [&](auto log_group) {
    constexpr int kLog = decltype(log_group)::value;
    if (blocked)
      quantize_kernel<DT, BF16S, true, true, kLog><<<grid, 256, 0, s>>>(w, R, C, S, blocks, c, sc);
    else if (C % 8 == 0)
      quantize_kernel<DT, BF16S, false, true, kLog><<<grid, 256, 0, s>>>(w, R, C, S, blocks, c, sc);
    else
      quantize_kernel<DT, BF16S, false, false, kLog><<<grid, 256, 0, s>>>(w, R, C, S, blocks, c, sc);
    return hipGetLastError();
  };
  if (group == 32) return launch(std::integral_constant<int, 5>{});
  if (group == 64) return launch(std::integral_constant<int, 6>{});
  return launch(std::integral_constant<int, 7>{});
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

bool matvec_fits(int64_t R, int64_t K, int64_t T, bool sparse) {
  return column_lds(R, K, T) || MatvecPlan(R, K, T, sparse).pieces < (int64_t)1 << 32;
}

size_t matvec_workspace_bytes(int64_t R, int64_t K, int64_t T, bool sparse) {
  return column_lds(R, K, T) ? 0 : (size_t)MatvecPlan(R, K, T, sparse).bytes;
}

hipError_t launch_matvec(const void* codes, const void* scales, const void* meta, int64_t R,
                         int64_t K, int group, const void* X, int64_t T, int dt, void* Y, int y_dt,
                         void* workspace, hipStream_t s) {
  const int64_t C = meta ? K / 2 : K;
  const MatvecPlan p(R, K, T, meta != nullptr);
  MatvecArgs a;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.meta = static_cast<const uint8_t*>(meta);
  a.x = static_cast<const uint16_t*>(X);
  a.y = Y;
  a.R = R;
  a.T = T;
  a.K = K;
  a.S = (int)((C + kBlockCols - 1) / kBlockCols);
  a.steps = (int)((C + 31) / 32);
  a.groups = (int)((C + group - 1) / group);
  a.slice = p.slice;
  a.log_along = p.log_along;
  a.part = static_cast<float4_t*>(workspace);
  const int lg = log2_of(group);
  if (dt == kBF16)
    return meta ? launch_matvec_group<true, true>(a, p, lg, y_dt, s)
                : launch_matvec_group<true, false>(a, p, lg, y_dt, s);
  return meta ? launch_matvec_group<false, true>(a, p, lg, y_dt, s)
              : launch_matvec_group<false, false>(a, p, lg, y_dt, s);
}

}  // namespace nm
