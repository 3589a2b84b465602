// nm_thin.hip -- nm_spmm_act for few tokens and small matrices (gfx950), 2:4, 1:2, 1:4 and 4:8, every type.
//
// The tiled kernels of nm_spmm.hip give a workgroup 128 rows or more and walk K in one barrier a
// step, so with few rows and columns most units have nothing to do and the rest wait.  Here a
// workgroup has 16 RG rows and 16 NT columns, and its eight waves take the steps of 64 K in turn, each
// with the next step's loads in flight, no barrier and no LDS until their sums are joined there in wave
// order.  Both operands come from memory as the structured-sparse instruction (v_smfmac_f32_16x16x64)
// wants them: the compressed rows as they lie, and X from a transposed copy in which a lane's K are
// contiguous, made by a first small launch; where few workgroups read X, they load its numbers one by
// one instead, and one column as it lies.  fp8 and int8 become bf16 exactly on the way (int8 sums are
// exact: fp32 holds 1024 K of products of up to 2^14, then they move to int32).  1:2 places become
// 2:4's by their bits, a 1:4 group a pair with a zero.  What the sparse instruction cannot have is
// expanded in registers: 4:8 for v_mfma_f32_16x16x32, fp32 for v_mfma_f32_16x16x4_f32.
//
// Bound by the first loads' latency on small matrices and by the reads of W on large ones: bf16, one
// column, 1024 x 4096 5.1 us, 4096 x 4096 6.2, 8192 x 4096 8.5 (4.4 TB/s of W; the tiled kernels take 41
// for the middle one); 1000 x 1024, 517 columns 9.4 and 4.1 for X's copy, against 53 in tiles; 4:8 2358 x 1856, 6 columns 7.4 against 40.
#include <algorithm>
#include <type_traits>

#include "nm_act.h"
#include "nm_launch.h"
#include "nm_tiles.h"

namespace nm {
namespace {

constexpr int kThinWaves = 8;
enum { kP24, kP12, kP14, kP48 };  // patterns

// ---- X, transposed -------------------------------------------------------------------

// v in 16 bits: as it is (16-bit types), exactly as bf16 (8-bit types).
template <int DT>
__device__ __forceinline__ uint32_t to_half(uint32_t raw) {
  if constexpr (DT == kI8) return f32_to_bf16((float)(int8_t)raw);
  else if constexpr (DT == kFP8) return f32_to_bf16(e4m3_to_f32(raw));
  else return raw;
}

template <int DT>
struct ThinElem {
  typedef std::conditional_t<DT == kF32, float, std::conditional_t<DT == kI8 || DT == kFP8, uint8_t,
                                                                   uint16_t>> type;
  typedef std::conditional_t<DT == kF32, uint32_t, uint16_t> turned;  // of X's copy
};

struct TurnArgs {
  const void* x;      // K x T
  int64_t K, T, Tp;   // Tp: columns with the zeros after them
  void* xt;           // Tp / 16 x K / 64 blocks of 16 columns x 64 K
};

// 64 x 64 of X a workgroup, through LDS.  A block of X's copy holds 16 columns and 64 K as the product's
// lanes read it, each load of a wave 1 KB in one run: piece i of lane 16 q + l, 16 bytes at
// 64 i + 16 q + l, has of column l the K 32 i + 8 q .. + 7, in fp32 16 q + 4 i .. + 3.
template <int DT>
__global__ void __launch_bounds__(256) turn_kernel(TurnArgs p) {
  typedef typename ThinElem<DT>::type E;
  typedef typename ThinElem<DT>::turned O;
  constexpr int kPer = 16 / sizeof(O), kPieces = 64 / kPer;  // of 16 bytes, a column
  __shared__ O tile[64][DT == kF32 ? 65 : 66];  // [column][k]
  const E* x = static_cast<const E*>(p.x);
  const int64_t k0 = (int64_t)blockIdx.x * 64, t0 = (int64_t)blockIdx.y * 64;
  const int c = threadIdx.x & 63, r = threadIdx.x >> 6;
  E in[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {  // (loads without conditions, or each would be waited for)
    const int64_t k = k0 + r + 4 * i;
    in[i] = x[min(k, p.K - 1) * p.T + min(t0 + c, p.T - 1)];
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (t0 + c >= p.T || k0 + r + 4 * i >= p.K) in[i] = E(0);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (DT == kF32) tile[c][r + 4 * i] = __float_as_uint(in[i]);
    else tile[c][r + 4 * i] = (uint16_t)to_half<DT>(in[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 64 * kPieces / 256; ++i) {
    const int at = i * 256 + threadIdx.x, b = at / (16 * kPieces), in_b = at % (16 * kPieces);
    const int piece = in_b >> 6, q = (in_b >> 4) & 3, col = 16 * b + (in_b & 15);
    const int k = DT == kF32 ? 16 * q + 4 * piece : 32 * piece + 8 * q;
    if (t0 + col >= p.Tp) continue;
    u32x4_t w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (DT == kF32) w[e] = tile[col][k + e];
      else w[e] = tile[col][k + 2 * e] | (uint32_t)tile[col][k + 2 * e + 1] << 16;
    }
    const int64_t block = (t0 / 16 + b) * ((p.K + 63) / 64) + blockIdx.x;
    static_cast<u32x4_t*>(p.xt)[block * (16 * kPieces) + in_b] = w;
  }
}

// ---- the product ---------------------------------------------------------------------------------

struct ThinArgs {
  const uint8_t* values;
  const uint8_t* meta;
  const void* xt;
  int64_t R, K, T, Tp;
  int64_t row_values, row_meta;  // of the row layout: values, bytes of metadata
  Epilogue ep;
};

// Sixteen K of a row as they lie: 8 values (1:4: 4) and their places.
template <int DT, int PAT>
struct ThinRaw {
  typedef typename ThinElem<DT>::type E;
  static __device__ __forceinline__ int values_at(int q) { return q * kBytes; }  // of the lane's, in bytes
  static __device__ __forceinline__ int places_at(int q) { return q * (PAT == kP24 ? 2 : 1); }
  static constexpr int kValues = PAT == kP14 ? 4 : 8;
  static constexpr int kBytes = kValues * (int)sizeof(E);
  uint32_t w[kBytes / 4];
  uint32_t places;

  // The row's values and places at any address, its sixteen K ending after `left` values (none or fewer
  // than kValues, whole groups; zeros at place 0 after them): the row layout where K is not whole steps.
  __device__ __forceinline__ void load_ragged(const uint8_t* v, const uint8_t* m, int64_t left) {
    typedef uint32_t one_t __attribute__((aligned(1)));
    typedef uint16_t half_t __attribute__((aligned(1)));
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) w[i] = 0u;
    places = 0u;
    if (left >= kValues) {
#pragma unroll
      for (int i = 0; i < kBytes / 4; ++i) w[i] = reinterpret_cast<const one_t*>(v)[i];
      places = PAT == kP24 ? *reinterpret_cast<const half_t*>(m) : *m;
    } else if (left > 0) {
#pragma unroll
      for (int i = 0; i < kValues; ++i) {
        if (i >= left) continue;
        if constexpr (sizeof(E) == 4) w[i] = reinterpret_cast<const one_t*>(v)[i];
        else if constexpr (sizeof(E) == 2) w[i / 2] |= (uint32_t)reinterpret_cast<const half_t*>(v)[i] << (16 * (i & 1));
        else w[i / 4] |= (uint32_t)v[i] << (8 * (i & 3));
      }
      places = *m;  // rows of metadata are whole words: a second byte only where values need it
      if (PAT == kP24 && left > 4) places |= (uint32_t)m[1] << 8;
    }
  }

  // values: the row's first of the sixteen K; places: their first byte
  __device__ __forceinline__ void load(const uint8_t* v, const uint8_t* m) {
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const u32x4_t x = reinterpret_cast<const u32x4_t*>(v)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = x[e];
      }
    } else if constexpr (kBytes == 8) {
      const u32x2_t x = *reinterpret_cast<const u32x2_t*>(v);
      w[0] = x[0];
      w[1] = x[1];
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(v);
    }
    places = PAT == kP24 ? *reinterpret_cast<const uint16_t*>(m) : *m;
  }

  __device__ __forceinline__ uint32_t raw(int i) const {
    if constexpr (sizeof(E) == 4) return w[i];
    else if constexpr (sizeof(E) == 2) return (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
    else return (w[i / 4] >> (8 * (i & 3))) & 0xFFu;
  }

  // The A operand of the sparse instruction and its index word.
  __device__ __forceinline__ u32x4_t operand(uint32_t& ix) const {
    if constexpr (PAT == kP24) {
      ix = places;
    } else if constexpr (PAT == kP12) {  // bit i -> bit 2 i; the second of a pair is in the upper half
      uint32_t x = places;
      x = (x | (x << 4)) & 0x0F0Fu;
      x = (x | (x << 2)) & 0x3333u;
      ix = ((x | (x << 1)) & 0x5555u) | 0x8888u;
    } else {  // (value, 0) at places 0 and 1, or (0, value) at 0 and the value's
      ix = 0;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t p = (places >> (2 * g)) & 3u;
        ix |= (p == 0 ? 4u : p << 2) << (4 * g);
      }
    }
    if constexpr (sizeof(E) == 2 && PAT != kP14) return u32x4_t{w[0], w[1], w[2], w[3]};
    u32x4_t a;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if constexpr (PAT == kP14)
        a[g] = to_half<DT>(raw(g)) << (((places >> (2 * g)) & 3u) == 0 ? 0 : 16);
      else
        a[g] = to_half<DT>(raw(2 * g)) | to_half<DT>(raw(2 * g + 1)) << 16;
    }
    return a;
  }

  // fp32: the sixteen numbers of the dense row.
  __device__ __forceinline__ void expand(float (&d)[16]) const {
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (PAT == kP24) {
          const uint32_t p = places >> (4 * g);
          const float lo = (p & 3u) == (uint32_t)k ? __uint_as_float(w[2 * g]) : 0.f;
          d[4 * g + k] = ((p >> 2) & 3u) == (uint32_t)k ? __uint_as_float(w[2 * g + 1]) : lo;
        } else if constexpr (PAT == kP12) {
          const int i = 2 * g + k / 2;
          d[4 * g + k] = ((places >> i) & 1u) == (uint32_t)(k & 1) ? __uint_as_float(w[i]) : 0.f;
        } else {
          d[4 * g + k] = ((places >> (2 * g)) & 3u) == (uint32_t)k ? __uint_as_float(w[g]) : 0.f;
        }
      }
  }
};

// 4:8: two groups, of 4 values and 12 bits each: a lane's numbers of the two dense products of a step,
// groups q and 4 + q of it, or in fp32 2 q and 2 q + 1, next to one another.
template <int DT>
struct ThinRaw<DT, kP48> {
  typedef typename ThinElem<DT>::type E;
  static constexpr bool kF = DT == kF32;
  static constexpr int kGroup = 4 * (int)sizeof(E), kFar = kF ? kGroup : 4 * kGroup;  // bytes
  uint32_t w[2][kGroup / 4];
  uint32_t places[2];
  static __device__ __forceinline__ int values_at(int q) { return q * (kF ? 2 * kGroup : kGroup); }
  static __device__ __forceinline__ int places_at(int q) { return kF ? 3 * q : 3 * q / 2; }

  template <bool RAGGED>
  __device__ __forceinline__ void load_groups(const uint8_t* v, const uint8_t* m, int q, int64_t left) {
    typedef uint32_t one_t __attribute__((aligned(1)));
    typedef uint16_t half_t __attribute__((aligned(1)));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint8_t* at = v + j * kFar;
#pragma unroll
      for (int i = 0; i < kGroup / 4; ++i) w[j][i] = 0u;
      places[j] = 0u;
      if (RAGGED && left <= (kF ? 8 * q + 4 * j : 16 * j + 4 * q)) continue;
      if constexpr (RAGGED || kGroup == 4) {
#pragma unroll
        for (int i = 0; i < kGroup / 4; ++i) w[j][i] = reinterpret_cast<const one_t*>(at)[i];
      } else if constexpr (kGroup == 8) {
        const u32x2_t x = *reinterpret_cast<const u32x2_t*>(at);
        w[j][0] = x[0];
        w[j][1] = x[1];
      } else {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(at);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[j][i] = x[i];
      }
      const int shift = kF ? 4 * j : 4 * (q & 1);
      places[j] = (uint32_t)*reinterpret_cast<const half_t*>(m + (kF ? j : 6 * j)) >> shift;
    }
  }
  __device__ __forceinline__ void load(const uint8_t* v, const uint8_t* m, int q) {
    load_groups<false>(v, m, q, 0);
  }
  // left: the row's values from this step on (whole groups)
  __device__ __forceinline__ void load_ragged(const uint8_t* v, const uint8_t* m, int q, int64_t left) {
    load_groups<true>(v, m, q, left);
  }

  __device__ __forceinline__ uint32_t raw(int j, int i) const {
    if constexpr (sizeof(E) == 4) return w[j][i];
    else if constexpr (sizeof(E) == 2) return (w[j][i / 2] >> (16 * (i & 1))) & 0xFFFFu;
    else return (w[j][0] >> (8 * i)) & 0xFFu;
  }
  // The eight numbers of group j.
  __device__ __forceinline__ u32x4_t dense(int j) const {
    u32x4_t d{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p = (places[j] >> (3 * i)) & 7u, v = to_half<DT>(raw(j, i)) << (16 * (p & 1u));
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] |= (p >> 1) == (uint32_t)k ? v : 0u;
    }
    return d;
  }
  __device__ __forceinline__ void expand(float (&d)[16]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x = ((places[j] >> (3 * i)) & 7u) == (uint32_t)k ? __uint_as_float(w[j][i]) : x;
        d[8 * j + k] = x;
      }
  }
};

template <bool F16>
__device__ __forceinline__ float4_t thin_smfmac(const u32x4_t& a, const u32x4_t& b0, const u32x4_t& b1,
                                                const float4_t& c, uint32_t ix) {
  typedef uint32_t u32x8_t __attribute__((ext_vector_type(8)));
  const u32x8_t b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
  if constexpr (F16)
    return __builtin_amdgcn_smfmac_f32_16x16x64_f16(__builtin_bit_cast(f16x8_t, a),
                                                    __builtin_bit_cast(f16x16_t, b), c, (int)ix, 0, 0);
  else
    return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                     __builtin_bit_cast(bf16x16_t, b), c, (int)ix, 0,
                                                     0);
}

template <bool F16>
__device__ __forceinline__ float4_t thin_mfma(const u32x4_t& a, const u32x4_t& b, const float4_t& c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// RAGGED: the row layout, K not in whole steps (X's copy ends in zeros).  DIRECT: xt is X itself, whose
// numbers are loaded one by one.  COLS = 0: one column, X as it lies, in each of the instruction's
// sixteen.
template <int DT, int PAT, bool BLOCKED, bool RAGGED, bool DIRECT, int RG, int COLS>
__global__ void __launch_bounds__(64 * kThinWaves) thin_kernel(ThinArgs p) {
  typedef typename ThinElem<DT>::type E;
  typedef ThinRaw<DT, PAT> Raw;
  constexpr bool kF = DT == kF32, kOne = COLS == 0;
  constexpr int NT = kOne ? 1 : COLS;
  constexpr int kRows = 16 * RG, kCols = 16 * NT;
  constexpr int kRowValues = PAT == kP14 ? 16 : 32, kRowMeta = PAT == kP48 ? 12 : PAT == kP24 ? 8 : 4;  // a row and step
  constexpr int kPitch = kCols + 4;  // of the sums in LDS
  __shared__ __attribute__((aligned(16))) float sums[kThinWaves][kRows * kPitch];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int steps = (int)((p.K + 63) / 64);
  static_assert(!(RAGGED && (BLOCKED || DIRECT)), "blocks are whole steps, a copy ends in zeros");
  const int64_t r0 = (int64_t)blockIdx.x * kRows, t0 = (int64_t)blockIdx.y * kCols;
  const int64_t groups = (p.R + 15) / 16;

  // this lane's rows (past the matrix: its last group or row again) and columns of X
  const uint8_t *v[RG], *m[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    if constexpr (BLOCKED) {
      const int64_t b = min(r0 / 16 + g, groups - 1);
      v[g] = p.values + (b * steps * 16 + l16) * kRowValues * (int64_t)sizeof(E) + Raw::values_at(q);
      m[g] = p.meta + (b * steps * 16 + l16) * kRowMeta + Raw::places_at(q);
    } else {
      const int64_t row = min(r0 + 16 * g + l16, p.R - 1);
      v[g] = p.values + row * p.row_values * (int64_t)sizeof(E) + Raw::values_at(q);
      m[g] = p.meta + row * p.row_meta + Raw::places_at(q);
    }
  }
  constexpr int kVStep = (BLOCKED ? 16 : 1) * kRowValues * (int)sizeof(E);
  constexpr int kMStep = (BLOCKED ? 16 : 1) * kRowMeta;
  constexpr int kPieces = kF ? 4 : 2;  // of X's copy to a lane, step and fragment
  const u32x4_t* x = static_cast<const u32x4_t*>(p.xt) + (t0 / 16 * steps) * (64 * kPieces) + lane;
  const E* column = static_cast<const E*>(p.xt);

  const auto one_column = [](const E* k, int q, int i) {  // piece i of the lane, as the copy has it
    if constexpr (kF) return *reinterpret_cast<const u32x4_t*>(k + 16 * q + 4 * i);
    else if constexpr (sizeof(E) == 2) return *reinterpret_cast<const u32x4_t*>(k + 32 * i + 8 * q);
    else {
      const u32x2_t raw = *reinterpret_cast<const u32x2_t*>(k + 32 * i + 8 * q);
      u32x4_t h;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        h[e] = to_half<DT>((raw[e / 2] >> (16 * (e & 1))) & 0xFFu) |
               to_half<DT>((raw[e / 2] >> (16 * (e & 1) + 8)) & 0xFFu) << 16;
      return h;
    }
  };
  // DIRECT: number e of the lane's piece i is in row kPieceRows i + e of the step, from the quarter's on;
  // columns past the last one are the last one again, and not stored
  constexpr int kEach = kF ? 4 : 8, kPieceRows = kF ? 4 : 32;
  uint32_t direct[NT];
  if constexpr (DIRECT) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      direct[t] = (uint32_t)((kF ? 16 : 8) * q * p.T + min(t0 + 16 * t + l16, p.T - 1));
  }
  struct Step {
    Raw a[RG];
    u32x4_t b[DIRECT ? 1 : NT][kPieces];
    uint32_t one[DIRECT ? NT : 1][DIRECT ? 16 : 1];
  };
  const auto piece = [&](const Step& f, int t, int i) {
    if constexpr (DIRECT) {
      u32x4_t w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (kF) w[e] = f.one[t][4 * i + e];
        else w[e] = to_half<DT>(f.one[t][8 * i + 2 * e]) | to_half<DT>(f.one[t][8 * i + 2 * e + 1]) << 16;
      }
      return w;
    } else {
      return f.b[t][i];
    }
  };
  const auto load = [&](Step& f, int s) {
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const uint8_t *va = v[g] + (int64_t)s * kVStep, *ma = m[g] + (int64_t)s * kMStep;
      if constexpr (PAT == kP48 && RAGGED) f.a[g].load_ragged(va, ma, q, p.row_values - 32 * (int64_t)s);
      else if constexpr (PAT == kP48) f.a[g].load(va, ma, q);
      else if constexpr (RAGGED) f.a[g].load_ragged(va, ma, p.row_values - (4 * (int64_t)s + q) * Raw::kValues);
      else f.a[g].load(va, ma);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (DIRECT) {
        const E* at = column + 64 * (int64_t)s * p.T;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            const E* row = at + (kPieceRows * i + e) * p.T;
            if constexpr (kF) f.one[t][kEach * i + e] = __float_as_uint(row[direct[t]]);
            else f.one[t][kEach * i + e] = row[direct[t]];
          }
      } else if constexpr (kOne) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) f.b[t][i] = one_column(column + 64 * (int64_t)s, q, i);
      } else {
        const u32x4_t* at = x + ((int64_t)t * steps + s) * (64 * kPieces);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) f.b[t][i] = at[64 * i];
      }
    }
  };
  float4_t acc[RG][NT];
  int4 whole[DT == kI8 ? RG : 1][DT == kI8 ? NT : 1];  // int8: exact totals
#pragma unroll
  for (int g = 0; g < RG; ++g)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      acc[g][t] = float4_t{0.f, 0.f, 0.f, 0.f};
      if constexpr (DT == kI8) whole[g][t] = int4{0, 0, 0, 0};
    }
  Step next;
  if (wave < steps) load(next, wave);
  int count = 0;
  for (int s = wave; s < steps; s += kThinWaves) {
    const Step cur = next;
    if (s + kThinWaves < steps) load(next, s + kThinWaves);
    u32x4_t b[NT][kPieces];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) b[t][i] = piece(cur, t, i);
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      if constexpr (kF) {
        float d[16];
        cur.a[g].expand(d);
#pragma unroll
        for (int k = 0; k < 16; ++k)  // K 16 q + k in lane quarter q
#pragma unroll
          for (int t = 0; t < NT; ++t)
            acc[g][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(d[k], __uint_as_float(b[t][k / 4][k % 4]),
                                                             acc[g][t], 0, 0, 0);
      } else if constexpr (PAT == kP48) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const u32x4_t a = cur.a[g].dense(i);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[g][t] = thin_mfma<DT == kF16>(a, b[t][i], acc[g][t]);
        }
      } else {
        uint32_t ix;
        const u32x4_t a = cur.a[g].operand(ix);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[g][t] = thin_smfmac<DT == kF16>(a, b[t][0], b[t][1], acc[g][t], ix);
      }
    }
    if constexpr (DT == kI8) {
      if ((++count & 15) == 0 || s + kThinWaves >= steps) {
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            whole[g][t].x += (int)acc[g][t][0];
            whole[g][t].y += (int)acc[g][t][1];
            whole[g][t].z += (int)acc[g][t][2];
            whole[g][t].w += (int)acc[g][t][3];
            acc[g][t] = float4_t{0.f, 0.f, 0.f, 0.f};
          }
      }
    }
  }

  // lane (l16, q) holds rows 4 q .. + 3 of column l16 of each fragment
#pragma unroll
  for (int g = 0; g < RG; ++g)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float* d = sums[wave] + (16 * g + 4 * q) * kPitch + 16 * t + l16;
      if constexpr (DT == kI8) {
        d[0] = __int_as_float(whole[g][t].x);
        d[kPitch] = __int_as_float(whole[g][t].y);
        d[2 * kPitch] = __int_as_float(whole[g][t].z);
        d[3 * kPitch] = __int_as_float(whole[g][t].w);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i * kPitch] = acc[g][t][i];
      }
    }
  const int row = threadIdx.x / (2 * NT), col = threadIdx.x % (2 * NT) * 8;
  const int64_t r = r0 + row, t = t0 + col;
  const bool mine = row < kRows && r < p.R && t < p.T;
  const int64_t i = r * p.T + t, left = p.T - t;
  RawEight residual{};
  float scale = 1.f, bias = 0.f;
  if (mine) {
    if (p.ep.residual) residual = load_eight(p.ep.residual, y_type<DT>(p.ep), i, left);
    if (p.ep.scale) scale = p.ep.scale[r];
    if (p.ep.bias) bias = p.ep.bias[r];
  }
  __syncthreads();
  if (!mine) return;
  float y[8];
  if constexpr (DT == kI8) {
    int n[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kThinWaves; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] += __float_as_int(sums[w][row * kPitch + col + e]);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (float)n[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kThinWaves; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] += sums[w][row * kPitch + col + e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(y[e], scale, bias);
  if constexpr (DT == kF32 || DT == kBF16 || DT == kF16)
    if (p.ep.z) store_eight(p.ep.z, DT, i, left, y);
  act_values(p.ep.act, y);
  if (p.ep.residual) {
    float add[8];
    to_floats(residual, y_type<DT>(p.ep), add);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] += add[e];
  }
  store_eight(p.ep.y, y_type<DT>(p.ep), i, left, y);
}

template <int DT, int PAT, bool BLOCKED, bool RAGGED, bool DIRECT>
hipError_t launch_cols(const ThinArgs& p, const ThinPlan& plan, hipStream_t s) {
  const auto go = [&](auto rg, auto nt) {
    constexpr int RG = decltype(rg)::value, NT = decltype(nt)::value;
    const unsigned cols = NT == 0 ? 1u : (unsigned)(plan.Tp / (16 * (NT == 0 ? 1 : NT)));
    const dim3 grid((unsigned)((p.R + 16 * RG - 1) / (16 * RG)), cols);
    thin_kernel<DT, PAT, BLOCKED, RAGGED, DIRECT && NT != 0, RG, NT><<<grid, 64 * kThinWaves, 0, s>>>(p);
    return hipGetLastError();
  };
  typedef std::integral_constant<int, 1> One;
  if constexpr (DIRECT)
    if (p.T == 1) return go(One{}, std::integral_constant<int, 0>{});
  typedef std::integral_constant<int, 2> Two;
  if (plan.nt == 1) return go(One{}, One{});
  if constexpr (!DIRECT && DT != kF32)
    if (plan.nt == 4) return go(Two{}, std::integral_constant<int, 4>{});
  return go(Two{}, Two{});
}

template <int DT>
hipError_t launch_thin_as(ThinArgs p, const ThinPlan& plan, int pat, bool blocked, const void* X,
                          void* xt, hipStream_t s) {
  if (plan.direct) {
    p.xt = X;
  } else {
    const TurnArgs turn{X, p.K, p.T, p.Tp, xt};
    turn_kernel<DT><<<dim3((unsigned)((p.K + 63) / 64), (unsigned)((p.Tp + 63) / 64)), 256, 0, s>>>(turn);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const auto go = [&](auto pattern) {
    constexpr int PAT = decltype(pattern)::value;
    if (plan.direct)
      return blocked ? launch_cols<DT, PAT, true, false, true>(p, plan, s)
                     : launch_cols<DT, PAT, false, false, true>(p, plan, s);
    if (blocked) return launch_cols<DT, PAT, true, false, false>(p, plan, s);
    if (p.K % 64 == 0) return launch_cols<DT, PAT, false, false, false>(p, plan, s);
    return launch_cols<DT, PAT, false, true, false>(p, plan, s);
  };
  if (pat == kP24) return go(std::integral_constant<int, kP24>{});
  if (pat == kP12) return go(std::integral_constant<int, kP12>{});
  if (pat == kP48) return go(std::integral_constant<int, kP48>{});
  return go(std::integral_constant<int, kP14>{});
}

}  // namespace

hipError_t launch_thin(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n, int m,
                       bool blocked, const void* X, int64_t T, int dt, const Product& product,
                       void* workspace, hipStream_t s) {
  const ThinPlan plan(R, K, T, m, dt == kF32);
  void* xt = workspace;
  const ThinArgs p{static_cast<const uint8_t*>(values), reinterpret_cast<const uint8_t*>(meta), xt, R,
                   K, T, plan.Tp, K / m * n, ((K / m * n) * (m == 2 ? 1 : m == 4 ? 2 : 3) + 31) / 32 * 4,
                   epilogue_of(product)};
  const int pat = m == 8 ? kP48 : m == 2 ? kP12 : n == 2 ? kP24 : kP14;
  if (dt == kBF16) return launch_thin_as<kBF16>(p, plan, pat, blocked, X, xt, s);
  if (dt == kF16) return launch_thin_as<kF16>(p, plan, pat, blocked, X, xt, s);
  if (dt == kF32) return launch_thin_as<kF32>(p, plan, pat, blocked, X, xt, s);
  if (dt == kI8) return launch_thin_as<kI8>(p, plan, pat, blocked, X, xt, s);
  return launch_thin_as<kFP8>(p, plan, pat, blocked, X, xt, s);
}

}  // namespace nm
