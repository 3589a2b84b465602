// nm_orth.hip -- the orthogonalised update of a weight matrix (nm_orthogonalize): a fixed
// number of Newton-Schulz steps on X = G / (|G|_F + eps),
//   A = X X^T,   B = b A + c A A,   X <- a X + B X,
// on the shorter side of G (X^T X and X B when G is taller than wide), which bring the singular
// values of X near 1 and keep its singular vectors.  Every product is a dense product on the
// matrix cores (nm_gemm.h); A, B and the sums' scaling live in the epilogues.
//
// Numbers.  The matrix cores' operands are fp16, not bf16: X, A and B have singular values of
// at most about 3, so the wide exponent of bf16 buys nothing and its 8 bits cost a percent of
// the result.  All three are held times 2^8, which keeps entries of 2^-22 in fp16's normal
// range.  G itself is only scaled by a power of two (exact for bf16); the rest of its norm, a
// factor in fp32, goes into the first step's epilogues.  Where eps makes X far smaller than 1, each
// step multiplies it by about a until it is near 1; the X that is stored is kept at its first size
// meanwhile and a factor is carried beside it, since fp16 would lose it.  A is stored as it is: what
// it loses below 2^-33 is nothing beside the a of a X.
//   bf16 G: operands are one fp16, and the X that a X is formed from has the next four bits
//     beside it (one fp8 an entry): without them the small singular values lose most.
//   fp16 and fp32 G: each operand is two fp16, hi + lo (22 bits), and a product is hi hi +
//     hi lo + lo hi in the same accumulators, as exact as fp32 products.
// The norm is summed in fp64, so no finite G overflows or vanishes in it.
//
// Bound by the matrix cores on large G: a step of 4096 x 11008 in bf16 is 191 us of X X^T (970
// TFLOP/s of the half that is computed), 79 of A A and 356 of the update (1040; its 688 tiles are
// three rounds of 256 units for 2.7).  On small G by the chain of 3 launches a step: 256 x 384 takes
// 4.8 to 5.7 us for each, of which a launch after another is 1.6 and the rest one tile's latency.
#include <algorithm>
#include <cmath>

#include "nm_gemm.h"
#include "nm_tiles.h"

namespace nm {
namespace {

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

constexpr int kNormBlocks = 1024;
constexpr float kOrthScale = 256.f;
constexpr int kMaxSteps = 100;
constexpr float kCoefA = 3.4445f, kCoefB = -4.7750f, kCoefC = 2.0315f;

struct OrthHead {  // first bytes of the workspace
  double partial[kNormBlocks];
  float size[kMaxSteps];  // X of a step is `size` times the stored one
  float grow[kMaxSteps];  // this step's size over the next one's (1 for the result)
};

template <int DT>
__device__ __forceinline__ float load_f32(const void* p, int64_t i) {
  if constexpr (DT == kF32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == kF16) return f16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// Sums of squares in fp64 (exact squares of 16-bit numbers; the accumulation costs nothing beside
// the reads), 16 bytes a lane at a time.
template <int DT>
__global__ void __launch_bounds__(256) norm_kernel(const void* __restrict__ G, int64_t n,
                                                   OrthHead* head) {
  constexpr int kPer = DT == kF32 ? 4 : 8;
  __shared__ double part[4];
  double sum = 0;
  const int64_t whole = n / kPer, stride = (int64_t)gridDim.x * 256;
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
#pragma unroll 4
  for (int64_t i = first; i < whole; i += stride) {
    const u32x4_t v = static_cast<const u32x4_t*>(G)[i];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      double x;
      if constexpr (DT == kF32) x = __uint_as_float(v[e]);
      else if constexpr (DT == kF16) x = f16_to_f32((v[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
      else x = bf16_to_f32((v[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
      sum += x * x;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < n - whole * kPer) {
    const double x = load_f32<DT>(G, whole * kPer + threadIdx.x);
    sum += x * x;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) head->partial[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
  // one block may stand for several places that start_kernel adds
  for (int i = gridDim.x + blockIdx.x; threadIdx.x == 0 && i < kNormBlocks; i += gridDim.x)
    head->partial[i] = 0;
}

// X' = G 2^k (rp x kp, zeros past R x K) with 2^k |G|_F in (2^7, 2^8].
template <int DT, bool SPLIT>
__global__ void __launch_bounds__(256)
    start_kernel(const void* __restrict__ G, int64_t R, int64_t K, int64_t rp, int64_t kp, float eps,
                 int steps, OrthHead* head, _Float16* __restrict__ hi, _Float16* __restrict__ lo) {
  __shared__ double part[4];
  double sum = 0;
#pragma unroll
  for (int i = 0; i < kNormBlocks; i += 256) sum += head->partial[threadIdx.x + i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double norm = sqrt(part[0] + part[1] + part[2] + part[3]);
  int e = 0;
  if (norm > 0 && norm < INFINITY) frexp(norm, &e);  // norm = f 2^e, f in [1/2, 1)
  const int k = 8 - e;
  if (blockIdx.x == 0 && (int)threadIdx.x < steps) {  // a thread a step
    const int i = threadIdx.x;
    const auto after = [](double size) { return size > 0 ? fmin(1.0, size * kCoefA) : 1.0; };
    double size = norm > 0 ? ldexp(256.0, -k) / (norm + (double)eps) : 1.0;
    for (int j = 0; j < i && size != 1.0; ++j) size = after(size);
    head->size[i] = (float)size;
    head->grow[i] = (float)(i + 1 < steps ? size / after(size) : size);
  }
  const int64_t total = rp * kp / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = 4 * i / kp, c = 4 * i % kp;
    _Float16 h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = r < R && c + j < K ? ldexpf(load_f32<DT>(G, r * K + c + j), k) : 0.f;
      h[j] = (_Float16)x;
      l[j] = (_Float16)(x - (float)h[j]);
    }
    *reinterpret_cast<half4_t*>(hi + 4 * i) = half4_t{h[0], h[1], h[2], h[3]};
    if constexpr (SPLIT) *reinterpret_cast<half4_t*>(lo + 4 * i) = half4_t{l[0], l[1], l[2], l[3]};
  }
}

enum OrthKind { kGram, kSquare, kUpdate };

struct OrthArgs {
  GemmOperand a, b;
  int steps;
  GemmMap map;
  int64_t rows, cols;  // of the result, whole multiples of 64; its rows are `cols` apart
  const float *size, *grow;    // the step's (OrthHead)
  const _Float16 *from_hi, *from_lo;  // square: A; update: the X before
  _Float16 *hi, *lo;           // result (lo only with two parts)
  uint8_t* rest;               // one part: what hi lacks of X in fp8
  bool from_rest;              // whether the X before has any
  void* out;                   // the last update: the caller's result (R x K), else null
  int out_dt;
  int64_t R, K;
};


__device__ __forceinline__ float4_t widen(half4_t h) {
  return float4_t{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
}

// What fp16 lacks of a number, as fp8 (E4M3) times 2^10: at most 2^7 there, and seen down to 2^-19
// of the scaled X, whose entries are around 1.
[[maybe_unused]] constexpr float kRestScale = 1024.f;
__device__ __forceinline__ uint32_t pack_rest(float4_t r) {
  int w = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  w = __builtin_amdgcn_cvt_pk_fp8_f32(r[0] * kRestScale, r[1] * kRestScale, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(r[2] * kRestScale, r[3] * kRestScale, w, true);
#endif
  return (uint32_t)w;
}
__device__ __forceinline__ float4_t unpack_rest(uint32_t w) {
#if defined(__HIP_DEVICE_COMPILE__)
  const float2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const float2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return float4_t{a[0], a[1], b[0], b[1]} * (1.f / kRestScale);
#else
  return float4_t{};
#endif
}

// The epilogue works on 32 rows of a wave's part of the tile at a time, which pass through LDS in
// both directions, so that device memory sees 16-byte pieces of whole lines: as the lanes hold
// them, 8 bytes in each of 32 rows, they take four times the requests (4096 x 11008, one update:
// 445 us so, 392 staged).
template <class G, int KIND, bool SPLIT>
struct OrthEpilogue {
  static constexpr int kFN = G::kFN, kCols = 32 * kFN;
  static constexpr bool kReads = KIND != kGram, kMirrors = KIND != kUpdate;
  static constexpr bool kRest = KIND == kUpdate && !SPLIT;
  static constexpr bool kSecond = SPLIT || kRest;         // a second plane: lo or rest
  static constexpr int kSecondBytes = SPLIT ? 2 : 1;      // of an entry of it
  static constexpr int kPieces = 2 * kFN, kSecondPieces = kSecondBytes * kFN;  // a lane
  static constexpr int kPitch = 2 * kCols + 16, kSecondPitch = kSecondBytes * kCols + 16;
  static constexpr int kTurned = 64 + 16;                 // pitch of 32 rows of a column
  static constexpr int kSecondAt = 32 * kPitch;
  static constexpr int kTurnedAt = kSecondAt + (kSecond ? 32 * kSecondPitch : 0);
  static constexpr int kWaveBytes = kTurnedAt + (kMirrors ? (SPLIT ? 2 : 1) * kCols * kTurned : 0);
  static_assert(G::kWaves * kWaveBytes <= G::kLds, "the waves' parts fit");

  // What is read of A (square) or of the X before (update).
  struct Before {
    u32x4_t first[kPieces], second[kSecondPieces];
  };

  const OrthArgs& p;
  uint8_t* mine;
  int lane;
  int64_t row, col;  // of the wave's part
  float factor;      // size of X (gram), its growth (update)
  bool mirror;

  // f(k, row, column, 16-byte column) for each 16-byte piece of the lane in a plane of BYTES an
  // entry that lies in the result.
  template <int BYTES, typename F>
  __device__ __forceinline__ void pieces(int i, int64_t rows, int64_t cols, F f) const {
    constexpr int kRow = BYTES * kCols / 16;
#pragma unroll
    for (int k = 0; k < BYTES * kFN; ++k) {
      const int at = k * 64 + lane, r = at / kRow, c = at % kRow;
      if (row + 32 * i + r < rows && col + c * (16 / BYTES) < cols)
        f(k, row + 32 * i + r, col + c * (16 / BYTES), r, 16 * c);
    }
  }

  __device__ __forceinline__ void load(int i, Before& b) const {
    if constexpr (kReads) {
      pieces<2>(i, p.rows, p.cols, [&](int k, int64_t r, int64_t c, int, int) {
        b.first[k] = *reinterpret_cast<const u32x4_t*>(p.from_hi + r * p.cols + c);
      });
      if constexpr (SPLIT)
        pieces<2>(i, p.rows, p.cols, [&](int k, int64_t r, int64_t c, int, int) {
          b.second[k] = *reinterpret_cast<const u32x4_t*>(p.from_lo + r * p.cols + c);
        });
      else if constexpr (kRest)
        if (p.from_rest)
          pieces<1>(i, p.rows, p.cols, [&](int k, int64_t r, int64_t c, int, int) {
            b.second[k] = *reinterpret_cast<const u32x4_t*>(p.rest + r * p.cols + c);
          });
    }
  }

  __device__ __forceinline__ void store(int i, const typename G::Acc& acc, const Before& b) const {
    uint8_t* const first = mine;
    uint8_t* const second = mine + kSecondAt;
    uint8_t* const turned = mine + kTurnedAt;
    if constexpr (kReads) {
      pieces<2>(i, p.rows, p.cols, [&](int k, int64_t, int64_t, int r, int c) {
        *reinterpret_cast<u32x4_t*>(first + r * kPitch + c) = b.first[k];
      });
      if constexpr (kSecond)
        pieces<kSecondBytes>(i, p.rows, p.cols, [&](int k, int64_t, int64_t, int r, int c) {
          *reinterpret_cast<u32x4_t*>(second + r * kSecondPitch + c) = b.second[k];
        });
    }
    keep_lds_order();
    const bool last = KIND == kUpdate && p.out;
    const bool staged = !last || p.out_dt != kF32;
#pragma unroll
    for (int q = 0; q < 4 * kFN; ++q) {
      const float4_t v = G::quad(acc, i, q / 4, q % 4);
      const int r = lane & 31, c = 32 * (q / 4) + 8 * (q % 4) + 4 * (lane >> 5);
      half4_t* const at = reinterpret_cast<half4_t*>(first + r * kPitch + 2 * c);
      uint8_t* const at2 = second + r * kSecondPitch + kSecondBytes * c;
      float4_t y;
      if constexpr (KIND == kGram) {
        y = v * (factor * factor / kOrthScale);
      } else {
        float4_t x = widen(*at);
        if constexpr (SPLIT) x += widen(*reinterpret_cast<const half4_t*>(at2));
        else if (kRest && p.from_rest) x += unpack_rest(*reinterpret_cast<const uint32_t*>(at2));
        if constexpr (KIND == kSquare) y = kCoefB * x + (kCoefC / kOrthScale) * v;
        else y = factor * (kCoefA * x + (1.f / kOrthScale) * v);
      }
      if (last) {
        y *= 1.f / kOrthScale;
        if (staged) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = p.out_dt == kF16 ? f32_to_f16(y[e]) : f32_to_bf16(y[e]);
          *reinterpret_cast<u32x2_t*>(at) = u32x2_t{h[0] | h[1] << 16, h[2] | h[3] << 16};
          continue;
        }
        const int64_t to_row = row + 32 * i + r, to = to_row * p.K + col + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (to_row < p.R && col + c + e < p.K) store_from_f32<kF32>(p.out, to + e, y[e]);
        continue;
      }
      half4_t h, l;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = (_Float16)y[e];
        l[e] = (_Float16)(y[e] - (float)h[e]);
      }
      *at = h;
      if constexpr (SPLIT) *reinterpret_cast<half4_t*>(at2) = l;
      else if constexpr (kRest) *reinterpret_cast<uint32_t*>(at2) = pack_rest(y - widen(h));
      if (kMirrors && mirror) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          *reinterpret_cast<_Float16*>(turned + (c + e) * kTurned + 2 * r) = h[e];
          if constexpr (SPLIT)
            *reinterpret_cast<_Float16*>(turned + (kCols + c + e) * kTurned + 2 * r) = l[e];
        }
      }
    }
    keep_lds_order();
    if (!staged) return;
    if (last) {
      pieces<2>(i, p.R, p.K, [&](int, int64_t r, int64_t c, int lr, int lc) {
        store_piece(static_cast<uint16_t*>(p.out) + r * p.K + c, first + lr * kPitch + lc, p.K - c);
      });
      return;
    }
    pieces<2>(i, p.rows, p.cols, [&](int, int64_t r, int64_t c, int lr, int lc) {
      *reinterpret_cast<u32x4_t*>(p.hi + r * p.cols + c) =
          *reinterpret_cast<const u32x4_t*>(first + lr * kPitch + lc);
    });
    if constexpr (kSecond)
      pieces<kSecondBytes>(i, p.rows, p.cols, [&](int, int64_t r, int64_t c, int lr, int lc) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(second + lr * kSecondPitch + lc);
        if constexpr (SPLIT) *reinterpret_cast<u32x4_t*>(p.lo + r * p.cols + c) = v;
        else *reinterpret_cast<u32x4_t*>(p.rest + r * p.cols + c) = v;
      });
    if (kMirrors && mirror) {  // the same numbers above the diagonal, 32 of a row
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = (k * 64 + lane) / 4, r = (k * 64 + lane) % 4 * 8;
        if (col + c >= p.cols || row + 32 * i + r >= p.rows) continue;
        const int64_t to = (col + c) * p.cols + row + 32 * i + r;
        *reinterpret_cast<u32x4_t*>(p.hi + to) =
            *reinterpret_cast<const u32x4_t*>(turned + c * kTurned + 2 * r);
        if constexpr (SPLIT)
          *reinterpret_cast<u32x4_t*>(p.lo + to) =
              *reinterpret_cast<const u32x4_t*>(turned + (kCols + c) * kTurned + 2 * r);
      }
    }
  }
};

template <class G, int KIND, bool SPLIT>
__global__ void __launch_bounds__(G::kThreads) orth_kernel(OrthArgs p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  typedef OrthEpilogue<G, KIND, SPLIT> Epilogue;
  int tm, tn;
  if (!p.map.tile_of(blockIdx.x, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * G::kBM, n0 = (int64_t)tn * G::kBN;
  const int wave = threadIdx.x >> 6;
  const Epilogue epilogue{p, smem + wave * Epilogue::kWaveBytes, (int)threadIdx.x & 63,
                          m0 + wave / G::kWN * 32 * G::kFM, n0 + wave % G::kWN * 32 * G::kFN,
                          KIND == kGram ? *p.size : KIND == kUpdate ? *p.grow : 1.f, tm != tn};
  // A small tile's epilogue reads come ahead of its few steps, a large one's 32 rows ahead.
  constexpr bool kEarly = G::kFM == 1;
  typename Epilogue::Before before[2];
  if constexpr (kEarly) epilogue.load(0, before[0]);
  typename G::Acc acc;
  G::clear(acc);
  G::run(p.a, p.b, m0, n0, p.steps, (int64_t)p.steps * kGemmStep, smem, acc);
  if constexpr (!kEarly) epilogue.load(0, before[0]);
#pragma unroll
  for (int i = 0; i < G::kFM; ++i) {
    if (i + 1 < G::kFM) epilogue.load(i + 1, before[(i + 1) & 1]);
    epilogue.store(i, acc, before[i & 1]);
    keep_lds_order();
  }
}

template <class G, int KIND, bool SPLIT>
hipError_t launch_orth_tile(OrthArgs p, hipStream_t s) {
  // A and B are symmetric: their tiles above the diagonal are written by those below it
  p.map = make_gemm_map((p.rows + G::kBM - 1) / G::kBM, (p.cols + G::kBN - 1) / G::kBN, KIND != kUpdate);
  return G::template launch<orth_kernel<G, KIND, SPLIT>>(p, p.map.groups(), 1, s);
}

template <int KIND, bool AS, bool BS, bool SPLIT>
hipError_t launch_orth_product(const OrthArgs& p, hipStream_t s) {
  constexpr bool kLower = KIND != kUpdate;
  if constexpr (SPLIT) {
    const int tile = pick_orth_tile(kOrthSplitTiles, p.rows, p.cols, p.steps, kLower);
    if (tile == 128)
      return launch_orth_tile<Gemm<2, 4, 2, 1, AS, BS, false, true, 2, 2>, KIND, true>(p, s);
    return launch_orth_tile<Gemm<2, 2, 1, 1, AS, BS, false, true, 4, 2>, KIND, true>(p, s);
  } else {
    const int tile = pick_orth_tile(kOrthTiles, p.rows, p.cols, p.steps, kLower);
    if (tile == 256)
      return launch_orth_tile<Gemm<2, 4, 4, 2, AS, BS, false, true, 2>, KIND, false>(p, s);
    if (tile == 192)
      return launch_orth_tile<Gemm<2, 6, 3, 1, AS, BS, false, true, 3>, KIND, false>(p, s);
    if (tile == 128)
      return launch_orth_tile<Gemm<2, 4, 2, 1, AS, BS, false, true, 4>, KIND, false>(p, s);
    return launch_orth_tile<Gemm<2, 2, 1, 1, AS, BS, false, true, 4>, KIND, false>(p, s);
  }
}

// Workspace parts, in bytes.
struct OrthLayout {
  int64_t rp, kp, mp;  // padded sizes; mp: the shorter side
  bool tall, split;
  int64_t x_part, a_part;       // elements of one fp16 part
  int64_t head, x, rest, a, b, total;
  OrthLayout(int64_t R, int64_t K, int dt) {
    rp = pad64(R);
    kp = pad64(K);
    tall = R > K;
    mp = tall ? kp : rp;
    split = dt != kBF16;
    x_part = rp * kp;
    a_part = mp * mp;
    const int64_t parts = split ? 2 : 1;
    head = 0;
    x = (int64_t)((sizeof(OrthHead) + 255) / 256 * 256);
    rest = x + 2 * parts * x_part * 2;  // after two buffers of X
    a = rest + (split ? 0 : x_part);
    b = a + parts * a_part * 2;
    total = b + parts * a_part * 2;
  }
};

template <bool SPLIT>
hipError_t run_orth(const void* G, int dt, int64_t R, int64_t K, int steps, float eps, void* out,
                    uint8_t* ws, const OrthLayout& L, hipStream_t s) {
  OrthHead* head = reinterpret_cast<OrthHead*>(ws);
  _Float16* x[2];
  x[0] = reinterpret_cast<_Float16*>(ws + L.x);
  x[1] = x[0] + (SPLIT ? 2 : 1) * L.x_part;
  _Float16* A = reinterpret_cast<_Float16*>(ws + L.a);
  _Float16* B = reinterpret_cast<_Float16*>(ws + L.b);
  const int64_t x_lo = SPLIT ? L.x_part : 0, a_lo = SPLIT ? L.a_part : 0;

  const int64_t n = R * K;
  const unsigned blocks = (unsigned)std::min<int64_t>(kNormBlocks, (n + 2047) / 2048);
  if (dt == kF32) norm_kernel<kF32><<<blocks, 256, 0, s>>>(G, n, head);
  else if (dt == kF16) norm_kernel<kF16><<<blocks, 256, 0, s>>>(G, n, head);
  else norm_kernel<kBF16><<<blocks, 256, 0, s>>>(G, n, head);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t quads = L.rp * L.kp / 4;
  const unsigned grid = (unsigned)(quads / 256 < 2048 ? (quads + 255) / 256 : 2048);
  if (dt == kF32)
    start_kernel<kF32, SPLIT><<<grid, 256, 0, s>>>(G, R, K, L.rp, L.kp, eps, steps, head, x[0],
                                                     x[0] + x_lo);
  else if (dt == kF16)
    start_kernel<kF16, SPLIT><<<grid, 256, 0, s>>>(G, R, K, L.rp, L.kp, eps, steps, head, x[0],
                                                     x[0] + x_lo);
  else
    start_kernel<kBF16, SPLIT><<<grid, 256, 0, s>>>(G, R, K, L.rp, L.kp, eps, steps, head, x[0],
                                                     x[0] + x_lo);
  if ((e = hipGetLastError()) != hipSuccess) return e;

  auto op = [](const _Float16* p, int64_t ld, int64_t rows, int64_t lo) {
    return GemmOperand{reinterpret_cast<const uint16_t*>(p), ld, rows, lo};
  };
  for (int i = 0; i < steps; ++i) {
    const _Float16* from = x[i & 1];
    OrthArgs p{};
    p.size = &head->size[i];
    p.grow = &head->grow[i];
    // A = X X^T, or X^T X (both operands then have k as their row index)
    p.a = p.b = op(from, L.kp, L.mp, x_lo);
    p.steps = (int)((L.tall ? L.rp : L.kp) / kGemmStep);
    p.rows = p.cols = L.mp;
    p.hi = A;
    p.lo = A + a_lo;
    e = L.tall ? launch_orth_product<kGram, true, true, SPLIT>(p, s)
               : launch_orth_product<kGram, false, false, SPLIT>(p, s);
    if (e != hipSuccess) return e;
    // B = b A + c A A (A is symmetric: its rows are its columns)
    p.a = p.b = op(A, L.mp, L.mp, a_lo);
    p.steps = (int)(L.mp / kGemmStep);
    p.from_hi = A;
    p.from_lo = A + a_lo;
    p.hi = B;
    p.lo = B + a_lo;
    if ((e = launch_orth_product<kSquare, false, false, SPLIT>(p, s)) != hipSuccess) return e;
    // X <- a X + B X, or a X + X B
    p.rows = L.rp;
    p.cols = L.kp;
    p.from_hi = from;
    p.from_lo = from + x_lo;
    p.rest = ws + L.rest;
    p.from_rest = i > 0;
    p.hi = x[(i + 1) & 1];
    p.lo = p.hi + x_lo;
    if (i + 1 == steps) {
      p.out = out;
      p.out_dt = dt;
      p.R = R;
      p.K = K;
    }
    if (L.tall) {
      p.a = op(from, L.kp, L.rp, x_lo);
      p.b = op(B, L.mp, L.mp, a_lo);
      e = launch_orth_product<kUpdate, false, false, SPLIT>(p, s);
    } else {
      p.a = op(B, L.mp, L.mp, a_lo);
      p.b = op(from, L.kp, L.kp, x_lo);
      e = launch_orth_product<kUpdate, false, true, SPLIT>(p, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t orth_workspace_bytes(int64_t R, int64_t K, int dt) {
  return (size_t)OrthLayout(R, K, dt).total;
}

hipError_t launch_orthogonalize(const void* G, int dt, int64_t R, int64_t K, int steps, float eps,
                                void* out, void* workspace, hipStream_t s) {
  const OrthLayout L(R, K, dt);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return L.split ? run_orth<true>(G, dt, R, K, steps, eps, out, ws, L, s)
                 : run_orth<false>(G, dt, R, K, steps, eps, out, ws, L, s);
}

}  // namespace nm
