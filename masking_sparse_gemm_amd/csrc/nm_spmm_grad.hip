// nm_spmm_grad.hip -- what nm_spmm_act needs around its product (rows of X made whole 16-byte
// pieces), and its gradient (nm_spmm_act_grad).
//
//   dZ = act'(Z) dY,   dbias[r] = sum over t of dZ[r, t],   dW = dZ X^T,   dX = W^T dZ
//
// dZ is one pass over Z and dY that also adds up its rows (bound by memory).  It leaves in 16 bits,
// as the operand of the other two: where the sizes are not whole multiples of 64 into a padded copy,
// and not at all where there is no activation and the sizes are whole.  That rounding is the same
// relative size as those of dW and dX themselves, and the matrix cores take no wider operand: two parts
// of 16 bits would double both products' time, to take dW's and dX's error against 64 bits from 2.3e-3 to
// 1.7e-3 in bf16 and from 2.9e-4 to 2.1e-4 in fp16, which is what their own rounding leaves.
//
// fp16's range is too short for it: a slope far below 1 on a dY near 2^-24 would leave nothing, and relu's
// square passes 65504.  So there, where a slope changes dY (all but none and relu), each product has its
// own copy of dZ over a power of two: dW of the row, dX of the column, whose largest finite dY (relu's
// square: dZ) then lies in 2^14 .. 2^15, and the fp32 sums are brought back before they are rounded.  What
// is below 2^-28 of that largest loses bits, what is below 2^-39 of it is lost.  The columns' largest take
// a pass of their own; the rows' are taken where the copies are written.  dW is the gradient of the
// dense weight, as SR-STE takes it.  W^T has no structure that the sparse instruction could use (W's
// groups run along its rows), so W is decompressed and both products are dense (nm_gemm.h).
//
// What the products need (dZ, X and W in whole steps) goes out in one launch where W is small, and both
// products in one, dX's long sums first: alone, each leaves units idle at its end (1000 x 768, 333
// columns: 30 us a call in launches of their own, 21 so).
//
// Bound by the matrix cores where matrices are large: bf16 11008 x 4096, 2048 columns, dZ 26 us and W 24.5,
// both at the memory's rate, the products 314 in a replayed graph (1180 TFLOP/s; a library's product of
// 8192^3 on the same card 1199) and 350 under a profiler.  By load latency and launches where they are
// small: 6.8 and 10.0 us for 1000 x 768, 333 columns, in fp16 with a smooth activation 6.2, 8.2 and 10.1.
#include <algorithm>

#include "nm_act.h"
#include "nm_gemm.h"
#include "nm_grid.h"
#include "nm_tiles.h"

namespace nm {
namespace {

int64_t whole256(int64_t n) { return (n + 255) / 256 * 256; }

// ---- rows made longer, with zeros --------------------------------------------------------------

struct WidenArgs {
  const uint8_t* in;  // rows x width elements
  uint8_t* out;       // out_rows x out_width, rows of whole 16-byte pieces
  int64_t rows, width, out_rows, out_width;
};

typedef uint32_t u32x4_byte_t __attribute__((ext_vector_type(4), aligned(1)));

// E: an element's storage.  A thread a 16-byte piece of the output.
template <typename E>
__device__ __forceinline__ void widen_pieces(const WidenArgs& p, int64_t first, int64_t stride) {
  constexpr int kPer = 16 / sizeof(E);
  const int64_t pieces = p.out_width / kPer, total = p.out_rows * pieces;
  for (int64_t i = first; i < total; i += stride) {
    const int64_t r = i / pieces, c = i % pieces * kPer;
    u32x4_t v{0, 0, 0, 0};
    if (r < p.rows && c < p.width) {
      const E* x = reinterpret_cast<const E*>(p.in) + r * p.width + c;
      if (c + kPer <= p.width) {
        v = *reinterpret_cast<const u32x4_byte_t*>(x);
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          constexpr int kBits = 8 * sizeof(E), kIn = 32 / kBits;
          if (c + e < p.width) v[e / kIn] |= (uint32_t)x[e] << (kBits * (e % kIn));
        }
      }
    }
    reinterpret_cast<u32x4_t*>(p.out)[i] = v;
  }
}
template <typename E>
__global__ void __launch_bounds__(256) widen_kernel(WidenArgs p) {
  widen_pieces<E>(p, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

hipError_t widen(const void* in, int64_t rows, int64_t width, void* out, int64_t out_rows,
                 int64_t out_width, int elem, hipStream_t s) {
  const WidenArgs p{static_cast<const uint8_t*>(in), static_cast<uint8_t*>(out), rows, width,
                    out_rows, out_width};
  const int64_t pieces = out_rows * out_width * elem / 16;
  if (pieces == 0) return hipSuccess;
  const unsigned grid = stride_grid(pieces, 256);
  if (elem == 1) widen_kernel<uint8_t><<<grid, 256, 0, s>>>(p);
  else if (elem == 2) widen_kernel<uint16_t><<<grid, 256, 0, s>>>(p);
  else widen_kernel<uint32_t><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

int elem_of(int dt) { return dt == kF32 ? 4 : dt == kI8 || dt == kFP8 ? 1 : 2; }
int64_t whole_row(int64_t T, int dt) {
  const int64_t per = 16 / elem_of(dt);
  return (T + per - 1) / per * per;
}

// ---- dZ ----------------------------------------------------------------------------------------

struct SlopeArgs {
  const void *z, *dy;  // R x T; z null without an activation
  int64_t R, T;
  int act;
  uint16_t* padded;    // Rp x Tp with zeros, or null
  int64_t Rp, Tp;
  uint16_t* dz;        // R x T, or null
  float* dbias;        // R, or null
  // of the scaled copies alone: padded is dW's (or null), over row_back, which is written here
  uint16_t* padded_x;     // dX's, over col_back, or null
  float* row_back;        // R
  const float* col_back;  // Tp
};

// What brings numbers back that leave with `most` in 2^14 .. 2^15, and what takes them there; both are
// powers of two.
__device__ __forceinline__ float back_of(float most) {
  const int e = (int)(__float_as_uint(most) >> 23) - 127;
  return __uint_as_float((uint32_t)(max(-80, min(e, 40)) - 14 + 127) << 23);
}
__device__ __forceinline__ float inverse_of(float power) {
  return __uint_as_float(0x7F000000u - __float_as_uint(power));
}

// dZ's numbers at (row, c) .. c + 7 in fp32, those past the matrix 0.
template <int DT>
__device__ __forceinline__ void load_slopes(const SlopeArgs& p, int64_t row, int64_t c, RawEight& d,
                                            RawEight& z) {
  const int64_t left = row < p.R ? p.T - c : 0;
  d = RawEight{};
  z = RawEight{};
  if (left > 0) {
    d = load_eight(p.dy, DT, row * p.T + c, left);
    if (p.act != kActNone) z = load_eight(p.z, DT, row * p.T + c, left);
  }
}
template <int DT>
__device__ __forceinline__ void slopes_of(const SlopeArgs& p, const RawEight& d, const RawEight& z,
                                          float (&v)[8]) {
  float x[8];
  to_floats(d, DT, v);
  to_floats(z, DT, x);
  act_slopes(p.act, x, v);
}

// The largest finite sizes of eight columns: of dY (no slope is above 1.13 in size), or of relu's square's
// dZ.  fp16 numbers' sizes are in the order of their bits; 0x400 more makes infinities and NaN negative.
template <bool SQUARE>
struct Largest {
  typedef short short2_t __attribute__((ext_vector_type(2)));
  short2_t bits[4];
  float numbers[8];
  __device__ __forceinline__ Largest() {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      numbers[e] = 0.f;
      bits[e / 2] = short2_t{0x400, 0x400};
    }
  }
  __device__ __forceinline__ void add(const SlopeArgs& p, const RawEight& d, const RawEight& z) {
    if constexpr (SQUARE) {
      float v[8];
      slopes_of<kF16>(p, d, z, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) numbers[e] = fabsf(v[e]) < INFINITY ? fmaxf(numbers[e], fabsf(v[e])) : numbers[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        bits[e] = __builtin_elementwise_max(
            bits[e], __builtin_bit_cast(short2_t, d.lo[e] & 0x7FFF7FFFu) + short2_t{0x400, 0x400});
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (SQUARE) return numbers[e];
    else return f16_to_f32((uint32_t)(bits[e / 2][e & 1] - 0x400));
  }
};
// Eight columns from c <= T - 8 on, without a condition, for which the loads would wait for one another; all
// T of them where there are fewer.
template <bool SQUARE>
__device__ __forceinline__ void load_sizes(const SlopeArgs& p, int64_t row, int64_t c, RawEight& d,
                                           RawEight& z) {
  const int64_t left = p.T < 8 ? p.T : 8;
  d = load_eight(p.dy, kF16, row * p.T + c, left);
  z = RawEight{};
  if constexpr (SQUARE) z = load_eight(p.z, kF16, row * p.T + c, left);
}
__device__ __forceinline__ int64_t held_column(const SlopeArgs& p, int64_t c) {
  return min(c, max((int64_t)0, p.T - 8));
}

// What brings the columns of dX's copy back: strips of 32 columns, `chunk` rows a workgroup, eight columns
// of every 256th row a work-item, 1024 rows in flight at once.  One chunk: `back` itself; more: their
// largest, joined by the next kernel.  (1000 rows, 333 columns 6.2 us; 11008, 2048 columns 20 and 5 for the join;
// the slopes themselves instead of the sizes of dY, 55 us for the first.)
struct ExtentArgs {
  SlopeArgs slope;
  int64_t chunk;
  float* out;  // Tp numbers a chunk
};
template <bool SQUARE>
__global__ void __launch_bounds__(1024) extent_kernel(ExtentArgs p) {
  __shared__ float part[16][32];
  constexpr int kBatch = 4;  // rows in flight
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * 32, c = held_column(p.slope, t0 + 8 * (lane & 3));
  const int64_t end = min(p.slope.R, ((int64_t)blockIdx.y + 1) * p.chunk);
  Largest<SQUARE> most;
  for (int64_t r0 = (int64_t)blockIdx.y * p.chunk + 16 * wave + (lane >> 2); r0 < end;
       r0 += 256 * kBatch) {
    RawEight d[kBatch], z[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)  // (rows past the chunk are its last one again)
      load_sizes<SQUARE>(p.slope, min(r0 + 256 * k, end - 1), c, d[k], z[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) most.add(p.slope, d[k], z[k]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float m = most.at(e);
#pragma unroll
    for (int d = 4; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    // (columns that several lanes have come out the same in each of them)
    if (lane < 4 && c + e >= t0) part[wave][c + e - t0] = m;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  float all = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) all = fmaxf(all, part[w][lane]);
  const int64_t t = t0 + lane;  // below Tp, a multiple of 64
  if (t >= p.slope.T) all = 0.f;
  p.out[(int64_t)blockIdx.y * p.slope.Tp + t] = gridDim.y == 1 ? back_of(all) : all;
}
__global__ void __launch_bounds__(256)
    join_extents_kernel(const float* __restrict__ most, int chunks, int64_t Tp, float* __restrict__ back) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= Tp) return;
  float all = 0.f;
  for (int k0 = 0; k0 < chunks; k0 += 16) {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = most[min(k0 + k, chunks - 1) * Tp + t];
#pragma unroll
    for (int k = 0; k < 16; ++k) all = fmaxf(all, v[k]);
  }
  back[t] = back_of(all);
}
// Chunks of rows: one where the rows are few (a launch less), 1024 rows each where they are many.
inline int64_t extent_chunks(int64_t R) { return R <= 2048 ? 1 : std::min<int64_t>(64, (R + 1023) / 1024); }

// The largest size in a row, of which this work-item takes pieces first, first + stride, ...
template <bool SQUARE>
__device__ __forceinline__ float row_largest(const SlopeArgs& p, int64_t row, int64_t first, int64_t stride) {
  constexpr int kBatch = 4;
  Largest<SQUARE> most;
  for (int64_t c0 = first; row < p.R && c0 < p.T; c0 += kBatch * stride) {
    RawEight d[kBatch], z[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      load_sizes<SQUARE>(p, row, held_column(p, c0 + k * stride), d[k], z[k]);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) most.add(p, d[k], z[k]);
  }
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, most.at(e));
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  return m;
}

// WPR waves of a workgroup's four to a row; its sums are joined in wave order.
template <bool BF16, int WPR, bool SCALED>
__device__ __forceinline__ void slope_rows(const SlopeArgs& p, int64_t group, float* part) {
  constexpr int DT = BF16 ? kBF16 : kF16, kRows = 4 / WPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = group * kRows + wave / WPR;
  const bool copies = p.padded || (SCALED && p.padded_x);
  const int64_t width = copies ? p.Tp : p.T, rows = copies ? p.Rp : p.R;
  constexpr int kBatch = 4;  // pieces in flight
  float up = 1.f;
  if constexpr (SCALED) {
    if (p.padded) {
      const int64_t first = ((int64_t)(wave % WPR) * 64 + lane) * 8;
      float most = p.act == kActRelu2 ? row_largest<true>(p, row, first, WPR * 512)
                                      : row_largest<false>(p, row, first, WPR * 512);
      if constexpr (WPR > 1) {
        if (lane == 0) part[4 + wave] = most;
        __syncthreads();
        most = fmaxf(fmaxf(part[4], part[5]), fmaxf(part[6], part[7]));
      }
      const float back = back_of(most);
      up = inverse_of(back);
      if (lane == 0 && wave % WPR == 0 && row < p.R) p.row_back[row] = back;
    }
  }
  float sum = 0.f;
  if (row < rows) {
    for (int64_t c0 = ((int64_t)(wave % WPR) * 64 + lane) * 8; c0 < width; c0 += kBatch * WPR * 512) {
      RawEight d[kBatch], z[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) load_slopes<DT>(p, row, c0 + k * WPR * 512, d[k], z[k]);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * WPR * 512;
        if (c >= width) continue;
        float v[8];
        slopes_of<DT>(p, d[k], z[k], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[e];
        if constexpr (SCALED) {
          float w[8];
          if (p.padded) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = v[e] * up;
            *reinterpret_cast<u32x4_t*>(p.padded + row * p.Tp + c) = pack_eight(w, DT);
          }
          if (p.padded_x) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4_t back = *reinterpret_cast<const float4_t*>(p.col_back + c + 4 * h);
#pragma unroll
              for (int e = 0; e < 4; ++e) w[4 * h + e] = v[4 * h + e] * inverse_of(back[e]);
            }
            *reinterpret_cast<u32x4_t*>(p.padded_x + row * p.Tp + c) = pack_eight(w, DT);
          }
        } else if (p.padded) {
          *reinterpret_cast<u32x4_t*>(p.padded + row * p.Tp + c) = pack_eight(v, DT);
        }
        if (p.dz && row < p.R && c < p.T) store_eight(p.dz, DT, row * p.T + c, p.T - c, v);
      }
    }
  }
  if (!p.dbias) return;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if constexpr (WPR > 1) {
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0 && row < p.R) {
      float all = 0.f;
      for (int w = 0; w < WPR; ++w) all += part[w];
      p.dbias[row] = all;
    }
  } else if (lane == 0 && row < p.R) {
    p.dbias[row] = sum;
  }
}

template <bool BF16, int WPR, bool SCALED>
__global__ void __launch_bounds__(256) slope_kernel(SlopeArgs p) {
  __shared__ float part[8];
  slope_rows<BF16, WPR, SCALED>(p, blockIdx.x, part);
}

// ---- W ---------------------------------------------------------------------------------------------

// The dense W of a pair of any pattern and layout, 16 bits, rows of Kp numbers with zeros after the K-th
// and rows of zeros after the R-th: a thread eight of them.  For small matrices and widths that are not
// multiples of 8; the others are decompressed by nm_compress.hip's kernels, which are specialised for each
// pattern, and have only the rows of zeros from here.  (Rows read twice instead would meet dZ's zeros, and
// an infinity in the last one would be NaN.)
struct ExpandArgs {
  const uint16_t* values;
  const uint8_t* meta;
  int64_t R, K, Kp;
  int64_t begin, end;  // rows that are written
  int n, m, bits;
  bool blocked;
  uint16_t* out;
};
__device__ __forceinline__ void expand_pieces(const ExpandArgs& p, int64_t first, int64_t stride) {
  const int64_t pieces = p.Kp / 8, total = p.end * pieces, row_values = p.K / p.m * p.n;
  const int per = 64 / p.m * p.n;  // values of a row and step of the blocked layout
  const int64_t meta_row = (row_values * p.bits + 31) / 32 * 4;
  for (int64_t i = p.begin * pieces + first; i < total; i += stride) {
    const int64_t r = i / pieces;
    const int k0 = (int)(i % pieces * 8);
    uint64_t half[2] = {0, 0};  // numbers 0 .. 3 and 4 .. 7
    const int groups = 8 / p.m;
    for (int g = 0; g < groups && r < p.R && k0 + g * p.m < p.K; ++g) {
      const int64_t f0 = (int64_t)(k0 / p.m + g) * p.n;  // the group's first value in its row
      int64_t vi, bit;
      const uint8_t* places;
      if (p.blocked) {
        const int64_t block = ((r >> 4) * (p.K / 64) + f0 / per) * 16 + (r & 15);
        vi = block * per + f0 % per;
        places = p.meta + block * (per * p.bits / 8);
        bit = f0 % per * p.bits;
      } else {
        vi = r * row_values + f0;
        places = p.meta + r * meta_row;
        bit = f0 * p.bits;
      }
      for (int j = 0; j < p.n; ++j, bit += p.bits) {
        const int shift = (int)(bit & 7);
        uint32_t field = places[bit >> 3] >> shift;
        if (shift + p.bits > 8) field |= (uint32_t)places[(bit >> 3) + 1] << (8 - shift);
        const int at = g * p.m + (int)(field & (uint32_t)(p.m - 1));
        // (as the decompression has it: the later value of a place that is given twice)
        const uint64_t v = p.values[vi + j], mask = (uint64_t)0xFFFF << (16 * (at & 3));
        const uint64_t put = v << (16 * (at & 3));
        if (at < 4) half[0] = (half[0] & ~mask) | put;
        else half[1] = (half[1] & ~mask) | put;
      }
    }
    reinterpret_cast<u32x4_t*>(p.out)[i] =
        u32x4_t{(uint32_t)half[0], (uint32_t)(half[0] >> 32), (uint32_t)half[1], (uint32_t)(half[1] >> 32)};
  }
}

// All that the products need in one launch: workgroups for dZ's rows, then for X, then for W.
struct PrepareArgs {
  SlopeArgs slope;
  WidenArgs x;
  ExpandArgs w;
  unsigned slope_groups, x_groups, w_groups;
};
template <bool BF16, bool SCALED>
__global__ void __launch_bounds__(256) prepare_kernel(PrepareArgs p) {
  __shared__ float part[8];
  const unsigned b = blockIdx.x;
  if (b < p.slope_groups) {
    slope_rows<BF16, 1, SCALED>(p.slope, b, part);
  } else if (b < p.slope_groups + p.x_groups) {
    widen_pieces<uint16_t>(p.x, (int64_t)(b - p.slope_groups) * 256 + threadIdx.x,
                           (int64_t)p.x_groups * 256);
  } else {
    expand_pieces(p.w, (int64_t)(b - p.slope_groups - p.x_groups) * 256 + threadIdx.x,
                  (int64_t)p.w_groups * 256);
  }
}

// ---- the products ------------------------------------------------------------------------------

struct GradProduct {
  GemmOperand a, b;
  int64_t klen;      // of a strided a
  int steps, per;    // steps of 64, of which each split takes `per`
  GemmMap map;
  int groups, splits;
  int64_t rows, cols;
  uint16_t* out;     // rows x cols
  float* sums;       // splits x rows x ld, where there is more than one
  int64_t ld;        // cols to whole fours
  const float* back; // fp16: what brings its rows (dW) or columns (dX) back, or null
};

template <class G, bool BF16>
__device__ __forceinline__ void grad_tile(const GradProduct& p, int group, uint8_t* smem) {
  const int split = group / p.groups;
  int tm, tn;
  if (!p.map.tile_of(group % p.groups, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * G::kBM, n0 = (int64_t)tn * G::kBN;
  const int s0 = split * p.per, steps = min(p.per, p.steps - s0);
  GemmOperand a = p.a, b = p.b;
  a.p += (int64_t)s0 * kGemmStep * (G::kAS ? a.ld : 1);
  b.p += (int64_t)s0 * kGemmStep * (G::kBS ? b.ld : 1);
  typename G::Acc acc;
  G::clear(acc);
  G::run(a, b, m0, n0, steps, p.klen - (int64_t)s0 * kGemmStep, smem, acc);
  if constexpr (!BF16) {
    if (p.back) {
#pragma unroll
      for (int i = 0; !G::kAS && i < G::kFM; ++i) {
        const int64_t row = G::row0(m0) + 32 * i;
        const float f = row < p.rows ? p.back[row] : 1.f;
#pragma unroll
        for (int j = 0; j < G::kFN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] *= f;
      }
#pragma unroll
      for (int q = 0; G::kAS && q < 4 * G::kFN; ++q) {
        const int64_t col = G::col0(n0) + 32 * (q / 4) + 8 * (q % 4);
        float4_t f{1.f, 1.f, 1.f, 1.f};
        if (col < p.b.rows) f = *reinterpret_cast<const float4_t*>(p.back + col);
#pragma unroll
        for (int i = 0; i < G::kFM; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][q / 4][4 * (q % 4) + e] *= f[e];
        keep_lds_order();  // one piece at a time: there are no registers for all of them
      }
    }
  }
  if (p.splits == 1) {
    G::template store16<BF16>(acc, m0, n0, smem, p.out, p.cols, p.rows, p.cols);
    return;
  }
  float* out = p.sums + (int64_t)split * p.rows * p.ld;
  const int64_t row0 = G::row0(m0), col0 = G::col0(n0);
#pragma unroll
  for (int i = 0; i < G::kFM; ++i)
#pragma unroll
    for (int q = 0; q < 4 * G::kFN; ++q) {
      const int64_t row = row0 + 32 * i, col = col0 + 32 * (q / 4) + 8 * (q % 4);
      if (row < p.rows && col < p.ld)
        *reinterpret_cast<float4_t*>(out + row * p.ld + col) = G::quad(acc, i, q / 4, q % 4);
    }
}

struct GradProducts {
  GradProduct x, w;
};
template <class GX, class GW, bool BF16>
__global__ void __launch_bounds__(GX::kThreads) grad_products_kernel(GradProducts p) {
  static_assert(GX::kThreads == GW::kThreads && GX::kLds == GW::kLds, "one launch for both");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int b = blockIdx.x, first_w = p.x.groups * p.x.splits;
  if (b < first_w) grad_tile<GX, BF16>(p.x, b, smem);
  else grad_tile<GW, BF16>(p.w, b - first_w, smem);
}

// Sums of the splits, in split order.
template <bool BF16>
__global__ void __launch_bounds__(256) join_splits_kernel(GradProduct p) {
  const int64_t total = p.rows * p.ld / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    float4_t v = reinterpret_cast<const float4_t*>(p.sums)[i];
    for (int z = 1; z < p.splits; ++z) {
      const float4_t b = reinterpret_cast<const float4_t*>(p.sums)[z * total + i];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += b[e];
    }
    const int64_t r = 4 * i / p.ld, c = 4 * i % p.ld;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < p.cols) store_from_f32<BF16 ? kBF16 : kF16>(p.out, r * p.cols + c + e, v[e]);
  }
}

// Entries of W up to which it is expanded in the launch that prepares the rest: 1000 x 768 in 3.5 us of
// its own, and a launch less; past it the specialised kernels' rate counts.
constexpr int64_t kSmallW = 4 << 20;

// Where everything lies in the workspace.
struct SpmmGradLayout {
  int64_t Rp, Tp, Kp;           // Kp: row length of the dense W
  bool scaled;                  // each product has its own copy of dZ
  bool pad_z, pad_x;            // dZ goes to a padded copy; X is copied
  int64_t chunks = 0;           // of the rows, for the columns' largest
  SpmmGradCut cut;
  int64_t z, zx, row_back, col_back, most, x, w, sums_x, sums_w, total;
  SpmmGradLayout(int64_t R, int64_t K, int64_t T, bool want_w, bool want_x, bool want_z, bool act,
                 bool scale)
      : Rp(pad64(R)), Tp(pad64(T)), Kp(K % 8 == 0 ? K : pad64(K)), cut(R, K, T, want_w, want_x) {
    const bool whole = Rp == R && Tp == T, product = want_w || want_x;
    scaled = scale && product && R > 0 && T > 0;
    pad_z = product && !scaled && (!whole || (act && !want_z));
    pad_x = want_w && Tp != T;
    if (scaled && want_x) chunks = extent_chunks(R);
    z = 0;
    zx = z + (pad_z || (scaled && want_w) ? whole256(Rp * Tp * 2) : 0);
    row_back = zx + (scaled && want_x ? whole256(Rp * Tp * 2) : 0);
    col_back = row_back + (scaled && want_w ? whole256(R * 4) : 0);
    most = col_back + (scaled && want_x ? whole256(Tp * 4) : 0);
    x = most + (chunks > 1 ? whole256(chunks * Tp * 4) : 0);
    w = x + (pad_x ? whole256(K * Tp * 2) : 0);
    sums_x = w + (want_x ? whole256(Rp * Kp * 2) : 0);
    sums_w = sums_x + (cut.splits_x > 1 ? whole256(cut.splits_x * K * ((T + 3) / 4 * 4) * 4) : 0);
    total = sums_w + (cut.splits_w > 1 ? whole256(cut.splits_w * R * ((K + 3) / 4 * 4) * 4) : 0);
  }
};

template <class GX, class GW, bool BF16>
hipError_t launch_products(GradProducts& p, bool want_x, bool want_w, hipStream_t s) {
  const auto size = [](GradProduct& q, int64_t bm, int64_t bn, bool want) {
    q.groups = 0;
    if (!want) return 0;
    q.map = make_gemm_map((q.rows + bm - 1) / bm, (q.cols + bn - 1) / bn);
    q.groups = q.map.groups();
    q.per = (q.steps + q.splits - 1) / q.splits;
    return q.groups * q.splits;
  };
  const int groups = size(p.x, GX::kBM, GX::kBN, want_x) + size(p.w, GW::kBM, GW::kBN, want_w);
  hipError_t e = GX::template launch<grad_products_kernel<GX, GW, BF16>>(p, groups, 1, s);
  for (const GradProduct* q : {&p.x, &p.w}) {
    if (e != hipSuccess || q->groups == 0 || q->splits == 1) continue;
    join_splits_kernel<BF16><<<stride_grid(q->rows * q->ld / 4, 256), 256, 0, s>>>(*q);
    e = hipGetLastError();
  }
  return e;
}

template <bool BF16, int WPR>
hipError_t launch_slopes(const SlopeArgs& p, unsigned groups, bool scaled, hipStream_t s) {
  if constexpr (!BF16)
    if (scaled) {
      slope_kernel<BF16, WPR, true><<<groups, 256, 0, s>>>(p);
      return hipGetLastError();
    }
  slope_kernel<BF16, WPR, false><<<groups, 256, 0, s>>>(p);
  return hipGetLastError();
}
template <bool BF16>
hipError_t launch_prepare(const PrepareArgs& p, unsigned groups, bool scaled, hipStream_t s) {
  if constexpr (!BF16)
    if (scaled) {
      prepare_kernel<BF16, true><<<groups, 256, 0, s>>>(p);
      return hipGetLastError();
    }
  prepare_kernel<BF16, false><<<groups, 256, 0, s>>>(p);
  return hipGetLastError();
}

// Whether dZ's rounding can leave its type's range: in fp16, where a slope changes dY.
bool scaled_grad(bool bf16, int act) { return !bf16 && act != kActNone && act != kActRelu; }

template <bool BF16>
hipError_t run_spmm_act_grad(const SpmmGradCall& c, uint8_t* ws, hipStream_t s) {
  const int64_t R = c.R, K = c.K, T = c.T;
  // (an empty result is not wanted)
  const bool want_w = c.dW && R * K > 0, want_x = c.dX && K * T > 0, act = c.act != kActNone;
  const SpmmGradLayout L(R, K, T, want_w, want_x, c.dZ != nullptr, act, scaled_grad(BF16, c.act));
  const uint16_t* dz = static_cast<const uint16_t*>(act ? c.dZ : c.dY);
  const uint16_t* dz_x = dz;
  const uint16_t* x = static_cast<const uint16_t*>(c.X);
  hipError_t e;
  PrepareArgs a{};
  if (R > 0 && (L.scaled || L.pad_z || c.dZ || c.dbias)) {
    a.slope = SlopeArgs{c.Z, c.dY, R, T, c.act, nullptr, L.Rp, L.Tp, static_cast<uint16_t*>(c.dZ), c.dbias,
                        nullptr, nullptr, nullptr};
    if (L.pad_z) dz = dz_x = a.slope.padded = reinterpret_cast<uint16_t*>(ws + L.z);
    if (L.scaled && want_w) {
      dz = a.slope.padded = reinterpret_cast<uint16_t*>(ws + L.z);
      a.slope.row_back = reinterpret_cast<float*>(ws + L.row_back);
    }
    if (L.scaled && want_x) {
      dz_x = a.slope.padded_x = reinterpret_cast<uint16_t*>(ws + L.zx);
      float* back = reinterpret_cast<float*>(ws + L.col_back);
      a.slope.col_back = back;
      float* most = L.chunks > 1 ? reinterpret_cast<float*>(ws + L.most) : back;
      const ExtentArgs extent{a.slope, (R + L.chunks - 1) / L.chunks, most};
      const dim3 grid((unsigned)(L.Tp / 32), (unsigned)L.chunks);
      if (c.act == kActRelu2) extent_kernel<true><<<grid, 1024, 0, s>>>(extent);
      else extent_kernel<false><<<grid, 1024, 0, s>>>(extent);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      if (L.chunks > 1) {
        join_extents_kernel<<<(unsigned)((L.Tp + 255) / 256), 256, 0, s>>>(most, (int)L.chunks, L.Tp, back);
        if ((e = hipGetLastError()) != hipSuccess) return e;
      }
    }
    const int64_t rows = L.pad_z || L.scaled ? L.Rp : R;
    if (rows >= 2048 || T <= 512) {  // a wave a row fills the device where rows are many or short
      a.slope_groups = (unsigned)((rows + 3) / 4);
    } else {
      e = launch_slopes<BF16, 4>(a.slope, (unsigned)rows, L.scaled, s);
      if (e != hipSuccess) return e;
    }
  }
  if (L.pad_x) {
    a.x = WidenArgs{static_cast<const uint8_t*>(c.X), ws + L.x, K, T, K, L.Tp};
    a.x_groups = stride_grid(K * L.Tp / 8, 256);
    x = reinterpret_cast<const uint16_t*>(ws + L.x);
  }
  if (want_x && R > 0) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + L.w);
    const bool large = R * K > kSmallW && L.Kp == K;
    if (large) {
      e = launch_decompress(c.values, c.meta, 2, R, K, c.n, c.m, c.blocked, to, s);
      if (e != hipSuccess) return e;
    }
    const int64_t begin = large ? R : 0;
    if (begin < L.Rp) {
      a.w = ExpandArgs{static_cast<const uint16_t*>(c.values), reinterpret_cast<const uint8_t*>(c.meta), R,
                       K, L.Kp, begin, L.Rp, c.n, c.m, c.m == 2 ? 1 : c.m == 4 ? 2 : 3, c.blocked, to};
      a.w_groups = stride_grid((L.Rp - begin) * L.Kp / 8, 256);
    }
  }
  const unsigned groups = a.slope_groups + a.x_groups + a.w_groups;
  if (groups > 0) {
    e = groups == a.slope_groups ? launch_slopes<BF16, 1>(a.slope, groups, L.scaled, s)
                                 : launch_prepare<BF16>(a, groups, L.scaled, s);
    if (e != hipSuccess) return e;
  }
  if (!want_w && !want_x) return hipSuccess;
  GradProducts p{};
  p.x.a = GemmOperand{reinterpret_cast<const uint16_t*>(ws + L.w), L.Kp, L.Kp, 0};
  p.x.b = GemmOperand{dz_x, L.Tp, L.Tp, 0};
  p.x.klen = L.Rp;
  p.x.steps = (int)(L.Rp / kGemmStep);
  p.x.splits = L.cut.splits_x;
  p.x.rows = K;
  p.x.cols = T;
  p.x.out = static_cast<uint16_t*>(c.dX);
  p.x.sums = reinterpret_cast<float*>(ws + L.sums_x);
  p.x.ld = (T + 3) / 4 * 4;
  p.x.back = a.slope.col_back;
  p.w.a = GemmOperand{dz, L.Tp, R, 0};
  p.w.b = GemmOperand{x, L.Tp, K, 0};
  p.w.klen = L.Tp;
  p.w.steps = (int)(L.Tp / kGemmStep);
  p.w.splits = L.cut.splits_w;
  p.w.rows = R;
  p.w.cols = K;
  p.w.out = static_cast<uint16_t*>(c.dW);
  p.w.sums = reinterpret_cast<float*>(ws + L.sums_w);
  p.w.ld = (K + 3) / 4 * 4;
  p.w.back = a.slope.row_back;
  if (L.cut.tile == kTile256)
    return launch_products<Gemm<2, 4, 4, 2, true, true, BF16, true, 2>,
                           Gemm<2, 4, 4, 2, false, false, BF16, true, 2>, BF16>(p, want_x, want_w, s);
  if (L.cut.tile == kTile128)
    return launch_products<Gemm<2, 4, 2, 1, true, true, BF16, true, 2>,
                           Gemm<2, 4, 2, 1, false, false, BF16, true, 2>, BF16>(p, want_x, want_w, s);
  return launch_products<Gemm<2, 2, 2, 1, true, true, BF16, true, 3>,
                         Gemm<2, 2, 2, 1, false, false, BF16, true, 3>, BF16>(p, want_x, want_w, s);
}

}  // namespace

size_t spmm_act_workspace_bytes(int64_t R, int64_t K, int n, int m, int64_t T, int dt) {
  if (thin_preferred(R, K, n, m, T, elem_of(dt))) {
    const ThinPlan plan(R, K, T, m, dt == kF32);
    return plan.direct ? 0 : (size_t)(plan.Tp * pad64(K) * (dt == kF32 ? 4 : 2));
  }
  const int64_t ldx = whole_row(T, dt);
  return ldx == T ? 0 : (size_t)whole256(K * ldx * elem_of(dt));
}

hipError_t run_spmm_act(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n, int m,
                        bool blocked, const void* X, int64_t T, int dt, Product p, void* workspace,
                        hipStream_t s) {
  if (thin_preferred(R, K, n, m, T, elem_of(dt)))
    return launch_thin(values, meta, R, K, n, m, blocked, X, T, dt, p, workspace, s);
  p.ldx = whole_row(T, dt);
  if (p.ldx != T && K > 0) {
    const hipError_t e = widen(X, K, T, workspace, K, p.ldx, elem_of(dt), s);
    if (e != hipSuccess) return e;
    X = workspace;
  }
  return launch_spmm_act(values, meta, R, K, n, m, blocked, X, T, dt, p, s);
}

size_t spmm_act_grad_workspace_bytes(int64_t R, int64_t K, int64_t T, bool bf16, int act, bool want_w,
                                     bool want_x, bool want_z) {
  return (size_t)SpmmGradLayout(R, K, T, want_w, want_x, want_z, act != kActNone, scaled_grad(bf16, act)).total;
}

hipError_t launch_spmm_act_grad(const SpmmGradCall& c, void* workspace, hipStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return c.bf16 ? run_spmm_act_grad<true>(c, ws, s) : run_spmm_act_grad<false>(c, ws, s);
}

}  // namespace nm
