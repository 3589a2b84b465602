// nm_spmm_grad.hip -- what nm_spmm_act needs around its product (rows of X made whole 16-byte
// pieces), and its gradient (nm_spmm_act_grad).
//
//   dZ = act'(Z) dY,   dbias[r] = sum over t of dZ[r, t],   dW = dZ X^T,   dX = W^T dZ
//
// dZ is one pass over Z and dY that also adds up its rows (bound by memory).  It leaves in 16 bits,
// as the operand of the other two: where the sizes are not whole multiples of 64 into a padded copy,
// and not at all where there is no activation and the sizes are whole.  dW is the gradient of the
// dense weight, as SR-STE takes it.  W^T has no structure that the sparse instruction could use (W's
// groups run along its rows), so W is decompressed and both products are dense (nm_gemm.h).
//
// What the products need (dZ, X and W in whole steps) goes out in one launch where W is small, and both
// products in one, dX's long sums first: alone, each leaves units idle at its end (1000 x 768, 333
// columns: 30 us a call in launches of their own, 21 so).
//
// Bound by the matrix cores where matrices are large: bf16 11008 x 4096, 2048 columns, dZ 25.6 us and W
// 24.8, both at the memory's rate, the products 328-336 (1100-1130 TFLOP/s; a library's product of 8192^3
// on the same card 1215).  By launches where they are small: 6.9 and 9.9 us for 1000 x 768, 333 columns.
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
};

// WPR waves of a workgroup's four to a row; its sums are joined in wave order.
template <bool BF16, int WPR>
__device__ __forceinline__ void slope_rows(const SlopeArgs& p, int64_t group, float* part) {
  constexpr int DT = BF16 ? kBF16 : kF16, kRows = 4 / WPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = group * kRows + wave / WPR;
  const int64_t width = p.padded ? p.Tp : p.T, rows = p.padded ? p.Rp : p.R;
  float sum = 0.f;
  if (row < rows) {
    constexpr int kBatch = 4;  // pieces in flight
    for (int64_t c0 = ((int64_t)(wave % WPR) * 64 + lane) * 8; c0 < width; c0 += kBatch * WPR * 512) {
      RawEight d[kBatch], z[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * WPR * 512, left = row < p.R ? p.T - c : 0;
        d[k] = RawEight{};
        z[k] = RawEight{};
        if (left > 0) {
          d[k] = load_eight(p.dy, DT, row * p.T + c, left);
          if (p.act != kActNone) z[k] = load_eight(p.z, DT, row * p.T + c, left);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + k * WPR * 512;
        if (c >= width) continue;
        float v[8], x[8];
        to_floats(d[k], DT, v);
        to_floats(z[k], DT, x);
        act_slopes(p.act, x, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[e];
        if (p.padded) *reinterpret_cast<u32x4_t*>(p.padded + row * p.Tp + c) = pack_eight(v, DT);
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

template <bool BF16, int WPR>
__global__ void __launch_bounds__(256) slope_kernel(SlopeArgs p) {
  __shared__ float part[4];
  slope_rows<BF16, WPR>(p, blockIdx.x, part);
}

// ---- W ---------------------------------------------------------------------------------------------

// The dense W of a pair of any pattern and layout, 16 bits, rows of Kp numbers with zeros after the K-th:
// a thread eight of them.  For small matrices and widths that are not multiples of 8; the others are
// decompressed by nm_compress.hip's kernels, which are specialised for each pattern.
struct ExpandArgs {
  const uint16_t* values;
  const uint8_t* meta;
  int64_t R, K, Kp;
  int n, m, bits;
  bool blocked;
  uint16_t* out;
};
__device__ __forceinline__ void expand_pieces(const ExpandArgs& p, int64_t first, int64_t stride) {
  const int64_t pieces = p.Kp / 8, total = p.R * pieces, row_values = p.K / p.m * p.n;
  const int per = 64 / p.m * p.n;  // values of a row and step of the blocked layout
  const int64_t meta_row = (row_values * p.bits + 31) / 32 * 4;
  for (int64_t i = first; i < total; i += stride) {
    const int64_t r = i / pieces;
    const int k0 = (int)(i % pieces * 8);
    uint64_t half[2] = {0, 0};  // numbers 0 .. 3 and 4 .. 7
    const int groups = 8 / p.m;
    for (int g = 0; g < groups && k0 + g * p.m < p.K; ++g) {
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
template <bool BF16>
__global__ void __launch_bounds__(256) prepare_kernel(PrepareArgs p) {
  __shared__ float part[4];
  const unsigned b = blockIdx.x;
  if (b < p.slope_groups) {
    slope_rows<BF16, 1>(p.slope, b, part);
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
  bool pad_z, pad_x;            // dZ goes to a padded copy; X is copied
  SpmmGradCut cut;
  int64_t z, x, w, sums_x, sums_w, total;
  SpmmGradLayout(int64_t R, int64_t K, int64_t T, bool want_w, bool want_x, bool want_z, bool act)
      : Rp(pad64(R)), Tp(pad64(T)), Kp(K % 8 == 0 ? K : pad64(K)), cut(R, K, T, want_w, want_x) {
    const bool whole = Rp == R && Tp == T, product = want_w || want_x;
    pad_z = product && (!whole || (act && !want_z));
    pad_x = want_w && Tp != T;
    z = 0;
    x = z + (pad_z ? whole256(Rp * Tp * 2) : 0);
    w = x + (pad_x ? whole256(K * Tp * 2) : 0);
    sums_x = w + (want_x ? whole256(R * Kp * 2) : 0);
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

template <bool BF16>
hipError_t run_spmm_act_grad(const SpmmGradCall& c, uint8_t* ws, hipStream_t s) {
  const int64_t R = c.R, K = c.K, T = c.T;
  // (an empty result is not wanted)
  const bool want_w = c.dW && R * K > 0, want_x = c.dX && K * T > 0, act = c.act != kActNone;
  const SpmmGradLayout L(R, K, T, want_w, want_x, c.dZ != nullptr, act);
  const uint16_t* dz = static_cast<const uint16_t*>(act ? c.dZ : c.dY);
  const uint16_t* x = static_cast<const uint16_t*>(c.X);
  hipError_t e;
  PrepareArgs a{};
  if (R > 0 && (L.pad_z || c.dZ || c.dbias)) {
    a.slope = SlopeArgs{c.Z, c.dY, R, T, c.act, nullptr, L.Rp, L.Tp, static_cast<uint16_t*>(c.dZ), c.dbias};
    if (L.pad_z) {
      a.slope.padded = reinterpret_cast<uint16_t*>(ws + L.z);
      dz = a.slope.padded;
    }
    const int64_t rows = a.slope.padded ? L.Rp : R;
    if (rows >= 2048 || T <= 512) {  // a wave a row fills the device where rows are many or short
      a.slope_groups = (unsigned)((rows + 3) / 4);
    } else {
      slope_kernel<BF16, 4><<<(unsigned)rows, 256, 0, s>>>(a.slope);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  if (L.pad_x) {
    a.x = WidenArgs{static_cast<const uint8_t*>(c.X), ws + L.x, K, T, K, L.Tp};
    a.x_groups = stride_grid(K * L.Tp / 8, 256);
    x = reinterpret_cast<const uint16_t*>(ws + L.x);
  }
  if (want_x && R > 0) {
    uint16_t* to = reinterpret_cast<uint16_t*>(ws + L.w);
    if (R * K > kSmallW && L.Kp == K) {
      e = launch_decompress(c.values, c.meta, 2, R, K, c.n, c.m, c.blocked, to, s);
      if (e != hipSuccess) return e;
    } else {
      a.w = ExpandArgs{static_cast<const uint16_t*>(c.values), reinterpret_cast<const uint8_t*>(c.meta), R,
                       K, L.Kp, c.n, c.m, c.m == 2 ? 1 : c.m == 4 ? 2 : 3, c.blocked, to};
      a.w_groups = stride_grid(R * L.Kp / 8, 256);
    }
  }
  const unsigned groups = a.slope_groups + a.x_groups + a.w_groups;
  if (groups > 0) {
    if (groups == a.slope_groups) slope_kernel<BF16, 1><<<groups, 256, 0, s>>>(a.slope);
    else prepare_kernel<BF16><<<groups, 256, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!want_w && !want_x) return hipSuccess;
  GradProducts p{};
  p.x.a = GemmOperand{reinterpret_cast<const uint16_t*>(ws + L.w), L.Kp, L.Kp, 0};
  p.x.b = GemmOperand{dz, L.Tp, L.Tp, 0};
  p.x.klen = R;
  p.x.steps = (int)(L.Rp / kGemmStep);
  p.x.splits = L.cut.splits_x;
  p.x.rows = K;
  p.x.cols = T;
  p.x.out = static_cast<uint16_t*>(c.dX);
  p.x.sums = reinterpret_cast<float*>(ws + L.sums_x);
  p.x.ld = (T + 3) / 4 * 4;
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

size_t spmm_act_grad_workspace_bytes(int64_t R, int64_t K, int64_t T, bool want_w, bool want_x,
                                     bool want_z, bool act) {
  return (size_t)SpmmGradLayout(R, K, T, want_w, want_x, want_z, act).total;
}

hipError_t launch_spmm_act_grad(const SpmmGradCall& c, void* workspace, hipStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return c.bf16 ? run_spmm_act_grad<true>(c, ws, s) : run_spmm_act_grad<false>(c, ws, s);
}

}  // namespace nm
