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
// factor rho in fp32, goes into the first step's epilogues.
//   bf16 G: operands are one fp16, and the X that a X is formed from is carried in fp32.
//   fp16 and fp32 G: each operand is two fp16, hi + lo (22 bits), and a product is hi hi +
//     hi lo + lo hi in the same accumulators, as exact as fp32 products.
// The norm is summed in fp64, so no finite G overflows or vanishes in it.
#include <cmath>

#include "nm_gemm.h"

namespace nm {
namespace {

constexpr int kNormBlocks = 512;
constexpr float kOrthScale = 256.f;

struct OrthHead {  // first bytes of the workspace
  double partial[kNormBlocks];
  float rho;
};

template <int DT>
__device__ __forceinline__ float load_f32(const void* p, int64_t i) {
  if constexpr (DT == kF32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == kF16) return f16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

template <int DT>
__global__ void __launch_bounds__(256) norm_kernel(const void* __restrict__ G, int64_t n,
                                                   OrthHead* head) {
  __shared__ double part[4];
  double sum = 0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)kNormBlocks * 256) {
    const double x = load_f32<DT>(G, i);
    sum += x * x;
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) head->partial[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X' = G 2^k (rp x kp, zeros past R x K) with 2^k |G|_F in (2^7, 2^8].
template <int DT, bool SPLIT>
__global__ void __launch_bounds__(256)
    start_kernel(const void* __restrict__ G, int64_t R, int64_t K, int64_t rp, int64_t kp, float eps,
                 OrthHead* head, _Float16* __restrict__ hi, _Float16* __restrict__ lo) {
  __shared__ double part[4];
  double sum = head->partial[threadIdx.x] + head->partial[threadIdx.x + 256];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double norm = sqrt(part[0] + part[1] + part[2] + part[3]);
  int e = 0;
  if (norm > 0 && norm < INFINITY) frexp(norm, &e);  // norm = f 2^e, f in [1/2, 1)
  const int k = 8 - e;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    head->rho = norm > 0 ? (float)(ldexp(256.0, -k) / (norm + (double)eps)) : 1.f;
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
    typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
    *reinterpret_cast<half4_t*>(hi + 4 * i) = half4_t{h[0], h[1], h[2], h[3]};
    if constexpr (SPLIT) *reinterpret_cast<half4_t*>(lo + 4 * i) = half4_t{l[0], l[1], l[2], l[3]};
  }
}

enum OrthKind { kGram, kSquare, kUpdate };

struct OrthArgs {
  GemmOperand a, b;
  int64_t a_lo, b_lo;  // element offset from an operand's hi part to its lo part
  int steps, segments;
  GemmMap map;
  int64_t rows, cols;  // of the result, whole multiples of 64; its rows are `cols` apart
  float ca, cb, cc;
  const float* rho;            // the first step's factor, else null
  const _Float16 *from_hi, *from_lo;  // square: A; update: the X before
  const float* from;           // update: the X before in fp32, or null
  _Float16 *hi, *lo;           // result (lo only with two parts)
  float* keep;                 // update: the X after in fp32, or null
  void* out;                   // the last update: the caller's result (R x K), else null
  int out_dt;
  int64_t R, K;
};

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float4_t widen(half4_t h) {
  return float4_t{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
}

template <int KIND, bool SPLIT>
__device__ __forceinline__ void orth_store(const OrthArgs& p, float rho, int64_t row, int64_t col,
                                           float4_t v) {
  if (row >= p.rows || col >= p.cols) return;
  const int64_t at = row * p.cols + col;
  float4_t r;
  if constexpr (KIND == kGram) {
    const float f = rho * rho / kOrthScale;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = v[i] * f;
  } else {
    float4_t x;
    if (KIND == kUpdate && !SPLIT && p.from) {
      x = *reinterpret_cast<const float4_t*>(p.from + at);
    } else {
      x = widen(*reinterpret_cast<const half4_t*>(p.from_hi + at));
      if constexpr (SPLIT) {
        const float4_t l = widen(*reinterpret_cast<const half4_t*>(p.from_lo + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += l[i];
      }
    }
    if constexpr (KIND == kSquare) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = p.cb * x[i] + (p.cc / kOrthScale) * v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = rho * (p.ca * x[i] + v[i] * (1.f / kOrthScale));
    }
  }
  if (KIND == kUpdate && p.out) {
    if (row >= p.R) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (col + i >= p.K) continue;
      const float y = r[i] * (1.f / kOrthScale);
      const int64_t o = row * p.K + col + i;
      if (p.out_dt == kF32) store_from_f32<kF32>(p.out, o, y);
      else if (p.out_dt == kF16) store_from_f32<kF16>(p.out, o, y);
      else store_from_f32<kBF16>(p.out, o, y);
    }
    return;
  }
  half4_t h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = (_Float16)r[i];
  *reinterpret_cast<half4_t*>(p.hi + at) = h;
  if constexpr (SPLIT) {
    half4_t l;
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = (_Float16)(r[i] - (float)h[i]);
    *reinterpret_cast<half4_t*>(p.lo + at) = l;
  } else if (KIND == kUpdate) {
    *reinterpret_cast<float4_t*>(p.keep + at) = r;
  }
}

template <class G, int KIND, bool SPLIT>
__global__ void __launch_bounds__(G::kThreads) orth_kernel(OrthArgs p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  int tm, tn;
  if (!p.map.tile_of(blockIdx.x, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * G::kBM, n0 = (int64_t)tn * G::kBN;
  typename G::Acc acc;
  G::clear(acc);
  G::run(p.a, p.b, m0, n0, p.steps, (int64_t)p.steps * kGemmStep, smem, acc, p.segments, p.a_lo,
         p.b_lo);
  const float rho = p.rho ? *p.rho : 1.f;
  G::each4(acc, m0, n0, [&](int64_t row, int64_t col, float4_t v) {
    orth_store<KIND, SPLIT>(p, rho, row, col, v);
  });
}

template <class G, int KIND, bool SPLIT>
hipError_t launch_orth_tile(OrthArgs p, hipStream_t s) {
  p.map = make_gemm_map((p.rows + G::kBM - 1) / G::kBM, (p.cols + G::kBN - 1) / G::kBN);
  return G::template launch<orth_kernel<G, KIND, SPLIT>>(p, p.map, 1, s);
}

template <int KIND, bool AS, bool BS, bool SPLIT>
hipError_t launch_orth_product(const OrthArgs& p, hipStream_t s) {
  const int64_t big = ((p.rows + 255) / 256) * ((p.cols + 255) / 256);
  const int64_t mid = ((p.rows + 127) / 128) * ((p.cols + 127) / 128);
  if (big >= 128) return launch_orth_tile<Gemm<2, 4, 4, 2, AS, BS, false, true>, KIND, SPLIT>(p, s);
  if (mid >= 128) return launch_orth_tile<Gemm<2, 2, 2, 2, AS, BS, false, true>, KIND, SPLIT>(p, s);
  return launch_orth_tile<Gemm<2, 2, 1, 1, AS, BS, false, true>, KIND, SPLIT>(p, s);
}

int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// Workspace parts, in bytes.
struct OrthLayout {
  int64_t rp, kp, mp;  // padded sizes; mp: the shorter side
  bool tall, split;
  int64_t x_part, a_part;       // elements of one fp16 part
  int64_t head, x, keep, a, b, total;
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
    keep = x + 2 * parts * x_part * 2;  // two buffers of X
    a = keep + (split ? 0 : x_part * 4);
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
  float* keep = reinterpret_cast<float*>(ws + L.keep);
  const int64_t x_lo = SPLIT ? L.x_part : 0, a_lo = SPLIT ? L.a_part : 0;

  const int64_t n = R * K;
  if (dt == kF32) norm_kernel<kF32><<<kNormBlocks, 256, 0, s>>>(G, n, head);
  else if (dt == kF16) norm_kernel<kF16><<<kNormBlocks, 256, 0, s>>>(G, n, head);
  else norm_kernel<kBF16><<<kNormBlocks, 256, 0, s>>>(G, n, head);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t quads = L.rp * L.kp / 4;
  const unsigned grid = (unsigned)(quads / 256 < 2048 ? (quads + 255) / 256 : 2048);
  if (dt == kF32)
    start_kernel<kF32, SPLIT><<<grid, 256, 0, s>>>(G, R, K, L.rp, L.kp, eps, head, x[0], x[0] + x_lo);
  else if (dt == kF16)
    start_kernel<kF16, SPLIT><<<grid, 256, 0, s>>>(G, R, K, L.rp, L.kp, eps, head, x[0], x[0] + x_lo);
  else
    start_kernel<kBF16, SPLIT><<<grid, 256, 0, s>>>(G, R, K, L.rp, L.kp, eps, head, x[0], x[0] + x_lo);
  if ((e = hipGetLastError()) != hipSuccess) return e;

  auto op = [](const _Float16* p, int64_t ld, int64_t rows) {
    return GemmOperand{reinterpret_cast<const uint16_t*>(p), ld, rows};
  };
  for (int i = 0; i < steps; ++i) {
    const _Float16* from = x[i & 1];
    OrthArgs p{};
    p.segments = SPLIT ? 3 : 1;
    p.ca = 3.4445f;
    p.cb = -4.7750f;
    p.cc = 2.0315f;
    p.rho = i == 0 ? &head->rho : nullptr;
    // A = X X^T, or X^T X (both operands then have k as their row index)
    p.a = p.b = op(from, L.kp, L.mp);
    p.a_lo = p.b_lo = x_lo;
    p.steps = (int)((L.tall ? L.rp : L.kp) / kGemmStep);
    p.rows = p.cols = L.mp;
    p.hi = A;
    p.lo = A + a_lo;
    e = L.tall ? launch_orth_product<kGram, true, true, SPLIT>(p, s)
               : launch_orth_product<kGram, false, false, SPLIT>(p, s);
    if (e != hipSuccess) return e;
    // B = b A + c A A (A is symmetric: its rows are its columns)
    p.a = p.b = op(A, L.mp, L.mp);
    p.a_lo = p.b_lo = a_lo;
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
    p.from = i == 0 || SPLIT ? nullptr : keep;
    p.hi = x[(i + 1) & 1];
    p.lo = p.hi + x_lo;
    p.keep = keep;
    if (i + 1 == steps) {
      p.out = out;
      p.out_dt = dt;
      p.R = R;
      p.K = K;
    }
    if (L.tall) {
      p.a = op(from, L.kp, L.rp);
      p.b = op(B, L.mp, L.mp);
      p.a_lo = x_lo;
      p.b_lo = a_lo;
      e = launch_orth_product<kUpdate, false, false, SPLIT>(p, s);
    } else {
      p.a = op(B, L.mp, L.mp);
      p.b = op(from, L.kp, L.kp);
      p.a_lo = a_lo;
      p.b_lo = x_lo;
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
