// nm_act.h -- activations, their slopes, and the epilogue of a product Y = act(s Z + b) + residual
// (gfx950): what nm_spmm_act, nm_matvec_act and nm_spmm_act_grad share.
//
// All of it is fp32 on the product's fp32 (int8: int32) sums, rounded once where Z and Y are stored.
// Exponentials and reciprocals are the hardware's (v_exp_f32, v_rcp_f32: one unit in the last place of what
// they are given: an exponent a that was rounded before is 2^-22 a of a relative error at most),
// so a sigmoid takes four instructions and the epilogue's arithmetic hides under its memory traffic
// (bf16 11008 x 4096, 2048 columns, in turn on warm caches: the product alone 107 us, with silu, Z kept,
// 124, of which the stores are most; 4096 x 11008 with a residual 94 and 101).
#pragma once

#include "nm_launch.h"
#include "nm_mfma.h"

namespace nm {
namespace {

// The order of nm_act in include/nm.h.
enum { kActNone, kActRelu, kActRelu2, kActSilu, kActGelu, kActGeluTanh, kActs };

constexpr float kActLog2e = 1.44269504088896340736f;
constexpr float kRoot2Pi = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kCubic = 0.044715f;                  // of the tanh form of GELU

// 1 / (1 + e^-z): 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kActLog2e * z));
}

// The normal distribution function of z, and e^(-z^2 / 2).  The tail Phi(-u), u = |z|, is
// e^(-u^2 / 2) t p(t) with t = 1 / (1 + 0.28 u): p is a polynomial of degree 8 fitted to
// e^(u^2 / 2) Phi(-u) / t for u in 0 .. 60 by weighted least squares (relative error 9.2e-8, 4e-7 as
// evaluated here), so the tail keeps a relative accuracy, which 1 + erf loses: that and 2^-22 u^2 / 2 at
// most, since u^2 / 2 is rounded before the exponential (2e-6 at u = 4, 1e-5 at 9).
__device__ __forceinline__ float normal_cdf(float z, float& gauss) {
  const float u = fabsf(z), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28f, u, 1.f));
  gauss = __builtin_amdgcn_exp2f(z * z * (-0.5f * kActLog2e));
  float p = 0.025919387f;
  p = __builtin_fmaf(p, t, -0.098323286f);
  p = __builtin_fmaf(p, t, 0.10007188f);
  p = __builtin_fmaf(p, t, -0.012975537f);
  p = __builtin_fmaf(p, t, 0.075940855f);
  p = __builtin_fmaf(p, t, 0.08275791f);
  p = __builtin_fmaf(p, t, 0.103213914f);
  p = __builtin_fmaf(p, t, 0.11169085f);
  p = __builtin_fmaf(p, t, 0.11170407f);
  const float tail = p * t * gauss;
  return z < 0.f ? tail : 1.f - tail;
}

// z times a share of it; a share of 0 gives -0 for z = -infinity too (a NaN is in the share as well).
__device__ __forceinline__ float share_of(float z, float s) { return fmaxf(z, -3.402823466e38f) * s; }

// act(v) of N numbers; the choice is the same for the whole launch, so it is made once for all of them.
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];
      break;
    case kActRelu2:
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = v[e] < 0.f ? 0.f : v[e] * v[e];
      break;
    case kActSilu:
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = share_of(v[e], sigmoid(v[e]));
      break;
    case kActGelu:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float gauss;
        v[e] = share_of(v[e], normal_cdf(v[e], gauss));
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int e = 0; e < N; ++e) {  // (1 + tanh y) / 2 = sigmoid(2 y)
        const float z = v[e];
        v[e] = share_of(z, sigmoid(2.f * kRoot2Pi * z * __builtin_fmaf(kCubic * z, z, 1.f)));
      }
      break;
    default: break;
  }
}

// d[e] = act'(z[e]) d[e].  Past |z| = 100 the smooth slopes are 0 or 1 in fp32: z is held there, so
// that no infinity meets a zero.
__device__ __forceinline__ float hold_100(float z) { return fminf(fmaxf(z, -100.f), 100.f); }

template <int N>
__device__ __forceinline__ void act_slopes(int act, const float (&z)[N], float (&d)[N]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = z[e] > 0.f ? d[e] : 0.f;
      break;
    case kActRelu2:
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = z[e] > 0.f ? 2.f * z[e] * d[e] : 0.f;
      break;
    case kActSilu:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float h = hold_100(z[e]), s = sigmoid(h);
        const float slope = s * __builtin_fmaf(h, 1.f - s, 1.f);
        d[e] *= z[e] != z[e] ? z[e] : slope;
      }
      break;
    case kActGelu:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float gauss;
        const float h = hold_100(z[e]), cdf = normal_cdf(h, gauss);
        const float slope = __builtin_fmaf(h * 0.39894228040143267794f, gauss, cdf);
        d[e] *= z[e] != z[e] ? z[e] : slope;
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float h = hold_100(z[e]);
        const float s = sigmoid(2.f * kRoot2Pi * h * __builtin_fmaf(kCubic * h, h, 1.f));
        const float inner = 2.f * kRoot2Pi * __builtin_fmaf(3.f * kCubic * h, h, 1.f);
        const float slope = __builtin_fmaf(h * s * (1.f - s), inner, s);
        d[e] *= z[e] != z[e] ? z[e] : slope;
      }
      break;
    default: break;
  }
}

// ---- eight numbers of a row, of a type known at run time -------------------------------------

typedef float float4_any_t __attribute__((ext_vector_type(4), aligned(4)));

// Raw numbers i .. i + 7 of `p` (the first `left` of them; zeros after), 4 or 2 bytes each, at any
// element address.
struct RawEight {
  u32x4_t lo, hi;  // 16-bit numbers fill lo alone
};
__device__ __forceinline__ RawEight load_eight(const void* p, int dt, int64_t i, int64_t left) {
  RawEight r{u32x4_t{0, 0, 0, 0}, u32x4_t{0, 0, 0, 0}};
  if (dt == kF32) {
    const uint32_t* q = static_cast<const uint32_t*>(p) + i;
    typedef uint32_t any_t __attribute__((ext_vector_type(4), aligned(4)));
    if (left >= 8) {
      r.lo = *reinterpret_cast<const any_t*>(q);
      r.hi = *reinterpret_cast<const any_t*>(q + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e < left) r.lo[e] = q[e];
        if (e + 4 < left) r.hi[e] = q[e + 4];
      }
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (left >= 8) {
      r.lo = *reinterpret_cast<const u32x4_any_t*>(q);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) r.lo[e / 2] |= (uint32_t)q[e] << (16 * (e & 1));
    }
  }
  return r;
}

__device__ __forceinline__ void to_floats(const RawEight& r, int dt, float (&v)[8]) {
  if (dt == kF32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __uint_as_float(r.lo[e]);
      v[e + 4] = __uint_as_float(r.hi[e]);
    }
  } else if (dt == kBF16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = bf16_to_f32((r.lo[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f16_to_f32((r.lo[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
  }
}

__device__ __forceinline__ u32x4_t pack_eight(const float (&v)[8], int dt) {
  u32x4_t w;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = dt == kBF16 ? f32_to_bf16(v[2 * e]) | f32_to_bf16(v[2 * e + 1]) << 16
                       : f32_to_f16(v[2 * e]) | f32_to_f16(v[2 * e + 1]) << 16;
  return w;
}

// The first `left` of v to numbers i .. of `p`, rounded once.
__device__ __forceinline__ void store_eight(void* p, int dt, int64_t i, int64_t left,
                                            const float (&v)[8]) {
  if (dt == kF32) {
    float* q = static_cast<float*>(p) + i;
    if (left >= 8) {
      *reinterpret_cast<float4_any_t*>(q) = float4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<float4_any_t*>(q + 4) = float4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) q[e] = v[e];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    const u32x4_t w = pack_eight(v, dt);
    if (left >= 8) {
      *reinterpret_cast<u32x4_any_t*>(q) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) q[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
  }
}

// ---- the epilogue ------------------------------------------------------------------------------

// A product's output type that stands for "what the Epilogue says".
constexpr int kAct = 6;

struct Epilogue {
  const float* scale;    // of a row, or null
  const float* bias;     // of a row, or null
  const void* residual;  // in y's type, or null; may be y
  void* y;
  void* z;               // act's argument, in z_dt, or null
  int64_t ldx;           // row length of X, at least the product's T
  int act, y_dt, z_dt;
};

inline Epilogue epilogue_of(const Product& p) {
  return Epilogue{p.scale, p.bias, p.residual, p.y, p.z, p.ldx, p.act, p.y_dt, p.z_dt};
}

// What a product kernel's output argument is, and the row length of its X.
template <int YT>
struct OutOf {
  typedef void* __restrict__ type;
};
template <>
struct OutOf<kAct> {
  typedef Epilogue type;
};
template <typename I>
__device__ __forceinline__ I x_stride(const void*, I T) { return T; }
template <typename I>
__device__ __forceinline__ I x_stride(const Epilogue& ep, I) { return (I)ep.ldx; }

// One result: row, column and sum.
__device__ __forceinline__ void finish_one(const Epilogue& ep, int64_t row, int64_t col, int64_t T,
                                           float sum) {
  float v[1] = {sum};
  if (ep.scale) v[0] *= ep.scale[row];
  if (ep.bias) v[0] += ep.bias[row];
  const int64_t i = row * T + col;
  const auto put = [&](void* p, int dt, float x) {
    if (dt == kF32) store_from_f32<kF32>(p, i, x);
    else if (dt == kBF16) store_from_f32<kBF16>(p, i, x);
    else store_from_f32<kF16>(p, i, x);
  };
  if (ep.z) put(ep.z, ep.z_dt, v[0]);
  act_values(ep.act, v);
  if (ep.residual) {
    if (ep.y_dt == kF32) {
      v[0] += static_cast<const float*>(ep.residual)[i];
    } else {
      const uint32_t h = static_cast<const uint16_t*>(ep.residual)[i];
      v[0] += ep.y_dt == kBF16 ? bf16_to_f32(h) : f16_to_f32(h);
    }
  }
  put(ep.y, ep.y_dt, v[0]);
}

// 64 rows x 64 columns of sums in LDS, fp32, row-major, kSlabPitch floats a row (padded against bank
// conflicts), finished by one wave.  A lane takes eight columns from 8 (lane % 8) of rows
// 8 k + lane / 8, k = 0 .. 7, in two groups of four; a group's residual, scales and biases are loaded
// (GroupInputs) before the group ahead of it is worked on, the first ones before the slab is written.
// DT: the product's type, which Z has, and Y if it is not fp32 (8-bit products: any Y).
constexpr int kSlabPitch = 68;
constexpr int kSlabBytes = 64 * kSlabPitch * 4;

struct GroupInputs {
  RawEight residual[4];
  float scale[4], bias[4];
};

template <int DT>
__device__ __forceinline__ int y_type(const Epilogue& ep) {
  if constexpr (DT == kF32) return kF32;
  else if constexpr (DT == kBF16 || DT == kF16) return ep.y_dt == kF32 ? kF32 : DT;
  else return ep.y_dt;
}

template <int DT>
__device__ __forceinline__ void group_load(GroupInputs& in, const Epilogue& ep, int64_t row0,
                                           int64_t col0, int64_t R, int64_t T, int lane) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t row = row0 + 8 * k + (lane >> 3), col = col0 + 8 * (lane & 7);
    const bool live = row < R && col < T;
    in.scale[k] = ep.scale && live ? ep.scale[row] : 1.f;
    in.bias[k] = ep.bias && live ? ep.bias[row] : 0.f;
    if (ep.residual && live)
      in.residual[k] = load_eight(ep.residual, y_type<DT>(ep), row * T + col, T - col);
  }
}

template <int DT>
__device__ __forceinline__ void group_finish(const GroupInputs& in, const float* slab,
                                             const Epilogue& ep, int64_t row0, int64_t col0, int64_t R,
                                             int64_t T, int lane) {
  const int64_t row = row0 + (lane >> 3), col = col0 + 8 * (lane & 7), left = T - col;
  const float* sums = slab + (lane >> 3) * kSlabPitch + 8 * (lane & 7);
  float v[4][8];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4_t a = *reinterpret_cast<const float4_t*>(sums + 8 * k * kSlabPitch + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k][4 * h + e] = __builtin_fmaf(a[e], in.scale[k], in.bias[k]);
    }
  if (left <= 0) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (row + 8 * k >= R) break;
    const int64_t i = (row + 8 * k) * T + col;
    if constexpr (DT == kF32 || DT == kBF16 || DT == kF16)
      if (ep.z) store_eight(ep.z, DT, i, left, v[k]);
    act_values(ep.act, v[k]);
    if (ep.residual) {
      float x[8];
      to_floats(in.residual[k], y_type<DT>(ep), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] += x[e];
    }
    store_eight(ep.y, y_type<DT>(ep), i, left, v[k]);
  }
}

// The slab's two groups (their code once); `first` are the first one's inputs.
template <int DT>
__device__ __forceinline__ void slab_finish(const GroupInputs& first, const float* slab,
                                            const Epilogue& ep, int64_t row0, int64_t col0, int64_t R,
                                            int64_t T, int lane) {
  GroupInputs in = first;
#pragma unroll 1
  for (int g = 0; g < 2; ++g) {
    const GroupInputs now = in;
    if (g == 0) group_load<DT>(in, ep, row0 + 32, col0, R, T, lane);
    group_finish<DT>(now, slab + g * 32 * kSlabPitch, ep, row0 + 32 * g, col0, R, T, lane);
  }
}

// Two fragments down of 32 rows x 64 columns (layout as of store_block_128x64) to LDS.
template <typename AccV>
__device__ __forceinline__ void slab_write(const AccV (&a)[2], const AccV (&b)[2], float* slab,
                                           int lane) {
  const int l32 = lane & 31, q = lane >> 5;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float* d = slab + (8 * (i / 4) + 4 * q + (i % 4)) * kSlabPitch + 32 * f + l32;
      d[0] = (float)a[f][i];
      d[32 * kSlabPitch] = (float)b[f][i];
    }
}

// LDS serves a wave in order: between its writes and its other lanes' reads only the compiler has to
// keep it.
__device__ __forceinline__ void keep_order() { asm volatile("" ::: "memory"); }

// Stores a wave's 64 x 64 block through its own kSlabBytes of LDS.
template <int DT, typename AccV>
__device__ __forceinline__ void finish_block(const AccV (&acc)[2][2], uint8_t* lds, const Epilogue& ep,
                                             int64_t row0, int64_t col0, int64_t R, int64_t T,
                                             int lane) {
  float* slab = reinterpret_cast<float*>(lds);
  GroupInputs in;
  group_load<DT>(in, ep, row0, col0, R, T, lane);
  slab_write(acc[0], acc[1], slab, lane);
  keep_order();
  slab_finish<DT>(in, slab, ep, row0, col0, R, T, lane);
}

// The same for a workgroup of four waves that hold 128 x 64 blocks each and four that do not: the
// blocks go to LDS whole, and all eight waves finish half of one each, since the activation's
// arithmetic would keep four waves longer than their stores (bf16 11008 x 4096, 2048 columns, silu,
// Z kept: 175 us a call with four, 139 with eight).  Wave w has block w % 4 and half w / 4.
constexpr int kBlockBytes = 2 * kSlabBytes;
__device__ __forceinline__ float* slab_of(uint8_t* smem, int wave) {
  return reinterpret_cast<float*>(smem + (wave & 3) * kBlockBytes + (wave >> 2) * kSlabBytes);
}
template <int DT>
__device__ __forceinline__ void finish_half(uint8_t* smem, const Epilogue& ep, int m0, int t0, int R,
                                            int T, int wave, int lane) {
  const int row0 = m0 + ((wave & 3) >> 1) * 128 + (wave >> 2) * 64, col0 = t0 + (wave & 1) * 64;
  GroupInputs in;
  group_load<DT>(in, ep, row0, col0, R, T, lane);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // every block is in LDS
  slab_finish<DT>(in, slab_of(smem, wave), ep, row0, col0, R, T, lane);
}

}  // namespace
}  // namespace nm
