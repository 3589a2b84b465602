// nm_xent.hip -- softmax cross entropy of the logits L = W X (V x T) over a large vocabulary
// V (nm_xent), and its gradient (nm_xent_grad), without ever storing the logits.
//
//   lse[t] = log sum over v of exp L[v, t],   loss[t] = lse[t] - L[y_t, t]
//   P[v, t] = (exp(L[v, t] - lse[t]) - [v = y_t]) g[t],   dW = P X^T,   dX = W^T P
//
// Loss: the product's tiles (nm_gemm.h) end in an epilogue that reduces each wave's rows of a
// column to their maximum and the sum of exp(. - maximum); a second kernel joins those.
//
// Gradient: the vocabulary is taken in pieces whose P fits a bounded workspace.  For each piece
// the logits are multiplied again and leave the epilogue as P in 16 bits (the operand the next
// two products need; the rounding is the same relative size as that of dW and dX themselves), then
// dW of the piece is one product, and W^T P is added to fp32 sums of dX.  g is taken over its largest,
// times 2^14, before the rounding, and the products are scaled back in fp32.  fp16: a token whose g
// is below 2^-14 of the largest keeps its P at 2^0 for a probability of 1, so that its column of dX
// loses no more to underflow than any other's, and brings the rest of its g to dW as a power of two
// on its column of X.
//
// Bound by the matrix cores where tokens are many: 32768 x 4096 with 2048 tokens in bf16 takes 469
// us for the loss's product (1170 TFLOP/s), and for the gradient's three, in two pieces, 464, 467 and
// 466 us (1180), with 43 us of copies and joins beside them.  With few tokens the loss is bound by the
// read of W (32000 x 768, 61 tokens: 13.8 us, 3.6 TB/s) and the launches.
//
// Tokens with a target outside 0 .. V - 1 are left out: their loss is 0 and their column of X
// is read as zeros in the gradient, so that not even infinities or NaN in it reach dW.
#include <algorithm>

#include "nm_gemm.h"
#include "nm_grid.h"
#include "nm_tiles.h"

namespace nm {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
int64_t pad256b(int64_t n) { return (n + 255) / 256 * 256; }

struct TokenArgs {  // of the tokens, padded to a whole number of 64
  int* y;           // target, -1 where left out
  float* lse;
  float* g;         // what P's column is times: g times 2^14 over the largest, over `down`
  float* down;      // fp16: what X's column is times for dW, a power of two up to 1
  float* back;      // what brings dX's column back
  float* all_back;  // one number: what brings dW back
  int* any_down;    // one number: whether a token's `down` is below 1
};

// One workgroup: the largest finite |g| of the tokens that count, then all g over it, times 2^14.  A
// mean's equal g become 2^14, so that the entries of P at the targets, just below 2^14 in size, lie
// where 16-bit numbers are densest for their size.  DOWN (fp16, whose normal numbers end at 2^-14): a
// smaller g keeps its P between 2^0 and 2^1 at least.
template <bool DOWN>
__device__ __forceinline__ void prepare_tokens(const int64_t* __restrict__ target,
                                               const float* __restrict__ lse,
                                               const float* __restrict__ gout, int64_t V, int64_t T,
                                               int64_t Tp, const TokenArgs& out) {
  __shared__ float part[4];
  __shared__ int any;
  if (threadIdx.x == 0) any = 0;
  float top = 0.f;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < T; t += 256)
    if (target[t] >= 0 && target[t] < V && fabsf(gout[t]) < INFINITY) top = fmaxf(top, fabsf(gout[t]));
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, part[i]);
  const bool scaled = top > 0.f;
  const float back = scaled ? top * 0x1p-14f : 1.f;
  int top_e;
  const float top_m = frexpf(top, &top_e);
  bool mine = false;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < Tp; t += 256) {
    const bool live = t < T && target[t] >= 0 && target[t] < V;
    const float g = live ? gout[t] : 0.f;
    float p = scaled ? g / top * 0x1p14f : g;
    out.y[t] = live ? (int)target[t] : -1;
    out.lse[t] = live ? lse[t] : 0.f;
    if constexpr (DOWN) {
      int e = 0;
      if (g != 0.f && fabsf(p) < 1.f) {  // g = m 2^e with m in [1/2, 1)
        const float m = frexpf(g, &e);
        p = m / top_m;
        e -= top_e - 14;
        if (fabsf(p) < 1.f) {
          p *= 2.f;
          --e;
        }
        mine |= e < 0;
      }
      out.down[t] = ldexpf(1.f, e > -100 ? e : -100);  // of fp16 nothing is left there
      out.back[t] = ldexpf(back, e);
    } else {
      out.back[t] = back;
    }
    out.g[t] = p;
  }
  if (threadIdx.x == 0) *out.all_back = back;
  if constexpr (DOWN) {
    if (mine) atomicOr(&any, 1);
    __syncthreads();
    if (threadIdx.x == 0) *out.any_down = any;
  }
}

struct PadArgs {
  const uint16_t* in;  // rows x cols
  int64_t rows, cols;
  uint16_t* out;       // rp x cp, zeros past the input
  int64_t rp, cp;
  // the gradient's copy of X: zeros at the columns of tokens left out, and the last workgroup
  // prepares the tokens
  const int64_t* target;
  const float *lse, *gout;
  int64_t V;
  TokenArgs tok;
};

// A thread keeps its eight columns and walks down the rows.
template <bool TOKENS, bool DOWN = false>
__global__ void __launch_bounds__(256) pad_kernel(PadArgs p) {
  const int64_t blocks = gridDim.x - (TOKENS ? 1 : 0);
  if (TOKENS && blockIdx.x == blocks) {
    prepare_tokens<DOWN>(p.target, p.lse, p.gout, p.V, p.cols, p.cp, p.tok);
    return;
  }
  const int64_t chunks = p.cp / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t stride = blocks * 256 / chunks, c = i % chunks * 8;
  if (i / chunks >= stride) return;
  uint32_t keep[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bool take = c + e < p.cols;
    if (TOKENS && take) take = p.target[c + e] >= 0 && p.target[c + e] < p.V;
    const uint32_t half = take ? 0xFFFFu << (16 * (e & 1)) : 0u;
    keep[e / 2] = e & 1 ? keep[e / 2] | half : half;
  }
#pragma unroll 4
  for (int64_t r = i / chunks; r < p.rp; r += stride) {
    u32x4_t v{0, 0, 0, 0};
    if (r < p.rows) {
      const uint16_t* x = p.in + r * p.cols + c;
      if (c + 8 <= p.cols) {
        v = *reinterpret_cast<const u32x4_any_t*>(x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < p.cols) v[e / 2] |= (uint32_t)x[e] << (16 * (e & 1));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] &= keep[e];
    *reinterpret_cast<u32x4_t*>(p.out + r * p.cp + c) = v;
  }
}

// A chunk to a thread until two workgroups to a unit, more rows a thread from there, since each
// thread reads its columns' targets first (4096 x 2048: 17 us with 512 workgroups, 23 with 2048);
// and no fewer threads than a row has chunks.
template <bool TOKENS, bool DOWN = false>
hipError_t launch_pad(const PadArgs& p, hipStream_t s) {
  const int64_t chunks = p.cp / 8, least = (chunks + 255) / 256;
  int64_t blocks = (p.rp * chunks + 255) / 256;
  if (blocks > 512) blocks = 512;
  if (blocks < least) blocks = least;
  if (p.rp * chunks > 0 || TOKENS)
    pad_kernel<TOKENS, DOWN><<<(unsigned)(blocks + (TOKENS ? 1 : 0)), 256, 0, s>>>(p);
  return hipGetLastError();
}

template <class G>
struct TileTag {
  typedef G type;
};
template <bool AS, bool BS, bool BF16, bool SWAP, typename F>
hipError_t with_tile(int tile, F&& f) {
  if (tile == kTile256) return f(TileTag<Gemm<2, 4, 4, 2, AS, BS, BF16, SWAP, 2>>{});
  if (tile == kTile128) return f(TileTag<Gemm<2, 4, 2, 1, AS, BS, BF16, SWAP, 2>>{});
  return f(TileTag<Gemm<2, 2, 2, 1, AS, BS, BF16, SWAP, 3>>{});
}

// ---- loss ------------------------------------------------------------------------------

struct StatsArgs {
  GemmOperand w, x;
  int steps;
  GemmMap map;
  int64_t V, T;
  const int64_t* target;
  float *top, *sum;  // [rows of waves][T]
  float* hit;        // [T]: the target's logit
};

// What exponents are taken relative to: the maximum, or 0 where that is an infinity, so that logits
// of -infinity add 0 and one of +infinity makes the sum and its logarithm +infinity.
__device__ __forceinline__ float base_of(float top) { return fabsf(top) < INFINITY ? top : 0.f; }

template <class G>
__global__ void __launch_bounds__(G::kThreads) stats_kernel(StatsArgs p) {
  constexpr int FM = G::kFM, FN = G::kFN, WM = G::kWM, WN = G::kWN;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  int tm, tn;
  if (!p.map.tile_of(blockIdx.x, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * G::kBM, n0 = (int64_t)tn * G::kBN;
  typename G::Acc acc;
  G::clear(acc);
  G::run(p.w, p.x, m0, n0, p.steps, (int64_t)p.steps * kGemmStep, smem, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / WN, wn = wave % WN;
  const int64_t row0 = m0 + wm * 32 * FM + 4 * (lane >> 5);
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t t = n0 + wn * 32 * FN + 32 * j + (lane & 31);
    const bool in = t < p.T;
    // the target as a row of this lane's: its registers hold rows 32 i + 8 g + e
    const int64_t y = in ? p.target[t] : -1;
    const int64_t yr = y - row0;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int off = 32 * i + 8 * (r / 4) + r % 4;
        if (in && y < p.V && yr == off) p.hit[t] = acc[i][j][r];
        if (row0 + off >= p.V) acc[i][j][r] = -INFINITY;
        m = fmaxf(m, acc[i][j][r]);
      }
    m = fmaxf(m, __shfl_xor(m, 32));
    const float shift = base_of(m) * kLog2e;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], kLog2e, -shift));
    s += __shfl_xor(s, 32);
    if (in && lane < 32) {
      const int64_t at = ((int64_t)tm * WM + wm) * p.T + t;
      p.top[at] = m;
      p.sum[at] = s;
    }
  }
}

// 32 tokens a workgroup, 32 threads a token; each joins every 32nd partial, then they join.
__global__ void __launch_bounds__(1024)
    join_kernel(const float* __restrict__ top, const float* __restrict__ sum, int64_t parts,
                int64_t T, int64_t V, const int64_t* __restrict__ target,
                const float* __restrict__ hit, float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float ms[32][33], ss[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * 32 + x;
  float m = -INFINITY, s = 0.f;
  if (t < T) {
    // eight loads of each kind in flight at a time
    for (int64_t i = y; i < parts; i += 8 * 32) {
      float mi[8], si[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool in = i + 32 * k < parts;
        mi[k] = in ? top[(i + 32 * k) * T + t] : -INFINITY;
        si[k] = in ? sum[(i + 32 * k) * T + t] : 0.f;
      }
      float n = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) n = fmaxf(n, mi[k]);
      const float sh = base_of(n);
      s *= __builtin_amdgcn_exp2f((m - sh) * kLog2e);
#pragma unroll
      for (int k = 0; k < 8; ++k) s += si[k] * __builtin_amdgcn_exp2f((mi[k] - sh) * kLog2e);
      m = n;
    }
  }
  ms[y][x] = m;
  ss[y][x] = s;
  __syncthreads();
  if (y == 0 && t < T) {
    float top_all = -INFINITY;
    for (int i = 0; i < 32; ++i) top_all = fmaxf(top_all, ms[i][x]);
    const float sh = base_of(top_all);
    float total = 0.f;
    for (int i = 0; i < 32; ++i) total += ss[i][x] * __builtin_amdgcn_exp2f((ms[i][x] - sh) * kLog2e);
    const float l = sh + __builtin_amdgcn_logf(total) * kLn2;
    lse[t] = l;
    const int64_t yt = target[t];
    loss[t] = yt >= 0 && yt < V ? l - hit[t] : 0.f;
  }
}

struct LossLayout {
  int64_t Kp, Tp;
  bool copy_x, copy_w;
  int tile;
  int64_t x, w, top, sum, hit, total, parts;
  LossLayout(int64_t V, int64_t K, int64_t T) {
    Kp = pad64(K);
    copy_w = K % 64 != 0;
    copy_x = copy_w || T % 8 != 0;
    Tp = copy_x ? pad64(T) : T;
    tile = pick_tile(V, T, Kp / kGemmStep);
    parts = (V + kTileM[tile] - 1) / kTileM[tile] * 2;  // every tile has two rows of waves
    x = 0;
    w = x + (copy_x ? pad256b(Kp * Tp * 2) : 0);
    top = w + (copy_w ? pad256b(V * Kp * 2) : 0);
    sum = top + pad256b(parts * T * 4);
    hit = sum + pad256b(parts * T * 4);
    total = hit + pad256b(T * 4);
  }
};

// ---- gradient --------------------------------------------------------------------------

// fp16: the X that dW is formed from where a token's column is brought down, rows x Tp.
struct DownArgs {
  const uint16_t* x;
  int64_t rows, Tp;
  const float* down;
  const int* any;    // without any, X itself is used
  uint16_t* out;
};
__device__ __forceinline__ void bring_down(const DownArgs& p, int64_t first, int64_t stride) {
  if (*p.any == 0) return;
  for (int64_t i = first; i < p.rows * p.Tp / 8; i += stride) {
    const int64_t t = 8 * i % p.Tp;
    u32x4_t v = reinterpret_cast<const u32x4_t*>(p.x)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = f32_to_f16(f16_to_f32(v[e] & 0xFFFFu) * p.down[t + 2 * e]) |
             f32_to_f16(f16_to_f32(v[e] >> 16) * p.down[t + 2 * e + 1]) << 16;
    reinterpret_cast<u32x4_t*>(p.out)[i] = v;
  }
}

struct ProbArgs {
  GemmOperand w, x;  // w from the piece's first row on
  int steps;
  GemmMap map;
  int64_t v0, V;     // the piece's first row; rows of W
  int64_t rows, Tp;  // of P, padded
  TokenArgs tok;
  uint16_t* P;       // rows x Tp
  int groups;        // workgroups of the product; those past them (fp16, first piece) bring X down
  DownArgs down;
};

template <class G, bool BF16>
__global__ void __launch_bounds__(G::kThreads) prob_kernel(ProbArgs p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  if (!BF16 && (int)blockIdx.x >= p.groups) {
    bring_down(p.down, (int64_t)(blockIdx.x - p.groups) * G::kThreads + threadIdx.x,
               (int64_t)(gridDim.x - p.groups) * G::kThreads);
    return;
  }
  int tm, tn;
  if (!p.map.tile_of(blockIdx.x, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * G::kBM, n0 = (int64_t)tn * G::kBN;
  typename G::Acc acc;
  G::clear(acc);
  G::run(p.w, p.x, m0, n0, p.steps, (int64_t)p.steps * kGemmStep, smem, acc);
  const int64_t row0 = G::row0(m0), col0 = G::col0(n0);
#pragma unroll
  for (int j = 0; j < G::kFN; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t col = col0 + 32 * j + 8 * c;
      float4_t lse{}, g{};
      int4 y{-1, -1, -1, -1};
      if (col < p.Tp) {
        lse = *reinterpret_cast<const float4_t*>(p.tok.lse + col);
        g = *reinterpret_cast<const float4_t*>(p.tok.g + col);
        y = *reinterpret_cast<const int4*>(p.tok.y + col);
      }
      const int ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < G::kFM; ++i) {
        const int v = (int)(p.v0 + row0 + 32 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f((acc[i][j][4 * c + e] - lse[e]) * kLog2e);
          acc[i][j][4 * c + e] =
              v < p.V && ys[e] >= 0 ? (x - (v == ys[e] ? 1.f : 0.f)) * g[e] : 0.f;
        }
      }
    }
  G::template store16<BF16>(acc, m0, n0, smem, p.P, p.Tp, p.rows, p.Tp);
}

struct GradXArgs {
  GemmOperand w, q;  // W's piece and P, both with v as their row index
  int64_t klen;      // rows of the piece
  int steps, per;    // steps of 64 of them; of which each split takes `per`
  GemmMap map;
  int64_t K, Tp;
  float* sums;       // [splits][K][Tp]
  bool add;          // to what earlier pieces left there
};

template <class G>
__device__ __forceinline__ void grad_x_tile(const GradXArgs& p, int group, int split,
                                            uint8_t* smem) {
  int tm, tn;
  if (!p.map.tile_of(group, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * G::kBM, n0 = (int64_t)tn * G::kBN;
  const int s0 = split * p.per, steps = min(p.per, p.steps - s0);
  GemmOperand w = p.w, q = p.q;
  w.p += (int64_t)s0 * kGemmStep * w.ld;
  q.p += (int64_t)s0 * kGemmStep * q.ld;
  typename G::Acc acc;
  G::clear(acc);
  if (steps > 0) G::run(w, q, m0, n0, steps, p.klen - (int64_t)s0 * kGemmStep, smem, acc);
  float* out = p.sums + (int64_t)split * p.K * p.Tp;
  const int64_t row0 = G::row0(m0), col0 = G::col0(n0);
#pragma unroll
  for (int i = 0; i < G::kFM; ++i) {
    const int64_t row = row0 + 32 * i;
    float4_t before[4 * G::kFN];  // read together: between the stores each would be waited for
    if (p.add) {
#pragma unroll
      for (int q = 0; q < 4 * G::kFN; ++q) {
        const int64_t col = col0 + 32 * (q / 4) + 8 * (q % 4);
        if (row < p.K && col < p.Tp)
          before[q] = *reinterpret_cast<const float4_t*>(out + row * p.Tp + col);
      }
    }
#pragma unroll
    for (int q = 0; q < 4 * G::kFN; ++q) {
      const int64_t col = col0 + 32 * (q / 4) + 8 * (q % 4);
      if (row >= p.K || col >= p.Tp) continue;
      float4_t v = G::quad(acc, i, q / 4, q % 4);
      if (p.add) v += before[q];
      *reinterpret_cast<float4_t*>(out + row * p.Tp + col) = v;
    }
  }
}

struct GradWArgs {
  GemmOperand q, x;
  int steps;
  GemmMap map;
  int64_t rows, K;  // rows of W in the piece
  const float* back;
  const uint16_t* x_down;  // fp16: the X to use if *any_down
  const int* any_down;
  uint16_t* dW;     // from the piece's first row on
};

template <class G, bool BF16>
__device__ __forceinline__ void grad_w_tile(const GradWArgs& p, int group, uint8_t* smem) {
  int tm, tn;
  if (!p.map.tile_of(group, tm, tn)) return;
  const int64_t m0 = (int64_t)tm * G::kBM, n0 = (int64_t)tn * G::kBN;
  typename G::Acc acc;
  G::clear(acc);
  GemmOperand x = p.x;
  if (!BF16 && __builtin_amdgcn_readfirstlane(*p.any_down)) x.p = p.x_down;
  G::run(p.q, x, m0, n0, p.steps, (int64_t)p.steps * kGemmStep, smem, acc);
  const float back = *p.back;
#pragma unroll
  for (int i = 0; i < G::kFM; ++i)
#pragma unroll
    for (int j = 0; j < G::kFN; ++j) acc[i][j] *= back;
  G::template store16<BF16>(acc, m0, n0, smem, p.dW, p.K, p.rows, p.K);
}

template <class G>
__global__ void __launch_bounds__(G::kThreads) grad_x_kernel(GradXArgs p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  grad_x_tile<G>(p, blockIdx.x, blockIdx.y, smem);
}
template <class G, bool BF16>
__global__ void __launch_bounds__(G::kThreads) grad_w_kernel(GradWArgs p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  grad_w_tile<G, BF16>(p, blockIdx.x, smem);
}

// Both in one launch, dX's longer sums first: where each alone has few tiles, the units that one
// leaves idle take the other's.
struct GradArgs {
  GradXArgs x;
  GradWArgs w;
  int groups_x, splits;  // workgroups for each split of dX
};
template <class GX, class GW, bool BF16>
__global__ void __launch_bounds__(GX::kThreads) grad_kernel(GradArgs p) {
  static_assert(GX::kThreads == GW::kThreads && GX::kLds == GW::kLds, "one launch for both");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int b = blockIdx.x, first_w = p.groups_x * p.splits;
  if (b < first_w) grad_x_tile<GX>(p.x, b % p.groups_x, b / p.groups_x, smem);
  else grad_w_tile<GW, BF16>(p.w, b - first_w, smem);
}

// dX from its sums; zeros at the tokens left out, also where a word's row of W is not finite and made
// NaN of their P of zeros.
template <bool BF16>
__global__ void __launch_bounds__(256)
    finish_x_kernel(const float* __restrict__ sums, int splits, int64_t K, int64_t T, int64_t Tp,
                    const float* __restrict__ back, const int* __restrict__ y,
                    uint16_t* __restrict__ dX) {
  const int64_t total = K * Tp / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    float4_t v = reinterpret_cast<const float4_t*>(sums)[i];
    for (int z = 1; z < splits; ++z) {
      const float4_t b = reinterpret_cast<const float4_t*>(sums)[z * total + i];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += b[e];
    }
    const int64_t k = 4 * i / Tp, t = 4 * i % Tp;
    const int4 y4 = *reinterpret_cast<const int4*>(y + t);
    const float4_t f = *reinterpret_cast<const float4_t*>(back + t);
    const int ys[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (t + e < T)
        store_from_f32<BF16 ? kBF16 : kF16>(dX, k * T + t + e, ys[e] >= 0 ? v[e] * f[e] : 0.f);
  }
}

struct GradLayout {
  int64_t Kp, Tp, piece;  // piece: rows of W at a time
  bool copy_w;
  int tile_x, splits;     // of dX
  int64_t x, x_down, w, tok_y, tok_lse, tok_g, tok_down, tok_back, all_back, P, sums, total;
  GradLayout(int64_t V, int64_t K, int64_t T) {
    Kp = pad64(K);
    Tp = pad64(T);
    copy_w = K % 64 != 0;
    const XentGradCut cut(V, K, T);
    piece = cut.piece;
    tile_x = cut.tile_x;
    splits = cut.splits;
    x = 0;
    x_down = x + pad256b(Kp * Tp * 2);
    w = x_down + pad256b(Kp * Tp * 2);
    tok_y = w + (copy_w ? pad256b(V * Kp * 2) : 0);
    tok_lse = tok_y + pad256b(Tp * 4);
    tok_g = tok_lse + pad256b(Tp * 4);
    tok_down = tok_g + pad256b(Tp * 4);
    tok_back = tok_down + pad256b(Tp * 4);
    all_back = tok_back + pad256b(Tp * 4);  // and any_down
    P = all_back + 256;
    sums = P + pad256b(pad64(piece) * Tp * 2);
    total = sums + pad256b((int64_t)splits * K * Tp * 4);
  }
};

__global__ void __launch_bounds__(256) zero_kernel(uint16_t* out, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    out[i] = 0;
}

template <bool BF16>
hipError_t run_grad(const uint16_t* W, const uint16_t* X, int64_t V, int64_t K, int64_t T,
                    const int64_t* target, const float* lse, const float* gout, uint16_t* dW,
                    uint16_t* dX, uint8_t* ws, hipStream_t s) {
  if (T == 0) {  // no token: dX is empty
    zero_kernel<<<stride_grid(V * K, 256), 256, 0, s>>>(dW, V * K);
    return hipGetLastError();
  }
  const GradLayout L(V, K, T);
  uint16_t* Xp = reinterpret_cast<uint16_t*>(ws + L.x);
  uint16_t* P = reinterpret_cast<uint16_t*>(ws + L.P);
  float* sums = reinterpret_cast<float*>(ws + L.sums);
  uint16_t* x_down = reinterpret_cast<uint16_t*>(ws + L.x_down);
  const TokenArgs tok{reinterpret_cast<int*>(ws + L.tok_y),
                      reinterpret_cast<float*>(ws + L.tok_lse),
                      reinterpret_cast<float*>(ws + L.tok_g),
                      reinterpret_cast<float*>(ws + L.tok_down),
                      reinterpret_cast<float*>(ws + L.tok_back),
                      reinterpret_cast<float*>(ws + L.all_back),
                      reinterpret_cast<int*>(ws + L.all_back) + 1};
  const PadArgs pad_x{X, K, T, Xp, L.Kp, L.Tp, target, lse, gout, V, tok};
  hipError_t e;
  if ((e = launch_pad<true, !BF16>(pad_x, s)) != hipSuccess) return e;
  const uint16_t* Wp = W;
  if (L.copy_w) {
    uint16_t* w = reinterpret_cast<uint16_t*>(ws + L.w);
    if ((e = launch_pad<false>(PadArgs{W, V, K, w, V, L.Kp}, s)) != hipSuccess) return e;
    Wp = w;
  }
  const int64_t ldw = L.Kp;
  for (int64_t v0 = 0; v0 < V; v0 += L.piece) {
    const int64_t rows = V - v0 < L.piece ? V - v0 : L.piece, rp = pad64(rows);
    ProbArgs a{};
    a.w = GemmOperand{Wp + v0 * ldw, ldw, rows, 0};
    a.x = GemmOperand{Xp, L.Tp, L.Tp, 0};
    a.steps = (int)(L.Kp / kGemmStep);
    a.v0 = v0;
    a.V = V;
    a.rows = rp;
    a.Tp = L.Tp;
    a.tok = tok;
    a.P = P;
    a.down = DownArgs{Xp, L.Kp, L.Tp, tok.down, tok.any_down, x_down};
    const int down = BF16 || v0 > 0 ? 0 : (int)std::min<int64_t>(L.Kp * L.Tp / 8 / 256, 256);
    e = with_tile<false, true, BF16, true>(pick_tile(rp, L.Tp, a.steps), [&](auto tag) {
      typedef typename decltype(tag)::type G;
      a.map = make_gemm_map((rp + G::kBM - 1) / G::kBM, (L.Tp + G::kBN - 1) / G::kBN);
      a.groups = a.map.groups();
      return G::template launch<prob_kernel<G, BF16>>(a, a.groups + down, 1, s);
    });
    if (e != hipSuccess) return e;

    GradWArgs b{};
    b.q = GemmOperand{P, L.Tp, rp, 0};
    b.x = GemmOperand{Xp, L.Tp, L.Kp, 0};
    b.steps = (int)(L.Tp / kGemmStep);
    b.rows = rows;
    b.K = K;
    b.back = tok.all_back;
    b.x_down = x_down;
    b.any_down = tok.any_down;
    b.dW = dW + v0 * K;
    GradXArgs c{};
    c.w = GemmOperand{Wp + v0 * ldw, ldw, L.Kp, 0};
    c.q = GemmOperand{P, L.Tp, L.Tp, 0};
    c.klen = rows;
    c.steps = (int)(rp / kGemmStep);
    c.per = (c.steps + L.splits - 1) / L.splits;
    c.K = K;
    c.Tp = L.Tp;
    c.sums = sums;
    c.add = v0 > 0;
    const int tile_w = pick_tile(rows, K, b.steps);
    if (tile_w == kTile128 && L.tile_x == kTile128) {
      typedef Gemm<2, 4, 2, 1, true, true, BF16, true, 2> GX;
      typedef Gemm<2, 4, 2, 1, false, false, BF16, true, 2> GW;
      GradArgs both{c, b, 0, L.splits};
      both.x.map = make_gemm_map((K + 127) / 128, (L.Tp + 127) / 128);
      both.w.map = make_gemm_map((rows + 127) / 128, (K + 127) / 128);
      both.groups_x = both.x.map.groups();
      e = GX::template launch<grad_kernel<GX, GW, BF16>>(
          both, both.groups_x * L.splits + both.w.map.groups(), 1, s);
      if (e != hipSuccess) return e;
      continue;
    }
    e = with_tile<true, true, BF16, true>(L.tile_x, [&](auto tag) {
      typedef typename decltype(tag)::type G;
      c.map = make_gemm_map((K + G::kBM - 1) / G::kBM, (L.Tp + G::kBN - 1) / G::kBN);
      return G::template launch<grad_x_kernel<G>>(c, c.map.groups(), L.splits, s);
    });
    if (e != hipSuccess) return e;
    e = with_tile<false, false, BF16, true>(tile_w, [&](auto tag) {
      typedef typename decltype(tag)::type G;
      b.map = make_gemm_map((rows + G::kBM - 1) / G::kBM, (K + G::kBN - 1) / G::kBN);
      return G::template launch<grad_w_kernel<G, BF16>>(b, b.map.groups(), 1, s);
    });
    if (e != hipSuccess) return e;
  }
  finish_x_kernel<BF16><<<stride_grid(K * L.Tp / 4, 256), 256, 0, s>>>(sums, L.splits, K, T, L.Tp,
                                                                     tok.back, tok.y, dX);
  return hipGetLastError();
}

}  // namespace

size_t xent_workspace_bytes(int64_t V, int64_t K, int64_t T) {
  return (size_t)LossLayout(V, K, T).total;
}
size_t xent_grad_workspace_bytes(int64_t V, int64_t K, int64_t T) {
  return (size_t)GradLayout(V, K, T).total;
}

hipError_t launch_xent(const void* W, const void* X, int dt, int64_t V, int64_t K, int64_t T,
                       const int64_t* target, float* loss, float* lse, void* workspace,
                       hipStream_t s) {
  const LossLayout L(V, K, T);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  StatsArgs p{};
  const uint16_t* w = static_cast<const uint16_t*>(W);
  const uint16_t* x = static_cast<const uint16_t*>(X);
  hipError_t e;
  if (L.copy_x) {
    uint16_t* c = reinterpret_cast<uint16_t*>(ws + L.x);
    if ((e = launch_pad<false>(PadArgs{x, K, T, c, L.Kp, L.Tp}, s)) != hipSuccess) return e;
    x = c;
  }
  if (L.copy_w) {
    uint16_t* c = reinterpret_cast<uint16_t*>(ws + L.w);
    if ((e = launch_pad<false>(PadArgs{w, V, K, c, V, L.Kp}, s)) != hipSuccess) return e;
    w = c;
  }
  p.w = GemmOperand{w, L.Kp, V, 0};
  p.x = GemmOperand{x, L.Tp, L.Tp, 0};
  p.steps = (int)(L.Kp / kGemmStep);
  p.V = V;
  p.T = T;
  p.target = target;
  p.top = reinterpret_cast<float*>(ws + L.top);
  p.sum = reinterpret_cast<float*>(ws + L.sum);
  p.hit = reinterpret_cast<float*>(ws + L.hit);
  const auto launch = [&](auto tag) {
    typedef typename decltype(tag)::type G;
    p.map = make_gemm_map((V + G::kBM - 1) / G::kBM, (T + G::kBN - 1) / G::kBN);
    return G::template launch<stats_kernel<G>>(p, p.map.groups(), 1, s);
  };
  e = dt == kBF16 ? with_tile<false, true, true, false>(L.tile, launch)
                  : with_tile<false, true, false, false>(L.tile, launch);
  if (e != hipSuccess) return e;
  join_kernel<<<(unsigned)((T + 31) / 32), 1024, 0, s>>>(p.top, p.sum, L.parts, T, V, target, p.hit,
                                                       loss, lse);
  return hipGetLastError();
}

hipError_t launch_xent_grad(const void* W, const void* X, int dt, int64_t V, int64_t K, int64_t T,
                            const int64_t* target, const float* lse, const float* gout, void* dW,
                            void* dX, void* workspace, hipStream_t s) {
  const uint16_t* w = static_cast<const uint16_t*>(W);
  const uint16_t* x = static_cast<const uint16_t*>(X);
  uint16_t* a = static_cast<uint16_t*>(dW);
  uint16_t* b = static_cast<uint16_t*>(dX);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return dt == kBF16 ? run_grad<true>(w, x, V, K, T, target, lse, gout, a, b, ws, s)
                     : run_grad<false>(w, x, V, K, T, target, lse, gout, a, b, ws, s);
}

}  // namespace nm
