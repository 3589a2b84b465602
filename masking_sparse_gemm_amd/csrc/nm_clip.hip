// nm_clip.hip -- the global norm of many tensors (nm_grad_norm) and clipping by it (nm_clip_grads).
//
//   norm = sqrt(sum over all tensors and entries of g^2),   out = g min(1, max_norm / norm)
//
// The tensors' addresses and sizes travel as kernel arguments, kTable of them a launch, so nothing is
// copied to the device and a captured graph keeps them.  Entries are taken in chunks of 32 KB, by
// workgroups in turn, each of which walks on through the tensors from its last chunk.  Squares are
// added eight at a time in fp32 and then in fp64 (all in fp64 where eight squares leave fp32's range),
// and the workgroups' sums are joined in a fixed order by every workgroup of the second pass: two
// launches for up to kTable tensors.
//
// Bound by memory, the first pass by reads, the second by a read and a write.  The second pass takes
// the chunks last first, since what the first pass read last is still in the 256 MB cache, and writes
// past the caches, so that it stays there (405 M bf16 gradients 442 -> 423 us, 128 of them the first pass
// at 6.3 TB/s, 294 the second at 5.5; 42 M in fp32 86 -> 81).
// Workgroups side by side have chunks side by side: a run of chunks to a workgroup took 498 us.
#include <algorithm>
#include <type_traits>

#include "nm_act.h"
#include "nm_launch.h"

namespace nm {
namespace {

constexpr int kTable = 112;       // tensors a launch: the arguments stay below 4 KB
constexpr int kSmallTable = 32;   // of a call with no more
constexpr int kPieces = 8;        // of 16 bytes to a work-item and chunk, all of them in flight at once
constexpr int kChunkBytes = 256 * 16 * kPieces;
constexpr int kMostGroups = 2048;

template <int N>
struct TensorTable {
  const void* in[N];
  void* out[N];
  int64_t count[N];
  uint32_t first[N + 1];  // chunk that a tensor begins with
  int dt[N];
  int tensors;
};
static_assert(sizeof(TensorTable<kTable>) < 3900, "kernel arguments");

template <int DT>
struct ClipElem {
  typedef std::conditional_t<DT == kF32, uint32_t, uint16_t> type;
  static constexpr int kPer = 16 / (int)sizeof(type), kChunk = kChunkBytes / (int)sizeof(type);
  typedef uint32_t any_t __attribute__((ext_vector_type(4), aligned(2)));
};
constexpr int64_t chunk_entries(int dt) { return kChunkBytes / (dt == kF32 ? 4 : 2); }

// Piece k of this work-item in a chunk: entries entry(k) and on.
template <int DT>
__device__ __forceinline__ int64_t entry(int k) {
  return (k * 256 + (int)threadIdx.x) * ClipElem<DT>::kPer;
}
// The pieces of a chunk: f(k, piece).  A whole chunk's loads are all in flight before the first is used.
template <int DT, typename F>
__device__ __forceinline__ void each_piece(const void* p, int64_t at, int64_t left, F&& f) {
  typedef typename ClipElem<DT>::type E;
  constexpr int kPer = ClipElem<DT>::kPer;
  const E* x = static_cast<const E*>(p) + at;
  if (left >= ClipElem<DT>::kChunk) {
    u32x4_t r[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
      r[k] = *reinterpret_cast<const typename ClipElem<DT>::any_t*>(x + entry<DT>(k));
#pragma unroll
    for (int k = 0; k < kPieces; ++k) f(k, r[k]);
    return;
  }
#pragma unroll 1
  for (int k = 0; k < kPieces; ++k) {
    const int64_t e = entry<DT>(k);
    if (e >= left) break;
    u32x4_t r{0, 0, 0, 0};
    if (e + kPer <= left) {
      r = *reinterpret_cast<const typename ClipElem<DT>::any_t*>(x + e);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (e + j < left) r[j * 4 / kPer] |= (uint32_t)x[e + j] << (DT == kF32 ? 0 : 16 * (j & 1));
    }
    f(k, r);
  }
}
template <int DT>
__device__ __forceinline__ float number(const u32x4_t& r, int j) {
  if constexpr (DT == kF32) return __uint_as_float(r[j]);
  else if constexpr (DT == kBF16) return bf16_to_f32((r[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
  else return f16_to_f32((r[j / 2] >> (16 * (j & 1))) & 0xFFFFu);
}

// Calls f with the type as a constant.
template <typename F>
__device__ __forceinline__ void by_type(int dt, F&& f) {
  if (dt == kF32) f(std::integral_constant<int, kF32>{});
  else if (dt == kBF16) f(std::integral_constant<int, kBF16>{});
  else f(std::integral_constant<int, kF16>{});
}

// Calls f(tensor, first entry, entries left in the tensor) for chunks blockIdx.x, + gridDim.x, ..., or
// for the same counted from the last one.
template <bool BACK, int N, typename F>
__device__ __forceinline__ void each_chunk(const TensorTable<N>& t, F&& f) {
  const uint32_t all = t.first[t.tensors];
  int i = BACK ? t.tensors - 1 : 0;
  for (uint32_t n = blockIdx.x; n < all; n += gridDim.x) {
    const uint32_t c = BACK ? all - 1 - n : n;
    if constexpr (BACK) {
      while (c < t.first[i]) --i;
    } else {
      while (c >= t.first[i + 1]) ++i;
    }
    const int64_t at = (int64_t)(c - t.first[i]) * (kChunkBytes / (t.dt[i] == kF32 ? 4 : 2));
    f(i, at, t.count[i] - at);
  }
}

__device__ __forceinline__ double add_lanes(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The sum of the workgroup's 256 work-items, in every one of them.
__device__ __forceinline__ double add_group(double v, double* part) {
  v = add_lanes(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return (part[0] + part[1]) + (part[2] + part[3]);
}

template <int N>
__global__ void __launch_bounds__(256) square_kernel(TensorTable<N> t, double* __restrict__ sums) {
  __shared__ double part[4];
  double total = 0;
  each_chunk<false>(t, [&](int i, int64_t at, int64_t left) {
    by_type(t.dt[i], [&](auto type) {
      constexpr int DT = decltype(type)::value, kPer = ClipElem<DT>::kPer;
      each_piece<DT>(t.in[i], at, left, [&](int, const u32x4_t& r) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) s = __builtin_fmaf(number<DT>(r, j), number<DT>(r, j), s);
        if (s >= 0x1p-100f && s < INFINITY) {  // then no square that counts left fp32's range
          total += (double)s;
        } else if (((DT == kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu) & (r[0] | r[1] | r[2] | r[3])) != 0u) {
#pragma unroll 1
          for (int j = 0; j < kPer; ++j) {
            double v = 0;  // (an index that is no constant would put r into memory)
#pragma unroll
            for (int q = 0; q < kPer; ++q) v = q == j ? (double)number<DT>(r, q) : v;
            total += v * v;
          }
        }
      });
    });
  });
  total = add_group(total, part);
  if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

__device__ __forceinline__ double norm_of(const double* __restrict__ sums, int count, double* part) {
  double v = 0;
  for (int i = threadIdx.x; i < count; i += 256) v += sums[i];
  return sqrt(add_group(v, part));
}

__global__ void __launch_bounds__(256)
    norm_kernel(const double* __restrict__ sums, int count, float* __restrict__ norm) {
  __shared__ double part[4];
  const float n = (float)norm_of(sums, count, part);
  if (threadIdx.x == 0) *norm = n;
}

template <int N>
__global__ void __launch_bounds__(256)
    clip_kernel(TensorTable<N> t, const double* __restrict__ sums, int count,
                const float* __restrict__ given, float max_norm, float* __restrict__ norm) {
  __shared__ double part[4];
  const double wide = given ? (double)*given : norm_of(sums, count, part);
  const float n = (float)wide;
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  // A norm that is no number leaves everything as it is.  One past fp32 does not: the sum of squares has
  // it.  A ratio below fp32's normal numbers goes as a number in 1/2 .. 1 and a power of two.
  const bool clip = n > max_norm && wide < (double)INFINITY;
  const bool small = clip && (n == INFINITY || max_norm / n < 0x1p-126f);
  const double ratio = (double)max_norm / (n == INFINITY ? wide : (double)n);
  int power = 0;
  float f = clip ? max_norm / n : 1.f;
  if (small) f = (float)frexp(ratio, &power);
  each_chunk<true>(t, [&](int i, int64_t at, int64_t left) {
    if (!clip && t.out[i] == t.in[i]) return;
    by_type(t.dt[i], [&](auto type) {
      constexpr int DT = decltype(type)::value, kPer = ClipElem<DT>::kPer;
      typedef typename ClipElem<DT>::type E;
      E* y = static_cast<E*>(t.out[i]) + at;
      each_piece<DT>(t.in[i], at, left, [&](int k, const u32x4_t& r) {
        u32x4_t w{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float v = __builtin_ldexpf(number<DT>(r, j) * f, power);
          if constexpr (DT == kF32) w[j] = __float_as_uint(v);
          else w[j / 2] |= (DT == kBF16 ? f32_to_bf16(v) : f32_to_f16(v)) << (16 * (j & 1));
        }
        if (!clip) w = r;
        const int64_t e = entry<DT>(k);
        if (e + kPer <= left) {
          // past the caches, where the rest of the gradients still is
          __builtin_nontemporal_store(w, reinterpret_cast<typename ClipElem<DT>::any_t*>(y + e));
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (e + j < left) y[e + j] = (E)(w[j * 4 / kPer] >> (DT == kF32 ? 0 : 16 * (j & 1)));
        }
      });
    });
  });
}

// The tables of a call: for each, a range of the non-empty tensors, and its workgroups.
int64_t chunks_of(int64_t count, int dt) {
  return (count + chunk_entries(dt) - 1) / chunk_entries(dt);
}

int64_t tables_of(const int64_t* counts, int64_t tensors) {
  int64_t live = 0;
  for (int64_t i = 0; i < tensors; ++i) live += counts[i] > 0;
  return (live + kTable - 1) / kTable;
}

int64_t most_groups(int64_t tables) {
  return tables > 0 ? std::max<int64_t>(256, kMostGroups / tables) : 0;
}

// Calls f(table, workgroups) for each table of N in turn.
template <int N, typename F>
hipError_t each_table(const void* const* grads, void* const* outs, const int64_t* counts,
                      const int* dts, int64_t tensors, int64_t most, F&& f) {
  TensorTable<N> t;
  t.tensors = 0;
  t.first[0] = 0;
  const auto flush = [&]() {
    if (t.tensors == 0) return hipSuccess;
    const int64_t all = t.first[t.tensors];
    const hipError_t e = f(t, (unsigned)std::min(all, most));
    t.tensors = 0;
    return e;
  };
  hipError_t e = hipSuccess;
  for (int64_t i = 0; i < tensors && e == hipSuccess; ++i) {
    if (counts[i] == 0) continue;
    t.in[t.tensors] = grads[i];
    t.out[t.tensors] = outs ? outs[i] : nullptr;
    t.count[t.tensors] = counts[i];
    t.dt[t.tensors] = dts[i];
    t.first[t.tensors + 1] = t.first[t.tensors] + (uint32_t)chunks_of(counts[i], dts[i]);
    if (++t.tensors == N) e = flush();
  }
  return e == hipSuccess ? flush() : e;
}

}  // namespace

size_t norm_workspace_bytes(const int64_t* counts, int64_t tensors) {
  const int64_t tables = tables_of(counts, tensors);
  return (size_t)(tables * most_groups(tables)) * sizeof(double);
}

namespace {
template <int N>
hipError_t clip_tables(const void* const* grads, void* const* outs, const int64_t* counts,
                       const int* dts, int64_t tensors, int64_t most, float max_norm,
                       const float* given, float* norm, double* sums, hipStream_t s) {
  int parts = 0;
  hipError_t e = hipSuccess;
  if (!given) {
    e = each_table<N>(grads, nullptr, counts, dts, tensors, most,
                      [&](const TensorTable<N>& t, unsigned groups) {
      square_kernel<N><<<groups, 256, 0, s>>>(t, sums + parts);
      parts += (int)groups;
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    if (!outs || most == 0) {
      norm_kernel<<<1, 256, 0, s>>>(sums, parts, norm);
      return hipGetLastError();
    }
  }
  float* write = given ? nullptr : norm;  // by the first table's kernel
  return each_table<N>(grads, outs, counts, dts, tensors, most,
                       [&](const TensorTable<N>& t, unsigned groups) {
    clip_kernel<N><<<groups, 256, 0, s>>>(t, sums, parts, given, max_norm, write);
    write = nullptr;
    return hipGetLastError();
  });
}
}  // namespace

hipError_t launch_clip(const void* const* grads, void* const* outs, const int64_t* counts,
                       const int* dts, int64_t tensors, float max_norm, const float* given,
                       float* norm, void* workspace, hipStream_t s) {
  const int64_t most = most_groups(tables_of(counts, tensors));
  double* sums = static_cast<double*>(workspace);
  return tensors <= kSmallTable
             ? clip_tables<kSmallTable>(grads, outs, counts, dts, tensors, most, max_norm, given, norm, sums, s)
             : clip_tables<kTable>(grads, outs, counts, dts, tensors, most, max_norm, given, norm, sums, s);
}

}  // namespace nm
