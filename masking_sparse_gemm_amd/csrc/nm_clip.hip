// nm_clip.hip -- the global norm of many tensors (nm_grad_norm) and clipping by it (nm_clip_grads).
//
//   norm = sqrt(sum over all tensors and entries of g^2),   out = g min(1, max_norm / norm)
//
// The tensors' addresses and sizes travel as kernel arguments, kTable of them a launch, so nothing is
// copied to the device and a captured graph keeps them.  Entries are taken in chunks of 8192; a
// workgroup has a run of chunks, so it looks its tensor up once and walks on from there.  Squares are
// added eight at a time in fp32 and then in fp64 (all in fp64 where eight squares leave fp32's range),
// and the workgroups' sums are joined in a fixed order by every workgroup of the second pass: two
// launches for up to kTable tensors.
//
// Bound by memory, the first pass by reads, the second by a read and a write.  The second pass takes
// the chunks last first: what the first pass read last is still in the 256 MB cache.
#include <algorithm>

#include "nm_act.h"
#include "nm_launch.h"

namespace nm {
namespace {

constexpr int kTable = 112;    // tensors a launch: the arguments stay below 4 KB
constexpr int kChunk = 8192;   // entries: 256 work-items x 4 pieces of eight
constexpr int kMostGroups = 2048;

struct TensorTable {
  const void* in[kTable];
  void* out[kTable];
  int64_t count[kTable];
  uint32_t first[kTable + 1];  // chunk that a tensor begins with
  uint8_t dt[kTable];
  int tensors;
  uint32_t per;                // chunks a workgroup
};
static_assert(sizeof(TensorTable) < 3900, "kernel arguments");

// Calls f(tensor, first entry, entries left in the tensor) for the chunks of run `run`.
template <typename F>
__device__ __forceinline__ void each_chunk(const TensorTable& t, uint32_t run, F&& f) {
  const uint32_t all = t.first[t.tensors], c0 = run * t.per, c1 = min(all, c0 + t.per);
  int lo = 0, hi = t.tensors - 1;  // the last tensor with first <= c0
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c0) lo = mid;
    else hi = mid - 1;
  }
  for (uint32_t c = c0; c < c1; ++c) {
    while (c >= t.first[lo + 1]) ++lo;
    const int64_t at = (int64_t)(c - t.first[lo]) * kChunk;
    f(lo, at, t.count[lo] - at);
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

__global__ void __launch_bounds__(256) square_kernel(TensorTable t, double* __restrict__ sums) {
  __shared__ double part[4];
  double total = 0;
  each_chunk(t, blockIdx.x, [&](int i, int64_t at, int64_t left) {
    RawEight r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t e = (k * 256 + threadIdx.x) * 8;
      r[k] = RawEight{};
      if (e < left) r[k] = load_eight(t.in[i], t.dt[i], at + e, left - e);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[8];
      to_floats(r[k], t.dt[i], v);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __builtin_fmaf(v[e], v[e], s);
      if (s >= 0x1p-100f && s < INFINITY) {  // then no square that counts left fp32's range
        total += (double)s;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) total += (double)v[e] * (double)v[e];
      }
    }
  });
  total = add_group(total, part);
  if (threadIdx.x == 0) sums[blockIdx.x] = total;
}

__device__ __forceinline__ float norm_of(const double* __restrict__ sums, int count, double* part) {
  double v = 0;
  for (int i = threadIdx.x; i < count; i += 256) v += sums[i];
  return (float)sqrt(add_group(v, part));
}

__global__ void __launch_bounds__(256)
    norm_kernel(const double* __restrict__ sums, int count, float* __restrict__ norm) {
  __shared__ double part[4];
  const float n = norm_of(sums, count, part);
  if (threadIdx.x == 0) *norm = n;
}

__global__ void __launch_bounds__(256)
    clip_kernel(TensorTable t, const double* __restrict__ sums, int count,
                const float* __restrict__ given, float max_norm, float* __restrict__ norm) {
  __shared__ double part[4];
  const float n = given ? *given : norm_of(sums, count, part);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  // a norm that is no number leaves everything as it is
  const bool clip = n > max_norm && n < INFINITY;
  const float f = clip ? max_norm / n : 1.f;
  each_chunk(t, gridDim.x - 1 - blockIdx.x, [&](int i, int64_t at, int64_t left) {
    if (!clip && t.out[i] == t.in[i]) return;
    const int dt = t.dt[i];
    RawEight r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t e = (k * 256 + threadIdx.x) * 8;
      r[k] = RawEight{};
      if (e < left) r[k] = load_eight(t.in[i], dt, at + e, left - e);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t e = (k * 256 + threadIdx.x) * 8;
      if (e >= left) continue;
      float v[8];
      to_floats(r[k], dt, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = clip ? v[j] * f : v[j];
      store_eight(t.out[i], dt, at + e, left - e, v);
    }
  });
}

// The tables of a call: for each, a range of the non-empty tensors, and its workgroups.
int64_t chunks_of(int64_t count) { return (count + kChunk - 1) / kChunk; }

int64_t tables_of(const int64_t* counts, int64_t tensors) {
  int64_t live = 0;
  for (int64_t i = 0; i < tensors; ++i) live += counts[i] > 0;
  return (live + kTable - 1) / kTable;
}

int64_t most_groups(int64_t tables) {
  return tables > 0 ? std::max<int64_t>(256, kMostGroups / tables) : 0;
}

// Calls f(table, workgroups) for each table in turn.
template <typename F>
hipError_t each_table(const void* const* grads, void* const* outs, const int64_t* counts,
                      const int* dts, int64_t tensors, int64_t most, F&& f) {
  TensorTable t;
  t.tensors = 0;
  t.first[0] = 0;
  const auto flush = [&]() {
    if (t.tensors == 0) return hipSuccess;
    const int64_t all = t.first[t.tensors];
    t.per = (uint32_t)((all + most - 1) / most);
    const hipError_t e = f(t, (unsigned)((all + t.per - 1) / t.per));
    t.tensors = 0;
    return e;
  };
  hipError_t e = hipSuccess;
  for (int64_t i = 0; i < tensors && e == hipSuccess; ++i) {
    if (counts[i] == 0) continue;
    t.in[t.tensors] = grads[i];
    t.out[t.tensors] = outs ? outs[i] : nullptr;
    t.count[t.tensors] = counts[i];
    t.dt[t.tensors] = (uint8_t)dts[i];
    t.first[t.tensors + 1] = t.first[t.tensors] + (uint32_t)chunks_of(counts[i]);
    if (++t.tensors == kTable) e = flush();
  }
  return e == hipSuccess ? flush() : e;
}

}  // namespace

size_t norm_workspace_bytes(const int64_t* counts, int64_t tensors) {
  const int64_t tables = tables_of(counts, tensors);
  return (size_t)(tables * most_groups(tables)) * sizeof(double);
}

hipError_t launch_clip(const void* const* grads, void* const* outs, const int64_t* counts,
                       const int* dts, int64_t tensors, float max_norm, const float* given,
                       float* norm, void* workspace, hipStream_t s) {
  const int64_t tables = tables_of(counts, tensors), most = most_groups(tables);
  double* sums = static_cast<double*>(workspace);
  int parts = 0;
  hipError_t e = hipSuccess;
  if (!given) {
    e = each_table(grads, nullptr, counts, dts, tensors, most, [&](const TensorTable& t, unsigned groups) {
      square_kernel<<<groups, 256, 0, s>>>(t, sums + parts);
      parts += (int)groups;
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    if (!outs || tables == 0) {
      norm_kernel<<<1, 256, 0, s>>>(sums, parts, norm);
      return hipGetLastError();
    }
  }
  float* write = given ? nullptr : norm;  // by the first table's kernel
  return each_table(grads, outs, counts, dts, tensors, most, [&](const TensorTable& t, unsigned groups) {
    clip_kernel<<<groups, 256, 0, s>>>(t, sums, parts, given, max_norm, write);
    write = nullptr;
    return hipGetLastError();
  });
}

}  // namespace nm
