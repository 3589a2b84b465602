// nm_logits.hip -- penalties for a sequence's own words, biases and masks on logits
// (nm_adjust_logits), V words x T sequences, a column a sequence.
//
// Of a word that stands in column t's tokens (seen), a times of them after its prompt:
//   x / repetition[t] where x > 0 and x repetition[t] where not, if seen;
//   - presence[t] if a > 0,  - frequency[t] a,  + bias,  -infinity where the mask has no bit.
//
// One pass over the logits, bound by memory on large ones and by the launch on small ones.  A word's
// counts are needed beside its logit, and a column's tokens come in any order.  Short histories: a
// workgroup has a tile of words x columns, reads all of its columns' tokens and counts its own words in
// LDS; every workgroup of a column reads that column's tokens again, from cache.  Long histories: the
// counts go through a table in the workspace (cleared, counted with atomics, read by the pass); integer
// sums come out the same in any order.  Either way bit 31 of a count stands for a word of the prompt.
// fp32 50257 x 64 with 96,000 tokens 15.7 us, of which reading and counting them is 5 (the logits alone
// are 5 at a copy's rate; all workgroups are there at once, so loads and stores do not overlap).
#include <algorithm>

#include "nm_grid.h"
#include "nm_launch.h"
#include "nm_mfma.h"
#include "nm_tiles.h"

namespace nm {
namespace {

constexpr int kCounts = 8448;              // in LDS: columns of one more than the tile's words, and copies
constexpr uint32_t kSeen = 0x80000000u;    // of a count: the word is in the prompt

struct LogitsArgs {
  LogitsCall c;
  int log_cols, log_cells, copies;
  uint32_t* counts;  // V x T, or null
};

// Column t's tokens: entries [begin, end), the answer's from `own` on; whatever `starts` and
// `prompts` hold, within the c.count tokens there are.
__device__ __forceinline__ void tokens_of(const LogitsCall& c, int64_t t, int64_t& begin,
                                          int64_t& own, int64_t& end) {
  const auto hold = [&](int64_t x) { return x < 0 ? (int64_t)0 : x > c.count ? c.count : x; };
  begin = hold(c.starts[t]);
  end = hold(c.starts[t + 1]);
  const int64_t skip = c.prompts ? hold(c.prompts[t]) : 0;
  own = begin + skip;
}

__global__ void __launch_bounds__(256) clear_counts_kernel(uint32_t* __restrict__ counts, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    counts[i] = 0u;
}

// Workgroups (x) share a column's (y, and on) tokens, kRun at a time.  A text's frequent words would
// queue at one address of the table, so a workgroup first counts in LDS, at a place given by the word's
// low bits, which the first word to come holds; only words that find theirs held go to the table at
// once.
constexpr int kRun = 8192, kPlaces = 4096;

__global__ void __launch_bounds__(1024) count_kernel(LogitsCall c, uint32_t* __restrict__ counts) {
  __shared__ int held[kPlaces];
  __shared__ uint32_t sums[kPlaces];
  const auto put = [&](int64_t v, int64_t t, uint32_t sum) {
    uint32_t* cell = counts + v * c.T + t;
    if (sum & kSeen) atomicOr(cell, kSeen);
    if (sum & ~kSeen) atomicAdd(cell, sum & ~kSeen);
  };
  for (int64_t t = blockIdx.y; t < c.T; t += gridDim.y) {
    int64_t begin, own, end;
    tokens_of(c, t, begin, own, end);
    for (int i = threadIdx.x; i < kPlaces; i += 1024) {
      held[i] = -1;
      sums[i] = 0u;
    }
    __syncthreads();
    for (int64_t i0 = begin + (int64_t)blockIdx.x * kRun; i0 < end; i0 += (int64_t)gridDim.x * kRun) {
      int64_t v[kRun / 1024];
#pragma unroll
      for (int j = 0; j < kRun / 1024; ++j)
        v[j] = c.tokens[min(i0 + j * 1024 + (int)threadIdx.x, end - 1)];
#pragma unroll
      for (int j = 0; j < kRun / 1024; ++j) {
        const int64_t i = i0 + j * 1024 + threadIdx.x;
        if (i >= end || v[j] < 0 || v[j] >= c.V) continue;
        const int place = (int)v[j] & (kPlaces - 1), word = (int)v[j];
        int who = held[place];
        if (who == -1) {
          who = atomicCAS(held + place, -1, word);
          if (who == -1) who = word;
        }
        if (who != word) put(word, t, i < own ? kSeen : 1u);
        else if (i < own) atomicOr(sums + place, kSeen);
        else atomicAdd(sums + place, 1u);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kPlaces; i += 1024)
      if (held[i] >= 0) put(held[i], t, sums[i]);
    __syncthreads();
  }
}

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (DT == kF32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == kBF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return f16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// HISTORY: 0 none, 1 counted here in LDS, 2 from the table.
template <int DT, int HISTORY>
__global__ void __launch_bounds__(kLogitsThreads, 8) adjust_kernel(LogitsArgs a) {
  __shared__ uint32_t cells[HISTORY == 1 ? kCounts : 1];
  __shared__ uint32_t bits[kLogitsCells / 32];
  __shared__ int64_t ranges[HISTORY == 1 ? 32 : 1][3];
  const LogitsCall& c = a.c;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int cols = 1 << a.log_cols, all = 1 << a.log_cells, words = all >> a.log_cols;
  const int64_t t0 = (int64_t)blockIdx.y * cols, v0 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * words;
  if (v0 >= c.V) return;
  const int64_t t = t0 + (tid & (cols - 1));  // this work-item's column
  const bool live = t < c.T;
  // the logits are under way while the tokens are counted
  float x[kLogitsEach];
  const auto place = [&](int k) {  // of entry k of this work-item, held within the matrix
    const int64_t v = v0 + ((tid + k * threads) >> a.log_cols);
    return min(v, c.V - 1) * c.T + min(t, c.T - 1);
  };
#pragma unroll
  for (int k = 0; k < kLogitsEach; ++k)
    if (tid + k * threads < all) x[k] = logit_at<DT>(c.logits, place(k));
  if constexpr (HISTORY == 1) {
    for (int i = tid; i < a.copies * cols * (words + 1); i += threads) cells[i] = 0u;
    if (tid < cols && live) tokens_of(c, t, ranges[tid][0], ranges[tid][1], ranges[tid][2]);
  }
  if (c.allowed) {  // words is a multiple of 32: whole words of the mask
    const int64_t row = (c.V + 31) / 32;
    for (int i = tid; i < all / 32; i += threads) {
      const int64_t col = t0 + (i & (cols - 1)), w = v0 / 32 + (i >> a.log_cols);
      bits[i] = col < c.T && w < row ? c.allowed[col * row + w] : 0u;
    }
  }
  __syncthreads();
  if constexpr (HISTORY == 1) {
    constexpr int kBatch = 6;
    const int lane = tid & 63, wave = tid >> 6, waves = threads >> 6;
    // a text's frequent words would have a wave's lanes wait for one another: several copies of the
    // counts, and a column's words on banks of their own
    uint32_t* copy = cells + (lane & (a.copies - 1)) * cols * (words + 1);
    // a wave a column, or several where columns are few
    const int shares = waves > cols ? waves >> a.log_cols : 1, share = waves > cols ? wave >> a.log_cols : 0;
    for (int k = waves > cols ? wave & (cols - 1) : wave; k < cols && t0 + k < c.T; k += waves) {
      const int64_t begin = ranges[k][0], own = ranges[k][1], end = ranges[k][2];
      for (int64_t i = begin + share * 64 + lane; i < end; i += kBatch * 64 * shares) {
        int64_t v[kBatch];  // (loads without conditions, or each would be waited for)
#pragma unroll
        for (int j = 0; j < kBatch; ++j) v[j] = c.tokens[min(i + 64 * shares * j, end - 1)];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          v[j] -= v0;
          if (i + 64 * shares * j >= end || v[j] < 0 || v[j] >= words || v[j] >= c.V - v0) continue;
          uint32_t* cell = copy + k * (words + 1) + (int)v[j];
          if (i + 64 * shares * j < own) atomicOr(cell, kSeen);
          else atomicAdd(cell, 1u);
        }
      }
    }
    __syncthreads();
  }
  if (!live) return;
  const float repetition = HISTORY && c.repetition ? c.repetition[t] : 1.f;
  const float presence = HISTORY && c.presence ? c.presence[t] : 0.f;
  const float frequency = HISTORY && c.frequency ? c.frequency[t] : 0.f;
  float b[kLogitsEach];
  uint32_t n[kLogitsEach];
#pragma unroll
  for (int k = 0; k < kLogitsEach; ++k) {
    if (tid + k * threads >= all) continue;
    const int64_t v = v0 + ((tid + k * threads) >> a.log_cols);
    if (c.bias) b[k] = c.bias[c.bias_each ? place(k) : min(v, c.V - 1)];
    if constexpr (HISTORY == 2) n[k] = a.counts[place(k)];
  }
#pragma unroll
  for (int k = 0; k < kLogitsEach; ++k) {
    const int i = tid + k * threads, w = i >> a.log_cols;
    const int64_t v = v0 + w;
    if (i >= all || v >= c.V) continue;
    float y = x[k];
    uint32_t count = 0;
    if constexpr (HISTORY == 2) count = n[k];
    if constexpr (HISTORY == 1) {
      uint32_t seen = 0;
      for (int q = 0; q < a.copies; ++q) {
        const uint32_t one = cells[(q * cols + (tid & (cols - 1))) * (words + 1) + w];
        seen |= one & kSeen;
        count += one & ~kSeen;
      }
      count |= seen;
    }
    if (HISTORY && count != 0) {
      if (c.repetition) y = y > 0.f ? y / repetition : y * repetition;
      const uint32_t own = count & ~kSeen;
      if (own != 0) y = (y - presence) - frequency * (float)own;
    }
    if (c.bias) y += b[k];
    if (c.allowed && !((bits[((w >> 5) << a.log_cols) + (tid & (cols - 1))] >> (w & 31)) & 1u))
      y = -INFINITY;
    store_from_f32<DT>(c.out, v * c.T + t, y);
  }
}

int64_t table_bytes(int64_t V, int64_t T) { return V * T * 4; }

template <int DT>
hipError_t launch_adjust(const LogitsArgs& a, const LogitsPlan& p, int history, hipStream_t s) {
  const dim3 grid((unsigned)p.grid_v, (unsigned)p.blocks_t, (unsigned)p.grid_z);
  if (history == 0) adjust_kernel<DT, 0><<<grid, p.threads, 0, s>>>(a);
  else if (history == 1) adjust_kernel<DT, 1><<<grid, p.threads, 0, s>>>(a);
  else adjust_kernel<DT, 2><<<grid, p.threads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t logits_workspace_bytes(int64_t V, int64_t T, int64_t count) {
  return count > 0 && LogitsPlan(V, T, count).table ? (size_t)table_bytes(V, T) : 0;
}

hipError_t launch_adjust_logits(const LogitsCall& c, void* workspace, hipStream_t s) {
  const bool any = c.count > 0 && (c.repetition || c.presence || c.frequency);
  const LogitsPlan p(c.V, c.T, c.count);
  LogitsArgs a{c, p.log_cols, p.log_cells, p.copies, nullptr};
  int history = any ? 1 : 0;
  if (any && p.table) {
    history = 2;
    a.counts = static_cast<uint32_t*>(workspace);
    clear_counts_kernel<<<stride_grid(c.V * c.T, 1024), 256, 0, s>>>(a.counts, c.V * c.T);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = std::min<int64_t>(c.T, 4096);
    const int64_t each = std::min((c.count / c.T + kRun - 1) / kRun, 2048 / cols);
    count_kernel<<<dim3((unsigned)std::max<int64_t>(1, each), (unsigned)cols), 1024, 0, s>>>(c, a.counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (c.dt == kF32) return launch_adjust<kF32>(a, p, history, s);
  if (c.dt == kBF16) return launch_adjust<kBF16>(a, p, history, s);
  return launch_adjust<kF16>(a, p, history, s);
}

}  // namespace nm
