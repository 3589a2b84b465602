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
#include <algorithm>

#include "nm_grid.h"
#include "nm_launch.h"
#include "nm_mfma.h"

namespace nm {
namespace {

constexpr int kMostCells = 8192;           // words x columns of a workgroup
constexpr int kMostThreads = 1024;
constexpr uint32_t kSeen = 0x80000000u;    // of a count: the word is in the prompt

// A workgroup's tile: 2^log_cols columns, 2^log_cells entries, `threads` work-items.
struct LogitsPlan {
  int log_cols, log_cells, threads;
  int64_t blocks_v, blocks_t;
  bool table;        // the counts go through the workspace
  LogitsPlan(int64_t V, int64_t T, int64_t count);
};

struct LogitsArgs {
  LogitsCall c;
  int log_cols, log_cells;
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

// Workgroups (x) share a column's (y, and on) tokens.
__global__ void __launch_bounds__(256) count_kernel(LogitsCall c, uint32_t* __restrict__ counts) {
  for (int64_t t = blockIdx.y; t < c.T; t += gridDim.y) {
    int64_t begin, own, end;
    tokens_of(c, t, begin, own, end);
    for (int64_t i = begin + (int64_t)blockIdx.x * 256 + threadIdx.x; i < end;
         i += (int64_t)gridDim.x * 256) {
      const int64_t v = c.tokens[i];
      if (v < 0 || v >= c.V) continue;
      if (i < own) atomicOr(counts + v * c.T + t, kSeen);
      else atomicAdd(counts + v * c.T + t, 1u);
    }
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
__global__ void __launch_bounds__(kMostThreads) adjust_kernel(LogitsArgs a) {
  __shared__ uint32_t cells[HISTORY == 1 ? kMostCells : 1];
  __shared__ uint32_t bits[kMostCells / 32];
  const LogitsCall& c = a.c;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int cols = 1 << a.log_cols, all = 1 << a.log_cells, words = all >> a.log_cols;
  const int64_t t0 = (int64_t)blockIdx.y * cols, v0 = (int64_t)blockIdx.x * words;
  const int64_t t = t0 + (tid & (cols - 1));  // this work-item's column
  const bool live = t < c.T;
  if constexpr (HISTORY == 1) {
    for (int i = tid; i < all; i += threads) cells[i] = 0u;
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
    constexpr int kBatch = 8;
    const int lane = tid & 63, wave = tid >> 6, waves = threads >> 6;
    // a wave a column, or several where columns are few
    const int shares = waves > cols ? waves >> a.log_cols : 1, share = waves > cols ? wave >> a.log_cols : 0;
    for (int k = waves > cols ? wave & (cols - 1) : wave; k < cols && t0 + k < c.T; k += waves) {
      int64_t begin, own, end;
      tokens_of(c, t0 + k, begin, own, end);
      for (int64_t i = begin + share * 64 + lane; i < end; i += kBatch * 64 * shares) {
        int64_t v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          v[j] = i + 64 * shares * j < end ? c.tokens[i + 64 * shares * j] - v0 : -1;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (v[j] < 0 || v[j] >= words || v[j] >= c.V - v0) continue;
          uint32_t* cell = cells + ((int)v[j] << a.log_cols) + k;
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
  const bool penalised = c.repetition != nullptr;
  constexpr int kBatch = 8;  // loads in flight
#pragma unroll 1
  for (int i0 = tid; i0 < all; i0 += kBatch * threads) {
    float x[kBatch], b[kBatch];
    uint32_t n[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * threads;
      const int64_t v = v0 + (i >> a.log_cols);
      const bool in = i < all && v < c.V;
      x[k] = in ? logit_at<DT>(c.logits, v * c.T + t) : 0.f;
      b[k] = in && c.bias ? c.bias[c.bias_each ? v * c.T + t : v] : 0.f;
      n[k] = 0;
      if constexpr (HISTORY == 1) n[k] = in ? cells[i] : 0u;
      if constexpr (HISTORY == 2) n[k] = in ? a.counts[v * c.T + t] : 0u;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * threads, w = i >> a.log_cols;
      const int64_t v = v0 + w;
      if (i >= all || v >= c.V) continue;
      float y = x[k];
      if (HISTORY && n[k] != 0) {
        if (penalised) y = y > 0.f ? y / repetition : y * repetition;
        const uint32_t own = n[k] & ~kSeen;
        if (own != 0) y = (y - presence) - frequency * (float)own;
      }
      if (c.bias) y += b[k];
      if (c.allowed && !((bits[((w >> 5) << a.log_cols) + (tid & (cols - 1))] >> (w & 31)) & 1u))
        y = -INFINITY;
      store_from_f32<DT>(c.out, v * c.T + t, y);
    }
  }
}

int64_t table_bytes(int64_t V, int64_t T) { return V * T * 4; }

// Columns: 16, whose 64 bytes (fp32) of a row are one request, or what there are, to a power of two.
// Entries: as many as fit, since every workgroup reads its columns' tokens, but few enough that all
// 256 units have a workgroup.
LogitsPlan::LogitsPlan(int64_t V, int64_t T, int64_t count) {
  log_cols = 0;
  while (log_cols < 4 && ((int64_t)1 << log_cols) < T) ++log_cols;
  const int64_t cols = (int64_t)1 << log_cols;
  blocks_t = (T + cols - 1) / cols;
  const int least = std::max(8, 5 + log_cols);  // whole words of the mask
  for (log_cells = 13; log_cells > least; --log_cells) {
    const int64_t words = ((int64_t)1 << log_cells) / cols;
    if ((V + words - 1) / words * blocks_t >= 256) break;
  }
  const int64_t words = ((int64_t)1 << log_cells) / cols;
  blocks_v = (V + words - 1) / words;
  const int64_t each = count / std::max<int64_t>(1, T);  // tokens of a column
  threads = log_cells >= 13 || each > 2048 ? kMostThreads : 256;
  // in LDS each of blocks_v workgroups reads a column's tokens; through the table they are read once,
  // and the table is written and read, with two more launches
  table = (double)blocks_v * (double)count * 8 > 3.0 * (double)table_bytes(V, T) + 64e6;
}

template <int DT>
hipError_t launch_adjust(const LogitsArgs& a, const LogitsPlan& p, int history, hipStream_t s) {
  const dim3 grid((unsigned)p.blocks_v, (unsigned)p.blocks_t);
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
  LogitsArgs a{c, p.log_cols, p.log_cells, nullptr};
  int history = any ? 1 : 0;
  if (any && p.table) {
    history = 2;
    a.counts = static_cast<uint32_t*>(workspace);
    clear_counts_kernel<<<stride_grid(c.V * c.T, 1024), 256, 0, s>>>(a.counts, c.V * c.T);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = std::min<int64_t>(c.T, 4096);
    const int64_t each = std::min((c.count / c.T + 1023) / 1024, 4096 / cols);
    count_kernel<<<dim3((unsigned)std::max<int64_t>(1, each), (unsigned)cols), 256, 0, s>>>(c, a.counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (c.dt == kF32) return launch_adjust<kF32>(a, p, history, s);
  if (c.dt == kBF16) return launch_adjust<kBF16>(a, p, history, s);
  return launch_adjust<kF16>(a, p, history, s);
}

}  // namespace nm
