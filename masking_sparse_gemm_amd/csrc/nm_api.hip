// nm_api.hip -- the C ABI declared in include/nm.h: argument checks and dispatch.
//
// Every check runs on the host before any HIP call, so a rejected call touches
// neither the device nor the outputs.  The global state is a per-device record of
// whether the device is a gfx950, filled on first use, and the per-device address of
// the static scratch buffer behind nm_perm_gains_static, looked up on first use.
#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/nm.h"
#include "nm_launch.h"

namespace {

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = unsupported device
std::atomic<int> g_device_ok[kMaxDevices];

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A pointer may be NULL only when the array it addresses is empty.
bool missing(const void* p, int64_t count) { return p == nullptr && count > 0; }

int meta_bits_of(int m) { return m == 2 ? 1 : m == 4 ? 2 : m == 8 ? 3 : -1; }

int elem_bytes(nm_dtype dt) { return dt == NM_F32 ? 4 : (dt == NM_I8 || dt == NM_FP8) ? 1 : 2; }

// Element types of W for the selection and the products; NM_I32 is an output type only.
bool valid_dtype(int dt) {
  return dt == NM_F32 || dt == NM_F16 || dt == NM_BF16 || dt == NM_I8 || dt == NM_FP8;
}
bool float_dtype(int dt) { return dt == NM_F32 || dt == NM_F16 || dt == NM_BF16; }

// The blocked layout stores a lane's 16 elements of a block as whole 32-bit words of values:
// for byte elements (int8, fp8), 16 N / M bytes must divide by 4.
bool blocked_pattern_ok(nm_dtype dt, int n, int m) {
  return elem_bytes(dt) != 1 || (16 * n / m) % 4 == 0;
}

nm_status check_pattern(int n, int m) {
  if (meta_bits_of(m) < 0 || n < 1 || n > m) return NM_ERR_PATTERN;
  return NM_OK;
}

nm_status check_shape(int64_t R, int64_t K, int m) {
  if (R < 0 || K < 0 || K % m != 0) return NM_ERR_SHAPE;
  // below 2^36 elements (128 GiB of 16-bit W) every launch of the element-wise passes has
  // fewer than 2^32 work-items: their fast kernels give each work-item at least 16 elements,
  // and the per-group fallbacks loop over a capped grid
  if (R > 0 && K >= ((int64_t)1 << 36) / R + ((((int64_t)1 << 36) % R) != 0)) return NM_ERR_SHAPE;
  return NM_OK;
}

nm_status check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return NM_ERR_DEVICE;
  int state = g_device_ok[dev].load(std::memory_order_acquire);
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return NM_ERR_DEVICE;
    state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_device_ok[dev].store(state, std::memory_order_release);
  }
  return state == 1 ? NM_OK : NM_ERR_DEVICE;
}

// Do the byte ranges [a, a + a_bytes) and [b, b + b_bytes) share a byte?
bool overlaps(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes > 0 && b_bytes > 0 && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
bool overlaps(const void* a, const void* b, int64_t bytes) { return overlaps(a, bytes, b, bytes); }

nm_status from_hip(hipError_t e) { return e == hipSuccess ? NM_OK : NM_ERR_DEVICE; }

// NM_LAYOUT_BLOCKED cuts K into steps of 64: each step then holds a whole number of
// groups (M divides 64) and of metadata bytes (64 N / M fields of log2(M) bits).
nm_status check_layout(int layout, int64_t K) {
  if (layout == NM_LAYOUT_ROWS) return NM_OK;
  if (layout == NM_LAYOUT_BLOCKED && K % 64 == 0) return NM_OK;
  return NM_ERR_LAYOUT;
}

int64_t padded_rows(int64_t R, int layout) { return layout == NM_LAYOUT_BLOCKED ? (R + 15) / 16 * 16 : R; }

// Bytes of metadata per row: the row's whole words (ROWS) or its K/64 step slices (BLOCKED).
int64_t meta_row_bytes(int64_t K, int n, int m, int layout) {
  const int64_t bits = (K / m) * n * meta_bits_of(m);
  return layout == NM_LAYOUT_BLOCKED ? bits / 8 : (bits + 31) / 32 * 4;
}

}  // namespace

extern "C" {

int nm_abi_version(void) { return NM_ABI_VERSION; }

const char* nm_status_str(nm_status s) {
  switch (s) {
    case NM_OK: return "ok";
    case NM_ERR_NULL: return "null pointer";
    case NM_ERR_SHAPE: return "bad shape (negative size, K not a multiple of M, R*K >= 2^36 or past the call's limits)";
    case NM_ERR_PATTERN: return "bad N:M pattern (need 1 <= N <= M, M in {2,4,8})";
    case NM_ERR_DTYPE: return "bad dtype (unknown, or output neither input dtype nor fp32)";
    case NM_ERR_ALIGN: return "pointer not 16-byte aligned";
    case NM_ERR_UNSUPPORTED: return "unsupported combination";
    case NM_ERR_DEVICE: return "device error (no gfx950 device, or launch failed)";
    case NM_ERR_LAYOUT: return "bad layout (unknown, or blocked layout with K not a multiple of 64)";
    case NM_ERR_ALIAS: return "an output overlaps an input it may not replace";
    case NM_ERR_SCRATCH: return "the call needs more scratch than the static buffer or the given workspace";
  }
  return "unknown status";
}

size_t nm_values_bytes(int64_t R, int64_t K, int n, int m, nm_dtype dt, nm_layout layout) {
  if (!valid_dtype(dt) || check_pattern(n, m) != NM_OK || check_shape(R, K, m) != NM_OK ||
      check_layout(layout, K) != NM_OK)
    return 0;
  if (layout == NM_LAYOUT_BLOCKED && !blocked_pattern_ok(dt, n, m)) return 0;
  return (size_t)(padded_rows(R, layout) * (K / m * n) * elem_bytes(dt));
}

size_t nm_meta_bytes(int64_t R, int64_t K, int n, int m, nm_layout layout) {
  if (check_pattern(n, m) != NM_OK || check_shape(R, K, m) != NM_OK ||
      check_layout(layout, K) != NM_OK)
    return 0;
  return (size_t)(padded_rows(R, layout) * meta_row_bytes(K, n, m, layout));
}

int64_t nm_check_meta(const uint32_t* meta_host, int64_t R, int64_t K, int n, int m,
                      nm_layout layout) {
  if (check_pattern(n, m) != NM_OK || check_shape(R, K, m) != NM_OK ||
      check_layout(layout, K) != NM_OK)
    return -2;
  if (R * K == 0) return -1;
  if (meta_host == nullptr) return -2;
  const int b = meta_bits_of(m);
  const int64_t G = K / m, row_bits = G * n * b;
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(meta_host);
  const int64_t row_bytes = meta_row_bytes(K, n, m, layout);
  std::vector<uint8_t> row((size_t)row_bytes + 2);  // + 2: a field read may look past the end
  for (int64_t r = 0; r < R; ++r) {
    if (layout == NM_LAYOUT_ROWS) {
      std::memcpy(row.data(), bytes + r * row_bytes, (size_t)row_bytes);
    } else {  // the row's slice of every 64-wide step, from block (r / 16, s)
      const int64_t S = K / 64, B = row_bytes / S;
      for (int64_t st = 0; st < S; ++st)
        std::memcpy(row.data() + st * B, bytes + (((r / 16) * S + st) * 16 + r % 16) * B, (size_t)B);
    }
    row[row_bytes] = row[row_bytes + 1] = 0;
    auto field = [&](int64_t f) {  // b bits at bit f * b, least significant first
      const int64_t bit = f * b;
      const uint32_t v = row[bit / 8] | (uint32_t)row[bit / 8 + 1] << 8;
      return (int)((v >> (bit % 8)) & ((1u << b) - 1u));
    };
    for (int64_t g = 0; g < G; ++g) {
      int prev = -1;
      for (int j = 0; j < n; ++j) {
        const int p = field(g * n + j);
        if (p <= prev) return r * G + g;
        prev = p;
      }
    }
    for (int64_t bit = row_bits; bit < row_bytes * 8; ++bit)
      if ((row[bit / 8] >> (bit % 8)) & 1u) return r * G + G - 1;
  }
  return -1;
}

int64_t nm_meta_words_per_row(int64_t K, int n, int m) {
  if (check_pattern(n, m) != NM_OK || K < 0 || K % m != 0) return -1;
  return ((K / m) * n * meta_bits_of(m) + 31) / 32;
}

nm_status nm_mask(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m, uint8_t* mask,
                  nm_stream_t stream) {
  if (!valid_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (missing(W, R * K) || missing(mask, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (!aligned16(W) || !aligned16(mask)) return NM_ERR_ALIGN;
  if (overlaps(mask, R * K, W, R * K * elem_bytes(dt))) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_select(W, (int)dt, R, K, n, m, false, nullptr, nullptr, mask,
                                    static_cast<hipStream_t>(stream)));
}

nm_status nm_compress(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m,
                      nm_layout layout, void* values, uint32_t* meta, nm_stream_t stream) {
  if (!valid_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if ((st = check_layout(layout, K)) != NM_OK) return st;
  if (layout == NM_LAYOUT_BLOCKED && !blocked_pattern_ok(dt, n, m)) return NM_ERR_UNSUPPORTED;
  if (missing(W, R * K) || missing(values, R * K) || missing(meta, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (!aligned16(W) || !aligned16(values) || !aligned16(meta)) return NM_ERR_ALIGN;
  {
    const int64_t w_bytes = R * K * elem_bytes(dt);
    const int64_t v_bytes = (int64_t)nm_values_bytes(R, K, n, m, dt, layout);
    const int64_t m_bytes = (int64_t)nm_meta_bytes(R, K, n, m, layout);
    if (overlaps(values, v_bytes, W, w_bytes) || overlaps(meta, m_bytes, W, w_bytes) ||
        overlaps(values, v_bytes, meta, m_bytes))
      return NM_ERR_ALIAS;
  }
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_select(W, (int)dt, R, K, n, m, layout == NM_LAYOUT_BLOCKED,
                                    values, meta, nullptr, static_cast<hipStream_t>(stream)));
}

nm_status nm_mask_compress(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m,
                           nm_layout layout, uint8_t* mask, void* values, uint32_t* meta,
                           nm_stream_t stream) {
  if (!valid_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if ((st = check_layout(layout, K)) != NM_OK) return st;
  if (layout == NM_LAYOUT_BLOCKED && !blocked_pattern_ok(dt, n, m)) return NM_ERR_UNSUPPORTED;
  if (missing(W, R * K) || missing(mask, R * K) || missing(values, R * K) ||
      missing(meta, R * K))
    return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (!aligned16(W) || !aligned16(mask) || !aligned16(values) || !aligned16(meta))
    return NM_ERR_ALIGN;
  const int64_t w_bytes = R * K * elem_bytes(dt), mask_bytes = R * K;
  const int64_t v_bytes = (int64_t)nm_values_bytes(R, K, n, m, dt, layout);
  const int64_t m_bytes = (int64_t)nm_meta_bytes(R, K, n, m, layout);
  if (overlaps(mask, mask_bytes, W, w_bytes) || overlaps(values, v_bytes, W, w_bytes) ||
      overlaps(meta, m_bytes, W, w_bytes) || overlaps(mask, mask_bytes, values, v_bytes) ||
      overlaps(mask, mask_bytes, meta, m_bytes) || overlaps(values, v_bytes, meta, m_bytes))
    return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_select(W, (int)dt, R, K, n, m, layout == NM_LAYOUT_BLOCKED, values,
                                    meta, mask, static_cast<hipStream_t>(stream)));
}

nm_status nm_decompress(const void* values, const uint32_t* meta, nm_dtype dt, int64_t R,
                        int64_t K, int n, int m, nm_layout layout, void* W_out,
                        nm_stream_t stream) {
  if (!valid_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if ((st = check_layout(layout, K)) != NM_OK) return st;
  if (layout == NM_LAYOUT_BLOCKED && !blocked_pattern_ok(dt, n, m)) return NM_ERR_UNSUPPORTED;
  if (missing(values, R * K) || missing(meta, R * K) || missing(W_out, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (!aligned16(values) || !aligned16(meta) || !aligned16(W_out)) return NM_ERR_ALIGN;
  {
    const int64_t w_bytes = R * K * elem_bytes(dt);
    if (overlaps(W_out, w_bytes, values, (int64_t)nm_values_bytes(R, K, n, m, dt, layout)) ||
        overlaps(W_out, w_bytes, meta, (int64_t)nm_meta_bytes(R, K, n, m, layout)))
      return NM_ERR_ALIAS;
  }
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_decompress(values, meta, elem_bytes(dt), R, K, n, m,
                                        layout == NM_LAYOUT_BLOCKED, W_out,
                                        static_cast<hipStream_t>(stream)));
}

nm_status nm_spmm(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n, int m,
                  nm_layout layout, const void* X, int64_t T, nm_dtype dt, void* Y,
                  nm_dtype y_dt, nm_stream_t stream) {
  if (dt == NM_I8) {
    if (y_dt != NM_I32) return NM_ERR_DTYPE;
  } else if (dt == NM_FP8) {
    if (y_dt != NM_F32 && y_dt != NM_BF16) return NM_ERR_DTYPE;
  } else if (!float_dtype(dt) || !float_dtype(y_dt) || (y_dt != dt && y_dt != NM_F32)) {
    return NM_ERR_DTYPE;
  }
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (dt == NM_I8 && K >= (int64_t)1 << 17) return NM_ERR_SHAPE;  // int32 sums stay exact
  if ((st = check_layout(layout, K)) != NM_OK) return st;
  if (layout == NM_LAYOUT_BLOCKED && !blocked_pattern_ok(dt, n, m)) return NM_ERR_UNSUPPORTED;
  if (T < 0 || (K > 0 && T > ((int64_t)1 << 40) / K) || (R > 0 && T > ((int64_t)1 << 40) / R))
    return NM_ERR_SHAPE;
  if (missing(values, R * K) || missing(meta, R * K) || missing(X, K * T) || missing(Y, R * T))
    return NM_ERR_NULL;
  if (R * T == 0) return NM_OK;
  if (!aligned16(values) || !aligned16(meta) || !aligned16(X) || !aligned16(Y)) return NM_ERR_ALIGN;
  {
    // Y is written while other workgroups still read values, meta and X
    const int64_t y_bytes = R * T * ((y_dt == NM_F32 || y_dt == NM_I32) ? 4 : 2);
    if (overlaps(Y, y_bytes, X, K * T * elem_bytes(dt)) ||
        overlaps(Y, y_bytes, values, (int64_t)nm_values_bytes(R, K, n, m, dt, layout)) ||
        overlaps(Y, y_bytes, meta, (int64_t)nm_meta_bytes(R, K, n, m, layout)))
      return NM_ERR_ALIAS;
  }
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_spmm(values, meta, R, K, n, m, layout == NM_LAYOUT_BLOCKED, X, T,
                                  (int)dt, Y, (int)y_dt, static_cast<hipStream_t>(stream)));
}

nm_status nm_tmask(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m, uint8_t* mask,
                   nm_stream_t stream) {
  if (!float_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (R % m != 0) return NM_ERR_SHAPE;
  if (missing(W, R * K) || missing(mask, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (overlaps(W, R * K * elem_bytes(dt), mask, R * K)) return NM_ERR_ALIAS;
  if (!aligned16(W) || !aligned16(mask)) return NM_ERR_ALIGN;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_tmask(W, elem_bytes(dt), R, K, n, m, false, mask,
                                   static_cast<hipStream_t>(stream)));
}

nm_status nm_tprune(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m, void* W_out,
                    nm_stream_t stream) {
  if (!float_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (R % m != 0) return NM_ERR_SHAPE;
  if (missing(W, R * K) || missing(W_out, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (W_out != W && overlaps(W, W_out, R * K * elem_bytes(dt))) return NM_ERR_ALIAS;
  if (!aligned16(W) || !aligned16(W_out)) return NM_ERR_ALIGN;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_tmask(W, elem_bytes(dt), R, K, n, m, true, W_out,
                                   static_cast<hipStream_t>(stream)));
}

nm_status nm_compress_t(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m,
                        nm_layout layout, void* values, uint32_t* meta, nm_stream_t stream) {
  if (!float_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(K, R, m)) != NM_OK) return st;  // the transpose is K x R
  if ((st = check_layout(layout, R)) != NM_OK) return st;
  if (missing(W, R * K) || missing(values, R * K) || missing(meta, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  const int64_t wb = R * K * elem_bytes(dt);
  if (overlaps(W, wb, values, (int64_t)nm_values_bytes(K, R, n, m, dt, layout)) ||
      overlaps(W, wb, meta, (int64_t)nm_meta_bytes(K, R, n, m, layout)))
    return NM_ERR_ALIAS;
  if (!aligned16(W) || !aligned16(values) || !aligned16(meta)) return NM_ERR_ALIGN;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_select_t(W, elem_bytes(dt), R, K, n, m, layout == NM_LAYOUT_BLOCKED,
                                      values, meta, static_cast<hipStream_t>(stream)));
}

nm_status nm_prune(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m, void* W_out,
                   nm_stream_t stream) {
  if (!float_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (missing(W, R * K) || missing(W_out, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (W_out != W && overlaps(W, W_out, R * K * elem_bytes(dt))) return NM_ERR_ALIAS;
  if (!aligned16(W) || !aligned16(W_out)) return NM_ERR_ALIGN;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_prune(W, (int)dt, R, K, n, m, W_out,
                                   static_cast<hipStream_t>(stream)));
}

nm_status nm_srste_grad(const void* W, const void* G, nm_dtype dt, int64_t R, int64_t K, int n,
                        int m, float decay, void* G_out, nm_stream_t stream) {
  if (!float_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (missing(W, R * K) || missing(G, R * K) || missing(G_out, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  const int64_t bytes = R * K * elem_bytes(dt);
  if (overlaps(W, G_out, bytes) || (G_out != G && overlaps(G, G_out, bytes))) return NM_ERR_ALIAS;
  if (!aligned16(W) || !aligned16(G) || !aligned16(G_out)) return NM_ERR_ALIGN;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_srste_grad(W, G, (int)dt, R, K, n, m, decay, G_out,
                                        static_cast<hipStream_t>(stream)));
}

size_t nm_perm_workspace_bytes(int64_t R, int64_t K, int n, int m) {
  if (check_pattern(n, m) != NM_OK || check_shape(R, K, m) != NM_OK) return 0;
  if (R * K >= ((int64_t)1 << 31)) return 0;
  return nm::perm_workspace_bytes(R, K, m);
}

namespace {
nm_status check_perm_args(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m,
                          const void* workspace, size_t workspace_bytes) {
  if (!valid_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (R * K >= ((int64_t)1 << 31)) return NM_ERR_SHAPE;  // 32-bit gather indices
  if (missing(W, R * K) || missing(workspace, R * K)) return NM_ERR_NULL;
  if (R * K > 0 && workspace_bytes < nm::perm_workspace_bytes(R, K, m)) return NM_ERR_SHAPE;
  if (!aligned16(W) || !aligned16(workspace)) return NM_ERR_ALIGN;
  return NM_OK;
}
}  // namespace

nm_status nm_perm_gains(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m,
                        const int32_t* perm, float* gain, int32_t* pick, void* workspace,
                        size_t workspace_bytes, nm_stream_t stream) {
  nm_status st = check_perm_args(W, dt, R, K, n, m, workspace, workspace_bytes);
  if (st != NM_OK) return st;
  const int64_t G = K / m;
  if (missing(perm, K) || missing(gain, G * G) || missing(pick, G * G)) return NM_ERR_NULL;
  if (R * K == 0 || G < 2) return NM_OK;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_perm_gains(W, (int)dt, R, K, n, m, perm, gain, pick, workspace,
                                        static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// The scratch buffer of nm_perm_gains_static.  Each device holds its own copy at its own
// address; in host code the name is only the host-side handle of the symbol, so kernels get
// the device address that hipGetSymbolAddress returns for the current device.
static __device__ __align__(256) uint8_t scratch[NM_STATIC_SCRATCH_BYTES];

std::mutex g_scratch_mu;
std::atomic<void*> g_scratch_ptr[kMaxDevices];

// Device address of `scratch` on device `dev` (the current device), looked up once per
// device; nullptr if the lookup fails.
void* scratch_on(int dev) {
  void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
  if (p != nullptr) return p;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess) {
      (void)hipGetLastError();
      return nullptr;
    }
    g_scratch_ptr[dev].store(p, std::memory_order_release);
  }
  return p;
}

}  // namespace

extern "C" {

nm_status nm_perm_gains_static(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m,
                               const int32_t* perm, float* gain, int32_t* pick,
                               nm_stream_t stream) {
  if (!valid_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (R * K >= ((int64_t)1 << 31)) return NM_ERR_SHAPE;  // 32-bit gather indices, as nm_perm_gains
  const int64_t G = K / m;
  if (missing(W, R * K) || missing(perm, K) || missing(gain, G * G) || missing(pick, G * G))
    return NM_ERR_NULL;
  // the kernels use only the permuted fp32 copy of W: the first part of the workspace
  if ((size_t)(R * K) * 4 > NM_STATIC_SCRATCH_BYTES) return NM_ERR_SCRATCH;
  if (!aligned16(W)) return NM_ERR_ALIGN;
  if (R * K == 0 || G < 2) return NM_OK;
  if ((st = check_device()) != NM_OK) return st;
  int dev = 0, sdev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return NM_ERR_DEVICE;
  if (stream != nullptr &&
      (hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev) != hipSuccess || sdev != dev))
    return NM_ERR_DEVICE;
  void* ws = scratch_on(dev);
  if (ws == nullptr) return NM_ERR_DEVICE;
  return from_hip(nm::launch_perm_gains(W, (int)dt, R, K, n, m, perm, gain, pick, ws,
                                        static_cast<hipStream_t>(stream)));
}

nm_status nm_perm_search(const void* W, nm_dtype dt, int64_t R, int64_t K, int n, int m,
                         int max_rounds, int32_t* perm, int* rounds, void* workspace,
                         size_t workspace_bytes, nm_stream_t stream) {
  nm_status st = check_perm_args(W, dt, R, K, n, m, workspace, workspace_bytes);
  if (st != NM_OK) return st;
  if (missing(perm, K)) return NM_ERR_NULL;
  if (max_rounds < 0) return NM_ERR_SHAPE;
  // perm must be a permutation of 0 .. K-1
  std::vector<uint8_t> seen((size_t)K, 0);
  for (int64_t i = 0; i < K; ++i) {
    if (perm[i] < 0 || perm[i] >= K || seen[(size_t)perm[i]]) return NM_ERR_SHAPE;
    seen[(size_t)perm[i]] = 1;
  }
  if (rounds) *rounds = 0;
  if (R * K == 0 || K / m < 2 || max_rounds == 0) return NM_OK;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::run_perm_search(W, (int)dt, R, K, n, m, max_rounds, perm, rounds,
                                      workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

bool half_dtype(int dt) { return dt == NM_F16 || dt == NM_BF16; }
bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }

int64_t codes_bytes(int64_t R, int64_t C) { return (R + 15) / 16 * ((C + 127) / 128) * 1024; }
int64_t scales_bytes(int64_t R, int64_t C, int group) {
  return (R + 15) / 16 * ((C + group - 1) / group) * 32;
}

// The stored matrix of nm_quantize and nm_dequantize: sizes, layout and group.
nm_status check_codes(int64_t R, int64_t C, int layout, int group) {
  const nm_status st = check_shape(R, C, 1);
  if (st != NM_OK) return st;
  if (!group_ok(group)) return NM_ERR_UNSUPPORTED;
  if (layout == NM_LAYOUT_BLOCKED ? C % 32 != 0 : layout != NM_LAYOUT_ROWS) return NM_ERR_LAYOUT;
  return NM_OK;
}

constexpr int64_t kMaxSide = (int64_t)1 << 22;  // 64 rows of 16-bit numbers within 32-bit offsets

nm_status check_xent(nm_dtype dt, int64_t V, int64_t K, int64_t T) {
  if (!half_dtype(dt)) return NM_ERR_DTYPE;
  if (V < 0 || K < 0 || T < 0 || V >= (int64_t)1 << 31 || K >= kMaxSide || T >= kMaxSide ||
      (V == 0 && T > 0))
    return NM_ERR_SHAPE;
  // below 2^36 logits and entries of X every launch has fewer than 2^32 work-items
  nm_status st = check_shape(V, K, 1);
  if (st == NM_OK) st = check_shape(V, T, 1);
  return st == NM_OK ? check_shape(K, T, 1) : st;
}

nm_status check_workspace(const void* p, size_t have, size_t need) {
  if (have < need) return NM_ERR_SCRATCH;
  if (need > 0 && p == nullptr) return NM_ERR_NULL;
  return aligned16(p) ? NM_OK : NM_ERR_ALIGN;
}

struct Range {
  const void* p;
  int64_t bytes;
};
// Does a written range overlap another of the call's ranges (the written ones come first)?
bool any_alias(const Range* r, int written, int all) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < all; ++j)
      if (overlaps(r[i].p, r[i].bytes, r[j].p, r[j].bytes)) return true;
  return false;
}

}  // namespace

extern "C" {

size_t nm_codes_bytes(int64_t R, int64_t C) {
  return check_shape(R, C, 1) == NM_OK ? (size_t)codes_bytes(R, C) : 0;
}

size_t nm_scales_bytes(int64_t R, int64_t C, int group) {
  return check_shape(R, C, 1) == NM_OK && group_ok(group) ? (size_t)scales_bytes(R, C, group) : 0;
}

nm_status nm_quantize(const void* W, nm_dtype dt, int64_t R, int64_t C, nm_layout layout, int group,
                      void* codes, void* scales, nm_dtype scale_dt, nm_stream_t stream) {
  if (!float_dtype(dt) || !half_dtype(scale_dt)) return NM_ERR_DTYPE;
  nm_status st = check_codes(R, C, layout, group);
  if (st != NM_OK) return st;
  if (missing(W, R * C) || missing(codes, R * C) || missing(scales, R * C)) return NM_ERR_NULL;
  if (R * C == 0) return NM_OK;
  if (!aligned16(W) || !aligned16(codes) || !aligned16(scales)) return NM_ERR_ALIGN;
  const Range r[] = {{codes, codes_bytes(R, C)},
                     {scales, scales_bytes(R, C, group)},
                     {W, padded_rows(R, layout) * C * elem_bytes(dt)}};
  if (any_alias(r, 2, 3)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_quantize(W, (int)dt, R, C, layout == NM_LAYOUT_BLOCKED, group, codes,
                                      scales, (int)scale_dt, static_cast<hipStream_t>(stream)));
}

nm_status nm_dequantize(const void* codes, const void* scales, nm_dtype scale_dt, int64_t R,
                        int64_t C, nm_layout layout, int group, void* W_out, nm_stream_t stream) {
  if (!half_dtype(scale_dt)) return NM_ERR_DTYPE;
  nm_status st = check_codes(R, C, layout, group);
  if (st != NM_OK) return st;
  if (missing(W_out, R * C) || missing(codes, R * C) || missing(scales, R * C)) return NM_ERR_NULL;
  if (R * C == 0) return NM_OK;
  if (!aligned16(W_out) || !aligned16(codes) || !aligned16(scales)) return NM_ERR_ALIGN;
  const Range r[] = {{W_out, padded_rows(R, layout) * C * 2},
                     {codes, codes_bytes(R, C)},
                     {scales, scales_bytes(R, C, group)}};
  if (any_alias(r, 1, 3)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_dequantize(codes, scales, (int)scale_dt, R, C,
                                        layout == NM_LAYOUT_BLOCKED, group, W_out,
                                        static_cast<hipStream_t>(stream)));
}

namespace {
nm_status check_matvec(int64_t R, int64_t K, int64_t T, bool sparse) {
  // the products' launches have at most 512 work-items for 16 rows along x, a slice for 1024 rows of X
  // or more along y and a workgroup for 16 columns or more along z; the slices' join is checked apart
  if (T < 0 || T >= kMaxSide / 4 || K >= (int64_t)1 << 25 || R >= (int64_t)1 << 26)
    return NM_ERR_SHAPE;
  const nm_status st = check_shape(R, K, 1);
  const bool small = (R + 15) * (T + 31) < (int64_t)1 << 34;
  return st != NM_OK || small || nm::matvec_fits(R, K, T, sparse) ? st : NM_ERR_SHAPE;
}
}  // namespace

size_t nm_matvec_workspace_bytes(int64_t R, int64_t K, int64_t T, int sparse) {
  if (check_matvec(R, K, T, sparse != 0) != NM_OK || R * T == 0) return 0;
  return nm::matvec_workspace_bytes(R, K, T, sparse != 0);
}

nm_status nm_matvec(const void* codes, const void* scales, const uint32_t* meta, int64_t R,
                    int64_t K, int group, const void* X, int64_t T, nm_dtype dt, void* Y,
                    nm_dtype y_dt, void* workspace, size_t workspace_bytes, nm_stream_t stream) {
  if (!half_dtype(dt) || (y_dt != dt && y_dt != NM_F32)) return NM_ERR_DTYPE;
  nm_status st = check_matvec(R, K, T, meta != nullptr);
  if (st != NM_OK) return st;
  if (!group_ok(group)) return NM_ERR_UNSUPPORTED;
  if (meta != nullptr && K % 64 != 0) return NM_ERR_LAYOUT;
  if (missing(codes, R * K) || missing(scales, R * K) || missing(X, K * T) || missing(Y, R * T))
    return NM_ERR_NULL;
  if (R * T == 0) return NM_OK;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(meta) || !aligned16(X) || !aligned16(Y))
    return NM_ERR_ALIGN;
  const size_t need = nm::matvec_workspace_bytes(R, K, T, meta != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const int64_t C = meta != nullptr ? K / 2 : K;
  const Range r[] = {{Y, R * T * elem_bytes(y_dt)},
                     {workspace, (int64_t)need},
                     {codes, codes_bytes(R, C)},
                     {scales, scales_bytes(R, C, group)},
                     {meta, meta != nullptr ? (R + 15) / 16 * 16 * (K / 8) : 0},
                     {X, K * T * 2}};
  if (any_alias(r, 2, 6)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_matvec(codes, scales, meta, R, K, group, X, T, (int)dt, Y, (int)y_dt,
                                    workspace, static_cast<hipStream_t>(stream)));
}

size_t nm_xent_workspace_bytes(int64_t V, int64_t K, int64_t T) {
  return check_xent(NM_BF16, V, K, T) == NM_OK ? nm::xent_workspace_bytes(V, K, T) : 0;
}

size_t nm_xent_grad_workspace_bytes(int64_t V, int64_t K, int64_t T) {
  return check_xent(NM_BF16, V, K, T) == NM_OK && V * K * T > 0
             ? nm::xent_grad_workspace_bytes(V, K, T)
             : 0;
}

nm_status nm_xent(const void* W, const void* X, nm_dtype dt, int64_t V, int64_t K, int64_t T,
                  const int64_t* target, float* loss, float* lse, void* workspace,
                  size_t workspace_bytes, nm_stream_t stream) {
  nm_status st = check_xent(dt, V, K, T);
  if (st != NM_OK) return st;
  if (missing(W, V * K) || missing(X, K * T) || missing(target, T) || missing(loss, T) ||
      missing(lse, T))
    return NM_ERR_NULL;
  if (T == 0) return NM_OK;
  if (!aligned16(W) || !aligned16(X) || !aligned16(target) || !aligned16(loss) || !aligned16(lse))
    return NM_ERR_ALIGN;
  const size_t need = nm::xent_workspace_bytes(V, K, T);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Range r[] = {{loss, T * 4}, {lse, T * 4},     {workspace, (int64_t)need},
                     {W, V * K * 2}, {X, K * T * 2}, {target, T * 8}};
  if (any_alias(r, 3, 6)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_xent(W, X, (int)dt, V, K, T, target, loss, lse, workspace,
                                  static_cast<hipStream_t>(stream)));
}

nm_status nm_xent_grad(const void* W, const void* X, nm_dtype dt, int64_t V, int64_t K, int64_t T,
                       const int64_t* target, const float* lse, const float* gout, void* dW,
                       void* dX, void* workspace, size_t workspace_bytes, nm_stream_t stream) {
  nm_status st = check_xent(dt, V, K, T);
  if (st != NM_OK) return st;
  if (missing(W, V * K) || missing(X, K * T) || missing(target, T) || missing(lse, T) ||
      missing(gout, T) || missing(dW, V * K) || missing(dX, K * T))
    return NM_ERR_NULL;
  if (K == 0 || V == 0) return NM_OK;  // both results are empty
  if (!aligned16(W) || !aligned16(X) || !aligned16(target) || !aligned16(lse) || !aligned16(gout) ||
      !aligned16(dW) || !aligned16(dX))
    return NM_ERR_ALIGN;
  const size_t need = T > 0 ? nm::xent_grad_workspace_bytes(V, K, T) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Range r[] = {{dW, V * K * 2}, {dX, K * T * 2},  {workspace, (int64_t)need}, {W, V * K * 2},
                     {X, K * T * 2},  {target, T * 8}, {lse, T * 4},              {gout, T * 4}};
  if (any_alias(r, 3, 8)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_xent_grad(W, X, (int)dt, V, K, T, target, lse, gout, dW, dX, workspace,
                                       static_cast<hipStream_t>(stream)));
}

namespace {
nm_status check_orth(nm_dtype dt, int64_t R, int64_t K) {
  if (!float_dtype(dt)) return NM_ERR_DTYPE;
  if (R < 0 || K < 0 || R >= kMaxSide || K >= kMaxSide) return NM_ERR_SHAPE;
  return check_shape(R, K, 1);
}
}  // namespace

size_t nm_orthogonalize_workspace_bytes(int64_t R, int64_t K, nm_dtype dt) {
  return check_orth(dt, R, K) == NM_OK && R * K > 0 ? nm::orth_workspace_bytes(R, K, (int)dt) : 0;
}

nm_status nm_orthogonalize(const void* G, nm_dtype dt, int64_t R, int64_t K, int steps, float eps,
                           void* out, void* workspace, size_t workspace_bytes, nm_stream_t stream) {
  nm_status st = check_orth(dt, R, K);
  if (st != NM_OK) return st;
  if (steps < 1 || steps > 100 || !(eps >= 0.f)) return NM_ERR_SHAPE;
  if (missing(G, R * K) || missing(out, R * K)) return NM_ERR_NULL;
  if (R * K == 0) return NM_OK;
  if (!aligned16(G) || !aligned16(out)) return NM_ERR_ALIGN;
  const size_t need = nm::orth_workspace_bytes(R, K, (int)dt);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const int64_t bytes = R * K * elem_bytes(dt);
  const Range r[] = {{workspace, (int64_t)need}, {G, bytes}, {out, bytes}};
  if (any_alias(r, 1, 3) || (out != G && overlaps(out, G, bytes))) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_orthogonalize(G, (int)dt, R, K, steps, eps, out, workspace,
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

bool act_ok(int act) { return act >= NM_ACT_NONE && act <= NM_ACT_GELU_TANH; }

// What a result of a product with an epilogue may be rounded to.
bool act_types_ok(int dt, int y_dt) {
  if (!valid_dtype(dt) || !float_dtype(y_dt)) return false;
  return elem_bytes((nm_dtype)dt) == 1 || y_dt == dt || y_dt == NM_F32;
}

bool below(int64_t a, int64_t b, int64_t most) { return a == 0 || b <= most / a; }

}  // namespace

extern "C" {

size_t nm_spmm_act_workspace_bytes(int64_t R, int64_t K, int n, int m, int64_t T, nm_dtype dt) {
  if (!valid_dtype(dt) || check_pattern(n, m) != NM_OK || check_shape(R, K, m) != NM_OK || T < 0 ||
      !below(K, T, (int64_t)1 << 40) || !below(R, T, (int64_t)1 << 40) || R * T == 0)
    return 0;
  return nm::spmm_act_workspace_bytes(R, K, n, m, T, (int)dt);
}

nm_status nm_spmm_act(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n, int m,
                      nm_layout layout, const void* X, int64_t T, nm_dtype dt, const float* scale,
                      const float* bias, nm_act act, const void* residual, void* Z, void* Y,
                      nm_dtype y_dt, void* workspace, size_t workspace_bytes, nm_stream_t stream) {
  if (!act_types_ok(dt, y_dt)) return NM_ERR_DTYPE;
  const bool eight = elem_bytes(dt) == 1;
  if (eight ? Z != nullptr : scale != nullptr) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if (dt == NM_I8 && K >= (int64_t)1 << 17) return NM_ERR_SHAPE;  // int32 sums stay exact
  if ((st = check_layout(layout, K)) != NM_OK) return st;
  if (layout == NM_LAYOUT_BLOCKED && !blocked_pattern_ok(dt, n, m)) return NM_ERR_UNSUPPORTED;
  if (!act_ok(act)) return NM_ERR_UNSUPPORTED;
  if (T < 0 || !below(K, T, (int64_t)1 << 40) || !below(R, T, (int64_t)1 << 40)) return NM_ERR_SHAPE;
  if (missing(values, R * K) || missing(meta, R * K) || missing(X, K * T) || missing(Y, R * T))
    return NM_ERR_NULL;
  if (R * T == 0) return NM_OK;
  if (!aligned16(values) || !aligned16(meta) || !aligned16(X) || !aligned16(Y) || !aligned16(scale) ||
      !aligned16(bias) || !aligned16(residual) || !aligned16(Z))
    return NM_ERR_ALIGN;
  const size_t need = nm::spmm_act_workspace_bytes(R, K, n, m, T, (int)dt);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const int64_t y_bytes = R * T * elem_bytes(y_dt);
  const Range r[] = {{Y, y_bytes},
                     {Z, Z ? R * T * elem_bytes(dt) : 0},
                     {workspace, (int64_t)need},
                     {values, (int64_t)nm_values_bytes(R, K, n, m, dt, layout)},
                     {meta, (int64_t)nm_meta_bytes(R, K, n, m, layout)},
                     {X, K * T * elem_bytes(dt)},
                     {scale, scale ? R * 4 : 0},
                     {bias, bias ? R * 4 : 0},
                     {residual, residual && residual != Y ? y_bytes : 0}};
  if (any_alias(r, 3, 9)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  nm::Product p{};
  p.scale = scale;
  p.bias = bias;
  p.residual = residual;
  p.y = Y;
  p.z = Z;
  p.act = (int)act;
  p.y_dt = (int)y_dt;
  p.z_dt = (int)dt;
  return from_hip(nm::run_spmm_act(values, meta, R, K, n, m, layout == NM_LAYOUT_BLOCKED, X, T, (int)dt,
                                   p, workspace, static_cast<hipStream_t>(stream)));
}

namespace {
nm_status check_spmm_grad(int64_t R, int64_t K, int64_t T) {
  if (R < 0 || K < 0 || T < 0 || R >= kMaxSide || K >= kMaxSide || T >= kMaxSide) return NM_ERR_SHAPE;
  nm_status st = check_shape(R, K, 1);
  if (st == NM_OK) st = check_shape(R, T, 1);
  return st == NM_OK ? check_shape(K, T, 1) : st;
}
}  // namespace

size_t nm_spmm_act_grad_workspace_bytes(int64_t R, int64_t K, int64_t T, nm_act act, int want_dW,
                                        int want_dX, int want_dZ) {
  return nm_spmm_act_grad_dt_workspace_bytes(R, K, T, NM_BF16, act, want_dW, want_dX, want_dZ);
}

size_t nm_spmm_act_grad_dt_workspace_bytes(int64_t R, int64_t K, int64_t T, nm_dtype dt, nm_act act,
                                           int want_dW, int want_dX, int want_dZ) {
  if (!half_dtype(dt) || check_spmm_grad(R, K, T) != NM_OK || !act_ok(act)) return 0;
  return nm::spmm_act_grad_workspace_bytes(R, K, T, dt == NM_BF16, (int)act, want_dW && R * K > 0,
                                           want_dX && K * T > 0, want_dZ != 0);
}

nm_status nm_spmm_act_grad(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n,
                           int m, nm_layout layout, const void* X, int64_t T, nm_dtype dt, nm_act act,
                           const void* Z, const void* dY, void* dW, void* dX, float* dbias, void* dZ,
                           void* workspace, size_t workspace_bytes, nm_stream_t stream) {
  if (!half_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_pattern(n, m);
  if (st != NM_OK) return st;
  if ((st = check_shape(R, K, m)) != NM_OK) return st;
  if ((st = check_spmm_grad(R, K, T)) != NM_OK) return st;
  if ((st = check_layout(layout, K)) != NM_OK) return st;
  if (!act_ok(act)) return NM_ERR_UNSUPPORTED;
  if (missing(dY, R * T) || (act != NM_ACT_NONE && missing(Z, R * T)) || (dW && missing(X, K * T)) ||
      (dX && (missing(values, R * K) || missing(meta, R * K))))
    return NM_ERR_NULL;
  if (!aligned16(values) || !aligned16(meta) || !aligned16(X) || !aligned16(Z) || !aligned16(dY) ||
      !aligned16(dW) || !aligned16(dX) || !aligned16(dbias) || !aligned16(dZ))
    return NM_ERR_ALIGN;
  const size_t need = nm_spmm_act_grad_dt_workspace_bytes(R, K, T, dt, act, dW != nullptr, dX != nullptr,
                                                          dZ != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Range r[] = {{dW, dW ? R * K * 2 : 0},
                     {dX, dX ? K * T * 2 : 0},
                     {dbias, dbias ? R * 4 : 0},
                     {dZ, dZ ? R * T * 2 : 0},
                     {workspace, (int64_t)need},
                     {values, dX ? (int64_t)nm_values_bytes(R, K, n, m, dt, layout) : 0},
                     {meta, dX ? (int64_t)nm_meta_bytes(R, K, n, m, layout) : 0},
                     {X, dW ? K * T * 2 : 0},
                     {Z, act != NM_ACT_NONE ? R * T * 2 : 0},
                     {dY, R * T * 2}};
  if (any_alias(r, 5, 10)) return NM_ERR_ALIAS;
  if (R * K + R * T + K * T == 0 && (R == 0 || dbias == nullptr)) return NM_OK;
  if ((st = check_device()) != NM_OK) return st;
  const nm::SpmmGradCall c{values, meta, R, K, n, m, layout == NM_LAYOUT_BLOCKED, X, T, dt == NM_BF16,
                           (int)act, Z, dY, dW, dX, dbias, dZ};
  return from_hip(nm::launch_spmm_act_grad(c, workspace, static_cast<hipStream_t>(stream)));
}

nm_status nm_matvec_act(const void* codes, const void* scales, const uint32_t* meta, int64_t R,
                        int64_t K, int group, const void* X, int64_t T, nm_dtype dt, const float* bias,
                        nm_act act, const void* residual, void* Y, nm_dtype y_dt, void* workspace,
                        size_t workspace_bytes, nm_stream_t stream) {
  if (!half_dtype(dt) || (y_dt != dt && y_dt != NM_F32)) return NM_ERR_DTYPE;
  nm_status st = check_matvec(R, K, T, meta != nullptr);
  if (st != NM_OK) return st;
  if (!group_ok(group) || !act_ok(act)) return NM_ERR_UNSUPPORTED;
  if (meta != nullptr && K % 64 != 0) return NM_ERR_LAYOUT;
  if (missing(codes, R * K) || missing(scales, R * K) || missing(X, K * T) || missing(Y, R * T))
    return NM_ERR_NULL;
  if (R * T == 0) return NM_OK;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(meta) || !aligned16(X) || !aligned16(Y) ||
      !aligned16(bias) || !aligned16(residual))
    return NM_ERR_ALIGN;
  const size_t need = nm::matvec_workspace_bytes(R, K, T, meta != nullptr);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const int64_t C = meta != nullptr ? K / 2 : K, y_bytes = R * T * elem_bytes(y_dt);
  const Range r[] = {{Y, y_bytes},
                     {workspace, (int64_t)need},
                     {codes, codes_bytes(R, C)},
                     {scales, scales_bytes(R, C, group)},
                     {meta, meta != nullptr ? (R + 15) / 16 * 16 * (K / 8) : 0},
                     {X, K * T * 2},
                     {bias, bias ? R * 4 : 0},
                     {residual, residual && residual != Y ? y_bytes : 0}};
  if (any_alias(r, 2, 8)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  nm::Product p{};
  p.bias = bias;
  p.residual = residual;
  p.y = Y;
  p.act = (int)act;
  p.y_dt = (int)y_dt;
  return from_hip(nm::launch_matvec_act(codes, scales, meta, R, K, group, X, T, (int)dt, p, workspace,
                                        static_cast<hipStream_t>(stream)));
}

namespace {

constexpr int64_t kMostTensors = (int64_t)1 << 20, kMostEntries = (int64_t)1 << 40;

nm_status check_tensors(const void* const* grads, void* const* outs, const int64_t* counts,
                        const nm_dtype* dts, int64_t tensors, bool write) {
  if (tensors < 0 || tensors > kMostTensors) return NM_ERR_SHAPE;
  if (tensors == 0) return NM_OK;
  if (counts == nullptr || dts == nullptr || grads == nullptr || (write && outs == nullptr))
    return NM_ERR_NULL;
  for (int64_t i = 0; i < tensors; ++i) {
    if (!float_dtype(dts[i])) return NM_ERR_DTYPE;
    if (counts[i] < 0 || counts[i] >= kMostEntries) return NM_ERR_SHAPE;
    if (missing(grads[i], counts[i]) || (write && missing(outs[i], counts[i]))) return NM_ERR_NULL;
    const uintptr_t mask = (uintptr_t)elem_bytes(dts[i]) - 1;
    if (counts[i] > 0 && ((reinterpret_cast<uintptr_t>(grads[i]) & mask) ||
                          (write && (reinterpret_cast<uintptr_t>(outs[i]) & mask))))
      return NM_ERR_ALIGN;
  }
  return NM_OK;
}

// Does what is written overlap anything else?  All ranges in the order of their starts: a written
// one may not begin before the end of any earlier one, a read one not before that of a written one.
bool tensors_alias(const void* const* grads, void* const* outs, const int64_t* counts,
                   const nm_dtype* dts, int64_t tensors, const Range* more, int n_more, int written) {
  struct Span {
    uintptr_t begin, end;
    bool write;
  };
  std::vector<Span> all;
  all.reserve((size_t)(2 * tensors) + (size_t)n_more);
  const auto add = [&](const void* p, int64_t bytes, bool write) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    if (p != nullptr && bytes > 0) all.push_back(Span{b, b + (uintptr_t)bytes, write});
  };
  for (int64_t i = 0; i < tensors; ++i) {
    const int64_t bytes = counts[i] * elem_bytes(dts[i]);
    if (outs) add(outs[i], bytes, true);
    if (!outs || outs[i] != grads[i]) add(grads[i], bytes, false);
  }
  for (int i = 0; i < n_more; ++i) add(more[i].p, more[i].bytes, i < written);
  std::sort(all.begin(), all.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any_end = 0, write_end = 0;
  for (const Span& s : all) {
    if (s.begin < (s.write ? any_end : write_end)) return true;
    any_end = std::max(any_end, s.end);
    if (s.write) write_end = std::max(write_end, s.end);
  }
  return false;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

size_t nm_grad_norm_workspace_bytes(const int64_t* counts, int64_t tensors) {
  if (tensors <= 0 || tensors > kMostTensors || counts == nullptr) return 0;
  return nm::norm_workspace_bytes(counts, tensors);
}

nm_status nm_grad_norm(const void* const* grads, const int64_t* counts, const nm_dtype* dts,
                       int64_t tensors, float* norm, void* workspace, size_t workspace_bytes,
                       nm_stream_t stream) try {
  nm_status st = check_tensors(grads, nullptr, counts, dts, tensors, false);
  if (st != NM_OK) return st;
  if (norm == nullptr) return NM_ERR_NULL;
  if (!aligned4(norm)) return NM_ERR_ALIGN;
  const size_t need = nm_grad_norm_workspace_bytes(counts, tensors);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Range more[] = {{norm, 4}, {workspace, (int64_t)need}};
  if (tensors_alias(grads, nullptr, counts, dts, tensors, more, 2, 2)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_clip(grads, nullptr, counts, reinterpret_cast<const int*>(dts), tensors, 0.f,
                                  nullptr, norm, workspace, static_cast<hipStream_t>(stream)));
} catch (const std::bad_alloc&) {
  return NM_ERR_SHAPE;  // no host memory to check that many tensors
}

nm_status nm_clip_grads(const void* const* grads, void* const* outs, const int64_t* counts,
                        const nm_dtype* dts, int64_t tensors, float max_norm, const float* given,
                        float* norm, void* workspace, size_t workspace_bytes, nm_stream_t stream) try {
  nm_status st = check_tensors(grads, outs, counts, dts, tensors, true);
  if (st != NM_OK) return st;
  if (!(max_norm >= 0.f)) return NM_ERR_SHAPE;
  if (given == nullptr && norm == nullptr) return NM_ERR_NULL;
  if (!aligned4(norm) || !aligned4(given)) return NM_ERR_ALIGN;
  const size_t need = given ? 0 : nm_grad_norm_workspace_bytes(counts, tensors);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const Range more[] = {{given ? nullptr : norm, 4}, {workspace, (int64_t)need}, {given, 4}};
  if (tensors_alias(grads, outs, counts, dts, tensors, more, 3, 2)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  return from_hip(nm::launch_clip(grads, outs, counts, reinterpret_cast<const int*>(dts), tensors,
                                  max_norm, given, norm, workspace, static_cast<hipStream_t>(stream)));
} catch (const std::bad_alloc&) {
  return NM_ERR_SHAPE;
}

namespace {
nm_status check_logits(int64_t V, int64_t T, int64_t count) {
  const int64_t most = (int64_t)1 << 31;
  if (V < 0 || T < 0 || V >= most || T >= (int64_t)1 << 20 || count < 0 || count >= most)
    return NM_ERR_SHAPE;
  return check_shape(V, T, 1);
}
}  // namespace

size_t nm_adjust_logits_workspace_bytes(int64_t V, int64_t T, int64_t count) {
  return check_logits(V, T, count) == NM_OK && V * T > 0 ? nm::logits_workspace_bytes(V, T, count) : 0;
}

nm_status nm_adjust_logits(const void* logits, nm_dtype dt, int64_t V, int64_t T,
                           const int64_t* tokens, int64_t count, const int64_t* starts,
                           const int64_t* prompts, const float* repetition, const float* presence,
                           const float* frequency, const float* bias, int bias_each,
                           const uint32_t* allowed, void* out, void* workspace,
                           size_t workspace_bytes, nm_stream_t stream) {
  if (!float_dtype(dt)) return NM_ERR_DTYPE;
  nm_status st = check_logits(V, T, tokens ? count : 0);
  if (st != NM_OK) return st;
  if (missing(logits, V * T) || missing(out, V * T) || (tokens && missing(starts, T))) return NM_ERR_NULL;
  if (V * T == 0) return NM_OK;
  for (const void* p : {logits, (const void*)out, (const void*)tokens, (const void*)starts,
                        (const void*)prompts, (const void*)repetition, (const void*)presence,
                        (const void*)frequency, (const void*)bias, (const void*)allowed})
    if (!aligned16(p)) return NM_ERR_ALIGN;
  if (tokens == nullptr) count = 0;
  const size_t need = nm_adjust_logits_workspace_bytes(V, T, count);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != NM_OK) return st;
  const auto floats = [&](const float* p, int64_t n) { return Range{p, p ? n * 4 : 0}; };
  const int64_t bytes = V * T * elem_bytes(dt);
  const Range r[] = {{out, bytes},
                     {workspace, (int64_t)need},
                     {logits, logits != out ? bytes : 0},
                     {tokens, tokens ? count * 8 : 0},
                     {starts, tokens ? (T + 1) * 8 : 0},
                     {prompts, prompts ? T * 8 : 0},
                     floats(repetition, T),
                     floats(presence, T),
                     floats(frequency, T),
                     floats(bias, bias_each ? V * T : V),
                     {allowed, allowed ? T * ((V + 31) / 32) * 4 : 0}};
  if (any_alias(r, 2, 11)) return NM_ERR_ALIAS;
  if ((st = check_device()) != NM_OK) return st;
  const nm::LogitsCall c{logits, (int)dt, V, T, tokens, count, starts, prompts, repetition, presence,
                         frequency, bias, bias_each != 0, allowed, out};
  return from_hip(nm::launch_adjust_logits(c, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
