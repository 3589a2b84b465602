// nm_gemm.h -- the dense 16-bit matrix product on the matrix cores (gfx950) that the cross
// entropy and the orthogonalised update are built from: one workgroup's tile of
//   C[m, n] = sum over k of A(m, k) B(n, k),
// fp32 accumulators, which the calling kernel's epilogue then turns into what it needs.
//
// Either operand is stored with k contiguous (rows of k) or with k as the row index
// ("strided"), so no operand is ever transposed in memory.  The sum's length is a multiple of
// 64 (the callers pad with zeros); rows of m and n past the matrix read another of its rows
// and the epilogue drops them.  A strided operand's rows are whole 16-byte pieces (ld and the
// width are multiples of 8).
//
// Steps of 64 k of both operands are brought into LDS by direct loads, up to STAGES steps ahead of
// the step that is being multiplied: two stages for the large tiles, whose step is long, and
// as many as fit for the small ones, whose whole sum may then be in flight at once.  A wave owns
// 32 FM x 32 FN of the tile and uses v_mfma_f32_32x32x16.  LDS layouts of a stage, both free of
// bank conflicts for their reads:
//   k contiguous: 128 bytes a row of the tile, 16-byte chunk c at c ^ (row / 2 & 7); a fragment is
//     one 16-byte read per lane;
//   strided: a row of the tile's columns for each k, 32-byte pair p at p ^ 2 (k & 3); a
//     fragment is two transposing reads (ds_read_b64_tr_b16).
// Bound, large tiles: the power that the matrix cores draw and the waits at a step's end; 256 x 256
// tiles keep them busy 58 to 62 % of the time at a clock that the load pulls down to 1.8 to 1.9 GHz
// (32768 x 4096 x 2048 bf16 in 466 us, 1180 TFLOP/s).  Small tiles: the barrier and the LDS latency of each
// 16 k, 0.25 us a step of 64 x 64 against 0.06 of products.  Measured on the way: more stages than
// these change nothing, four waves on 128 x 128 and sixteen on 256 x 256 are 2 to 10 % slower, fewer
// bank conflicts and reads between products gave 5 %, the loop's inner steps without tests up to 8 %.
// PARTS = 2: each operand is a sum hi + lo of two 16-bit matrices, and hi hi + hi lo + lo hi is
// summed; the four tiles are loaded once a step.
#pragma once

#include <type_traits>

#include "nm_launch.h"
#include "nm_mfma.h"

namespace nm {
namespace {

constexpr int kGemmStep = 64;  // k per step

// Between a wave's writes to LDS and its other lanes' reads of them, both ways round: LDS serves a
// wave's accesses in order, so only the compiler has to keep it.
__device__ __forceinline__ void keep_lds_order() { asm volatile("" ::: "memory"); }

// The first `left` of eight 16-bit numbers in LDS to memory at any 2-byte address.
__device__ __forceinline__ void store_piece(uint16_t* to, const uint8_t* lds, int64_t left) {
  const u32x4_t v = *reinterpret_cast<const u32x4_t*>(lds);
  if (left >= 8) {
    *reinterpret_cast<u32x4_any_t*>(to) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) to[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
  }
}

// One operand: element (row, k) at p[row * ld + k], or at p[k * ld + row] if strided.  rows:
// rows of the whole matrix from p on (loads past them read the last one).
struct GemmOperand {
  const uint16_t* p;
  int64_t ld;
  int64_t rows;
  int64_t lo;  // elements from p to the lo part, where there is one
};

// Workgroups are dealt to the XCDs in turn; each XCD takes a contiguous run of tiles, walked
// in blocks of gm x gn so that the tiles it works on at once share rows of A and B in its L2.
struct GemmMap {
  int tiles_m, tiles_n, xcds, per_xcd, gm, gn;
  bool lower;  // only the tiles of a square result with tm >= tn
  __device__ __forceinline__ bool tile_of(int b, int& tm, int& tn) const {
    const int t = (b % xcds) * per_xcd + b / xcds;
    if (lower) {
      if (t >= tiles_m * (tiles_m + 1) / 2) return false;
      tm = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);  // within one of the row that holds t
      if (tm * (tm + 1) / 2 > t) --tm;
      if ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
      tn = t - tm * (tm + 1) / 2;
      return true;
    }
    if (t >= tiles_m * tiles_n) return false;
    const int g_m = t / (gm * tiles_n);
    const int rows = min(gm, tiles_m - g_m * gm);
    const int u = t - g_m * gm * tiles_n;
    const int g_n = u / (rows * gn);
    const int v = u - g_n * rows * gn;
    tm = g_m * gm + v % rows;
    tn = g_n * gn + v / rows;
    return true;
  }
  int groups() const { return per_xcd * xcds; }
};

inline GemmMap make_gemm_map(int64_t tiles_m, int64_t tiles_n, bool lower = false) {
  GemmMap map;
  map.tiles_m = (int)tiles_m;
  map.tiles_n = (int)tiles_n;
  map.lower = lower;
  map.xcds = xcd_count();
  const int64_t tiles = lower ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n;
  map.per_xcd = (int)((tiles + map.xcds - 1) / map.xcds);
  map.gn = tiles_n < 4 ? (int)tiles_n : 4;
  map.gm = 32 / map.gn;
  return map;
}

// WM x WN waves of 32 FM rows x 32 FN columns each; AS / BS: operand stored strided;
// SWAP: accumulators hold C transposed within a fragment (lane = row, registers = columns).
template <int WM, int WN, int FM, int FN, bool AS, bool BS, bool BF16, bool SWAP, int STAGES = 2,
          int PARTS = 1>
struct Gemm {
  static constexpr int kFM = FM, kFN = FN, kWM = WM, kWN = WN;
  static constexpr bool kAS = AS, kBS = BS;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kBM = 32 * FM * WM, kBN = 32 * FN * WN;
  static constexpr int kABytes = kBM * 2 * kGemmStep, kBBytes = kBN * 2 * kGemmStep;
  static constexpr int kStage = PARTS * (kABytes + kBBytes), kLds = STAGES * kStage;
  static constexpr int kALoads = kABytes / 1024 / kWaves, kBLoads = kBBytes / 1024 / kWaves;
  static constexpr int kLoads = PARTS * (kALoads + kBLoads);  // of a wave and step
  static_assert(kABytes % (1024 * kWaves) == 0 && kBBytes % (1024 * kWaves) == 0, "whole loads");
  static constexpr int kProducts = FM * FN * (2 * PARTS - 1);  // of a wave and 16 k
  static_assert(kLds <= 160 * 1024, "LDS");
  static_assert(STAGES >= 2 && (STAGES - 1) * kLoads <= 63, "vmcnt");

  typedef float16v_t Acc[FM][FN];

  // Byte offset from (row0, k = 0) of what lane `lane` reads in load `j` of wave `wave`; left:
  // rows of the matrix from row0 on, kleft: k's from the step's first one on.
  template <bool STRIDED, int ROWS>
  static __device__ __forceinline__ uint32_t source(int j, int wave, int lane, int64_t ld,
                                                    int64_t left, int64_t kleft) {
    const int slot = (j * kWaves + wave) * 64 + lane;  // 16-byte slot of the tile
    if constexpr (!STRIDED) {
      const int r = slot >> 3, c = (slot & 7) ^ ((r >> 1) & 7);
      const int64_t row = r < left ? r : left - 1;
      return (uint32_t)(row * ld * 2 + 16 * c);
    } else {
      constexpr int kChunks = ROWS / 8, kPairs = ROWS / 16;
      const int k = slot / kChunks, pc = slot % kChunks;
      const int c = 2 * ((pc >> 1) ^ (((k & 3) << 1) & (kPairs - 1))) + (pc & 1);
      const int64_t col = 8 * c < left ? 8 * c : 0;
      const int64_t row = k < kleft ? k : kleft - 1;
      return (uint32_t)((row * ld + col) * 2);
    }
  }

  // Byte offset within an operand's part of a stage of the calling lane's fragment `f` (32 rows
  // from 32 f of the wave's first row w0) for k 16 kk .. 16 kk + 15.
  template <bool STRIDED, int ROWS>
  static __device__ __forceinline__ u32x4_t fragment(const uint8_t* tile, int w0, int f, int kk,
                                                     int lane) {
    const int q = lane >> 5;
    if constexpr (!STRIDED) {
      const int r = w0 + 32 * f + (lane & 31);
      return *reinterpret_cast<const u32x4_t*>(tile + r * 128 + (((2 * kk + q) ^ ((r >> 1) & 7)) << 4));
    } else {
      [[maybe_unused]] constexpr int kPairs = ROWS / 16;
      const int l16 = lane & 15, half = (lane >> 4) & 1;
      [[maybe_unused]] const int k = 16 * kk + 8 * q + (l16 >> 2);
      [[maybe_unused]] const int p = (w0 + 32 * f + 16 * half) / 16;
#if defined(__HIP_DEVICE_COMPILE__)
      // rows k and k + 4 have the same swizzle
      const uint8_t* at =
          tile + k * (ROWS * 2) + ((p ^ (((k & 3) << 1) & (kPairs - 1))) << 5) + 8 * (l16 & 3);
      const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)at);
      const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(at + 4 * ROWS * 2));
      return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#else
      return u32x4_t{};
#endif
    }
  }

  static __device__ __forceinline__ float16v_t mfma(const u32x4_t& a, const u32x4_t& b,
                                                    const float16v_t& c) {
    const u32x4_t& x = SWAP ? b : a;
    const u32x4_t& y = SWAP ? a : b;
    if constexpr (BF16)
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, x),
                                                     __builtin_bit_cast(bf16x8_t, y), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, x),
                                                    __builtin_bit_cast(f16x8_t, y), c, 0, 0, 0);
  }

  // acc += the tile at (m0, n0) over `steps` steps.  klen: rows of a strided A (past them its last
  // step reads the last one again, against zeros of B); B always has whole steps.
  static __device__ __forceinline__ void run(const GemmOperand& a, const GemmOperand& b,
                                             int64_t m0, int64_t n0, int steps, int64_t klen,
                                             uint8_t* smem, Acc& acc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int64_t a_left = a.rows - m0, b_left = b.rows - n0;
    const uint16_t* a0 = a.p + (AS ? m0 : m0 * a.ld);
    const uint16_t* b0 = b.p + (BS ? n0 : n0 * b.ld);
    const int64_t a_step = AS ? kGemmStep * a.ld : kGemmStep;
    const int64_t b_step = BS ? kGemmStep * b.ld : kGemmStep;
    const bool ragged = AS && klen < (int64_t)steps * kGemmStep;
    uint32_t av[kALoads], bv[kBLoads];
#pragma unroll
    for (int j = 0; j < kALoads; ++j)
      av[j] = source<AS, kBM>(j, wave, lane, a.ld, a_left, kGemmStep);
#pragma unroll
    for (int j = 0; j < kBLoads; ++j)
      bv[j] = source<BS, kBN>(j, wave, lane, b.ld, b_left, kGemmStep);
    const uint32_t lds0 = lds_addr(smem);

    auto issue = [&](int t, int stage) {
      const uint16_t* pa = a0 + t * a_step;
      const uint16_t* pb = b0 + t * b_step;
      const uint32_t st = lds0 + stage * kStage + wave * 1024;
      if (ragged && t == steps - 1) {  // A's rows end inside this step
        const int64_t kleft = klen - (int64_t)t * kGemmStep;
#pragma unroll
        for (int j = 0; j < kALoads; ++j)
          global_to_lds_sv<16>(pa, source<AS, kBM>(j, wave, lane, a.ld, a_left, kleft),
                               st + j * kWaves * 1024);
      } else {
#pragma unroll
        for (int j = 0; j < kALoads; ++j) global_to_lds_sv<16>(pa, av[j], st + j * kWaves * 1024);
      }
#pragma unroll
      for (int j = 0; j < kBLoads; ++j)
        global_to_lds_sv<16>(pb, bv[j], st + PARTS * kABytes + j * kWaves * 1024);
      if constexpr (PARTS == 2) {
#pragma unroll
        for (int j = 0; j < kALoads; ++j)
          global_to_lds_sv<16>(pa + a.lo, av[j], st + kABytes + j * kWaves * 1024);
#pragma unroll
        for (int j = 0; j < kBLoads; ++j)
          global_to_lds_sv<16>(pb + b.lo, bv[j], st + 2 * kABytes + kBBytes + j * kWaves * 1024);
      }
    };

    struct Fragments {
      u32x4_t a[PARTS][FM], b[PARTS][FN];
    };
    auto read = [&](Fragments& f, int stage, int kk) {
      const uint8_t* ta = smem + stage * kStage;
      const uint8_t* tb = ta + PARTS * kABytes;
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
          f.a[q][i] = fragment<AS, kBM>(ta + q * kABytes, wm * 32 * FM, i, kk, lane);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          f.b[q][j] = fragment<BS, kBN>(tb + q * kBBytes, wn * 32 * FN, j, kk, lane);
      }
    };
    // Reads the fragments due after product m of kProducts: those that the next products need first
    // come first, and the last is read two products ahead where there are enough.
    auto read_after = [&](Fragments& f, int stage, int kk, int m) {
      constexpr int kAll = PARTS * (FM + FN), kOver = kProducts > kAll ? kProducts - 2 : kProducts;
      const uint8_t* ta = smem + stage * kStage;
      const uint8_t* tb = ta + PARTS * kABytes;
#pragma unroll
      for (int x = 0; x < kAll; ++x) {
        if (x * kOver / kAll != m) continue;
        const int q = x / (FM + FN), y = x % (FM + FN);  // a[0], all of b, the rest of a
        if (y > 0 && y <= FN)
          f.b[q][(y - 1) % FN] = fragment<BS, kBN>(tb + q * kBBytes, wn * 32 * FN, y - 1, kk, lane);
        else
          f.a[q][y == 0 ? 0 : (y - FN) % FM] =
              fragment<AS, kBM>(ta + q * kABytes, wm * 32 * FM, y == 0 ? 0 : y - FN, kk, lane);
      }
    };
    auto multiply_and_read = [&](const Fragments& f, Fragments& next, int stage, int kk) {
#pragma unroll
      for (int m = 0; m < kProducts; ++m) {
        const int q = m / (FM * FN), i = m / FN % FM, j = m % FN;
        acc[i][j] = mfma(f.a[q >> 1][i], f.b[q & 1][j], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
        read_after(next, stage, kk, m);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto multiply = [&](const Fragments& f) {
#pragma unroll
      for (int q = 0; q < 2 * PARTS - 1; ++q)  // hi hi, hi lo, lo hi
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = mfma(f.a[q >> 1][i], f.b[q & 1][j], acc[i][j]);
    };
    // Waits until all but the last `keep` steps' loads have landed (all of them where fewer steps
    // follow) and this wave's reads are done, then meets the other waves.
    auto meet = [&](auto keep, bool full) {
      if (full)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(keep)::value * kLoads)
                     : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    if (steps <= 0) return;
#pragma unroll
    for (int t = 0; t < STAGES; ++t)
      if (t < steps) issue(t, t);
    meet(std::integral_constant<int, STAGES - 1>{}, steps >= STAGES);
    Fragments f[2];
    read(f[0], 0, 0);
    int stage = 0;
    // inner: a step with at least STAGES + 1 more behind it, which needs no tests.
    auto step = [&](int s, auto inner) {
      constexpr bool kInner = decltype(inner)::value;
      const int next = stage + 1 == STAGES ? 0 : stage + 1;
      // the next 16 k's fragments are read while the matrix cores work on these
#pragma unroll
      for (int kk = 0; kk < 3; ++kk) {
        if constexpr (kProducts >= 3) {
          multiply_and_read(f[kk & 1], f[(kk + 1) & 1], stage, kk + 1);
        } else {
          read(f[(kk + 1) & 1], stage, kk + 1);
          __builtin_amdgcn_sched_barrier(0);
          multiply(f[kk & 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (kInner || s + 1 < steps) {
        // step s + 1 has landed; no wave reads this step's stage any more
        meet(std::integral_constant<int, STAGES - 2>{}, kInner || s + STAGES <= steps);
        read(f[0], next, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      multiply(f[1]);
      __builtin_amdgcn_sched_barrier(0);
      if (kInner || s + STAGES < steps) issue(s + STAGES, stage);  // behind the products just queued
      __builtin_amdgcn_sched_barrier(0);
      stage = next;
    };
    int s = 0;
    for (; s < steps - STAGES - 1; ++s) step(s, std::true_type{});
    for (; s < steps; ++s) step(s, std::false_type{});
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // smem may be reused
  }

  // Launches kKernel, which uses this tile's LDS, on groups x splits workgroups.
  template <auto kKernel, typename Args>
  static hipError_t launch(const Args& args, int groups, int splits, hipStream_t s) {
    static const hipError_t attr = hipFuncSetAttribute(
        reinterpret_cast<const void*>(kKernel), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (attr != hipSuccess) return attr;
    kKernel<<<dim3((unsigned)groups, (unsigned)splits), kThreads, kLds, s>>>(args);
    return hipGetLastError();
  }

  static __device__ __forceinline__ void clear(Acc& acc) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = float16v_t{};
  }

  // With SWAP a lane holds, for each i < FM, j < FN and g < 4, four consecutive columns of a row:
  // quad(acc, i, j, g) at row row0(m0) + 32 i, columns col0(n0) + 32 j + 8 g .. + 3.
  static __device__ __forceinline__ int64_t row0(int64_t m0) {
    return m0 + ((threadIdx.x >> 6) / WN) * 32 * FM + (threadIdx.x & 31);
  }
  static __device__ __forceinline__ int64_t col0(int64_t n0) {
    return n0 + ((threadIdx.x >> 6) % WN) * 32 * FN + 4 * ((threadIdx.x >> 5) & 1);
  }
  static __device__ __forceinline__ float4_t quad(const Acc& acc, int i, int j, int g) {
    static_assert(SWAP, "rows by lane");
    return float4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                    acc[i][j][4 * g + 3]};
  }

  // Stores the accumulators as 16-bit numbers, element (row, col) at out[row * ld + col] for row <
  // rows and col < cols.  Each wave's 32 rows pass through its own part of smem and leave in
  // 16-byte pieces of whole 128-byte lines (a row's last ones by element where `cols` ends inside a
  // piece): stored as the lanes hold them, 8 bytes in each of 32 rows, they take four times the
  // requests.
  template <bool TO_BF16>
  static __device__ __forceinline__ void store16(const Acc& acc, int64_t m0, int64_t n0,
                                                 uint8_t* smem, uint16_t* out, int64_t ld,
                                                 int64_t rows, int64_t cols) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int kPitch = 64 * FN + 16, kPieces = 4 * FN;  // bytes, 16-byte pieces a row
    static_assert(kWaves * 32 * kPitch <= kLds, "the waves' parts fit");
    uint8_t* mine = smem + wave * 32 * kPitch;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int64_t row = m0 + (wave / WN) * 32 * FM + 32 * i;
      const int64_t col = n0 + (wave % WN) * 32 * FN;
#pragma unroll
      for (int q = 0; q < 4 * FN; ++q) {
        const float4_t v = quad(acc, i, q / 4, q % 4);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = TO_BF16 ? f32_to_bf16(v[e]) : f32_to_f16(v[e]);
        const int c = 32 * (q / 4) + 8 * (q % 4) + 4 * (lane >> 5);
        *reinterpret_cast<u32x2_t*>(mine + (lane & 31) * kPitch + 2 * c) =
            u32x2_t{h[0] | h[1] << 16, h[2] | h[3] << 16};
      }
      keep_lds_order();
#pragma unroll
      for (int k = 0; k < 32 * kPieces / 64; ++k) {
        const int p = k * 64 + lane, r = p / kPieces, c = p % kPieces * 8;
        if (row + r < rows)
          store_piece(out + (row + r) * ld + col + c, mine + r * kPitch + 2 * c, cols - col - c);
      }
      keep_lds_order();
    }
  }
};

}  // namespace
}  // namespace nm
