// nm_spmm.hip -- Y = W_sparse * X for the compressed N:M format (gfx950).
//
// The product ("[리뷰] Accelerating Sparse Deep Neural Networks", section "Tensor
// Scores 상에서 구조적인 sparse GEMM") takes the compressed weight as the first
// operand and a dense K x T activation matrix as the second; the result is dense.
//
// 2:4 and 1:2 with 16-bit inputs run on gfx950's structured-sparse matrix cores
// (v_smfmac_f32_32x32x32_{bf16,f16}, and v_smfmac_f32_16x16x64 for small tiles).  The
// instruction takes, per lane, stored values of one row with an index word whose 2-bit
// fields give each value's position in its group of four, least significant first --
// exactly this library's 2:4 metadata -- so compressed rows feed the matrix cores with no
// conversion and the hardware gathers the matching rows of X.  1:2 metadata (one bit per
// value) is widened to that nibble form in registers: pairs of 1:2 groups are 2:4 groups
// with one value in each half.
//
// Kernels, chosen per shape by an estimate of rounds of workgroups times tile time:
//  * smfmac_ws_spmm_kernel (256 x 128 tiles, the large shapes): wave-specialised.  Four
//    producer waves bring every operand of a 64-wide K step (X rows, compressed values,
//    metadata) into a 4-stage LDS ring with direct global -> LDS loads; four consumer
//    waves (128 x 64 outputs each) read fragments from LDS -- X through
//    ds_read_b64_tr_b16, which hands each lane consecutive K rows of one column, the
//    K-major order of the B operand -- and issue the smfmac.  One barrier per step.
//  * smfmac32_spmm_kernel (256 x 256 tiles): the same fragment code with every wave
//    issuing its own loads, for short K; smfmac_spmm_kernel (128 x 128 tiles,
//    v_smfmac_f32_16x16x64) for small shapes.
//  * mfma48_ws_spmm_kernel: 4:8 (either layout) on the dense matrix cores, each 4:8 group
//    expanded in registers with byte permutes.
//  * smfmac_i8_ws_spmm_kernel: 2:4 and 1:2 int8 (exact int32) and fp8 (fixed-point sums per
//    run of 16 K inside the instruction, fp32 across runs)
//    on the 32x32x64 8-bit instructions.
//  * expand_mfma_spmm_kernel: every other pattern and shape, any element type; the
//    compressed rows are expanded in LDS (8-bit elements widened exactly to bf16; int8
//    sums kept exact in int32) and multiplied on the dense matrix cores
//    (v_mfma_f32_32x32x2_f32, v_mfma_f32_32x32x16_{bf16,f16}).

// The blocked layout (include/nm.h) makes every direct load of compressed values or
// metadata one contiguous run; the row layout is accepted by the same kernels at a lower
// rate.  Accumulators are fp32 (int32 for int8) and rounded once to the output type.
//
// This file is compiled three times, in parallel: as it is for nm_spmm, and through nm_spmm_act.hip
// and nm_spmm_act_any.hip (NM_SPMM_PART 1 and 2) for the same kernels with the output type kAct, whose
// epilogue is nm_act.h's.
#include <atomic>
#include <cstdlib>
#include <type_traits>

#include "nm_act.h"
#include "nm_launch.h"
#include "nm_mfma.h"

namespace nm {

namespace {

// ===========================================================================
// Structured-sparse matrix-core kernel (2:4, or 1:2 widened to 2:4).
// ===========================================================================

// STAGES: LDS ring depth (the step being computed + STAGES - 1 in flight)
template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES>
struct SmfmacTile {
  static constexpr int kStages = STAGES;
  static constexpr int kThreads = 64 * WAVES_M * WAVES_N;
  static constexpr int kWaves = WAVES_M * WAVES_N;
  static constexpr int kWM = BM / WAVES_M;
  static constexpr int kWN = BN / WAVES_N;
  static constexpr int kFM = kWM / 16;
  static constexpr int kFN = kWN / 16;
  // one stage of the LDS ring: X tile (64 K rows x BN), A values (BM rows x 64 bytes),
  // metadata (BM rows x 8 bytes: four 16-bit 2:4 units, or 1:2 bytes in the first half)
  static constexpr int kXRowBytes = BN * 2;
  static constexpr int kXChunks = BN / 8;
  static constexpr int kXBytes = kKStep * kXRowBytes;
  static constexpr int kABytes = BM * 64;
  static constexpr int kMBytes = BM * 8;
  static constexpr int kStageBytes = kXBytes + kABytes + kMBytes;
  // direct loads per wave and step (each moves 1 KB; metadata ones move 256 bytes)
  static constexpr int kXLoads = kXBytes / 1024 / kWaves;
  static constexpr int kALoads = kABytes / 1024 / kWaves;
  static constexpr int kMLoads = kMBytes / 256 / kWaves;
  static constexpr int kLoads = kXLoads + kALoads + kMLoads;
  static_assert(kWM % 16 == 0 && kWN % 16 == 0, "wave tile must be whole 16x16 fragments");
  static_assert(kXBytes % (1024 * kWaves) == 0 && kABytes % (1024 * kWaves) == 0 &&
                    kMBytes % (256 * kWaves) == 0,
                "every wave issues the same number of direct loads per step");
  static_assert(kXChunks >= 16, "the X swizzle needs at least 16 chunks per row");
  static_assert(kFM % 4 == 0, "A fragments are read four at a time");
  static_assert(kStages >= 2 && (kStages - 2) * kLoads <= 63, "vmcnt budget");
  static_assert(kStages * kStageBytes <= 160 * 1024, "LDS budget");
};

// 1:2 metadata bits (one per value) of 16 K positions -> four 2:4 nibbles.
__device__ __forceinline__ uint32_t widen_1_2(uint32_t x8) {
  uint32_t x = x8 & 0xFFu;  // bit i -> bit 2i
  x = (x | (x << 4)) & 0x0F0Fu;
  x = (x | (x << 2)) & 0x3333u;
  x = (x | (x << 1)) & 0x5555u;
  return x | 0x8888u;  // the second value of each pair sits in the upper half (2 + bit)
}

template <bool BF16>
__device__ __forceinline__ float4_t smfmac(const u32x4_t& a, const short16_t& b, const float4_t& c,
                                           uint32_t idx) {
  if constexpr (BF16) {
    return __builtin_amdgcn_smfmac_f32_16x16x64_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                     __builtin_bit_cast(bf16x16_t, b), c,
                                                     (int)idx, 0, 0);
  } else {
    return __builtin_amdgcn_smfmac_f32_16x16x64_f16(__builtin_bit_cast(f16x8_t, a),
                                                    __builtin_bit_cast(f16x16_t, b), c, (int)idx,
                                                    0, 0);
  }
}

// All LDS reads go through asm blocks that also wait for them: the compiler then sees no
// LDS read that might alias the in-flight direct loads (it would answer with a wait for
// every outstanding load), and no register that a pending load might still write.

// One B fragment (16 K rows x 16 columns, K-major per lane): four transposing reads at
// rows kb, kb + 4 (addresses a0, a1) and kb + 32, kb + 36 (the same + kFar bytes).
template <int kFar>
__device__ __forceinline__ short16_t lds_b_fragment(uint32_t a0, uint32_t a1) {
  short4_t b0, b1, b2, b3;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %4\n\t"
      "ds_read_b64_tr_b16 %1, %5\n\t"
      "ds_read_b64_tr_b16 %2, %4 offset:%6\n\t"
      "ds_read_b64_tr_b16 %3, %5 offset:%6\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(b0), "=&v"(b1), "=&v"(b2), "=&v"(b3)
      : "v"(a0), "v"(a1), "n"(kFar)
      : "memory");
  const short8_t lo = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
  const short8_t hi = __builtin_shufflevector(b2, b3, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
}

// Four A fragments (16 bytes each, 1 KB apart) and their metadata (128 bytes apart).
// kPat12 reads one byte of 1:2 metadata, otherwise a 16-bit 2:4 unit.
template <bool kPat12, int kAStride = 1024, int kMStride = 128>
__device__ __forceinline__ void lds_a_fragments4(uint32_t va, uint32_t ma, u32x4_t& a0,
                                                 u32x4_t& a1, u32x4_t& a2, u32x4_t& a3,
                                                 uint32_t& m0, uint32_t& m1, uint32_t& m2,
                                                 uint32_t& m3) {
  if constexpr (kPat12) {
    asm volatile(
        "ds_read_b128 %0, %8\n\t"
        "ds_read_b128 %1, %8 offset:%10\n\t"
        "ds_read_b128 %2, %8 offset:%11\n\t"
        "ds_read_b128 %3, %8 offset:%12\n\t"
        "ds_read_u8 %4, %9\n\t"
        "ds_read_u8 %5, %9 offset:%13\n\t"
        "ds_read_u8 %6, %9 offset:%14\n\t"
        "ds_read_u8 %7, %9 offset:%15\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a0), "=&v"(a1), "=&v"(a2), "=&v"(a3), "=&v"(m0), "=&v"(m1), "=&v"(m2), "=&v"(m3)
        : "v"(va), "v"(ma), "n"(kAStride), "n"(2 * kAStride), "n"(3 * kAStride), "n"(kMStride),
          "n"(2 * kMStride), "n"(3 * kMStride)
        : "memory");
  } else {
    asm volatile(
        "ds_read_b128 %0, %8\n\t"
        "ds_read_b128 %1, %8 offset:%10\n\t"
        "ds_read_b128 %2, %8 offset:%11\n\t"
        "ds_read_b128 %3, %8 offset:%12\n\t"
        "ds_read_u16 %4, %9\n\t"
        "ds_read_u16 %5, %9 offset:%13\n\t"
        "ds_read_u16 %6, %9 offset:%14\n\t"
        "ds_read_u16 %7, %9 offset:%15\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a0), "=&v"(a1), "=&v"(a2), "=&v"(a3), "=&v"(m0), "=&v"(m1), "=&v"(m2), "=&v"(m3)
        : "v"(va), "v"(ma), "n"(kAStride), "n"(2 * kAStride), "n"(3 * kAStride), "n"(kMStride),
          "n"(2 * kMStride), "n"(3 * kMStride)
        : "memory");
  }
}

// Wait until at most N direct loads of this wave are outstanding, then meet the other
// waves: the step whose loads completed is then visible in LDS for every wave.
template <int N>
__device__ __forceinline__ void wait_loads_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Byte offset, for step 0, of one lane's direct load of compressed values: the load
// fills tile rows i0 .. i0+15 (64 value bytes per row and step), lane l taking row
// i0 + l/4 and the 16-byte chunk that lands at physical chunk l % 4 of that LDS row
// (logical chunk (l % 4) ^ ((row >> 2) & 3)).  Rows past the matrix read any valid row
// (their outputs are dropped).
template <bool kBlocked>
__device__ __forceinline__ int64_t values_source(int m0, int i0, int lane, int R, int K,
                                                 int nsteps) {
  const int i = i0 + (lane >> 2);
  const int lc = (lane & 3) ^ ((i >> 2) & 3);
  if constexpr (kBlocked) {  // one contiguous 1 KB block per 16 rows and step
    const int last = ((R + 15) >> 4) - 1;
    int g = (m0 + i0) >> 4;
    g = g < last ? g : last;
    return (int64_t)g * nsteps * 1024 + (lane >> 2) * 64 + 16 * lc;
  } else {  // row-major: 64 bytes per row and step
    int row = m0 + i;
    row = row < R ? row : R - 1;
    return (int64_t)row * K + 16 * lc;
  }
}
template <bool kBlocked>
constexpr int64_t values_step_bytes() { return kBlocked ? 1024 : 64; }

// The same for metadata: a load fills tile rows i0 .. i0+31 with 8 bytes each, two lanes
// per row (1:2 rows hold 4 bytes per step, which both lanes read).
template <bool kBlocked, bool kPat12>
__device__ __forceinline__ int64_t meta_source(int m0, int i0, int lane, int R, int K,
                                               int nsteps) {
  constexpr int kRowStep = kPat12 ? 4 : 8;  // metadata bytes per row and step
  const int i = i0 + (lane >> 1);
  const int half = kPat12 ? 0 : 4 * (lane & 1);
  if constexpr (kBlocked) {
    const int last = ((R + 15) >> 4) - 1;
    int g = (m0 + i) >> 4;
    g = g < last ? g : last;
    return (int64_t)g * nsteps * (16 * kRowStep) + (i & 15) * kRowStep + half;
  } else {
    int row = m0 + i;
    row = row < R ? row : R - 1;
    return (int64_t)row * (K / 64 * kRowStep) + half;
  }
}
template <bool kBlocked, bool kPat12>
constexpr int64_t meta_step_bytes() { return (kPat12 ? 4 : 8) * (kBlocked ? 16 : 1); }

// Which output tile a workgroup computes.  Workgroups are dispatched round-robin over
// the XCDs (each with its own L2), so workgroup b runs on XCD b % xcds.  Each XCD gets
// a contiguous run of `per_xcd` tiles of an order that walks groups of gm x gn tiles
// (row tiles x column tiles; column-major inside a group): the workgroups an XCD runs
// at the same time then cover a compact block of the output and share both their rows
// of A and their columns of X in that XCD's L2.
struct TileMap {
  int tiles_m, tiles_n, xcds, per_xcd, gm, gn;
  __device__ __forceinline__ bool tile_of(int b, int& tm, int& tn) const {
    const int t = (b % xcds) * per_xcd + b / xcds;
    if (t >= tiles_m * tiles_n) return false;
    // row-groups of gm row tiles (the last may be shorter), every earlier one full
    const int g_m = t / (gm * tiles_n);
    const int rows = min(gm, tiles_m - g_m * gm);
    const int u = t - g_m * gm * tiles_n;
    // inside it, column-groups of gn column tiles (the last may be narrower)
    const int g_n = u / (rows * gn);
    const int v = u - g_n * rows * gn;
    tm = g_m * gm + v % rows;
    tn = g_n * gn + v / rows;
    return true;
  }
};

// Workgroup b runs on XCD b % xcds; each XCD takes a contiguous run of per_xcd tiles,
// walked in groups of gm row tiles x gn column tiles so that the 32 workgroups an XCD runs
// at once share A stripes and X panels in its L2.  (8 x 4 and 4 x 8 groups time the same
// within noise on the LLaMA, BERT and sweep shapes, for every element type.)
[[maybe_unused]] TileMap make_tile_map(int tiles_m, int tiles_n, int xcds) {
  TileMap map;
  map.tiles_m = tiles_m;
  map.tiles_n = tiles_n;
  map.xcds = xcds;
  map.per_xcd = (tiles_m * tiles_n + xcds - 1) / xcds;
  map.gn = tiles_n < 4 ? tiles_n : 4;
  map.gm = 32 / map.gn;
  return map;
}

// Pipeline: K steps of 64 through a ring of kStages LDS stages, every operand brought in
// by direct global -> LDS loads issued kStages - 1 steps ahead (loads for steps past
// the end re-read the last step, so every step issues the same loads and the loop has no
// branches).  Per step each wave reads its A fragments and metadata once, then for each
// 16-column B fragment issues FM smfmac.
//
// LDS layouts within a stage (all conflict-free for the reads that follow):
//   X: K row r holds BN columns as 16-byte chunks, logical chunk c at physical chunk
//      c ^ (r & 15); a direct load of 1 KB fills 1024 / (2 BN) consecutive rows.
//   A: tile row i holds the 64 value bytes of this step (K/2 values per row of W in
//      global memory, 32 per step); 16-byte chunk c at physical chunk c ^ ((i >> 2) & 3).
//      One direct load fills rows 16 j .. 16 j + 15: exactly one fragment's rows.
//   meta: tile row i holds 8 bytes (2:4: four 16-bit units; 1:2: four bytes + pad).
template <bool BF16, bool kPat12, bool kBlocked, int YT, int BM, int BN, int WAVES_M, int WAVES_N,
          int STAGES>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N)
    smfmac_spmm_kernel(const uint16_t* __restrict__ values, const uint32_t* __restrict__ meta,
                       const uint16_t* __restrict__ X, typename OutOf<YT>::type Y, int R, int K, int T,
                       TileMap map) {
  using TL = SmfmacTile<BM, BN, WAVES_M, WAVES_N, STAGES>;
  constexpr int FM = TL::kFM, FN = TL::kFN, kStages = STAGES;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const int ldx = x_stride(Y, T);  // row length of X
  int tile_m, tile_n;
  if (!map.tile_of(blockIdx.x, tile_m, tile_n)) return;  // whole workgroup, before any load
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int m0 = tile_m * BM, t0 = tile_n * BN;
  const int l16 = lane & 15, q = lane >> 4;
  const int nsteps = K / kKStep;
  const int last_step = nsteps - 1;

  // ---- direct-load sources (byte offsets for step 0) and LDS destinations ----
  const uint8_t* xg = reinterpret_cast<const uint8_t*>(X);
  const uint8_t* vg = reinterpret_cast<const uint8_t*>(values);
  const uint8_t* mg = reinterpret_cast<const uint8_t*>(meta);
  int64_t x_src[TL::kXLoads];
  uint32_t x_dst[TL::kXLoads];
#pragma unroll
  for (int j = 0; j < TL::kXLoads; ++j) {
    const int w1k = j * TL::kWaves + wave;  // 1 KB window of the X tile
    const int slot = w1k * 64 + lane;       // 16-byte slot
    const int r = slot / TL::kXChunks, pc = slot % TL::kXChunks;
    const int lc = pc ^ (r & 15);
    int col = t0 + 8 * lc;
    col = col < T ? col : 0;  // columns past T: any valid address (outputs past T only)
    x_src[j] = ((int64_t)r * ldx + col) * 2;
    x_dst[j] = (uint32_t)(w1k * 1024);
  }
  int64_t a_src[TL::kALoads];
  uint32_t a_dst[TL::kALoads];
#pragma unroll
  for (int j = 0; j < TL::kALoads; ++j) {
    const int blk = j * TL::kWaves + wave;  // rows 16 blk .. 16 blk + 15 of the tile
    a_src[j] = values_source<kBlocked>(m0, 16 * blk, lane, R, K, nsteps);
    a_dst[j] = (uint32_t)(TL::kXBytes + blk * 1024);
  }
  int64_t m_src[TL::kMLoads];
  uint32_t m_dst[TL::kMLoads];
#pragma unroll
  for (int j = 0; j < TL::kMLoads; ++j) {
    const int blk = j * TL::kWaves + wave;  // rows 32 blk .. 32 blk + 31
    m_src[j] = meta_source<kBlocked, kPat12>(m0, 32 * blk, lane, R, K, nsteps);
    m_dst[j] = (uint32_t)(TL::kXBytes + TL::kABytes + blk * 256);
  }
  auto issue_step = [&](int step) {
    step = step < last_step ? step : last_step;
    uint8_t* st = smem + (step % kStages) * TL::kStageBytes;
    const int64_t kx = (int64_t)step * kKStep * ldx * 2;                      // X rows
    const int64_t ka = (int64_t)step * values_step_bytes<kBlocked>();       // values
    const int64_t km = (int64_t)step * meta_step_bytes<kBlocked, kPat12>();  // metadata
#pragma unroll
    for (int j = 0; j < TL::kXLoads; ++j) global_to_lds<16>(xg + x_src[j] + kx, st + x_dst[j]);
#pragma unroll
    for (int j = 0; j < TL::kALoads; ++j) global_to_lds<16>(vg + a_src[j] + ka, st + a_dst[j]);
#pragma unroll
    for (int j = 0; j < TL::kMLoads; ++j) global_to_lds<4>(mg + m_src[j] + km, st + m_dst[j]);
  };

  // ---- per-lane LDS read offsets within a stage ----
  // A fragment fm: tile row i = wm*kWM + 16 fm + l16, logical chunk q
  const int ia = wm * TL::kWM + l16;
  const uint32_t a_rd = (uint32_t)(TL::kXBytes + ia * 64 + ((q ^ ((ia >> 2) & 3)) << 4));
  const uint32_t m_rd = (uint32_t)(TL::kXBytes + TL::kABytes + ia * 8 + (kPat12 ? q : 2 * q));
  // B fragment fn: K rows {8q..8q+7} and {32+8q..32+8q+7}; lane i of a 16-lane block
  // reads K row kb + (i >> 2), logical columns 4 (i & 3) .. +3
  const int sw0 = 8 * (q & 1) | (l16 >> 2);  // (row & 15) for kb = 8q and 8q + 32
  const int sw1 = sw0 | 4;                   // (row & 15) for kb = 8q + 4 and 8q + 36
  const int rb = 8 * q + (l16 >> 2);
  const int half8 = 8 * (l16 & 1);
  uint32_t b_rd[FN][2];
#pragma unroll
  for (int fn = 0; fn < FN; ++fn) {
    const int lc = (wn * TL::kWN + fn * 16) / 8 + ((l16 & 3) >> 1);
    b_rd[fn][0] = (uint32_t)(rb * TL::kXRowBytes + ((lc ^ sw0) << 4) + half8);
    b_rd[fn][1] = (uint32_t)((rb + 4) * TL::kXRowBytes + ((lc ^ sw1) << 4) + half8);
  }

  float4_t acc[FM][FN];
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) acc[fm][fn] = float4_t{0.f, 0.f, 0.f, 0.f};

  // ---- prologue: steps 0 .. kStages-2 in flight ----
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue_step(k);

  const uint32_t smem_base = lds_addr(smem);
  for (int s = 0; s < nsteps; ++s) {
    // step s landed (steps s+1 .. s+kStages-2 may still be in flight); after the barrier
    // no wave reads stage (s-1) % kStages any more, which the next issue overwrites
    wait_loads_and_barrier<(kStages - 2) * TL::kLoads>();
    issue_step(s + kStages - 1);
    const uint32_t st = smem_base + (uint32_t)((s % kStages) * TL::kStageBytes);

    u32x4_t a[FM];
    uint32_t ix[FM];
#pragma unroll
    for (int f = 0; f < FM; f += 4)
      lds_a_fragments4<kPat12>(st + a_rd + f * 1024, st + m_rd + f * 128, a[f], a[f + 1],
                               a[f + 2], a[f + 3], ix[f], ix[f + 1], ix[f + 2], ix[f + 3]);
    if constexpr (kPat12) {
#pragma unroll
      for (int fm = 0; fm < FM; ++fm) ix[fm] = widen_1_2(ix[fm]);
    }
    short16_t b = lds_b_fragment<32 * TL::kXRowBytes>(st + b_rd[0][0], st + b_rd[0][1]);
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
#pragma unroll
      for (int fm = 0; fm < FM; ++fm) acc[fm][fn] = smfmac<BF16>(a[fm], b, acc[fm][fn], ix[fm]);
      if (fn + 1 < FN) {
        // the smfmacs above are queued before the next fragment's reads are issued, so
        // the matrix cores work through them while this wave waits for LDS
        __builtin_amdgcn_sched_barrier(0);
        b = lds_b_fragment<32 * TL::kXRowBytes>(st + b_rd[fn + 1][0], st + b_rd[fn + 1][1]);
      }
    }
  }
  // drain the loads issued for steps past the end before the wave exits
  wait_loads_and_barrier<0>();

  // ---- epilogue: lane holds rows 4q..4q+3, column l16 of each 16x16 fragment ----
  if constexpr (YT == kAct) {
    static_assert(FM == 4 && FN == 4, "a slab of 64 rows x 64 columns");
    static_assert(TL::kWaves * kSlabBytes <= kStages * TL::kStageBytes, "epilogue LDS");
    constexpr int kDT = BF16 ? kBF16 : kF16;
    float* slab = reinterpret_cast<float*>(smem + wave * kSlabBytes);
    const int row0 = m0 + wm * TL::kWM, col0 = t0 + wn * TL::kWN;
    GroupInputs in;
    group_load<kDT>(in, Y, row0, col0, R, T, lane);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < FN; ++fn)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          slab[(16 * fm + 4 * q + i) * kSlabPitch + 16 * fn + l16] = acc[fm][fn][i];
    keep_order();
    slab_finish<kDT>(in, slab, Y, row0, col0, R, T, lane);
    return;
  }
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
      const int col = t0 + wn * TL::kWN + fn * 16 + l16;
      if (col >= T) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = m0 + wm * TL::kWM + fm * 16 + 4 * q + i;
        if constexpr (YT != kAct)
          if (row < R) store_from_f32<YT>(Y, (int64_t)row * T + col, acc[fm][fn][i]);
      }
    }
  }
}

// ===========================================================================
// Structured-sparse matrix-core kernel, 32x32x32 form with hand-scheduled blocks.
//
// A wave owns 128 rows x 64 columns of the tile: four 32-row A fragments and two
// 32-column B fragments per 32-wide K substep (two substeps per 64-wide step).  The work
// of a step is cut into four blocks, one per (substep t, B fragment f); each block is one
// asm statement that first issues LDS reads of fragments needed later, then the four
// v_smfmac_f32_32x32x32 of this block (~130 matrix-core cycles), then waits for its
// reads, so the matrix cores work while the reads are in flight.  Each block reads the
// next block's B fragment; block (0,1) also reads this step's substep-1 A fragments and
// block (1,1) next step's substep-0 A fragments.  A register is thus rewritten only
// when the last smfmac that read it is at least one whole block back, and the B fragment
// of the previous block is passed in as a dummy input so that no read lands in it while
// that block's smfmac may still be reading it.  Accumulators live in AGPRs.
// ===========================================================================
template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES>
struct Smfmac32Tile {
  static constexpr int kThreads = 64 * WAVES_M * WAVES_N;
  static constexpr int kWaves = WAVES_M * WAVES_N;
  static constexpr int kStages = STAGES;
  static constexpr int kWM = BM / WAVES_M;
  static constexpr int kWN = BN / WAVES_N;
  static constexpr int kXRowBytes = BN * 2;
  static constexpr int kXChunks = BN / 8;
  static constexpr int kXBytes = kKStep * kXRowBytes;
  static constexpr int kABytes = BM * 64;
  static constexpr int kMBytes = BM * 8;
  static constexpr int kStageBytes = kXBytes + kABytes + kMBytes;
  static constexpr int kXLoads = kXBytes / 1024 / kWaves;
  static constexpr int kALoads = kABytes / 1024 / kWaves;
  static constexpr int kMLoads = kMBytes / 256 / kWaves;
  static constexpr int kLoads = kXLoads + kALoads + kMLoads;
  static_assert(kWM == 128, "a wave owns four 32-row A fragments");
  static_assert(kWN == 64, "a wave owns two 32-column B fragments");
  static_assert(kXBytes % (1024 * kWaves) == 0 && kABytes % (1024 * kWaves) == 0 &&
                    kMBytes % (256 * kWaves) == 0,
                "every wave issues the same number of direct loads per step");
  static_assert(BN >= 128, "the X swizzle needs at least 8 column pairs per row");
  static_assert(kStages >= 3 && (kStages - 2) * kLoads <= 63, "vmcnt budget");
  static_assert(kStages * kStageBytes <= 160 * 1024, "LDS budget");
};

struct AFrags {
  u32x4_t v[4];
  uint32_t ix[4];
};

// One block: the four smfmac of this block on accumulators c[0..3] (AGPRs), with the LDS
// reads of the next B fragment (rows kb, kb + 4 at b0, b1 and kb + 16, kb + 20 at + kFar)
// and, in the A form, of four A fragments (kAStride apart) and their index words (kMStride
// apart) issued between them.  The first smfmac goes ahead of every read: a wave issues in
// order, so reads placed first would hold its matrix core idle until the LDS queue had
// taken them all; issued behind a running smfmac they cost the matrix core nothing.
#define NM_SMF32(OP, C, A, I) OP " %[" C "], %[" A "], %[b], %[" I "]\n\t"
#define NM_SMFMAC32_BLOCK(OP)                                                              \
  "s_nop 2\n\t"                                                                            \
  NM_SMF32(OP, "c0", "a0", "i0")                                                           \
  "ds_read_b64_tr_b16 %[n0], %[b0]\n\t"                                                    \
  "ds_read_b64_tr_b16 %[n1], %[b1]\n\t"                                                    \
  NM_SMF32(OP, "c1", "a1", "i1")                                                           \
  "ds_read_b64_tr_b16 %[n2], %[b0] offset:%[far]\n\t"                                      \
  "ds_read_b64_tr_b16 %[n3], %[b1] offset:%[far]\n\t"                                      \
  NM_SMF32(OP, "c2", "a2", "i2")                                                           \
  NM_SMF32(OP, "c3", "a3", "i3")                                                           \
  "s_waitcnt lgkmcnt(0)"
#define NM_SMFMAC32_BLOCK_A(OP, MREAD)                                                     \
  "s_nop 2\n\t"                                                                            \
  NM_SMF32(OP, "c0", "a0", "i0")                                                           \
  "ds_read_b64_tr_b16 %[n0], %[b0]\n\t"                                                    \
  "ds_read_b64_tr_b16 %[n1], %[b1]\n\t"                                                    \
  "ds_read_b64_tr_b16 %[n2], %[b0] offset:%[far]\n\t"                                      \
  "ds_read_b64_tr_b16 %[n3], %[b1] offset:%[far]\n\t"                                      \
  NM_SMF32(OP, "c1", "a1", "i1")                                                           \
  "ds_read_b128 %[na0], %[aa]\n\t"                                                         \
  "ds_read_b128 %[na1], %[aa] offset:%[as1]\n\t"                                           \
  "ds_read_b128 %[na2], %[aa] offset:%[as2]\n\t"                                           \
  "ds_read_b128 %[na3], %[aa] offset:%[as3]\n\t"                                           \
  NM_SMF32(OP, "c2", "a2", "i2")                                                           \
  MREAD " %[ni0], %[ma]\n\t"                                                               \
  MREAD " %[ni1], %[ma] offset:%[ms1]\n\t"                                                 \
  MREAD " %[ni2], %[ma] offset:%[ms2]\n\t"                                                 \
  MREAD " %[ni3], %[ma] offset:%[ms3]\n\t"                                                 \
  NM_SMF32(OP, "c3", "a3", "i3")                                                           \
  "s_waitcnt lgkmcnt(0)"
#define NM_SMFMAC32_BOUTS                                                                  \
  [n0] "=&v"(n[0]), [n1] "=&v"(n[1]), [n2] "=&v"(n[2]), [n3] "=&v"(n[3])
#define NM_SMFMAC32_COUTS                                                                  \
  [c0] "+a"(c0), [c1] "+a"(c1), [c2] "+a"(c2), [c3] "+a"(c3)
#define NM_SMFMAC32_INS                                                                    \
  [a0] "v"(a.v[0]), [a1] "v"(a.v[1]), [a2] "v"(a.v[2]), [a3] "v"(a.v[3]),                  \
      [i0] "v"(a.ix[0]), [i1] "v"(a.ix[1]), [i2] "v"(a.ix[2]), [i3] "v"(a.ix[3]),          \
      [b] "v"(b), [keep] "v"(keep), [b0] "v"(b0), [b1] "v"(b1), [far] "n"(kFar)

template <bool BF16, int kFar>
__device__ __forceinline__ void smfmac32_block(float16v_t& c0, float16v_t& c1, float16v_t& c2,
                                               float16v_t& c3, const AFrags& a,
                                               const short16_t& b, const short16_t& keep,
                                               uint32_t b0, uint32_t b1, short4_t (&n)[4]) {
  if constexpr (BF16)
    asm volatile(NM_SMFMAC32_BLOCK("v_smfmac_f32_32x32x32_bf16")
                 : NM_SMFMAC32_BOUTS, NM_SMFMAC32_COUTS
                 : NM_SMFMAC32_INS
                 : "memory");
  else
    asm volatile(NM_SMFMAC32_BLOCK("v_smfmac_f32_32x32x32_f16")
                 : NM_SMFMAC32_BOUTS, NM_SMFMAC32_COUTS
                 : NM_SMFMAC32_INS
                 : "memory");
}

template <bool BF16, bool kPat12, int kFar, int kAStride, int kMStride>
__device__ __forceinline__ void smfmac32_block_a(float16v_t& c0, float16v_t& c1, float16v_t& c2,
                                                 float16v_t& c3, const AFrags& a,
                                                 const short16_t& b, const short16_t& keep,
                                                 uint32_t b0, uint32_t b1, short4_t (&n)[4],
                                                 uint32_t aa, uint32_t ma, AFrags& na) {
#define NM_SMFMAC32_A(OP, MREAD)                                                           \
  asm volatile(NM_SMFMAC32_BLOCK_A(OP, MREAD)                                           \
               : NM_SMFMAC32_BOUTS, [na0] "=&v"(na.v[0]), [na1] "=&v"(na.v[1]),            \
                 [na2] "=&v"(na.v[2]), [na3] "=&v"(na.v[3]), [ni0] "=&v"(na.ix[0]),        \
                 [ni1] "=&v"(na.ix[1]), [ni2] "=&v"(na.ix[2]), [ni3] "=&v"(na.ix[3]),      \
                 NM_SMFMAC32_COUTS                                                         \
               : NM_SMFMAC32_INS, [aa] "v"(aa), [ma] "v"(ma), [as1] "n"(kAStride),         \
                 [as2] "n"(2 * kAStride), [as3] "n"(3 * kAStride), [ms1] "n"(kMStride),    \
                 [ms2] "n"(2 * kMStride), [ms3] "n"(3 * kMStride)                          \
               : "memory")
  if constexpr (BF16) {
    if constexpr (kPat12)
      NM_SMFMAC32_A("v_smfmac_f32_32x32x32_bf16", "ds_read_u8");
    else
      NM_SMFMAC32_A("v_smfmac_f32_32x32x32_bf16", "ds_read_u16");
  } else {
    if constexpr (kPat12)
      NM_SMFMAC32_A("v_smfmac_f32_32x32x32_f16", "ds_read_u8");
    else
      NM_SMFMAC32_A("v_smfmac_f32_32x32x32_f16", "ds_read_u16");
  }
#undef NM_SMFMAC32_A
}
#undef NM_SMF32
#undef NM_SMFMAC32_BLOCK
#undef NM_SMFMAC32_BLOCK_A
#undef NM_SMFMAC32_BOUTS
#undef NM_SMFMAC32_COUTS
#undef NM_SMFMAC32_INS

__device__ __forceinline__ short16_t join_b(const short4_t (&n)[4]) {
  return __builtin_shufflevector(__builtin_shufflevector(n[0], n[1], 0, 1, 2, 3, 4, 5, 6, 7),
                                 __builtin_shufflevector(n[2], n[3], 0, 1, 2, 3, 4, 5, 6, 7),
                                 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
}

template <bool kPat12>
__device__ __forceinline__ void widen_frags(AFrags& a) {
  if constexpr (kPat12) {
#pragma unroll
    for (int fm = 0; fm < 4; ++fm) a.ix[fm] = widen_1_2(a.ix[fm]);
  }
}

template <bool BF16, bool kPat12, bool kBlocked, int YT, int BM, int BN, int WAVES_M, int WAVES_N,
          int STAGES>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N)
    smfmac32_spmm_kernel(const uint16_t* __restrict__ values, const uint32_t* __restrict__ meta,
                         const uint16_t* __restrict__ X, typename OutOf<YT>::type Y, int R, int K,
                         int T, TileMap map) {
  using TL = Smfmac32Tile<BM, BN, WAVES_M, WAVES_N, STAGES>;
  constexpr int kStages = STAGES;
  constexpr int kRB = TL::kXRowBytes;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const int ldx = x_stride(Y, T);  // row length of X
  int tile_m, tile_n;
  if (!map.tile_of(blockIdx.x, tile_m, tile_n)) return;  // whole workgroup, before any load
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int m0 = tile_m * BM, t0 = tile_n * BN;
  const int l32 = lane & 31, q = lane >> 5, l16 = lane & 15, blk = lane >> 4;
  const int nsteps = K / kKStep;
  const int last_step = nsteps - 1;

  // ---- direct-load sources and LDS destinations (as in smfmac_spmm_kernel, except that
  // X chunks are swizzled in 32-byte pairs: logical pair p of K row r sits at
  // p ^ xpair_swizzle(r))
  const uint8_t* xg = reinterpret_cast<const uint8_t*>(X);
  const uint8_t* vg = reinterpret_cast<const uint8_t*>(values);
  const uint8_t* mg = reinterpret_cast<const uint8_t*>(meta);
  int64_t x_src[TL::kXLoads];
  uint32_t x_dst[TL::kXLoads];
#pragma unroll
  for (int j = 0; j < TL::kXLoads; ++j) {
    const int w1k = j * TL::kWaves + wave;
    const int slot = w1k * 64 + lane;
    const int r = slot / TL::kXChunks, pc = slot % TL::kXChunks;
    const int lc = 2 * ((pc >> 1) ^ xpair_swizzle(r)) + (pc & 1);
    int col = t0 + 8 * lc;
    col = col < T ? col : 0;  // columns past T: any valid address (outputs past T only)
    x_src[j] = ((int64_t)r * ldx + col) * 2;
    x_dst[j] = (uint32_t)(w1k * 1024);
  }
  int64_t a_src[TL::kALoads];
  uint32_t a_dst[TL::kALoads];
#pragma unroll
  for (int j = 0; j < TL::kALoads; ++j) {
    const int b16 = j * TL::kWaves + wave;
    a_src[j] = values_source<kBlocked>(m0, 16 * b16, lane, R, K, nsteps);
    a_dst[j] = (uint32_t)(TL::kXBytes + b16 * 1024);
  }
  int64_t m_src[TL::kMLoads];
  uint32_t m_dst[TL::kMLoads];
#pragma unroll
  for (int j = 0; j < TL::kMLoads; ++j) {
    const int b32 = j * TL::kWaves + wave;
    m_src[j] = meta_source<kBlocked, kPat12>(m0, 32 * b32, lane, R, K, nsteps);
    m_dst[j] = (uint32_t)(TL::kXBytes + TL::kABytes + b32 * 256);
  }
  // The direct loads of one step, numbered 0 .. kLoads-1 (X, then values, then
  // metadata); issue_part<P> issues the P-th quarter of them.  The main loop spreads a
  // step's loads over its four smfmac blocks: issued all at once, right after the
  // barrier, they would hold every wave in the load-issue queue while the matrix cores
  // sit idle.
  auto issue_part = [&](auto part, int step) {
    constexpr int P = decltype(part)::value;
    constexpr int j0 = P * TL::kLoads / 4, j1 = (P + 1) * TL::kLoads / 4;
    step = step < last_step ? step : last_step;
    uint8_t* st = smem + (step % kStages) * TL::kStageBytes;
    const int64_t kx = (int64_t)step * kKStep * ldx * 2;
    const int64_t ka = (int64_t)step * values_step_bytes<kBlocked>();
    const int64_t km = (int64_t)step * meta_step_bytes<kBlocked, kPat12>();
#pragma unroll
    for (int j = 0; j < TL::kLoads; ++j) {
      if (j < j0 || j >= j1) continue;
      if (j < TL::kXLoads) {
        global_to_lds<16>(xg + x_src[j] + kx, st + x_dst[j]);
      } else if (j < TL::kXLoads + TL::kALoads) {
        const int a = j - TL::kXLoads;
        global_to_lds<16>(vg + a_src[a] + ka, st + a_dst[a]);
      } else {
        const int mi = j - TL::kXLoads - TL::kALoads;
        global_to_lds<4>(mg + m_src[mi] + km, st + m_dst[mi]);
      }
    }
  };
  auto issue_step = [&](int step) {
    issue_part(std::integral_constant<int, 0>{}, step);
    issue_part(std::integral_constant<int, 1>{}, step);
    issue_part(std::integral_constant<int, 2>{}, step);
    issue_part(std::integral_constant<int, 3>{}, step);
  };

  // ---- per-lane LDS read offsets within a stage ----
  // A fragment fm of substep t: tile row ia + 32 fm, 16-byte chunk (2t + q) ^ ((ia >> 2) & 3)
  const int ia = wm * TL::kWM + l32;
  const int aswz = (ia >> 2) & 3;
  const uint32_t a_rd0 = (uint32_t)(TL::kXBytes + ia * 64 + (((0 + q) ^ aswz) << 4));
  const uint32_t a_rd1 = (uint32_t)(TL::kXBytes + ia * 64 + (((2 + q) ^ aswz) << 4));
  // index word of substep t: unit 2t + q of the row's step (2:4: 16-bit units; 1:2: bytes)
  constexpr int kMT = kPat12 ? 2 : 4;  // byte distance from substep 0 to substep 1
  const uint32_t m_rd0 = (uint32_t)(TL::kXBytes + TL::kABytes + ia * 8 + (kPat12 ? q : 2 * q));
  const uint32_t m_rd1 = m_rd0 + kMT;
  // B fragment (t, f): K rows 32t + {8q..8q+7, 16+8q..16+8q+7}; lane i of a 16-lane block
  // reads K row kb + (i >> 2), columns 4 (i & 3) .. +3 of the block's 16 columns
  const int rb = 8 * q + (l16 >> 2);
  uint32_t b_rd[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int lp = (wn * TL::kWN + 32 * f + 16 * (blk & 1)) / 16;  // logical 32-byte pair
    b_rd[f][0] = (uint32_t)(rb * kRB + ((lp ^ xpair_swizzle(rb)) << 5) + 8 * (l16 & 3));
    b_rd[f][1] =
        (uint32_t)((rb + 4) * kRB + ((lp ^ xpair_swizzle(rb + 4)) << 5) + 8 * (l16 & 3));
  }
  constexpr int kFar = 16 * kRB;  // K rows +16
  constexpr int kSub = 32 * kRB;  // K rows +32 (substep 1)
  constexpr int kAS = 32 * 64;    // next 32-row A fragment
  constexpr int kMS = 32 * 8;     // its index words

  float16v_t acc[4][2];
#pragma unroll
  for (int fm = 0; fm < 4; ++fm)
#pragma unroll
    for (int f = 0; f < 2; ++f) acc[fm][f] = float16v_t{};

  // ---- prologue: steps 0 .. kStages-2 in flight; substep-0 A and the first B fragment of
  // step 0 in registers; step 1 landed and visible ----
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) issue_step(k);
  const uint32_t smem_base = lds_addr(smem);
  auto stage_of = [&](int step) {
    return smem_base + (uint32_t)((step % kStages) * TL::kStageBytes);
  };
  AFrags a0, a1;
  short16_t b, bk = short16_t{};
  short4_t n[4];
  wait_loads_and_barrier<(kStages - 2) * TL::kLoads>();  // step 0 landed
  {
    const uint32_t st = stage_of(0);
    lds_a_fragments4<kPat12, kAS, kMS>(st + a_rd0, st + m_rd0, a0.v[0], a0.v[1], a0.v[2],
                                       a0.v[3], a0.ix[0], a0.ix[1], a0.ix[2], a0.ix[3]);
    b = lds_b_fragment<kFar>(st + b_rd[0][0], st + b_rd[0][1]);
    widen_frags<kPat12>(a0);
  }
  wait_loads_and_barrier<(kStages - 3) * TL::kLoads>();  // step 1 landed

  for (int s = 0; s < nsteps; ++s) {
    // invariant: steps s and s+1 are in LDS and visible; a0 holds substep-0 A of step s;
    // b holds B(0,0) of step s; no wave reads stage (s-1) % kStages any more
    const int ahead = s + kStages - 1;  // the step whose loads this iteration issues
    const uint32_t st = stage_of(s), sn = stage_of(s + 1);
    // block (0,0): reads B(0,1)
    smfmac32_block<BF16, kFar>(acc[0][0], acc[1][0], acc[2][0], acc[3][0], a0, b, bk,
                               st + b_rd[1][0], st + b_rd[1][1], n);
    bk = b;
    b = join_b(n);
    issue_part(std::integral_constant<int, 0>{}, ahead);
    // block (0,1): reads B(1,0) and substep-1 A of this step
    smfmac32_block_a<BF16, kPat12, kFar, kAS, kMS>(
        acc[0][1], acc[1][1], acc[2][1], acc[3][1], a0, b, bk, st + b_rd[0][0] + kSub,
        st + b_rd[0][1] + kSub, n, st + a_rd1, st + m_rd1, a1);
    bk = b;
    b = join_b(n);
    widen_frags<kPat12>(a1);
    issue_part(std::integral_constant<int, 1>{}, ahead);
    // block (1,0): reads B(1,1)
    smfmac32_block<BF16, kFar>(acc[0][0], acc[1][0], acc[2][0], acc[3][0], a1, b, bk,
                               st + b_rd[1][0] + kSub, st + b_rd[1][1] + kSub, n);
    bk = b;
    b = join_b(n);
    issue_part(std::integral_constant<int, 2>{}, ahead);
    // block (1,1): reads next step's B(0,0) and substep-0 A (the last step reads a stage
    // that holds no useful data; the values are never used)
    smfmac32_block_a<BF16, kPat12, kFar, kAS, kMS>(
        acc[0][1], acc[1][1], acc[2][1], acc[3][1], a1, b, bk, sn + b_rd[0][0],
        sn + b_rd[0][1], n, sn + a_rd0, sn + m_rd0, a0);
    bk = b;
    b = join_b(n);
    widen_frags<kPat12>(a0);
    issue_part(std::integral_constant<int, 3>{}, ahead);
    // step s+2 landed (s+3 .. s+kStages-1 may still be in flight); after the barrier no
    // wave reads stage s % kStages any more
    wait_loads_and_barrier<(kStages - 3) * TL::kLoads>();
  }
  // drain the loads issued for steps past the end (every wave, then the barrier: no direct
  // load or fragment read touches LDS afterwards), and give the last smfmac results time
  // to land before plain instructions read the accumulators
  wait_loads_and_barrier<0>();
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  static_assert(TL::kWaves * kEpilogueBytes <= kStages * TL::kStageBytes, "epilogue LDS");
  store_block_128x64<YT>(acc, smem + wave * kEpilogueBytes, Y, m0 + wm * TL::kWM,
                         t0 + wn * TL::kWN, R, T, lane);
}

// The 2:4 consumer's whole K loop as one asm statement, so that LDS reads can stay in
// flight across blocks (the compiler would take an asm statement's outputs as written when
// the statement ends).  Fragments live in fixed registers: A of substep 0 (a0) in
// v64..v83, of substep 1 (a1) in v84..v103, the four B fragments of a step in v104..v127
// and v40..v47.  The loop is unrolled over the four ring slots: v48..v63 hold each lane
// offset plus the LDS address of slots 0-1 and of slots 2-3, and a read adds (slot & 1)
// stages and its own offset as the instruction's immediate, so a step does no address
// arithmetic.  Per step, block j issues its reads right behind
// its first smfmac, one block ahead of their use:
//   block 0 (a0 x B0): a1 fragments 0-1 and B2;   block 1 (a0 x B1): B3, a1 fragments 2-3;
//   block 2 (a1 x B2): next B0, next a0 0-1;       block 3 (a1 x B3): next B1, next a0 2-3.
// Each set is 8 LDS instructions, issued two behind each smfmac of the block so that the
// matrix core never waits on a run of LDS issue.  LDS reads complete in order, so
// "lgkmcnt(8)" before a block's first smfmac (blocks 0, 2) completes the set issued two
// blocks earlier, and "lgkmcnt(4)" before its third smfmac (four of its own reads issued)
// the set issued one block earlier.  A register is rewritten only by reads issued behind a
// later smfmac than every smfmac that reads it.  Reads of the next step's stage may be in flight at the step's barrier; the
// released stage (this step's) has no read in flight by then.  Everything has landed when
// the statement ends.
#define NM_WS24_LOOP(OP) \
  "s_waitcnt lgkmcnt(0)\n\t" \
  "v_add_u32 v48, %[base], %[ar0]\n\t" \
  "v_add_u32 v49, %[basehi], %[ar0]\n\t" \
  "v_add_u32 v50, %[base], %[ar1]\n\t" \
  "v_add_u32 v51, %[basehi], %[ar1]\n\t" \
  "v_add_u32 v52, %[base], %[mr0]\n\t" \
  "v_add_u32 v53, %[basehi], %[mr0]\n\t" \
  "v_add_u32 v54, %[base], %[mr1]\n\t" \
  "v_add_u32 v55, %[basehi], %[mr1]\n\t" \
  "v_add_u32 v56, %[base], %[b00]\n\t" \
  "v_add_u32 v57, %[basehi], %[b00]\n\t" \
  "v_add_u32 v58, %[base], %[b01]\n\t" \
  "v_add_u32 v59, %[basehi], %[b01]\n\t" \
  "v_add_u32 v60, %[base], %[b10]\n\t" \
  "v_add_u32 v61, %[basehi], %[b10]\n\t" \
  "v_add_u32 v62, %[base], %[b11]\n\t" \
  "v_add_u32 v63, %[basehi], %[b11]\n\t" \
  "ds_read_b64_tr_b16 v[104:105], v56\n\t" \
  "ds_read_b64_tr_b16 v[106:107], v58\n\t" \
  "ds_read_b64_tr_b16 v[108:109], v56 offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[110:111], v58 offset:4096\n\t" \
  "ds_read_b128 v[64:67], v48\n\t" \
  "ds_read_b128 v[68:71], v48 offset:2048\n\t" \
  "ds_read_u16 v80, v52\n\t" \
  "ds_read_u16 v81, v52 offset:256\n\t" \
  "ds_read_b64_tr_b16 v[112:113], v60\n\t" \
  "ds_read_b64_tr_b16 v[114:115], v62\n\t" \
  "ds_read_b64_tr_b16 v[116:117], v60 offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[118:119], v62 offset:4096\n\t" \
  "ds_read_b128 v[72:75], v48 offset:4096\n\t" \
  "ds_read_b128 v[76:79], v48 offset:6144\n\t" \
  "ds_read_u16 v82, v52 offset:512\n\t" \
  "ds_read_u16 v83, v52 offset:768\n\t" \
  "s_mov_b32 %[cnt], %[ns]\n\t" \
  "L_ws24_s0_%=:\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[64:67], v[104:111], v80\n\t" \
  "ds_read_b128 v[84:87], v50\n\t" \
  "ds_read_b128 v[88:91], v50 offset:2048\n\t" \
  OP " %[c10], v[68:71], v[104:111], v81\n\t" \
  "ds_read_u16 v100, v54\n\t" \
  "ds_read_u16 v101, v54 offset:256\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[72:75], v[104:111], v82\n\t" \
  "ds_read_b64_tr_b16 v[120:121], v56 offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[122:123], v58 offset:8192\n\t" \
  OP " %[c30], v[76:79], v[104:111], v83\n\t" \
  "ds_read_b64_tr_b16 v[124:125], v56 offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[126:127], v58 offset:12288\n\t" \
  OP " %[c01], v[64:67], v[112:119], v80\n\t" \
  "ds_read_b64_tr_b16 v[40:41], v60 offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[42:43], v62 offset:8192\n\t" \
  OP " %[c11], v[68:71], v[112:119], v81\n\t" \
  "ds_read_b64_tr_b16 v[44:45], v60 offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[46:47], v62 offset:12288\n\t" \
  OP " %[c21], v[72:75], v[112:119], v82\n\t" \
  "ds_read_b128 v[92:95], v50 offset:4096\n\t" \
  "ds_read_b128 v[96:99], v50 offset:6144\n\t" \
  OP " %[c31], v[76:79], v[112:119], v83\n\t" \
  "ds_read_u16 v102, v54 offset:512\n\t" \
  "ds_read_u16 v103, v54 offset:768\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[84:87], v[120:127], v100\n\t" \
  "ds_read_b64_tr_b16 v[104:105], v56 offset:34816\n\t" \
  "ds_read_b64_tr_b16 v[106:107], v58 offset:34816\n\t" \
  OP " %[c10], v[88:91], v[120:127], v101\n\t" \
  "ds_read_b64_tr_b16 v[108:109], v56 offset:38912\n\t" \
  "ds_read_b64_tr_b16 v[110:111], v58 offset:38912\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[92:95], v[120:127], v102\n\t" \
  "ds_read_b128 v[64:67], v48 offset:34816\n\t" \
  "ds_read_b128 v[68:71], v48 offset:36864\n\t" \
  OP " %[c30], v[96:99], v[120:127], v103\n\t" \
  "ds_read_u16 v80, v52 offset:34816\n\t" \
  "ds_read_u16 v81, v52 offset:35072\n\t" \
  OP " %[c01], v[84:87], v[40:47], v100\n\t" \
  "ds_read_b64_tr_b16 v[112:113], v60 offset:34816\n\t" \
  "ds_read_b64_tr_b16 v[114:115], v62 offset:34816\n\t" \
  OP " %[c11], v[88:91], v[40:47], v101\n\t" \
  "ds_read_b64_tr_b16 v[116:117], v60 offset:38912\n\t" \
  "ds_read_b64_tr_b16 v[118:119], v62 offset:38912\n\t" \
  OP " %[c21], v[92:95], v[40:47], v102\n\t" \
  "ds_read_b128 v[72:75], v48 offset:38912\n\t" \
  "ds_read_b128 v[76:79], v48 offset:40960\n\t" \
  OP " %[c31], v[96:99], v[40:47], v103\n\t" \
  "ds_read_u16 v82, v52 offset:35328\n\t" \
  "ds_read_u16 v83, v52 offset:35584\n\t" \
  "s_barrier\n\t" \
  "s_sub_u32 %[cnt], %[cnt], 1\n\t" \
  "s_cmp_eq_u32 %[cnt], 0\n\t" \
  "s_cbranch_scc1 L_ws24_end_%=\n\t" \
  "L_ws24_s1_%=:\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[64:67], v[104:111], v80\n\t" \
  "ds_read_b128 v[84:87], v50 offset:34816\n\t" \
  "ds_read_b128 v[88:91], v50 offset:36864\n\t" \
  OP " %[c10], v[68:71], v[104:111], v81\n\t" \
  "ds_read_u16 v100, v54 offset:34816\n\t" \
  "ds_read_u16 v101, v54 offset:35072\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[72:75], v[104:111], v82\n\t" \
  "ds_read_b64_tr_b16 v[120:121], v56 offset:43008\n\t" \
  "ds_read_b64_tr_b16 v[122:123], v58 offset:43008\n\t" \
  OP " %[c30], v[76:79], v[104:111], v83\n\t" \
  "ds_read_b64_tr_b16 v[124:125], v56 offset:47104\n\t" \
  "ds_read_b64_tr_b16 v[126:127], v58 offset:47104\n\t" \
  OP " %[c01], v[64:67], v[112:119], v80\n\t" \
  "ds_read_b64_tr_b16 v[40:41], v60 offset:43008\n\t" \
  "ds_read_b64_tr_b16 v[42:43], v62 offset:43008\n\t" \
  OP " %[c11], v[68:71], v[112:119], v81\n\t" \
  "ds_read_b64_tr_b16 v[44:45], v60 offset:47104\n\t" \
  "ds_read_b64_tr_b16 v[46:47], v62 offset:47104\n\t" \
  OP " %[c21], v[72:75], v[112:119], v82\n\t" \
  "ds_read_b128 v[92:95], v50 offset:38912\n\t" \
  "ds_read_b128 v[96:99], v50 offset:40960\n\t" \
  OP " %[c31], v[76:79], v[112:119], v83\n\t" \
  "ds_read_u16 v102, v54 offset:35328\n\t" \
  "ds_read_u16 v103, v54 offset:35584\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[84:87], v[120:127], v100\n\t" \
  "ds_read_b64_tr_b16 v[104:105], v57\n\t" \
  "ds_read_b64_tr_b16 v[106:107], v59\n\t" \
  OP " %[c10], v[88:91], v[120:127], v101\n\t" \
  "ds_read_b64_tr_b16 v[108:109], v57 offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[110:111], v59 offset:4096\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[92:95], v[120:127], v102\n\t" \
  "ds_read_b128 v[64:67], v49\n\t" \
  "ds_read_b128 v[68:71], v49 offset:2048\n\t" \
  OP " %[c30], v[96:99], v[120:127], v103\n\t" \
  "ds_read_u16 v80, v53\n\t" \
  "ds_read_u16 v81, v53 offset:256\n\t" \
  OP " %[c01], v[84:87], v[40:47], v100\n\t" \
  "ds_read_b64_tr_b16 v[112:113], v61\n\t" \
  "ds_read_b64_tr_b16 v[114:115], v63\n\t" \
  OP " %[c11], v[88:91], v[40:47], v101\n\t" \
  "ds_read_b64_tr_b16 v[116:117], v61 offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[118:119], v63 offset:4096\n\t" \
  OP " %[c21], v[92:95], v[40:47], v102\n\t" \
  "ds_read_b128 v[72:75], v49 offset:4096\n\t" \
  "ds_read_b128 v[76:79], v49 offset:6144\n\t" \
  OP " %[c31], v[96:99], v[40:47], v103\n\t" \
  "ds_read_u16 v82, v53 offset:512\n\t" \
  "ds_read_u16 v83, v53 offset:768\n\t" \
  "s_barrier\n\t" \
  "s_sub_u32 %[cnt], %[cnt], 1\n\t" \
  "s_cmp_eq_u32 %[cnt], 0\n\t" \
  "s_cbranch_scc1 L_ws24_end_%=\n\t" \
  "L_ws24_s2_%=:\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[64:67], v[104:111], v80\n\t" \
  "ds_read_b128 v[84:87], v51\n\t" \
  "ds_read_b128 v[88:91], v51 offset:2048\n\t" \
  OP " %[c10], v[68:71], v[104:111], v81\n\t" \
  "ds_read_u16 v100, v55\n\t" \
  "ds_read_u16 v101, v55 offset:256\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[72:75], v[104:111], v82\n\t" \
  "ds_read_b64_tr_b16 v[120:121], v57 offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[122:123], v59 offset:8192\n\t" \
  OP " %[c30], v[76:79], v[104:111], v83\n\t" \
  "ds_read_b64_tr_b16 v[124:125], v57 offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[126:127], v59 offset:12288\n\t" \
  OP " %[c01], v[64:67], v[112:119], v80\n\t" \
  "ds_read_b64_tr_b16 v[40:41], v61 offset:8192\n\t" \
  "ds_read_b64_tr_b16 v[42:43], v63 offset:8192\n\t" \
  OP " %[c11], v[68:71], v[112:119], v81\n\t" \
  "ds_read_b64_tr_b16 v[44:45], v61 offset:12288\n\t" \
  "ds_read_b64_tr_b16 v[46:47], v63 offset:12288\n\t" \
  OP " %[c21], v[72:75], v[112:119], v82\n\t" \
  "ds_read_b128 v[92:95], v51 offset:4096\n\t" \
  "ds_read_b128 v[96:99], v51 offset:6144\n\t" \
  OP " %[c31], v[76:79], v[112:119], v83\n\t" \
  "ds_read_u16 v102, v55 offset:512\n\t" \
  "ds_read_u16 v103, v55 offset:768\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[84:87], v[120:127], v100\n\t" \
  "ds_read_b64_tr_b16 v[104:105], v57 offset:34816\n\t" \
  "ds_read_b64_tr_b16 v[106:107], v59 offset:34816\n\t" \
  OP " %[c10], v[88:91], v[120:127], v101\n\t" \
  "ds_read_b64_tr_b16 v[108:109], v57 offset:38912\n\t" \
  "ds_read_b64_tr_b16 v[110:111], v59 offset:38912\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[92:95], v[120:127], v102\n\t" \
  "ds_read_b128 v[64:67], v49 offset:34816\n\t" \
  "ds_read_b128 v[68:71], v49 offset:36864\n\t" \
  OP " %[c30], v[96:99], v[120:127], v103\n\t" \
  "ds_read_u16 v80, v53 offset:34816\n\t" \
  "ds_read_u16 v81, v53 offset:35072\n\t" \
  OP " %[c01], v[84:87], v[40:47], v100\n\t" \
  "ds_read_b64_tr_b16 v[112:113], v61 offset:34816\n\t" \
  "ds_read_b64_tr_b16 v[114:115], v63 offset:34816\n\t" \
  OP " %[c11], v[88:91], v[40:47], v101\n\t" \
  "ds_read_b64_tr_b16 v[116:117], v61 offset:38912\n\t" \
  "ds_read_b64_tr_b16 v[118:119], v63 offset:38912\n\t" \
  OP " %[c21], v[92:95], v[40:47], v102\n\t" \
  "ds_read_b128 v[72:75], v49 offset:38912\n\t" \
  "ds_read_b128 v[76:79], v49 offset:40960\n\t" \
  OP " %[c31], v[96:99], v[40:47], v103\n\t" \
  "ds_read_u16 v82, v53 offset:35328\n\t" \
  "ds_read_u16 v83, v53 offset:35584\n\t" \
  "s_barrier\n\t" \
  "s_sub_u32 %[cnt], %[cnt], 1\n\t" \
  "s_cmp_eq_u32 %[cnt], 0\n\t" \
  "s_cbranch_scc1 L_ws24_end_%=\n\t" \
  "L_ws24_s3_%=:\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[64:67], v[104:111], v80\n\t" \
  "ds_read_b128 v[84:87], v51 offset:34816\n\t" \
  "ds_read_b128 v[88:91], v51 offset:36864\n\t" \
  OP " %[c10], v[68:71], v[104:111], v81\n\t" \
  "ds_read_u16 v100, v55 offset:34816\n\t" \
  "ds_read_u16 v101, v55 offset:35072\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[72:75], v[104:111], v82\n\t" \
  "ds_read_b64_tr_b16 v[120:121], v57 offset:43008\n\t" \
  "ds_read_b64_tr_b16 v[122:123], v59 offset:43008\n\t" \
  OP " %[c30], v[76:79], v[104:111], v83\n\t" \
  "ds_read_b64_tr_b16 v[124:125], v57 offset:47104\n\t" \
  "ds_read_b64_tr_b16 v[126:127], v59 offset:47104\n\t" \
  OP " %[c01], v[64:67], v[112:119], v80\n\t" \
  "ds_read_b64_tr_b16 v[40:41], v61 offset:43008\n\t" \
  "ds_read_b64_tr_b16 v[42:43], v63 offset:43008\n\t" \
  OP " %[c11], v[68:71], v[112:119], v81\n\t" \
  "ds_read_b64_tr_b16 v[44:45], v61 offset:47104\n\t" \
  "ds_read_b64_tr_b16 v[46:47], v63 offset:47104\n\t" \
  OP " %[c21], v[72:75], v[112:119], v82\n\t" \
  "ds_read_b128 v[92:95], v51 offset:38912\n\t" \
  "ds_read_b128 v[96:99], v51 offset:40960\n\t" \
  OP " %[c31], v[76:79], v[112:119], v83\n\t" \
  "ds_read_u16 v102, v55 offset:35328\n\t" \
  "ds_read_u16 v103, v55 offset:35584\n\t" \
  "s_waitcnt lgkmcnt(8)\n\t" \
  OP " %[c00], v[84:87], v[120:127], v100\n\t" \
  "ds_read_b64_tr_b16 v[104:105], v56\n\t" \
  "ds_read_b64_tr_b16 v[106:107], v58\n\t" \
  OP " %[c10], v[88:91], v[120:127], v101\n\t" \
  "ds_read_b64_tr_b16 v[108:109], v56 offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[110:111], v58 offset:4096\n\t" \
  "s_waitcnt lgkmcnt(4)\n\t" \
  OP " %[c20], v[92:95], v[120:127], v102\n\t" \
  "ds_read_b128 v[64:67], v48\n\t" \
  "ds_read_b128 v[68:71], v48 offset:2048\n\t" \
  OP " %[c30], v[96:99], v[120:127], v103\n\t" \
  "ds_read_u16 v80, v52\n\t" \
  "ds_read_u16 v81, v52 offset:256\n\t" \
  OP " %[c01], v[84:87], v[40:47], v100\n\t" \
  "ds_read_b64_tr_b16 v[112:113], v60\n\t" \
  "ds_read_b64_tr_b16 v[114:115], v62\n\t" \
  OP " %[c11], v[88:91], v[40:47], v101\n\t" \
  "ds_read_b64_tr_b16 v[116:117], v60 offset:4096\n\t" \
  "ds_read_b64_tr_b16 v[118:119], v62 offset:4096\n\t" \
  OP " %[c21], v[92:95], v[40:47], v102\n\t" \
  "ds_read_b128 v[72:75], v48 offset:4096\n\t" \
  "ds_read_b128 v[76:79], v48 offset:6144\n\t" \
  OP " %[c31], v[96:99], v[40:47], v103\n\t" \
  "ds_read_u16 v82, v52 offset:512\n\t" \
  "ds_read_u16 v83, v52 offset:768\n\t" \
  "s_barrier\n\t" \
  "s_sub_u32 %[cnt], %[cnt], 1\n\t" \
  "s_cmp_eq_u32 %[cnt], 0\n\t" \
  "s_cbranch_scc1 L_ws24_end_%=\n\t" \
  "s_branch L_ws24_s0_%=\n\t" \
  "L_ws24_end_%=:\n\t" \
  "s_waitcnt lgkmcnt(0)\n\t"

template <bool BF16, int kStageBytes, int kStages, int kFar, int kSub, int kAS, int kMS>
__device__ __forceinline__ void ws24_consumer_loop(float16v_t (&acc)[4][2], uint32_t base,
                                                   int nsteps, uint32_t ar0, uint32_t ar1,
                                                   uint32_t mr0, uint32_t mr1, uint32_t b00,
                                                   uint32_t b01, uint32_t b10, uint32_t b11) {
  // the loop text carries these as numbers (256 x 128 tiles, 64-wide steps, four slots)
  static_assert(kStageBytes == 34816 && kStages == 4 && kFar == 4096 && kSub == 8192 &&
                    kAS == 2048 && kMS == 256,
                "layout constants of the generated loop");
  uint32_t cnt;
  const uint32_t basehi = base + (uint32_t)(2 * kStageBytes);
#define NM_WS24_ASM(OPC)                                                                  \
  asm volatile(NM_WS24_LOOP(OPC)                                                          \
               : [c00] "+a"(acc[0][0]), [c10] "+a"(acc[1][0]), [c20] "+a"(acc[2][0]),     \
                 [c30] "+a"(acc[3][0]), [c01] "+a"(acc[0][1]), [c11] "+a"(acc[1][1]),     \
                 [c21] "+a"(acc[2][1]), [c31] "+a"(acc[3][1]), [cnt] "=&s"(cnt)           \
               : [base] "s"(base), [basehi] "s"(basehi), [ns] "s"(nsteps), [ar0] "v"(ar0), \
                 [ar1] "v"(ar1), [mr0] "v"(mr0), [mr1] "v"(mr1), [b00] "v"(b00),          \
                 [b01] "v"(b01), [b10] "v"(b10), [b11] "v"(b11)                           \
               : "memory", "scc", "v40", "v41", "v42", "v43", "v44", "v45", "v46", "v47", "v48", "v49", "v50", "v51", "v52", "v53", "v54", "v55", "v56", "v57", "v58", "v59", "v60", "v61", "v62", "v63", "v64", "v65", "v66", "v67", "v68", "v69", "v70", "v71", "v72", "v73", "v74", "v75", "v76", "v77", "v78", "v79", "v80", "v81", "v82", "v83", "v84", "v85", "v86", "v87", "v88", "v89", "v90", "v91", "v92", "v93", "v94", "v95", "v96", "v97", "v98", "v99", "v100", "v101", "v102", "v103", "v104", "v105", "v106", "v107", "v108", "v109", "v110", "v111", "v112", "v113", "v114", "v115", "v116", "v117", "v118", "v119", "v120", "v121", "v122", "v123", "v124", "v125", "v126", "v127")
  if constexpr (BF16)
    NM_WS24_ASM("v_smfmac_f32_32x32x32_bf16");
  else
    NM_WS24_ASM("v_smfmac_f32_32x32x32_f16");
#undef NM_WS24_ASM
}
#undef NM_WS24_LOOP

// ===========================================================================
// Wave-specialised form of the 32x32x32 kernel.  Each SIMD runs one consumer wave (LDS
// fragment reads and smfmac blocks, exactly as in smfmac32_spmm_kernel) and one producer
// wave (direct global -> LDS loads only).  A wave that issues direct loads stalls whenever
// the load queue is full; with the loads in their own waves those stalls no longer hold up
// a matrix core.  One barrier per step hands the stages over:
//   producer, iteration s: load step s+S-1 into the stage step s-1 used, then wait until
//     step s+2 has landed, then the barrier;
//   consumer, iteration s: compute step s (the last block also reads the first fragments
//     of step s+1), then the barrier.
// After barrier s, steps s+1 and s+2 are in LDS and visible, and no wave reads the stage
// of step s any more.  Both kinds of wave pass the same nsteps + 1 barriers.
// ===========================================================================
template <int BM, int BN, int CWAVES_M, int CWAVES_N, int PWAVES, int STAGES>
struct WsTile {
  static constexpr int kConsumers = CWAVES_M * CWAVES_N;
  static constexpr int kProducers = PWAVES;
  static constexpr int kThreads = 64 * (kConsumers + kProducers);
  static constexpr int kStages = STAGES;
  static constexpr int kWM = BM / CWAVES_M;
  static constexpr int kWN = BN / CWAVES_N;
  static constexpr int kXRowBytes = BN * 2;
  static constexpr int kXChunks = BN / 8;
  static constexpr int kXBytes = kKStep * kXRowBytes;
  static constexpr int kABytes = BM * 64;
  static constexpr int kMBytes = BM * 8;
  static constexpr int kStageBytes = kXBytes + kABytes + kMBytes;
  static constexpr int kXLoads = kXBytes / 1024 / kProducers;  // per producer wave and step
  static constexpr int kALoads = kABytes / 1024 / kProducers;
  static constexpr int kMLoads = kMBytes / 256 / kProducers;
  static constexpr int kLoads = kXLoads + kALoads + kMLoads;
  static_assert(kWM == 128 && kWN == 64, "a consumer owns 128 x 64 outputs");
  static_assert(kXBytes % (1024 * kProducers) == 0 && kABytes % (1024 * kProducers) == 0 &&
                    kMBytes % (256 * kProducers) == 0,
                "every producer issues the same number of direct loads per step");
  static_assert(BN >= 128, "the X swizzle needs at least 8 column pairs per row");
  static_assert(kStages >= 3 && (kStages - 2) * kLoads <= 63, "vmcnt budget");
  static_assert(kStages * kStageBytes <= 160 * 1024, "LDS budget");
};

template <bool BF16, bool kPat12, bool kBlocked, int YT, int BM, int BN, int CWAVES_M,
          int CWAVES_N, int PWAVES, int STAGES, int XB = 16>
__global__ void __launch_bounds__(64 * (CWAVES_M * CWAVES_N + PWAVES))
    smfmac_ws_spmm_kernel(const uint16_t* __restrict__ values, const uint32_t* __restrict__ meta,
                          const uint16_t* __restrict__ X, typename OutOf<YT>::type Y, int R, int K,
                          int T, TileMap map) {
  using TL = WsTile<BM, BN, CWAVES_M, CWAVES_N, PWAVES, STAGES>;
  constexpr int kStages = STAGES;
  constexpr int kRB = TL::kXRowBytes;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const int ldx = x_stride(Y, T);  // row length of X
  int tile_m, tile_n;
  if (!map.tile_of(blockIdx.x, tile_m, tile_n)) return;  // whole workgroup, before any load
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m0 = tile_m * BM, t0 = tile_n * BN;
  const int nsteps = K / kKStep;
  const int last_step = nsteps - 1;

  // X pieces per lane: 16 bytes when X rows are whole 16-byte pieces (T % 8 == 0), else 4
  // bytes (T even), which takes four times the load instructions
  static_assert(XB == 16 || (XB == 4 && BN * 2 == 64 * XB), "4-byte pieces: one row a load");
  constexpr int kXLoads = TL::kXBytes / (64 * XB) / TL::kProducers;
  if (wave >= TL::kConsumers) {
    // ---------------- producer ----------------
    // Every direct load reads at a wave-uniform base (scalar registers, advanced by one
    // step's bytes per step) plus a 32-bit per-lane offset that stays fixed for the whole
    // loop, so the loop issues its loads with no vector address arithmetic.  The per-lane
    // offsets stay below 2^32 because R, K and T are below 2^28 (the launcher's guard).
    static_assert(BN == 128 && TL::kProducers % 4 == 0, "X load windows of four K rows");
    const int pw = wave - TL::kConsumers;
    const uint8_t* xg = reinterpret_cast<const uint8_t*>(X);
    const uint8_t* vg = reinterpret_cast<const uint8_t*>(values);
    const uint8_t* mg = reinterpret_cast<const uint8_t*>(meta);
    const uint8_t* x_base[kXLoads];
    uint32_t x_off, x_dst[kXLoads];
    if constexpr (XB == 16) {
      // load j fills the 1 KB window w1k = j * kProducers + pw of the X tile: K rows
      // 4 w1k .. 4 w1k + 3, lane l taking row 4 w1k + l / 16 and physical chunk l % 16;
      // the row swizzle depends on r & 3 = (l / 16) & 3 only, so the lane offset is the
      // same for every j
      const int r = lane >> 4, pc = lane & 15;
      const int lc = 2 * ((pc >> 1) ^ xpair_swizzle(r)) + (pc & 1);
      int col = t0 + 8 * lc;
      col = col < T ? col : 0;  // columns past T: any valid address (outputs past T only)
      x_off = (uint32_t)(((int64_t)r * ldx + col) * 2);
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) {
        const int w1k = j * TL::kProducers + pw;
        x_base[j] = xg + (int64_t)(4 * w1k) * ldx * 2;
        x_dst[j] = (uint32_t)(w1k * 1024);
      }
    } else {
      // load j fills K row r = j * kProducers + pw: lane l lands at byte 4 l of the row,
      // physical pair l / 8, which holds logical pair (l / 8) ^ xpair_swizzle(r); r & 3 is
      // pw & 3 for every j
      const int lp = (lane >> 3) ^ xpair_swizzle(pw);
      int col = t0 + 16 * lp + 2 * (lane & 7);
      col = col < T ? col : 0;  // T even: col even, so every piece is 4-byte aligned
      x_off = (uint32_t)(col * 2);
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) {
        const int r = j * TL::kProducers + pw;
        x_base[j] = xg + (int64_t)r * ldx * 2;
        x_dst[j] = (uint32_t)(r * BN * 2);
      }
    }
    // compressed values: load j fills the 16 tile rows of block b16 = j * kProducers + pw
    // (the blocked layout's 1 KB block of those rows and the step; the row layout's
    // 64-byte pieces of each row); lane l takes row l / 4 of them and the chunk that lands
    // at physical chunk l % 4, logical chunk (l % 4) ^ ((l / 16) & 3)
    const uint8_t* a_base[TL::kALoads];
    uint32_t a_off, a_dst[TL::kALoads];
    {
      const int lc = (lane & 3) ^ ((lane >> 4) & 3);
      const int last = ((R + 15) >> 4) - 1;
      a_off = (uint32_t)((kBlocked ? (lane >> 2) * 64 : 0) + 16 * lc);
#pragma unroll
      for (int j = 0; j < TL::kALoads; ++j) {
        const int b16 = j * TL::kProducers + pw;
        if constexpr (kBlocked) {
          int g = (m0 >> 4) + b16;
          g = g < last ? g : last;  // rows past the matrix: any valid block
          a_base[j] = vg + (int64_t)g * nsteps * 1024;
        } else {
          a_base[j] = vg;  // row layout: the row is per lane (a_row below)
        }
        a_dst[j] = (uint32_t)(TL::kXBytes + b16 * 1024);
      }
    }
    // row layout: each lane's row, clamped to the matrix (its offset from W's start does
    // not fit the 32-bit lane offset, so it is kept as a 64-bit per-lane address)
    int64_t a_row[TL::kALoads];
#pragma unroll
    for (int j = 0; j < TL::kALoads; ++j) {
      if constexpr (!kBlocked) {
        int row = m0 + 16 * (j * TL::kProducers + pw) + (lane >> 2);
        row = row < R ? row : R - 1;
        a_row[j] = (int64_t)row * K;
      } else {
        a_row[j] = 0;
      }
    }
    int64_t m_src[TL::kMLoads];
    uint32_t m_dst[TL::kMLoads];
#pragma unroll
    for (int j = 0; j < TL::kMLoads; ++j) {
      const int b32 = j * TL::kProducers + pw;
      m_src[j] = meta_source<kBlocked, kPat12>(m0, 32 * b32, lane, R, K, nsteps);
      m_dst[j] = (uint32_t)(TL::kXBytes + TL::kABytes + b32 * 256);
    }
    // Blocked 2:4: the 128 metadata bytes of a 16-row block and step are contiguous, so
    // each producer fetches four blocks (512 bytes) with one 16-byte-per-lane load on half
    // its lanes, instead of two 4-byte-per-lane loads; the bytes land where those would.
    constexpr bool kWideMeta = kBlocked && !kPat12;
    static_assert(!kWideMeta || TL::kMBytes == 512 * TL::kProducers, "four blocks per producer");
    const uint8_t* m16_base = mg;
    uint32_t m16_off = 0, m16_dst = 0;
    if constexpr (kWideMeta) {
      const int last = ((R + 15) >> 4) - 1;
      int g0 = (m0 >> 4) + 4 * pw;
      g0 = g0 < last ? g0 : last;
      int g = (m0 >> 4) + 4 * pw + ((lane & 31) >> 3);
      g = g < last ? g : last;
      m16_base = mg + (int64_t)g0 * nsteps * 128;
      m16_off = (uint32_t)((g - g0) * nsteps * 128 + 16 * (lane & 7));
      m16_dst = (uint32_t)(TL::kXBytes + TL::kABytes + pw * 512);
    }
    auto issue_step = [&](int step) {
      // the step's own ring slot; past the end the loads re-read the last step's data into
      // it (a slot no wave reads any more), so every step issues the same loads
      const uint32_t sta = lds_addr(smem + (step % kStages) * TL::kStageBytes);
      step = step < last_step ? step : last_step;
      const int64_t kx = (int64_t)step * kKStep * ldx * 2;
      const int64_t ka = (int64_t)step * values_step_bytes<kBlocked>();
      const int64_t km = (int64_t)step * meta_step_bytes<kBlocked, kPat12>();
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) global_to_lds_sv<XB>(x_base[j] + kx, x_off, sta + x_dst[j]);
#pragma unroll
      for (int j = 0; j < TL::kALoads; ++j) {
        if constexpr (kBlocked)
          global_to_lds_sv<16>(a_base[j] + ka, a_off, sta + a_dst[j]);
        else
          global_to_lds_v<16>(vg + a_row[j] + ka + a_off, sta + a_dst[j]);
      }
      if constexpr (kWideMeta) {
        if (lane < 32) global_to_lds_sv<16>(m16_base + km, m16_off, sta + m16_dst);
      } else {
#pragma unroll
        for (int j = 0; j < TL::kMLoads; ++j) global_to_lds_v<4>(mg + m_src[j] + km, sta + m_dst[j]);
      }
    };
    // 1:2: once a step has landed, each producer rewrites the metadata rows it loaded
    // (four bytes per row, one bit per stored value) in place as the 2:4 instruction's
    // index units (four 16-bit units per row), so the consumers read both patterns alike.
    auto widen_step = [&](int step) {
      if constexpr (kPat12) {
        const int row = 32 * ((lane >> 5) * TL::kProducers + pw) + (lane & 31);
        const uint32_t a = lds_addr(smem + (step % kStages) * TL::kStageBytes + TL::kXBytes +
                                    TL::kABytes) + (uint32_t)(row * 8);
        uint32_t raw;
        asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(raw) : "v"(a) : "memory");
        const uint32_t w0 = widen_1_2(raw) | (widen_1_2(raw >> 8) << 16);
        const uint32_t w1 = widen_1_2(raw >> 16) | (widen_1_2(raw >> 24) << 16);
        asm volatile("ds_write_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)"
                     :
                     : "v"(a), "v"(u32x2_t{w0, w1})
                     : "memory");
      }
    };
    // direct loads one producer issues per step
    constexpr int kLoads = kXLoads + TL::kALoads + (kWideMeta ? 1 : TL::kMLoads);
    static_assert((kStages - 2) * kLoads <= 63, "vmcnt budget");
    static_assert(!kPat12 || TL::kMLoads * 32 * TL::kProducers == BM, "a metadata row per lane");
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue_step(k);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 3) * kLoads) : "memory");
    widen_step(0);  // steps 0 and 1 landed
    widen_step(1);
    asm volatile("s_barrier" ::: "memory");
    for (int s = 0; s < nsteps; ++s) {
      issue_step(s + kStages - 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 3) * kLoads) : "memory");
      widen_step(s + 2);  // step s+2 landed
      asm volatile("s_barrier" ::: "memory");
    }
    // loads past the end have landed before the consumers reuse LDS for the epilogue
    wait_loads_and_barrier<0>();
    if constexpr (YT == kAct) finish_half<BF16 ? kBF16 : kF16>(smem, Y, m0, t0, R, T, wave, lane);
    return;
  }

  // ---------------- consumer ----------------
  const int wm = wave / CWAVES_N, wn = wave % CWAVES_N;
  const int l32 = lane & 31, q = lane >> 5, l16 = lane & 15, blk = lane >> 4;
  const int ia = wm * TL::kWM + l32;
  const int aswz = (ia >> 2) & 3;
  const uint32_t a_rd0 = (uint32_t)(TL::kXBytes + ia * 64 + (((0 + q) ^ aswz) << 4));
  const uint32_t a_rd1 = (uint32_t)(TL::kXBytes + ia * 64 + (((2 + q) ^ aswz) << 4));
  // index units of the 2:4 instruction (1:2 rows are widened to them by the producers)
  const uint32_t m_rd0 = (uint32_t)(TL::kXBytes + TL::kABytes + ia * 8 + 2 * q);
  const uint32_t m_rd1 = m_rd0 + 4;
  const int rb = 8 * q + (l16 >> 2);
  uint32_t b_rd[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int lp = (wn * TL::kWN + 32 * f + 16 * (blk & 1)) / 16;
    b_rd[f][0] = (uint32_t)(rb * kRB + ((lp ^ xpair_swizzle(rb)) << 5) + 8 * (l16 & 3));
    b_rd[f][1] =
        (uint32_t)((rb + 4) * kRB + ((lp ^ xpair_swizzle(rb + 4)) << 5) + 8 * (l16 & 3));
  }
  constexpr int kFar = 16 * kRB;
  constexpr int kSub = 32 * kRB;
  constexpr int kAS = 32 * 64;
  constexpr int kMS = 32 * 8;

  float16v_t acc[4][2];
#pragma unroll
  for (int fm = 0; fm < 4; ++fm)
#pragma unroll
    for (int f = 0; f < 2; ++f) acc[fm][f] = float16v_t{};

  const uint32_t smem_base = lds_addr(smem);
  asm volatile("s_barrier" ::: "memory");  // steps 0 and 1 landed
  ws24_consumer_loop<BF16, TL::kStageBytes, kStages, kFar, kSub, kAS, kMS>(
      acc, smem_base, nsteps, a_rd0, a_rd1, m_rd0, m_rd1, b_rd[0][0], b_rd[0][1], b_rd[1][0],
      b_rd[1][1]);
  // the producers' last loads have landed (final barrier), and the last smfmac results
  // get time to land before plain instructions read the accumulators
  asm volatile("s_barrier\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  if constexpr (YT == kAct) {
    static_assert(CWAVES_M == 2 && CWAVES_N == 2 && PWAVES == 4, "blocks as finish_half has them");
    static_assert(4 * kBlockBytes <= kStages * TL::kStageBytes, "epilogue LDS");
    slab_write(acc[0], acc[1], slab_of(smem, wave), lane);
    slab_write(acc[2], acc[3], slab_of(smem, wave + 4), lane);
    finish_half<BF16 ? kBF16 : kF16>(smem, Y, m0, t0, R, T, wave, lane);
  } else {
    static_assert(TL::kConsumers * kEpilogueBytes <= kStages * TL::kStageBytes, "epilogue LDS");
    store_block_128x64<YT>(acc, smem + wave * kEpilogueBytes, Y, m0 + wm * TL::kWM,
                             t0 + wn * TL::kWN, R, T, lane);
  }
}

// ===========================================================================
// int8 2:4 and 1:2 on v_smfmac_i32_32x32x64_i8 (exact int32 sums).  Lane l of the instruction
// supplies row l % 32 of A as 16 stored bytes covering logical K [32 (l/32), +32) (8 groups,
// one 32-bit index word of 2-bit positions), and column l % 32 of B as 32 bytes, K
// {16 (l/32) + 0..15} and {32 + 16 (l/32) + 0..15}; the accumulator has the dense 32 x 32
// layout.  B comes out of the row-major X tile with ds_read_b64_tr_b8: inside each 16-lane
// block, lane i receives byte (i & 7) of the 8-byte chunks addressed by lanes (i >> 3) + 2j
// (j = 0..7), so with even lanes addressing 8 columns of 8 consecutive K rows and odd
// lanes the next 8 columns of the same rows, lane i gets 8 consecutive K of column i.
// One pipeline step is 128 of K: two blocked-layout steps, i.e. one contiguous 1 KB of
// values and 256 bytes of metadata per 16 rows (128 for 1:2), and 128 rows of X; the row
// layout lands the same LDS image from 64-byte pieces of each row.  Wave-specialised as
// smfmac_ws_spmm_kernel: producer waves issue the direct loads (4-stage ring, one barrier
// per step), each of four consumer waves owns 128 x 64 outputs (4 x 2 fragments).  The
// fp8 instantiation (v_smfmac_f32_32x32x64_fp8_fp8) has fp32 accumulators, but the
// instruction itself adds the products of each run of 16 consecutive K in fixed point
// aligned to the run's largest product (bits below 2^(e - 13) are dropped) before the run
// sum reaches the accumulator: not every product is summed in fp32.
// ===========================================================================
constexpr int kI8KStep = 128;

// Physical 16-byte chunk of logical chunk c in X tile row r (8 chunks per 128-byte row):
// the eight rows of one transposing read, and the two 16-row halves a wave reads at
// once, land on different banks.
__device__ __forceinline__ int xsw_i8(int r) { return ((r >> 1) ^ (r >> 4)) & 7; }

template <int BM, int BN, int CWAVES_M, int CWAVES_N, int PWAVES, int STAGES>
struct WsI8Tile {
  static constexpr int kConsumers = CWAVES_M * CWAVES_N;
  static constexpr int kProducers = PWAVES;
  static constexpr int kThreads = 64 * (kConsumers + kProducers);
  static constexpr int kStages = STAGES;
  static constexpr int kWM = BM / CWAVES_M;
  static constexpr int kWN = BN / CWAVES_N;
  static constexpr int kXBytes = kI8KStep * BN;   // 128 K rows of BN bytes
  static constexpr int kABytes = BM * 64;          // 64 stored bytes per row and step
  static constexpr int kMBytes = BM * 16;          // 16 metadata bytes per row and step
  static constexpr int kStageBytes = kXBytes + kABytes + kMBytes;
  static constexpr int kXLoads = kXBytes / 1024 / kProducers;
  static constexpr int kALoads = kABytes / 1024 / kProducers;
  static constexpr int kMLoads = kMBytes / 256 / kProducers;
  static constexpr int kLoads = kXLoads + kALoads + kMLoads;
  static_assert(BN == 128, "X rows are 8 swizzled 16-byte chunks");
  static_assert(kWM == 128 && kWN == 64, "a consumer owns 128 x 64 outputs");
  static_assert(kXBytes % (1024 * kProducers) == 0 && kABytes % (1024 * kProducers) == 0 &&
                    kMBytes % (256 * kProducers) == 0,
                "every producer issues the same number of direct loads per step");
  static_assert(kStages >= 3 && (kStages - 2) * kLoads <= 63, "vmcnt budget");
  static_assert(kStages * kStageBytes <= 160 * 1024, "LDS budget");
};

typedef int int16v_t __attribute__((ext_vector_type(16)));
typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef int int4v_t __attribute__((ext_vector_type(4)));
typedef int int2v_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) int2v_t lds_int2v_t;

template <bool kFp8, bool kBlocked, bool kPat12, int YT, int BM, int BN, int CWAVES_M,
          int CWAVES_N, int PWAVES, int STAGES>
__global__ void __launch_bounds__(64 * (CWAVES_M * CWAVES_N + PWAVES))
    smfmac_i8_ws_spmm_kernel(const uint8_t* __restrict__ values, const uint32_t* __restrict__ meta,
                             const uint8_t* __restrict__ X, typename OutOf<YT>::type Y, int R, int K,
                             int T, TileMap map) {
  using TL = WsI8Tile<BM, BN, CWAVES_M, CWAVES_N, PWAVES, STAGES>;
  constexpr int kStages = STAGES;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const int ldx = x_stride(Y, T);  // row length of X
  int tile_m, tile_n;
  if (!map.tile_of(blockIdx.x, tile_m, tile_n)) return;  // whole workgroup, before any load
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m0 = tile_m * BM, t0 = tile_n * BN;
  const int nsteps = K / kI8KStep;
  const int last_step = nsteps - 1;
  const int steps64 = K / 64;  // blocked-layout steps per row group

  if (wave >= TL::kConsumers) {
    // ---------------- producer ----------------
    const int pw = wave - TL::kConsumers;
    const int last_g = ((R + 15) >> 4) - 1;
    int64_t x_src[TL::kXLoads];
    uint32_t x_dst[TL::kXLoads];
#pragma unroll
    for (int j = 0; j < TL::kXLoads; ++j) {
      const int w1k = j * TL::kProducers + pw;  // 1 KB window: 8 rows of the X tile
      const int slot = w1k * 64 + lane;
      const int r = slot >> 3, pc = slot & 7;
      int col = t0 + 16 * (pc ^ xsw_i8(r));
      col = col < T ? col : 0;  // columns past T: any valid address (outputs past T only)
      x_src[j] = (int64_t)r * ldx + col;
      x_dst[j] = (uint32_t)(w1k * 1024);
    }
    // A stage holds, per 16-row group, the values as [64-wide half][row][32 bytes] (1 KB)
    // and the metadata as [half][row][8 bytes] (256 bytes; 1:2: [half][row][4 bytes] in its
    // first 128).  In the blocked layout both are one contiguous run per group and step; in
    // the row layout lane l fetches row (l % 32) / 2, half l / 32, 16-byte (values) or
    // 4-byte (metadata) piece l % 2 (1:2 metadata: lanes 0..31, row l % 16, half l / 16).
    int64_t a_src[TL::kALoads], m_src[TL::kMLoads];
    uint32_t a_dst[TL::kALoads], m_dst[TL::kMLoads];
    const int lrow = (lane & 31) >> 1, lh = lane >> 5, lp = lane & 1;
#pragma unroll
    for (int j = 0; j < TL::kALoads; ++j) {
      const int b16 = j * TL::kProducers + pw;  // row group of the tile
      if constexpr (kBlocked) {
        int g = (m0 >> 4) + b16;
        g = g < last_g ? g : last_g;  // rows past the matrix: any valid group
        a_src[j] = (int64_t)g * steps64 * 512 + 16 * lane;
      } else {
        int row = m0 + 16 * b16 + lrow;
        row = row < R ? row : R - 1;  // rows past the matrix: any valid row
        a_src[j] = (int64_t)row * (K / 2) + 32 * lh + 16 * lp;
      }
      a_dst[j] = (uint32_t)(TL::kXBytes + b16 * 1024);
    }
#pragma unroll
    for (int j = 0; j < TL::kMLoads; ++j) {
      const int b16 = j * TL::kProducers + pw;
      if constexpr (kBlocked) {
        int g = (m0 >> 4) + b16;
        g = g < last_g ? g : last_g;
        m_src[j] = (int64_t)g * steps64 * (kPat12 ? 64 : 128) + 4 * lane;
      } else if constexpr (kPat12) {
        int row = m0 + 16 * b16 + (lane & 15);
        row = row < R ? row : R - 1;
        m_src[j] = (int64_t)row * (K / 16) + 4 * ((lane >> 4) & 1);  // K / 64 words per row
      } else {
        int row = m0 + 16 * b16 + lrow;
        row = row < R ? row : R - 1;
        m_src[j] = (int64_t)row * (K / 8) + 8 * lh + 4 * lp;  // K / 32 words per row
      }
      m_dst[j] = (uint32_t)(TL::kXBytes + TL::kABytes + b16 * 256);
    }
    constexpr int64_t kAStep = kBlocked ? 1024 : 64;
    constexpr int64_t kMStep = kPat12 ? (kBlocked ? 128 : 8) : (kBlocked ? 256 : 16);
    const uint8_t* mg = reinterpret_cast<const uint8_t*>(meta);
    auto issue_step = [&](int step) {
      step = step < last_step ? step : last_step;  // past the end: re-read the last step
      uint8_t* st = smem + (step % kStages) * TL::kStageBytes;
      const int64_t kx = (int64_t)step * kI8KStep * ldx;
#pragma unroll
      for (int j = 0; j < TL::kXLoads; ++j) global_to_lds<16>(X + x_src[j] + kx, st + x_dst[j]);
#pragma unroll
      for (int j = 0; j < TL::kALoads; ++j)
        global_to_lds<16>(values + a_src[j] + step * kAStep, st + a_dst[j]);
#pragma unroll
      for (int j = 0; j < TL::kMLoads; ++j) {
        if constexpr (kPat12) {  // 128 bytes per group: half the lanes
          if (lane < 32) global_to_lds<4>(mg + m_src[j] + step * kMStep, st + m_dst[j]);
        } else {
          global_to_lds<4>(mg + m_src[j] + step * kMStep, st + m_dst[j]);
        }
      }
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue_step(k);
    wait_loads_and_barrier<(kStages - 3) * TL::kLoads>();  // steps 0 and 1 landed
    for (int s = 0; s < nsteps; ++s) {
      issue_step(s + kStages - 1);
      wait_loads_and_barrier<(kStages - 3) * TL::kLoads>();  // step s+2 landed
    }
    wait_loads_and_barrier<0>();  // no load in flight when the consumers reuse LDS
    if constexpr (YT == kAct) finish_half<kFp8 ? kFP8 : kI8>(smem, Y, m0, t0, R, T, wave, lane);
    return;
  }

  // ---------------- consumer ----------------
  const int wm = wave / CWAVES_N, wn = wave % CWAVES_N;
  const int l32 = lane & 31, q = lane >> 5, i16 = lane & 15, blk = lane >> 4;
  // A and index addresses of fragment fm in half h: row i = wm*128 + 32 fm + l32
  uint32_t a_off[4], m_off[4];
#pragma unroll
  for (int fm = 0; fm < 4; ++fm) {
    const int i = wm * TL::kWM + 32 * fm + l32;
    a_off[fm] = (uint32_t)(TL::kXBytes + (i >> 4) * 1024 + (i & 15) * 32 + 16 * q);
    m_off[fm] = (uint32_t)(TL::kXBytes + TL::kABytes + (i >> 4) * 256 +
                           (kPat12 ? (i & 15) * 4 + 2 * q : (i & 15) * 8 + 4 * q));
  }
  // B: piece p of fragment f in half h covers K rows 64h + 16q + 8(p & 1) + 32(p >> 1) + 0..7
  // of columns wn*64 + 32 f + 16 (blk & 1) + 0..15; this lane addresses row + (i16 >> 1),
  // 8-byte half (i16 & 1) of that 16-column chunk
  uint32_t b_off[2][2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int r = 64 * h + 16 * q + 8 * (p & 1) + 32 * (p >> 1) + (i16 >> 1);
        const int chunk = (wn * TL::kWN + 32 * f + 16 * (blk & 1)) >> 4;
        b_off[h][f][p] = (uint32_t)(r * BN + 16 * (chunk ^ xsw_i8(r)) + 8 * (i16 & 1));
      }

  using AccV = std::conditional_t<kFp8, float16v_t, int16v_t>;
  AccV acc[4][2];
#pragma unroll
  for (int fm = 0; fm < 4; ++fm)
#pragma unroll
    for (int f = 0; f < 2; ++f) acc[fm][f] = AccV{};

  // Fragments of one half step (64 of K): 4 A fragments with their index words and 2 B
  // fragments.  The next half step's fragments are read while this one's 8 smfmac run.
  struct Frags {
    int4v_t a[4];
    int ix[4];
    int8v_t b[2];
  };
  auto load_frags = [&](const uint8_t* st, int h) {
    Frags F;
#pragma unroll
    for (int fm = 0; fm < 4; ++fm) {
      F.a[fm] = *reinterpret_cast<const int4v_t*>(st + a_off[fm] + 512 * h);
      if constexpr (kPat12) {
        // 16 one-bit positions b_j of 1:2 groups j -> the 2:4 index word: value j sits in
        // group j / 2 of four at position 2 (j % 2) + b_j, i.e. bit j moves to bit 2j and
        // every odd field gets its bit 1
        uint32_t x = *reinterpret_cast<const uint16_t*>(st + m_off[fm] + 64 * h);
        x = (x | (x << 8)) & 0x00FF00FFu;
        x = (x | (x << 4)) & 0x0F0F0F0Fu;
        x = (x | (x << 2)) & 0x33333333u;
        x = (x | (x << 1)) & 0x55555555u;
        F.ix[fm] = (int)(x | 0x88888888u);
      } else {
        F.ix[fm] = *reinterpret_cast<const int*>(st + m_off[fm] + 128 * h);
      }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      int2v_t pc[4];
#pragma unroll
      for (int p = 0; p < 4; ++p)
        pc[p] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_int2v_t*)(st + b_off[h][f][p]));
      F.b[f] = int8v_t{pc[0][0], pc[0][1], pc[1][0], pc[1][1],
                       pc[2][0], pc[2][1], pc[3][0], pc[3][1]};
    }
    return F;
  };
  auto mma = [&](const Frags& F) {
#pragma unroll
    for (int fm = 0; fm < 4; ++fm)
#pragma unroll
      for (int f = 0; f < 2; ++f)
        if constexpr (kFp8)
          acc[fm][f] = __builtin_amdgcn_smfmac_f32_32x32x64_fp8_fp8(F.a[fm], F.b[f], acc[fm][f],
                                                                    F.ix[fm], 0, 0);
        else
          acc[fm][f] = __builtin_amdgcn_smfmac_i32_32x32x64_i8(F.a[fm], F.b[f], acc[fm][f],
                                                               F.ix[fm], 0, 0);
  };

  asm volatile("s_barrier" ::: "memory");  // steps 0 and 1 landed
  Frags cur = load_frags(smem, 0);
  for (int s = 0; s < nsteps; ++s) {
    const uint8_t* st = smem + (s % kStages) * TL::kStageBytes;
    const uint8_t* sn = smem + ((s + 1) % kStages) * TL::kStageBytes;
    Frags nxt = load_frags(st, 1);
    mma(cur);
    // step s+1 landed before the previous barrier; after the last step this reads a
    // stage of re-read data that is never used
    cur = load_frags(sn, 0);
    mma(nxt);
    asm volatile("s_barrier" ::: "memory");  // step s+2 landed; stage of step s released
  }
  asm volatile("s_barrier\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  if constexpr (YT == kAct) {
    static_assert(CWAVES_M == 2 && CWAVES_N == 2 && PWAVES == 4, "blocks as finish_half has them");
    static_assert(4 * kBlockBytes <= kStages * TL::kStageBytes, "epilogue LDS");
    slab_write(acc[0], acc[1], slab_of(smem, wave), lane);
    slab_write(acc[2], acc[3], slab_of(smem, wave + 4), lane);
    finish_half<kFp8 ? kFP8 : kI8>(smem, Y, m0, t0, R, T, wave, lane);
  } else {
    static_assert(TL::kConsumers * kEpilogueBytes <= kStages * TL::kStageBytes, "epilogue LDS");
    store_block_128x64<YT, AccV>(acc, smem + wave * kEpilogueBytes, Y, m0 + wm * TL::kWM,
                             t0 + wn * TL::kWN, R, T, lane);
  }
}

template <bool kFp8, bool kBlocked, bool kPat12, int YT>
hipError_t run_smfmac_8bit(const void* values, const uint32_t* meta, int64_t R, int64_t K,
                           const void* X, int64_t T, typename OutOf<YT>::type Y, hipStream_t s) {
  constexpr int BM = 256, BN = 128, ST = 4;
  using TL = WsI8Tile<BM, BN, 2, 2, 4, ST>;
  auto kernel = smfmac_i8_ws_spmm_kernel<kFp8, kBlocked, kPat12, YT, BM, BN, 2, 2, 4, ST>;
  const size_t lds = (size_t)ST * TL::kStageBytes;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (attr != hipSuccess) return attr;
  const TileMap map =
      make_tile_map((int)((R + BM - 1) / BM), (int)((T + BN - 1) / BN), xcd_count());
  kernel<<<map.xcds * map.per_xcd, TL::kThreads, lds, s>>>(
      static_cast<const uint8_t*>(values), meta, static_cast<const uint8_t*>(X), Y, (int)R,
      (int)K, (int)T, map);
  return hipGetLastError();
}

// ===========================================================================
// 4:8 on dense matrix cores (no structured-sparse instruction takes 4:8).  The blocked
// layout's values and metadata reach LDS exactly as for 2:4 (4:8 also keeps half the
// values; its metadata is 12 bytes per row and 64-wide step), and each consumer lane
// expands one 4:8 group into the dense A operand of v_mfma_f32_32x32x16: the A operand of a
// lane is 8 consecutive K of one row, i.e. exactly one group.  The 4 stored values become
// 8 slots with four v_perm_b32 byte selects whose selectors come from a 256-entry table
// indexed by the group's keep mask (one bit per kept position).  Inside a 64-wide step the
// contraction order is permuted so that lane half q of substep t takes group 4q + t (K
// 32q + 8t .. +7): a lane's four groups of a step are then one contiguous 32-byte run of
// values and 48 contiguous metadata bits, and B is read at the matching K rows.
// Wave-specialised like smfmac_ws_spmm_kernel: producer waves load, consumer waves expand
// and multiply, one barrier per step.  The producers, otherwise idle, also turn each
// landed step's 3-bit positions into one keep-mask byte per group (their own LDS region
// of the stage), which takes the mask building off the consumers' instruction stream.
// Producer, iteration s: load step s+3, wait for step s+2, build its keep masks, barrier;
// consumer, iteration s: step s (reading step s+1's keep masks for the next fragments).
// ===========================================================================
template <int BM, int BN, int CWAVES_M, int CWAVES_N, int PWAVES, int STAGES>
struct Ws48Tile {
  static constexpr int kConsumers = CWAVES_M * CWAVES_N;
  static constexpr int kProducers = PWAVES;
  static constexpr int kThreads = 64 * (kConsumers + kProducers);
  static constexpr int kStages = STAGES;
  static constexpr int kWM = BM / CWAVES_M;
  static constexpr int kWN = BN / CWAVES_N;
  static constexpr int kXRowBytes = BN * 2;
  static constexpr int kXChunks = BN / 8;
  static constexpr int kXBytes = kKStep * kXRowBytes;
  static constexpr int kABytes = BM * 64;
  static constexpr int kMRow = 12;  // metadata bytes per row and step
  static constexpr int kMBytes = BM * kMRow;
  static constexpr int kKmBytes = BM * 8;  // keep masks: one byte per group, 8 per row
  static constexpr int kStageBytes = kXBytes + kABytes + kMBytes + kKmBytes;
  static constexpr int kLutBytes = 256 * 16;
  static constexpr int kXLoads = kXBytes / 1024 / kProducers;
  static constexpr int kALoads = kABytes / 1024 / kProducers;
  static constexpr int kMLoads = kMBytes / 256 / kProducers;
  static constexpr int kLoads = kXLoads + kALoads + kMLoads;
  static_assert(kWM == 128 && kWN == 64, "a consumer owns 128 x 64 outputs");
  static_assert(kXBytes % (1024 * kProducers) == 0 && kABytes % (1024 * kProducers) == 0 &&
                    kMBytes % (256 * kProducers) == 0,
                "every producer issues the same number of direct loads per step");
  static_assert(BM == 64 * kProducers, "one producer lane per tile row builds its keep masks");
  static_assert(BN >= 128, "the X swizzle needs at least 8 column pairs per row");
  static_assert(kStages >= 4 && (kStages - 2) * kLoads <= 63, "vmcnt budget");
  static_assert(kStages * kStageBytes + kLutBytes <= 160 * 1024, "LDS budget");
};

template <bool BF16>
__device__ __forceinline__ float16v_t mfma32x32x16(const u32x4_t& a, const u32x4_t& b,
                                                   const float16v_t& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <bool BF16, bool kBlocked, int YT, int BM, int BN, int CWAVES_M, int CWAVES_N,
          int PWAVES, int STAGES, int XB = 16>
__global__ void __launch_bounds__(64 * (CWAVES_M * CWAVES_N + PWAVES))
    mfma48_ws_spmm_kernel(const uint16_t* __restrict__ values, const uint32_t* __restrict__ meta,
                          const uint16_t* __restrict__ X, typename OutOf<YT>::type Y, int R, int K,
                          int T, TileMap map) {
  using TL = Ws48Tile<BM, BN, CWAVES_M, CWAVES_N, PWAVES, STAGES>;
  constexpr int kStages = STAGES;
  constexpr int kRB = TL::kXRowBytes;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  const int ldx = x_stride(Y, T);  // row length of X
  int tile_m, tile_n;
  if (!map.tile_of(blockIdx.x, tile_m, tile_n)) return;  // whole workgroup, before any load
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m0 = tile_m * BM, t0 = tile_n * BN;
  const int nsteps = K / kKStep;
  const int last_step = nsteps - 1;
  const int last_group = ((R + 15) >> 4) - 1;

  if (wave >= TL::kConsumers) {
    // ---------------- producer ----------------
    const int pw = wave - TL::kConsumers;
    const uint8_t* xg = reinterpret_cast<const uint8_t*>(X);
    const uint8_t* vg = reinterpret_cast<const uint8_t*>(values);
    const uint8_t* mg = reinterpret_cast<const uint8_t*>(meta);
    // X pieces of 16 bytes, or of 4 bytes for even T that is not a multiple of 8 (as in
    // smfmac_ws_spmm_kernel)
    static_assert(XB == 16 || (XB == 4 && BN * 2 == 64 * XB), "4-byte pieces: one row a load");
    constexpr int kXLoads = TL::kXBytes / (64 * XB) / TL::kProducers;
    constexpr int kLoads = kXLoads + TL::kALoads + TL::kMLoads;
    static_assert((kStages - 2) * kLoads <= 63, "vmcnt budget");
    int64_t x_src[kXLoads];
    uint32_t x_dst[kXLoads];
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) {
      if constexpr (XB == 16) {
        const int w1k = j * TL::kProducers + pw;
        const int slot = w1k * 64 + lane;
        const int r = slot / TL::kXChunks, pc = slot % TL::kXChunks;
        const int lc = 2 * ((pc >> 1) ^ xpair_swizzle(r)) + (pc & 1);
        int col = t0 + 8 * lc;
        col = col < T ? col : 0;
        x_src[j] = ((int64_t)r * ldx + col) * 2;
        x_dst[j] = (uint32_t)(w1k * 1024);
      } else {
        const int r = j * TL::kProducers + pw;  // one K row per load
        const int lp = (lane >> 3) ^ xpair_swizzle(r);
        int col = t0 + 16 * lp + 2 * (lane & 7);
        col = col < T ? col : 0;
        x_src[j] = ((int64_t)r * ldx + col) * 2;
        x_dst[j] = (uint32_t)(r * BN * 2);
      }
    }
    int64_t a_src[TL::kALoads];
    uint32_t a_dst[TL::kALoads];
#pragma unroll
    for (int j = 0; j < TL::kALoads; ++j) {
      const int b16 = j * TL::kProducers + pw;
      a_src[j] = values_source<kBlocked>(m0, 16 * b16, lane, R, K, nsteps);
      a_dst[j] = (uint32_t)(TL::kXBytes + b16 * 1024);
    }
    // metadata: the tile's rows land back to back, 12 bytes each (tile row i at 12 i); in
    // the blocked layout that is the tile's 16 blocks of 16 rows x 12 bytes (192 bytes
    // each, nsteps * 192 bytes apart), in the row layout 12 bytes of each row (3K/16 bytes
    // apart).  A load covers 256 bytes of the run, four per lane.  Producer pw loads the
    // bytes of rows 64 pw .. 64 pw + 63 itself, so its own wait covers the rows whose keep
    // masks it builds.
    static_assert(64 * TL::kMRow == 256 * TL::kMLoads, "a producer's rows are whole loads");
    int64_t m_src[TL::kMLoads];
    uint32_t m_dst[TL::kMLoads];
#pragma unroll
    for (int j = 0; j < TL::kMLoads; ++j) {
      const int w256 = pw * TL::kMLoads + j;
      const int o = w256 * 256 + 4 * lane;
      if constexpr (kBlocked) {
        int g = m0 / 16 + o / 192;
        g = g < last_group ? g : last_group;
        m_src[j] = (int64_t)g * nsteps * 192 + o % 192;
      } else {
        int row = m0 + o / 12;
        row = row < R ? row : R - 1;  // rows past the matrix: any valid row
        m_src[j] = (int64_t)row * (3 * (int64_t)K / 16) + o % 12;
      }
      m_dst[j] = (uint32_t)(TL::kXBytes + TL::kABytes + w256 * 256);
    }
    auto issue_step = [&](int step) {
      step = step < last_step ? step : last_step;
      uint8_t* st = smem + (step % kStages) * TL::kStageBytes;
      const int64_t kx = (int64_t)step * kKStep * ldx * 2;
      const int64_t ka = (int64_t)step * values_step_bytes<kBlocked>();
      const int64_t km = (int64_t)step * (kBlocked ? 192 : 12);
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) global_to_lds<XB>(xg + x_src[j] + kx, st + x_dst[j]);
#pragma unroll
      for (int j = 0; j < TL::kALoads; ++j) global_to_lds<16>(vg + a_src[j] + ka, st + a_dst[j]);
#pragma unroll
      for (int j = 0; j < TL::kMLoads; ++j) global_to_lds<4>(mg + m_src[j] + km, st + m_dst[j]);
    };
    // keep masks of a landed step: lane l of producer pw takes tile row 64 pw + l (its 12
    // metadata bytes = eight 12-bit groups of four 3-bit positions).  LDS accesses go
    // through asm that waits for itself, so the compiler sees no LDS access that the
    // in-flight direct loads might alias.
    const uint32_t smem_base = lds_addr(smem);
    const int krow = 64 * pw + lane;
    auto build_keep_masks = [&](int step) {
      const uint32_t st = smem_base + (uint32_t)((step % kStages) * TL::kStageBytes);
      const uint32_t src = st + TL::kXBytes + TL::kABytes + krow * TL::kMRow;
      const uint32_t dst = st + TL::kXBytes + TL::kABytes + TL::kMBytes + krow * 8;
      uint32_t m0, m1, m2;
      asm volatile(
          "ds_read_b32 %0, %3\n\tds_read_b32 %1, %3 offset:4\n\tds_read_b32 %2, %3 offset:8\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(m0), "=&v"(m1), "=&v"(m2)
          : "v"(src)
          : "memory");
      const uint64_t lo = (uint64_t)m0 | ((uint64_t)m1 << 32);   // groups 0 .. 4
      const uint64_t hi = (uint64_t)m1 | ((uint64_t)m2 << 32);   // groups 5 .. 7 (from bit 32)
      uint32_t k[2] = {0u, 0u};
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const uint32_t bits = (uint32_t)(g < 5 ? lo >> (12 * g) : hi >> (12 * g - 32)) & 0xfffu;
        const uint32_t keep = (1u << (bits & 7)) | (1u << ((bits >> 3) & 7)) |
                              (1u << ((bits >> 6) & 7)) | (1u << ((bits >> 9) & 7));
        k[g >> 2] |= keep << (8 * (g & 3));
      }
      asm volatile("ds_write_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)"
                   :
                   : "v"(dst), "v"(u32x2_t{k[0], k[1]})
                   : "memory");
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue_step(k);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 3) * kLoads) : "memory");
    build_keep_masks(0);
    build_keep_masks(1);
    asm volatile("s_barrier" ::: "memory");  // steps 0 and 1 landed, their masks built
    for (int s = 0; s < nsteps; ++s) {
      issue_step(s + kStages - 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kStages - 3) * kLoads) : "memory");
      build_keep_masks(s + 2);  // past the end: stale data of an unused stage, never read
      asm volatile("s_barrier" ::: "memory");  // step s+2 landed and its masks built
    }
    wait_loads_and_barrier<0>();  // loads past the end landed before the epilogue
    if constexpr (YT == kAct) finish_half<BF16 ? kBF16 : kF16>(smem, Y, m0, t0, R, T, wave, lane);
    return;
  }

  // ---------------- consumer ----------------
  // expansion table: entry m (a keep mask) holds the v_perm_b32 selectors of output dwords
  // 0..3 (slots 2k, 2k+1): slot i kept -> bytes 2j, 2j+1 of the group's 8 value bytes, j the
  // rank of i among the kept positions; not kept -> 0x0c (a zero byte)
  uint8_t* lut = smem + kStages * TL::kStageBytes;
  {
    const int m = tid;  // 256 consumer threads, one entry each
    u32x4_t e;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t sel = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 2 * k + h;
        const uint32_t j = __builtin_popcount(m & ((1u << i) - 1u));
        const uint32_t pair = ((m >> i) & 1) ? (2 * j) | ((2 * j + 1) << 8) : 0x0c0cu;
        sel |= pair << (16 * h);
      }
      e[k] = sel;
    }
    *reinterpret_cast<u32x4_t*>(lut + 16 * m) = e;
  }
  const int wm = wave / CWAVES_N, wn = wave % CWAVES_N;
  const int l32 = lane & 31, q = lane >> 5, l16 = lane & 15, blk = lane >> 4;
  const int ia = wm * TL::kWM + l32;
  const int aswz = (ia >> 2) & 3;
  // values: chunks 2q and 2q+1 of the row (groups 4q .. 4q+3)
  const uint32_t a_rd0 = (uint32_t)(TL::kXBytes + ia * 64 + (((2 * q) ^ aswz) << 4));
  const uint32_t a_rd1 = (uint32_t)(TL::kXBytes + ia * 64 + (((2 * q + 1) ^ aswz) << 4));
  // keep masks of groups 4q .. 4q+3 of the row: one dword
  const uint32_t km_rd = (uint32_t)(TL::kXBytes + TL::kABytes + TL::kMBytes + ia * 8 + 4 * q);
  // B of substep t: K rows 32q + 8t + {0..3} and {4..7}
  const int rb = 32 * q + (l16 >> 2);
  uint32_t b_rd[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int lp = (wn * TL::kWN + 32 * f + 16 * (blk & 1)) / 16;
    b_rd[f][0] = (uint32_t)(rb * kRB + ((lp ^ xpair_swizzle(rb)) << 5) + 8 * (l16 & 3));
    b_rd[f][1] =
        (uint32_t)((rb + 4) * kRB + ((lp ^ xpair_swizzle(rb + 4)) << 5) + 8 * (l16 & 3));
  }
  float16v_t acc[4][2];
#pragma unroll
  for (int fm = 0; fm < 4; ++fm)
#pragma unroll
    for (int f = 0; f < 2; ++f) acc[fm][f] = float16v_t{};

  // Software pipeline over substeps u = 4 s + t: while substep u runs its eight matrix
  // instructions, the value dwords and expansion selectors of substep u+2 and the B
  // fragments of substep u+1 are being read (the selector reads index a table at random
  // and meet bank conflicts, so they get two substeps); step s+1's keep masks are read
  // at t = 1.
  auto vals_of = [&](const uint8_t* stg, int fm, int t) {  // group 4q + t of row ia + 32 fm
    return *reinterpret_cast<const u32x2_t*>(stg + (t < 2 ? a_rd0 : a_rd1) + fm * 32 * 64 +
                                             8 * (t & 1));
  };
  auto meta_of = [&](const uint8_t* stg, int fm) {  // keep masks of this lane's 4 groups
    return *reinterpret_cast<const uint32_t*>(stg + km_rd + fm * 32 * 8);
  };
  auto sel_of = [&](uint32_t masks, int t) {  // expansion selectors of group t
    return *reinterpret_cast<const u32x4_t*>(lut + 16 * ((masks >> (8 * t)) & 0xffu));
  };
  auto b_of = [&](const uint8_t* stg, int f, int t) {
    const short4_t lo =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(stg + b_rd[f][0] + 8 * t * kRB));
    const short4_t hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(stg + b_rd[f][1] + 8 * t * kRB));
    return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // table written; steps 0, 1 landed
  uint32_t mcur[4], mnext[4];
  u32x2_t vcur[4], vnext[4];
  u32x4_t scur[4], snext[4], bcur[2];
  {
    const uint8_t* st0 = smem;
#pragma unroll
    for (int fm = 0; fm < 4; ++fm) {
      mcur[fm] = meta_of(st0, fm);
      vcur[fm] = vals_of(st0, fm, 0);
      scur[fm] = sel_of(mcur[fm], 0);
      vnext[fm] = vals_of(st0, fm, 1);
      snext[fm] = sel_of(mcur[fm], 1);
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) bcur[f] = b_of(st0, f, 0);
  }
  for (int s = 0; s < nsteps; ++s) {
    const uint8_t* st = smem + (s % kStages) * TL::kStageBytes;
    const uint8_t* sn = smem + ((s + 1) % kStages) * TL::kStageBytes;  // landed; the last
    // step reads a stage that holds no useful data, and the values are never used
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t == 1) {
#pragma unroll
        for (int fm = 0; fm < 4; ++fm) mnext[fm] = meta_of(sn, fm);
      }
      const int t1 = (t + 1) & 3, t2 = (t + 2) & 3;
      const uint8_t* stg1 = t < 3 ? st : sn;  // substep u+1
      const uint8_t* stg2 = t < 2 ? st : sn;  // substep u+2
      u32x2_t vnn[4];
      u32x4_t snn[4], bnext[2];
#pragma unroll
      for (int fm = 0; fm < 4; ++fm) {
        vnn[fm] = vals_of(stg2, fm, t2);
        snn[fm] = sel_of(t < 2 ? mcur[fm] : mnext[fm], t2);
      }
#pragma unroll
      for (int f = 0; f < 2; ++f) bnext[f] = b_of(stg1, f, t1);
      // expand substep u and run its matrix instructions
      u32x4_t a[4];
#pragma unroll
      for (int fm = 0; fm < 4; ++fm) {
        const uint32_t d0 = vcur[fm][0], d1 = vcur[fm][1];
        a[fm] = u32x4_t{__builtin_amdgcn_perm(d1, d0, scur[fm][0]),
                        __builtin_amdgcn_perm(d1, d0, scur[fm][1]),
                        __builtin_amdgcn_perm(d1, d0, scur[fm][2]),
                        __builtin_amdgcn_perm(d1, d0, scur[fm][3])};
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int fm = 0; fm < 4; ++fm) acc[fm][f] = mfma32x32x16<BF16>(a[fm], bcur[f], acc[fm][f]);
#pragma unroll
      for (int fm = 0; fm < 4; ++fm) {
        vcur[fm] = vnext[fm];
        scur[fm] = snext[fm];
        vnext[fm] = vnn[fm];
        snext[fm] = snn[fm];
      }
      bcur[0] = bnext[0];
      bcur[1] = bnext[1];
    }
#pragma unroll
    for (int fm = 0; fm < 4; ++fm) mcur[fm] = mnext[fm];
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // stage of step s released
  }
  asm volatile("s_barrier" ::: "memory");  // the producers' last loads have landed
  if constexpr (YT == kAct) {
    static_assert(CWAVES_M == 2 && CWAVES_N == 2 && PWAVES == 4, "blocks as finish_half has them");
    static_assert(4 * kBlockBytes <= kStages * TL::kStageBytes, "epilogue LDS");
    slab_write(acc[0], acc[1], slab_of(smem, wave), lane);
    slab_write(acc[2], acc[3], slab_of(smem, wave + 4), lane);
    finish_half<BF16 ? kBF16 : kF16>(smem, Y, m0, t0, R, T, wave, lane);
  } else {
    static_assert(TL::kConsumers * kEpilogueBytes <= kStages * TL::kStageBytes, "epilogue LDS");
    store_block_128x64<YT>(acc, smem + wave * kEpilogueBytes, Y, m0 + wm * TL::kWM,
                             t0 + wn * TL::kWN, R, T, lane);
  }
}

// ===========================================================================
// Any N:M on the dense matrix cores: the compressed rows are expanded in LDS (zeros where
// pruned) and multiplied with v_mfma_f32_32x32x2_f32 (fp32) or
// v_mfma_f32_32x32x16_{bf16,f16} (16-bit patterns without a structured-sparse kernel, and
// fp8 and int8, whose values and X are widened exactly to bf16 on the way into LDS: an E4M3
// value has at most four significant bits and lies inside bf16's exponent range, an int8
// value is an integer below 2^8; products are then exact in fp32, fp8 sums stay in fp32 and
// int8 sums move to int32 every 512 of K).  This is the dense product of the decompressed tile, reading only the compressed pair, so
// it can at best match a dense GEMM.  The loads of step s+1 go to registers before step
// s's matrix instructions and into the other LDS stage after them (one barrier per step).
// Workgroup: 128 x 128 outputs, four waves of 64 x 64 (2 x 2 blocks of 32 x 32).
//  * fp32, K step 32: instruction i (0..15) pairs K 16q + i in lane half q (the contraction
//    order inside a step is free), so a lane's A operands of the step are one 16-float run
//    of its row and each B operand is one ds_read_b32.  X rows 16..31 swap adjacent
//    32-column blocks, so the two lane halves of a B read hit opposite halves of the banks.
//  * 16-bit, K step 64: substep t (0..3) gives lane half q K 32q + 8t + 0..7, one 16-byte
//    A read of its row; B comes from the row-major X tile through ds_read_b64_tr_b16, X
//    stored in 32-byte column pairs swizzled by xpair_swizzle as in the 2:4 kernels.
// A rows are 144 bytes (32 floats or 64 halves, then padding): conflict-free 16-byte reads.
// ===========================================================================
constexpr int kEM = 128, kEN = 128;
constexpr int kEARow = 36;                          // 32-bit words per A row in LDS
constexpr int kEStageWords = kEM * kEARow + 4096;   // A rows + 16 KB of X

__device__ __forceinline__ int ex_col(int c, int kk) {  // fp32: physical column of X entry
  return (((c >> 5) ^ ((kk >> 4) & 1)) << 5) | (c & 31);
}

template <int DT, int YT, int N, int M, bool kBlocked, bool kVecX>
__global__ void __launch_bounds__(256)
    expand_mfma_spmm_kernel(const void* __restrict__ values, const uint32_t* __restrict__ meta,
                            const void* __restrict__ X, typename OutOf<YT>::type Y, int64_t R,
                            int64_t K, int64_t T, int64_t tiles_n) {
  constexpr bool kF = DT == kF32;
  // fp8 and int8: widened to bf16 (exactly) when written to LDS.  int8 products are summed
  // exactly: fp32 partial sums of at most 512 products of magnitude <= 2^14 are integers
  // below 2^24, so every 8 steps (512 of K) they are moved into int32 accumulators.
  constexpr bool kI = DT == kI8;
  constexpr bool k8 = DT == kFP8 || kI;
  using E = std::conditional_t<kF, float, std::conditional_t<k8, uint8_t, uint16_t>>;
  constexpr int kEK = kF ? 32 : 64;          // K per step
  constexpr int kPerChunk = 16 / sizeof(E);  // X elements per 16-byte piece
  constexpr int kChunksPerRow = kEN / kPerChunk;
  constexpr int kXPieces = kEK * kEN * (int)sizeof(E) / 16 / 256;  // per thread and step
  constexpr int b = meta_bits(M);
  constexpr int kGPS = kEK / M;              // groups per row and step
  constexpr int kItems = kEM * kGPS / 256;   // (row, group) items per thread and step
  constexpr int64_t V = 64 / M * N;          // blocked layout: values per row per 64 of K
  static_assert(kItems * 256 == kEM * kGPS, "whole items per thread");
  static_assert(kXPieces * 256 * 16 == kEK * kEN * (int)sizeof(E), "whole X pieces");
  extern __shared__ __attribute__((aligned(16))) uint32_t ex_smem[];  // two stages
  const int64_t ldx = x_stride(Y, T);  // row length of X
  const E* vals = static_cast<const E*>(values);
  const E* Xe = static_cast<const E*>(X);
  auto widen8 = [](uint32_t code) {  // an 8-bit element as fp32 (exact)
    if constexpr (kI) return (float)(int8_t)code;
    else return e4m3_to_f32(code);
  };
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kEM;
  const int64_t t0 = (int64_t)(blockIdx.x % tiles_n) * kEN;
  const int64_t gpr = K / M, wpr = (gpr * N * b + 31) / 32;

  // prefetch registers: X pieces, each item's values and the (one or two) metadata words
  // holding its fields with the fields' bit offset; nothing fetched is used before the
  // stash, so the loads stay in flight across the step's matrix instructions
  u32x4_t xr[4];
  E vr[kItems][N];
  uint32_t mw0[kItems], mw1[kItems], msh[kItems];
  auto fetch = [&](int64_t k0) {
#pragma unroll
    for (int j = 0; j < kXPieces; ++j) {
      const int idx = j * 256 + tid, kk = idx / kChunksPerRow;
      const int c = kPerChunk * (idx % kChunksPerRow);
      const int64_t k = k0 + kk, col = t0 + c;
      if constexpr (kVecX) {  // rows of X are whole 16-byte pieces
        xr[j] = (k < K && col < T) ? *reinterpret_cast<const u32x4_t*>(Xe + k * ldx + col)
                                   : u32x4_t{0u, 0u, 0u, 0u};
      } else {  // any T: element loads, zeros past the last column
        uint32_t wv[4] = {0u, 0u, 0u, 0u};
        if (k < K) {
          const E* src = Xe + k * ldx + col;
#pragma unroll
          for (int e = 0; e < kPerChunk; ++e) {
            if (col + e < T) {
              if constexpr (kF) wv[e] = __float_as_uint(src[e]);
              else if constexpr (k8) wv[e >> 2] |= (uint32_t)src[e] << (8 * (e & 3));
              else wv[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
            }
          }
        }
        xr[j] = u32x4_t{wv[0], wv[1], wv[2], wv[3]};
      }
    }
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
      const int i = it * 256 + tid, r = i / kGPS, gl = i % kGPS;
      const int64_t row = m0 + r, g = k0 / M + gl;
#pragma unroll
      for (int j = 0; j < N; ++j) vr[it][j] = E(0);
      mw0[it] = mw1[it] = msh[it] = 0u;
      if (row < R && g < gpr) {
        // the group's N fields are consecutive in both layouts (a 64-wide step of the blocked
        // layout holds whole groups): first value index and first metadata bit
        const int64_t f0 = g * N;
        int64_t vi, bit;
        if constexpr (kBlocked) {
          const int64_t rr = ((row >> 4) * (K / 64) + f0 / V) * 16 + (row & 15);
          vi = rr * V + f0 % V;
          bit = (rr * V + f0 % V) * b;
        } else {
          vi = row * (gpr * N) + f0;
          bit = row * wpr * 32 + f0 * b;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) vr[it][j] = vals[vi + j];
        mw0[it] = meta[bit / 32];
        if ((bit % 32) + N * b > 32) mw1[it] = meta[bit / 32 + 1];
        msh[it] = (uint32_t)(bit % 32);
      }
    }
  };
  auto stash = [&](int stage) {
    uint32_t* As = ex_smem + stage * kEStageWords;
    uint32_t* Xs = As + kEM * kEARow;
#pragma unroll
    for (int j = 0; j < kXPieces; ++j) {
      const int idx = j * 256 + tid, kk = idx / kChunksPerRow, pc = idx % kChunksPerRow;
      if constexpr (kF) {
        *reinterpret_cast<u32x4_t*>(Xs + kk * kEN + ex_col(4 * pc, kk)) = xr[j];
      } else if constexpr (k8) {
        // 16 fp8 columns -> one 32-byte column pair of bf16
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t lo = (xr[j][e >> 1] >> (16 * (e & 1))) & 0xFFu;
          const uint32_t hi = (xr[j][e >> 1] >> (16 * (e & 1) + 8)) & 0xFFu;
          h[e] = (__float_as_uint(widen8(lo)) >> 16) | (__float_as_uint(widen8(hi)) & 0xFFFF0000u);
        }
        uint32_t* d = Xs + kk * (kEN / 2) + 8 * (pc ^ xpair_swizzle(kk));
        *reinterpret_cast<u32x4_t*>(d) = u32x4_t{h[0], h[1], h[2], h[3]};
        *reinterpret_cast<u32x4_t*>(d + 4) = u32x4_t{h[4], h[5], h[6], h[7]};
      } else {
        const int word = kk * (kEN / 2) + 4 * (2 * ((pc >> 1) ^ xpair_swizzle(kk)) + (pc & 1));
        *reinterpret_cast<u32x4_t*>(Xs + word) = xr[j];
      }
    }
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
      const int i = it * 256 + tid, r = i / kGPS, gl = i % kGPS;
      const uint32_t fields = (uint32_t)((((uint64_t)mw1[it] << 32) | mw0[it]) >> msh[it]);
      uint32_t o[M];  // element bits, zero where pruned
#pragma unroll
      for (int e = 0; e < M; ++e) o[e] = 0u;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int p = (int)((fields >> (j * b)) & ((1u << b) - 1u));
        uint32_t v;
        if constexpr (kF) v = __float_as_uint(vr[it][j]);
        else if constexpr (k8) v = __float_as_uint(widen8(vr[it][j])) >> 16;
        else v = vr[it][j];
#pragma unroll
        for (int e = 0; e < M; ++e) o[e] = (p == e) ? v : o[e];
      }
      if constexpr (kF) {
        uint32_t* dst = As + r * kEARow + gl * M;
        if constexpr (M == 2) {
          *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{o[0], o[1]};
        } else {
#pragma unroll
          for (int e = 0; e < M; e += 4)
            *reinterpret_cast<u32x4_t*>(dst + e) = u32x4_t{o[e], o[e + 1], o[e + 2], o[e + 3]};
        }
      } else {
        uint32_t pk[M / 2];
#pragma unroll
        for (int e = 0; e < M / 2; ++e) pk[e] = o[2 * e] | (o[2 * e + 1] << 16);
        uint32_t* dst = As + r * kEARow + gl * (M / 2);
        if constexpr (M == 2) {
          *dst = pk[0];
        } else if constexpr (M == 4) {
          *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{pk[0], pk[1]};
        } else {
          *reinterpret_cast<u32x4_t*>(dst) = u32x4_t{pk[0], pk[1], pk[2], pk[3]};
        }
      }
    }
  };

  const int q = lane >> 5, lr = lane & 31, wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, blk = lane >> 4;
  int a_off[2], b_off[2][2];  // 32-bit words (A, fp32 B) or bytes (16-bit B)
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    a_off[f] = (wm * 64 + f * 32 + lr) * kEARow + 16 * q;  // K 16q.. (fp32) or 32q.. (16-bit)
    if constexpr (kF) {
      b_off[f][0] = 16 * q * kEN + ex_col(wn * 64 + f * 32 + lr, 16 * q);
      b_off[f][1] = 0;
    } else {
      const int rb = 32 * q + (l16 >> 2), lp = (wn * 64 + 32 * f + 16 * (blk & 1)) / 16;
      b_off[f][0] = rb * (2 * kEN) + ((lp ^ xpair_swizzle(rb)) << 5) + 8 * (l16 & 3);
      b_off[f][1] = (rb + 4) * (2 * kEN) + ((lp ^ xpair_swizzle(rb + 4)) << 5) + 8 * (l16 & 3);
    }
  }
  float16v_t acc[2][2];
#pragma unroll
  for (int fm = 0; fm < 2; ++fm)
#pragma unroll
    for (int fn = 0; fn < 2; ++fn) acc[fm][fn] = float16v_t{};
  int acc_i[kI ? 2 : 1][kI ? 2 : 1][kI ? 16 : 1] = {};  // int8: exact totals

  // one barrier per step: step s+1 is written into the other stage while step s's matrix
  // instructions run; that stage was last read in step s-1, before the previous barrier
  fetch(0);
  stash(0);
  __syncthreads();
  int stage = 0;
  for (int64_t k0 = 0; k0 < K; k0 += kEK) {
    const bool more = k0 + kEK < K;
    if (more) fetch(k0 + kEK);
    const uint32_t* As = ex_smem + stage * kEStageWords;
    const uint32_t* Xs = As + kEM * kEARow;
    if constexpr (kF) {
      float4_t a[2][4];
#pragma unroll
      for (int fm = 0; fm < 2; ++fm)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[fm][j] = *reinterpret_cast<const float4_t*>(As + a_off[fm] + 4 * j);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float bv[2];
#pragma unroll
        for (int fn = 0; fn < 2; ++fn) bv[fn] = __uint_as_float(Xs[b_off[fn][0] + i * kEN]);
#pragma unroll
        for (int fm = 0; fm < 2; ++fm)
#pragma unroll
          for (int fn = 0; fn < 2; ++fn)
            acc[fm][fn] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[fm][i >> 2][i & 3], bv[fn],
                                                               acc[fm][fn], 0, 0, 0);
      }
    } else {
      const uint8_t* xb = reinterpret_cast<const uint8_t*>(Xs);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u32x4_t a[2], bb[2];
#pragma unroll
        for (int fm = 0; fm < 2; ++fm)
          a[fm] = *reinterpret_cast<const u32x4_t*>(As + a_off[fm] + 4 * t);
#pragma unroll
        for (int fn = 0; fn < 2; ++fn) {
          const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_short4_t*)(xb + b_off[fn][0] + 8 * t * 2 * kEN));
          const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_short4_t*)(xb + b_off[fn][1] + 8 * t * 2 * kEN));
          bb[fn] = __builtin_bit_cast(u32x4_t,
                                      __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
#pragma unroll
        for (int fm = 0; fm < 2; ++fm)
#pragma unroll
          for (int fn = 0; fn < 2; ++fn)
            acc[fm][fn] = mfma32x32x16<DT != kF16>(a[fm], bb[fn], acc[fm][fn]);
      }
    }
    if constexpr (kI) {
      if (!more || ((k0 / kEK) & 7) == 7) {  // 512 of K summed exactly in fp32
#pragma unroll
        for (int fm = 0; fm < 2; ++fm)
#pragma unroll
          for (int fn = 0; fn < 2; ++fn) {
#pragma unroll
            for (int e = 0; e < 16; ++e) acc_i[fm][fn][e] += (int)acc[fm][fn][e];
            acc[fm][fn] = float16v_t{};
          }
      }
    }
    if (more) stash(stage ^ 1);
    __syncthreads();
    stage ^= 1;
  }
  // accumulator layout: lane (q, lr) of block (fm, fn) holds column lr and, in register e,
  // row 8 (e / 4) + 4 q + e % 4
  if constexpr (YT == kAct) {  // every wave is past the loop's last barrier: LDS is free
    static_assert(4 * kSlabBytes <= 2 * kEStageWords * 4, "epilogue LDS");
    uint8_t* mine = reinterpret_cast<uint8_t*>(ex_smem) + wave * kSlabBytes;
    if constexpr (kI) {
      int16v_t sums[2][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) sums[i >> 1][i & 1][e] = acc_i[i >> 1][i & 1][e];
      finish_block<DT>(sums, mine, Y, m0 + wm * 64, t0 + wn * 64, R, T, lane);
    } else {
      finish_block<DT>(acc, mine, Y, m0 + wm * 64, t0 + wn * 64, R, T, lane);
    }
    return;
  }
#pragma unroll
  for (int fm = 0; fm < 2; ++fm)
#pragma unroll
    for (int fn = 0; fn < 2; ++fn) {
      const int64_t col = t0 + wn * 64 + fn * 32 + lr;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t row = m0 + wm * 64 + fm * 32 + 8 * (e >> 2) + 4 * q + (e & 3);
        if constexpr (YT != kAct) {
          if (row < R && col < T) {
            if constexpr (kI)
              static_cast<int32_t*>(Y)[row * T + col] = acc_i[fm][fn][e];
            else
              store_from_f32<YT>(Y, row * T + col, acc[fm][fn][e]);
          }
        }
      }
    }
}

template <int DT, int YT, bool kBlocked, bool kVecX>
hipError_t run_expand(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n,
                      int m, const void* X, int64_t T, typename OutOf<YT>::type Y, hipStream_t s) {
  const int64_t tiles_n = (T + kEN - 1) / kEN, tiles = (R + kEM - 1) / kEM * tiles_n;
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  constexpr size_t lds = 2 * kEStageWords * sizeof(uint32_t);
#define NM_E(NN, MM)                                                                       \
  if (n == NN && m == MM) {                                                                \
    auto kernel = expand_mfma_spmm_kernel<DT, YT, NN, MM, kBlocked, kVecX>;                \
    static const hipError_t attr =                                                         \
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),                         \
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);         \
    if (attr != hipSuccess) return attr;                                                   \
    kernel<<<(unsigned)tiles, 256, lds, s>>>(values, meta, X, Y, R, K, T, tiles_n);        \
    return hipGetLastError();                                                              \
  }
  NM_E(1, 2) NM_E(2, 2)
  NM_E(1, 4) NM_E(2, 4) NM_E(3, 4) NM_E(4, 4)
  NM_E(1, 8) NM_E(2, 8) NM_E(3, 8) NM_E(4, 8)
  NM_E(5, 8) NM_E(6, 8) NM_E(7, 8) NM_E(8, 8)
#undef NM_E
  return hipErrorInvalidValue;
}

// X rows of whole 16-byte pieces take vector loads, any other T element loads.
template <int DT, int YT>
hipError_t run_expand_layout(const void* values, const uint32_t* meta, int64_t R, int64_t K,
                             int n, int m, bool blocked, const void* X, int64_t T,
                             typename OutOf<YT>::type Y, hipStream_t s) {
  const bool vec = T % (DT == kF32 ? 4 : (DT == kFP8 || DT == kI8) ? 16 : 8) == 0;
  if (vec)
    return blocked ? run_expand<DT, YT, true, true>(values, meta, R, K, n, m, X, T, Y, s)
                   : run_expand<DT, YT, false, true>(values, meta, R, K, n, m, X, T, Y, s);
  return blocked ? run_expand<DT, YT, true, false>(values, meta, R, K, n, m, X, T, Y, s)
                 : run_expand<DT, YT, false, false>(values, meta, R, K, n, m, X, T, Y, s);
}

[[maybe_unused]] __global__ void zero_fill_kernel(uint32_t* __restrict__ p, int64_t words, int64_t tail_halves) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < words) p[i] = 0u;
  if (i == words && tail_halves) reinterpret_cast<uint16_t*>(p + words)[0] = 0;
}


// One matrix-core launch: kernel K32 (32x32x32 blocks) or the 16x16x64 kernel, with the
// XCD-aware tile order.
// Kernel forms: 0 = 16x16x64 smfmac kernel, 1 = 32x32x32 blocks, 2 = 32x32x32 blocks with
// producer waves (PW of them).
template <int KIND, int BM, int BN, int WM_, int WN_, int PW, int ST_>
using TileOf = std::conditional_t<
    KIND == 0, SmfmacTile<BM, BN, WM_, WN_, ST_>,
    std::conditional_t<KIND == 1, Smfmac32Tile<BM, BN, WM_, WN_, ST_>,
                       WsTile<BM, BN, WM_, WN_, PW, ST_>>>;

template <bool BF16, bool kPat12, bool kBlocked, int YT, int KIND, int BM, int BN, int WM_,
          int WN_, int PW, int ST_, int XB = 16>
hipError_t launch_tile(const void* values, const uint32_t* meta, int64_t R, int64_t K,
                       const void* X, int64_t T, typename OutOf<YT>::type Y, hipStream_t s) {
  using TL = TileOf<KIND, BM, BN, WM_, WN_, PW, ST_>;
  const int tiles_m = (int)((R + BM - 1) / BM), tiles_n = (int)((T + BN - 1) / BN);
  void (*kernel)(const uint16_t*, const uint32_t*, const uint16_t*, typename OutOf<YT>::type, int,
                 int, int, TileMap);
  if constexpr (KIND == 0)
    kernel = smfmac_spmm_kernel<BF16, kPat12, kBlocked, YT, BM, BN, WM_, WN_, ST_>;
  else if constexpr (KIND == 1)
    kernel = smfmac32_spmm_kernel<BF16, kPat12, kBlocked, YT, BM, BN, WM_, WN_, ST_>;
  else
    kernel = smfmac_ws_spmm_kernel<BF16, kPat12, kBlocked, YT, BM, BN, WM_, WN_, PW, ST_, XB>;
  const size_t lds = (size_t)ST_ * TL::kStageBytes;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (attr != hipSuccess) return attr;
  const TileMap map = make_tile_map(tiles_m, tiles_n, xcd_count());
  kernel<<<map.xcds * map.per_xcd, TL::kThreads, lds, s>>>(
      static_cast<const uint16_t*>(values), meta, static_cast<const uint16_t*>(X), Y, (int)R,
      (int)K, (int)T, map);
  return hipGetLastError();
}

// Three tile shapes; the launch picks the one with the smallest estimated time: rounds of
// workgroups over the device (ceil(tiles / CUs)) times the time of one tile, which is its
// work at the rate that shape sustains on long K loops (measured on MI355X with normally
// distributed data, effective TFLOP/s over the whole device) plus a fixed per-tile cost
// (pipeline fill and the epilogue).
struct TileChoice {
  int bm, bn;
  double rate;
};
constexpr int kNumTiles = 3;
constexpr TileChoice kTiles[kNumTiles] = {{256, 256, 1720.0}, {256, 128, 1900.0},
                                          {128, 128, 1150.0}};
constexpr double kTileFixedUs = 5.0;

[[maybe_unused]] int pick_tile(int64_t R, int64_t K, int64_t T, int first = 0) {
  // NM_SPMM_TILE=0/1/2 pins one shape (used by the tests to cover every shape)
  if (const char* e = getenv("NM_SPMM_TILE")) {
    if (e[0] >= '0' && e[0] < '0' + kNumTiles && e[1] == 0)
      return e[0] - '0' < first ? first : e[0] - '0';
  }
  int dev = 0, cus = 256;
  if (hipGetDevice(&dev) == hipSuccess)
    (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (cus <= 0) cus = 256;
  int best = first;
  double best_t = 0;
  for (int i = first; i < kNumTiles; ++i) {
    const TileChoice& c = kTiles[i];
    const int64_t tiles = ((R + c.bm - 1) / c.bm) * ((T + c.bn - 1) / c.bn);
    const double tile_us = 2.0 * c.bm * c.bn * (double)K / (c.rate * 1e6 / cus) + kTileFixedUs;
    const double t = (double)((tiles + cus - 1) / cus) * tile_us;
    if (i == first || t < best_t) {
      best = i;
      best_t = t;
    }
  }
  return best;
}

template <bool BF16, bool kPat12, bool kBlocked, int YT>
hipError_t run_smfmac(const void* values, const uint32_t* meta, int64_t R, int64_t K,
                      const void* X, int64_t T, typename OutOf<YT>::type Y, hipStream_t s) {
  if constexpr (YT != kAct) {  // (its X has whole pieces)
    if (T % 8 != 0)  // even T: the wave-specialised tile with 4-byte X pieces
      return launch_tile<BF16, kPat12, kBlocked, YT, 2, 256, 128, 2, 2, 4, 4, 4>(values, meta, R,
                                                                                K, X, T, Y, s);
  }
  // (256 x 256 tiles have no registers left for an epilogue: 16384 x 64, 1000 columns 23 us against
  // 19.5 in 256 x 128)
  switch (pick_tile(R, K, T, YT == kAct ? 1 : 0)) {
    case 0:
      if constexpr (YT != kAct)
        return launch_tile<BF16, kPat12, kBlocked, YT, 1, 256, 256, 2, 4, 0, 3>(values, meta, R, K,
                                                                               X, T, Y, s);
    case 1:
      return launch_tile<BF16, kPat12, kBlocked, YT, 2, 256, 128, 2, 2, 4, 4>(values, meta, R, K,
                                                                             X, T, Y, s);
    default:
      return launch_tile<BF16, kPat12, kBlocked, YT, 0, 128, 128, 2, 2, 0, 4>(values, meta, R, K,
                                                                             X, T, Y, s);
  }
}

// 4:8, 16-bit, either layout: dense matrix cores on expanded groups, 256 x 128 tiles.
template <bool BF16, bool kBlocked, int YT, int XB>
hipError_t run_mfma48(const void* values, const uint32_t* meta, int64_t R, int64_t K,
                      const void* X, int64_t T, typename OutOf<YT>::type Y, hipStream_t s) {
  constexpr int BM = 256, BN = 128, ST = 4;
  using TL = Ws48Tile<BM, BN, 2, 2, 4, ST>;
  const int tiles_m = (int)((R + BM - 1) / BM), tiles_n = (int)((T + BN - 1) / BN);
  auto kernel = mfma48_ws_spmm_kernel<BF16, kBlocked, YT, BM, BN, 2, 2, 4, ST, XB>;
  const size_t lds = (size_t)ST * TL::kStageBytes + TL::kLutBytes;
  static const hipError_t attr =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (attr != hipSuccess) return attr;
  const TileMap map = make_tile_map(tiles_m, tiles_n, xcd_count());
  kernel<<<map.xcds * map.per_xcd, TL::kThreads, lds, s>>>(
      static_cast<const uint16_t*>(values), meta, static_cast<const uint16_t*>(X), Y, (int)R,
      (int)K, (int)T, map);
  return hipGetLastError();
}

template <bool BF16, bool kPat12, int YT>
hipError_t run_smfmac_layout(const void* values, const uint32_t* meta, int64_t R, int64_t K,
                             bool blocked, const void* X, int64_t T, typename OutOf<YT>::type Y, hipStream_t s) {
  return blocked ? run_smfmac<BF16, kPat12, true, YT>(values, meta, R, K, X, T, Y, s)
                 : run_smfmac<BF16, kPat12, false, YT>(values, meta, R, K, X, T, Y, s);
}

}  // namespace

#ifndef NM_SPMM_PART

// XCDs of the current device: MI355X (gfx950) has 8, with 32 compute units each.
// Looked up once per device.
int xcd_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 1;
  int v = cached[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return 1;
    v = cus % 8 == 0 ? 8 : 1;
    cached[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

hipError_t launch_spmm(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n,
                       int m, bool blocked, const void* X, int64_t T, int dt, void* Y, int y_dt,
                       hipStream_t s) {
  if (R == 0 || T == 0) return hipSuccess;
  const bool pat24 = (n == 2 && m == 4), pat12 = (n == 1 && m == 2);
  const bool half = dt == kBF16 || dt == kF16;
  // the structured-sparse and 4:8 kernels: K in whole 64-wide steps, even T (X in 16-byte
  // pieces when T % 8 == 0, else 4-byte ones), 32-bit tile coordinates, and K and T below
  // 2^28 (the wave-specialised kernels' per-lane load offsets are 32-bit)
  const bool sparse_shape = K > 0 && K % kKStep == 0 && T % 2 == 0 && R < (1 << 30) &&
                            T < (1 << 28) && K < (1 << 28);
  if (half && n == 4 && m == 8 && sparse_shape) {
#define NM_48(BF, YT)                                                                   \
  if (T % 8 != 0)                                                                       \
    return blocked ? run_mfma48<BF, true, YT, 4>(values, meta, R, K, X, T, Y, s)        \
                   : run_mfma48<BF, false, YT, 4>(values, meta, R, K, X, T, Y, s);      \
  return blocked ? run_mfma48<BF, true, YT, 16>(values, meta, R, K, X, T, Y, s)         \
                 : run_mfma48<BF, false, YT, 16>(values, meta, R, K, X, T, Y, s);
    if (dt == kBF16) {
      if (y_dt == kF32) { NM_48(true, kF32) }
      NM_48(true, kBF16)
    }
    if (y_dt == kF32) { NM_48(false, kF32) }
    NM_48(false, kF16)
#undef NM_48
  }
  if (half && pat24 && blocked && sk_shape_ok(R, K, T)) {
    // large shapes: 256 x 256 tiles split over the compute units (nm_spmm_sk.hip), with
    // a workspace for the partial tiles taken from the stream-ordered pool for this call.
    // NM_SPMM_TILE=3 selects this kernel on any shape it takes, 0..2 pin the others.
    const char* pin = getenv("NM_SPMM_TILE");
    const bool use = pin ? (pin[0] == '3' && pin[1] == 0) : sk_preferred(R, K, T);
    if (use) {
      const int groups = sk_groups(R, K, T);
      const int64_t ws_bytes = sk_workspace_bytes(R, T, groups);
      if (ws_bytes == 0) return launch_spmm_sk(values, meta, R, K, X, T, dt, Y, y_dt, nullptr,
                                               groups, s);
      void* ws = nullptr;
      if (hipMallocAsync(&ws, (size_t)ws_bytes, s) == hipSuccess) {
        const hipError_t e =
            launch_spmm_sk(values, meta, R, K, X, T, dt, Y, y_dt, ws, groups, s);
        const hipError_t f = hipFreeAsync(ws, s);
        return e != hipSuccess ? e : f;
      }
      (void)hipGetLastError();  // no workspace: the kernels below need none
    }
  }
  if (half && (pat24 || pat12) && sparse_shape) {
    const bool yf32 = y_dt == kF32;
#define NM_S(BF, P12)                                                                       \
  return yf32 ? run_smfmac_layout<BF, P12, kF32>(values, meta, R, K, blocked, X, T, Y, s)   \
              : run_smfmac_layout<BF, P12, (BF ? kBF16 : kF16)>(values, meta, R, K, blocked, X, \
                                                                T, Y, s);
    if (dt == kBF16) {
      if (pat24) { NM_S(true, false) } else { NM_S(true, true) }
    } else {
      if (pat24) { NM_S(false, false) } else { NM_S(false, true) }
    }
#undef NM_S
  }
  if (K == 0) {
    // empty contraction: Y = 0, written by a fill kernel (safe under stream capture)
    const int ybytes = (y_dt == kF32 || y_dt == kI32) ? 4 : 2;
    const int64_t words = R * T * ybytes / 4;
    const int64_t tail_halves = (R * T * ybytes % 4) / 2;
    zero_fill_kernel<<<(unsigned)((words + 255) / 256 + 1), 256, 0, s>>>(
        static_cast<uint32_t*>(Y), words, tail_halves);
    return hipGetLastError();
  }
  // the 8-bit matrix-core kernel: 2:4 and 1:2, either layout, K a multiple of 128 (two
  // blocked steps), T a multiple of 16 (16-byte X loads), 32-bit X offsets
  const bool tiled_8bit = (pat24 || pat12) && K % kI8KStep == 0 && T % 16 == 0 &&
                          R < (1 << 30) && T < (1 << 30) && K < (1 << 30);
#define NM_8(FP8, YT)                                                                     \
  return blocked ? (pat12 ? run_smfmac_8bit<FP8, true, true, YT>(values, meta, R, K, X, T, Y, s)  \
                          : run_smfmac_8bit<FP8, true, false, YT>(values, meta, R, K, X, T, Y, s)) \
                 : (pat12 ? run_smfmac_8bit<FP8, false, true, YT>(values, meta, R, K, X, T, Y, s) \
                          : run_smfmac_8bit<FP8, false, false, YT>(values, meta, R, K, X, T, Y, s));
  if (dt == kI8) {
    if (tiled_8bit) { NM_8(false, kI32) }
    // other patterns and shapes: the expansion kernel on the bf16 matrix cores, exact
    return run_expand_layout<kI8, kI32>(values, meta, R, K, n, m, blocked, X, T, Y, s);
  }
  if (dt == kFP8) {  // the same kernel on the fp8 instruction (fixed-point runs of 16 K)
    const bool yf32 = y_dt == kF32;
    if (tiled_8bit) {
      if (yf32) { NM_8(true, kF32) }
      NM_8(true, kBF16)
    }
#undef NM_8
    // other patterns and shapes: the expansion kernel, fp8 widened to bf16 (exact) and
    // summed in fp32 on the bf16 matrix cores
    return yf32 ? run_expand_layout<kFP8, kF32>(values, meta, R, K, n, m, blocked, X, T, Y, s)
                : run_expand_layout<kFP8, kBF16>(values, meta, R, K, n, m, blocked, X, T, Y, s);
  }
  // 16-bit and fp32 cases the kernels above do not take: the expansion kernel
  if (dt == kF32)
    return run_expand_layout<kF32, kF32>(values, meta, R, K, n, m, blocked, X, T, Y, s);
  if (dt == kBF16)
    return y_dt == kF32
               ? run_expand_layout<kBF16, kF32>(values, meta, R, K, n, m, blocked, X, T, Y, s)
               : run_expand_layout<kBF16, kBF16>(values, meta, R, K, n, m, blocked, X, T, Y, s);
  return y_dt == kF32
             ? run_expand_layout<kF16, kF32>(values, meta, R, K, n, m, blocked, X, T, Y, s)
             : run_expand_layout<kF16, kF16>(values, meta, R, K, n, m, blocked, X, T, Y, s);
}

#elif NM_SPMM_PART == 1

// The product with its epilogue on the matrix-core kernels above, X's rows of ep.ldx numbers in whole
// 16-byte pieces; what they do not take goes to the expansion kernel (launch_expand_act).
hipError_t launch_spmm_act(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n,
                           int m, bool blocked, const void* X, int64_t T, int dt, const Product& p,
                           hipStream_t s) {
  const Epilogue Y = epilogue_of(p);
  const bool pat24 = (n == 2 && m == 4), pat12 = (n == 1 && m == 2);
  const bool half = dt == kBF16 || dt == kF16, b = dt == kBF16;
  // sizes as launch_spmm
  const bool sparse_shape =
      K > 0 && K % kKStep == 0 && R < (1 << 30) && Y.ldx < (1 << 28) && K < (1 << 28);
  if (half && sparse_shape && n == 4 && m == 8) {
#define NM_48(BF, BL) return run_mfma48<BF, BL, kAct, 16>(values, meta, R, K, X, T, Y, s)
    if (b) {
      if (blocked) NM_48(true, true);
      NM_48(true, false);
    }
    if (blocked) NM_48(false, true);
    NM_48(false, false);
#undef NM_48
  }
  if (half && sparse_shape && (pat24 || pat12)) {
#define NM_S(BF, P12) return run_smfmac_layout<BF, P12, kAct>(values, meta, R, K, blocked, X, T, Y, s)
    if (b) {
      if (pat24) NM_S(true, false);
      NM_S(true, true);
    }
    if (pat24) NM_S(false, false);
    NM_S(false, true);
#undef NM_S
  }
  const bool tiled_8bit = (dt == kI8 || dt == kFP8) && (pat24 || pat12) && K > 0 &&
                          K % kI8KStep == 0 && R < (1 << 30) && Y.ldx < (1 << 30) && K < (1 << 30);
  if (tiled_8bit) {
#define NM_8(FP8, BL, P12) return run_smfmac_8bit<FP8, BL, P12, kAct>(values, meta, R, K, X, T, Y, s)
    if (dt == kFP8) {
      if (blocked) {
        if (pat12) NM_8(true, true, true);
        NM_8(true, true, false);
      }
      if (pat12) NM_8(true, false, true);
      NM_8(true, false, false);
    }
    if (blocked) {
      if (pat12) NM_8(false, true, true);
      NM_8(false, true, false);
    }
    if (pat12) NM_8(false, false, true);
    NM_8(false, false, false);
#undef NM_8
  }
  return launch_expand_act(values, meta, R, K, n, m, blocked, X, T, dt, p, s);
}

#else

hipError_t launch_expand_act(const void* values, const uint32_t* meta, int64_t R, int64_t K, int n,
                             int m, bool blocked, const void* X, int64_t T, int dt, const Product& p,
                             hipStream_t s) {
  const Epilogue Y = epilogue_of(p);
#define NM_E(DT)                                                                            \
  return blocked ? run_expand<DT, kAct, true, true>(values, meta, R, K, n, m, X, T, Y, s)   \
                 : run_expand<DT, kAct, false, true>(values, meta, R, K, n, m, X, T, Y, s)
  if (dt == kF32) NM_E(kF32);
  if (dt == kBF16) NM_E(kBF16);
  if (dt == kF16) NM_E(kF16);
  if (dt == kI8) NM_E(kI8);
  NM_E(kFP8);
#undef NM_E
}

#endif

}  // namespace nm
