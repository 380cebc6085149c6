// Grouped MXFP4 x MXFP4 GEMM for gfx950: the kernel template and its launcher.
//
//   C[r][n] = sum over blocks b of 2^(ea[r][b] + eb[n][b]) * sum_i qa[r][b,i] qb[n][b,i]
//
// v_mfma_scale_f32_32x32x64_f8f6f4 computes exactly this on the stored bytes: a lane holds
// the 32 codes (16 bytes) of one row's block and the block's E8M0 byte.  Nothing is decoded,
// so the kernel moves 0.53 bytes per operand element from HBM to the matrix unit.  A loop of
// this instruction alone reaches 8.1 PFLOP/s on this card (the 16x16x128 form 4.3).
//
// Operand roles.  With the rows of A (tokens) as the instruction's first operand a lane holds
// one output column of 16 tokens: FP32 and BF16 rows leave as 128- and 64-byte pieces.  Where
// the SwiGLU result is quantised (TRANS) the roles are swapped: a lane then holds 16 columns of
// one token, and weight row n of a 32-row fragment sits at the operand row that makes them
// consecutive (frag_row), so that an MX block is two lanes' registers.
//
// Data flow: HBM / L2 -> LDS by 16-byte DMA (stages of K = 128 or 256: 64 or 128 bytes of codes
// and 4 or 8 scale bytes per row, a ring of kStages) -> registers (16-byte LDS reads, one per
// lane and 64 K) -> MFMA.
//
// Pipeline.  Stage s of a tile lives in ring slot s mod kStages.  A stage is two or four K = 64
// steps; before its last step every wave waits for its own loads of the next stage, the
// workgroup meets, and the slot just read is refilled: with this tile's stage s + kStages, or, in the
// tile's last kStages stages, with the next tile's stage of that slot, so that loads run
// across tile ends and under the epilogue.  A step's operands are read while the step before
// multiplies, each weight fragment into the registers that the one just used leaves.  Every stage
// issues the same number of loads (a load with nothing to fetch has an offset behind the buffer)
// and every epilogue the same number of branch-free stores, so a wait counts exactly what may
// still be under way.
//
// Measured: 8192 x 8192 x 8192 3.3-3.5 PFLOP/s; 768 rows of 128 experts 43 us, 5.0 TB/s of weights.
// Gate and up of 131072 skewed rows of 128 experts (K 2048, N 768) 290 to 330 us with BF16 rows (by
// inputs and clock), 272 with the re-quantised result alone, 300 with both, 454 with it and FP32
// rows.  No unit is full there: by counters the matrix cores are busy for 34 % of the cycles (2.8 of
// the 8.1 PFLOP/s above), 0.69 GB are moved at 2.4 TB/s, and a wave waits for 40 % of its cycles,
// for the next stage's loads and at the barriers, with one other wave on its SIMD.
// With K = 768 a tile is three stages, and its stores bound it: loads return in order behind them, so
// the third stage waits for them (FP32 weight gradients of 64 experts, 403 MB: 105 us, 70 without
// stores).  More and shorter stages in the same LDS (four of K = 128 instead of two of 256, large
// tile) were slower throughout: weight gradients 115, BF16 rows of K = 768 60 for 55, gate and up
// 358 for 320, 8192 x 8192 x 8192 396 for 318.
#pragma once

#include <algorithm>
#include <type_traits>

#include "grouped_tiles.h"
#include "mx_device.h"
#include "mx_internal.h"
#include "nv4_internal.h"
#include "../../include/nv4moe.h"

namespace nv4 {
namespace {

// WAVES_M x WAVES_N waves of FM x FN 32 x 32 fragments; a ring of STAGES stages of STEPS K = 64
// steps each
template <int WAVES_M, int WAVES_N, int FM, int FN, int STEPS, int STAGES, int WAVES_PER_SIMD>
struct MxTile {
  static constexpr int kWavesM = WAVES_M, kWavesN = WAVES_N, kFM = FM, kFN = FN;
  static constexpr int kSteps = STEPS, kStages = STAGES, kWavesPerSimd = WAVES_PER_SIMD;
  static constexpr int NW = WAVES_M * WAVES_N, NT = NW * 64;
  static constexpr int BM = WAVES_M * FM * 32;  // rows of A (tokens)
  static constexpr int BN = WAVES_N * FN * 32;  // rows of B (weights)
  static constexpr int BK = STEPS * 64;
  static constexpr int kRow = STEPS * 32;        // code bytes of a row per stage
  static constexpr int kChunks = STEPS * 2;      // 16-byte chunks of them: one block each
  static constexpr int kDwords = STEPS / 2;      // scale dwords of a row per stage
  static constexpr int kCodes = (BM + BN) * kRow;
  static constexpr int kCodeRows = 1024 / kRow;  // rows of one code DMA (64 lanes x 16 bytes)
  static constexpr int kCodeBlocks = (BM + BN) / kCodeRows;
  static constexpr int kCodeDma = (kCodeBlocks + NW - 1) / NW;  // per wave; surplus ones load rows behind the tile
  static constexpr int kScaleRows = 64 / kDwords;  // rows of one scale DMA (64 lanes x 4 bytes)
  static constexpr int kScaleBlocks = (BM + BN + kScaleRows - 1) / kScaleRows;
  static constexpr int kScaleDma = (kScaleBlocks + NW - 1) / NW;
  static constexpr int kDma = kCodeDma + kScaleDma;  // the same for every wave
  // (room for the surplus DMAs of either kind)
  static constexpr int kScaleBase = NW * kCodeDma * 1024;
  static constexpr int kStageBytes = kScaleBase + NW * kScaleDma * 256;
  // tile rows whose codes, and whose scales, one wave loads: a lane looks one of each up
  static constexpr int kWaveCodeRows = kCodeDma * kCodeRows, kWaveScaleRows = kScaleDma * kScaleRows;
  static_assert(kWaveCodeRows <= 64 && kWaveScaleRows <= 64, "a lane for each row");
  static constexpr bool kSameRows = kWaveCodeRows == kWaveScaleRows;
  // The smallest tile is for a few rows per expert in the mean: then hardly another tile reads its
  // part of B, which is streamed past the caches and leaves them to A.  Cached -> streamed, eight
  // layers' weights in turn (128 experts, 1536 x 2048): 768 rows 49.2 -> 44.1 us, 4096 rows 48.7 ->
  // 44.4.  With uneven loads several tiles of an expert stream the same weights, and the gain
  // goes: one expert with two thirds of 768 rows 53.1 -> 50.8, with half of 4096 56.2 -> 54.7, 4096 rows
  // by Zipf's law (1.1) 55.8 -> 55.6.  One layer's weights again and again, which the 256 MB
  // cache would hold, lose by it: 37.5 -> 42.4, uneven 42.8 to 45.0 -> 49.8 to 54.4.
  static constexpr bool kStreamB = BM == 64;
  // every wave loads rows of one operand only
  static constexpr bool kOneSide = kSameRows && BN % kWaveCodeRows == 0 && BM % kWaveCodeRows == 0;
  static_assert(STEPS == 2 || STEPS == 4, "stages of K = 128 or 256");
  static_assert(BN % 64 == 0 && (BM + BN) % kCodeRows == 0, "DMA blocks of one operand");
};

// Ring position of chunk q of tile row r: the 16 rows of one LDS read pass cover all 64 banks
// (rows of 64 bytes: 4 to a bank sweep; of 128: 2).
template <class Cfg>
__device__ __forceinline__ int mx_swz(int q, int r) {
  return Cfg::kSteps == 2 ? q ^ ((r >> 2) & 3) : q ^ ((r >> 1) & 7);
}

// four code dwords as the instruction's operand (FP4 reads the first four of eight)
__device__ __forceinline__ i32x8 mx_operand(int4 v) { return i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0}; }

template <class Cfg, int GROUP, int EPI, bool OUT_F32, bool TRANS>
__global__ __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(Cfg::kWavesPerSimd)))
void k_mx_gemm(MxGemmArgs g) {
  constexpr int BM = Cfg::BM, BN = Cfg::BN, FM = Cfg::kFM, FN = Cfg::kFN, NT = Cfg::NT, S = Cfg::kStages;
  constexpr bool SWIGLU = EPI == NV4_EPI_SWIGLU;
  static_assert(!TRANS || SWIGLU, "the quantised result is the SwiGLU's");
  // the ring's slots are separate arrays and every access names its slot at compile time: the
  // compiler then knows that the reads of one slot do not depend on the loads into another
  __shared__ __attribute__((aligned(1024))) uint8_t ring0[Cfg::kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t ring1[Cfg::kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t ring2[S > 2 ? Cfg::kStageBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t ring3[S > 3 ? Cfg::kStageBytes : 16];
  static_assert(S >= 2 && S <= 4, "ring of 2 to 4 slots");
  __shared__ int tab[kMxMaxExperts + 1];
  __shared__ int off[kMxMaxExperts + 1];
  __shared__ int rows_c[Cfg::NW][64], rows_s[Cfg::kSameRows ? 1 : Cfg::NW][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Cfg::kWavesN, wn = wave % Cfg::kWavesN;
  const int h = lane >> 5, l32 = lane & 31;
  const int64_t ld = g.K / 2, sld = (g.K / kMxBlock + 3) / 4 * 4;
  const uint32_t a_bytes = (uint32_t)(g.a_rows * ld), a_sbytes = (uint32_t)(g.a_rows * sld);
  // B is addressed from the tile's expert, so that only one expert's part must stay below 4 GiB
  const int64_t b_rows = GROUP == NV4_GROUP_M ? (SWIGLU ? 2 : 1) * g.N : g.b_rows;
  const uint32_t b_bytes = (uint32_t)(b_rows * ld), b_sbytes = (uint32_t)(b_rows * sld);

  // ---- tile space (offsets below zero or decreasing are outside the contract: taken as empty)
  for (int e = tid; e <= g.E; e += NT) off[e] = std::max(g.offsets[e], 0);
  __syncthreads();
  MxTiles<Cfg, GROUP, EPI, MxGemmArgs> tiles{g, off, tab, 0, 0, 0, 0, 0, 0};
  tiles_setup(g, off, tab, reinterpret_cast<int *>(ring0), tiles);

  // ---- loads: this lane's byte offsets of the loading tile's rows (K offset not included)
  uint32_t off_c[Cfg::kCodeDma], off_s[Cfg::kScaleDma];
  const int qrow = lane / Cfg::kChunks, qpos = lane % Cfg::kChunks;    // row and ring position in a code DMA
  const int srow = lane / Cfg::kDwords, sdw = lane % Cfg::kDwords;     // row and dword in a scale DMA
  MxJob cj{};   // the tile being multiplied
  MxJob pj{};   // the loading tile: the same, and the next one towards its end
  bool p_live;  // there is one with at least one stage
  const bool gather = GROUP == NV4_GROUP_M && g.a_rows_index != nullptr;
  // Row indices of a tile come through LDS as well: each wave loads its lanes' own (a row of B
  // or none has the offset behind the buffer) well before they are needed.
  const auto load_index = [&](const MxJob &j) MX_INLINE {
    const auto one = [&](int r, int *dst) MX_INLINE {
      const int row = j.m0 + (r - BN);
      mx_dma4(g.a_rows_index, (uint32_t)g.M_cap * 4u, reinterpret_cast<uint8_t *>(dst),
              r >= BN && r < BN + BM && row < j.m_end ? (uint32_t)row * 4u : kNoRow);
    };
    one(wave * Cfg::kWaveCodeRows + lane, rows_c[wave]);
    if constexpr (!Cfg::kSameRows) one(wave * Cfg::kWaveScaleRows + lane, rows_s[wave]);
  };
  // operand row of tile row r, or -1; idx: what load_index brought
  const auto p_row = [&](int r, const int *idx) MX_INLINE -> int {
    int row = pj.m0 + (r - BN);
    row = r < BN + BM && row < pj.m_end ? row : -1;
    if (gather && row >= 0) row = min(max(mx_table(idx + lane), 0), (int)g.a_rows - 1);
    if (Cfg::kOneSide ? wave * Cfg::kWaveCodeRows < BN : r < BN) row = mx_b_row<Cfg, GROUP, EPI, TRANS>(g, pj, r);
    return row;
  };
  const uint8_t *b_codes = g.b_codes, *b_scales = g.b_scales;  // the expert's
  const auto p_setup = [&]() MX_INLINE {
    if (GROUP == NV4_GROUP_M) {
      const int64_t first = (int64_t)pj.e * b_rows;
      b_codes = g.b_codes + first * ld;
      b_scales = g.b_scales + first * sld;
    }
    const int mc = p_row(wave * Cfg::kWaveCodeRows + lane, rows_c[wave]);
    const int ms = Cfg::kSameRows ? mc : p_row(wave * Cfg::kWaveScaleRows + lane, rows_s[wave]);
#pragma unroll
    for (int i = 0; i < Cfg::kCodeDma; ++i) {
      const int in = i * Cfg::kCodeRows + qrow, row = __shfl(mc, in, 64);
      off_c[i] = row < 0 ? kNoRow
                         : (uint32_t)row * (uint32_t)ld +
                               (uint32_t)(mx_swz<Cfg>(qpos, wave * Cfg::kWaveCodeRows + in) * 16);
    }
#pragma unroll
    for (int i = 0; i < Cfg::kScaleDma; ++i) {
      const int row = __shfl(ms, i * Cfg::kScaleRows + srow, 64);
      off_s[i] = row < 0 ? kNoRow : (uint32_t)row * (uint32_t)sld + (uint32_t)(sdw * 4);
    }
  };
  // the loading tile becomes tile `it`, if there is one
  const auto p_next = [&](int it) MX_INLINE {
    p_live = tiles.has(it);
    if (p_live) pj = tiles.get(it);
    p_live = p_live && pj.nst > 0;
  };
  // one stage of the loading tile into a ring slot (live: there is such a stage)
  const auto load_stage = [&](uint8_t *dst, int p_st, bool live, bool of_next) MX_INLINE {
    const int k_lo = of_next ? pj.k_lo : cj.k_lo, k_len = of_next ? pj.k_len : cj.k_len;
    const uint32_t kc = (uint32_t)(k_lo + p_st * Cfg::BK) / 2, ks = kc / 16;
    const int left = live ? k_len - p_st * Cfg::BK : 0;  // elements of this stage (may exceed BK)
#pragma unroll
    for (int i = 0; i < Cfg::kCodeDma; ++i) {
      const int b = wave * Cfg::kCodeDma + i;
      const bool in_k = mx_swz<Cfg>(qpos, b * Cfg::kCodeRows + qrow) * 32 < left;
      // (saturating: without a row the sum stays behind the buffer)
      const uint32_t v = in_k ? __builtin_elementwise_add_sat(off_c[i], kc) : kNoRow;
      const bool isb = b * Cfg::kCodeRows < BN;
      if (isb) mx_dma16<Cfg::kStreamB>(b_codes, b_bytes, dst + b * 1024, v);
      else mx_dma16(g.a_codes, a_bytes, dst + b * 1024, v);
    }
#pragma unroll
    for (int i = 0; i < Cfg::kScaleDma; ++i) {
      const int b = wave * Cfg::kScaleDma + i;
      const uint32_t v = sdw * 128 < left ? __builtin_elementwise_add_sat(off_s[i], ks) : kNoRow;
      const bool isb = b * Cfg::kScaleRows < BN;
      mx_dma4(isb ? b_scales : g.a_scales, isb ? b_sbytes : a_sbytes, dst + Cfg::kScaleBase + b * 256, v);
    }
  };

  p_next(0);
  if (gather) {
    load_index(pj);
    mx_wait_vm<0>();
  }
  p_setup();
  load_stage(ring0, 0, p_live && 0 < pj.nst, true);
  load_stage(ring1, 1, p_live && 1 < pj.nst, true);
  if constexpr (S > 2) load_stage(ring2, 2, p_live && 2 < pj.nst, true);
  if constexpr (S > 3) load_stage(ring3, 3, p_live && 3 < pj.nst, true);

  // ---- fragments of one K = 64 step.  Lane half h takes the chunks h KS .. h KS + KS - 1 of a
  // stage's rows, one per step: their scale bytes are then bytes 0 .. KS - 1 of what one LDS
  // read of the lane gives (K is permuted alike for both operands).
  constexpr int KS = Cfg::kSteps;
  int4 wf[FN], tf[2][FM];
  uint32_t ws[FN] = {}, ts[FM] = {};
  const int w_row = wn * FN * 32 + l32, t_row = BN + wm * FM * 32 + l32;
  const auto chunk = [&](const uint8_t *st, int row, int step) MX_INLINE {
    // (rows of different fragments differ by multiples of 32: one swizzle)
    return *reinterpret_cast<const int4 *>(st + row * Cfg::kRow + mx_swz<Cfg>(h * KS + step, l32) * 16);
  };
  const auto scale = [&](const uint8_t *st, int row) MX_INLINE -> uint32_t {
    const uint8_t *p = st + Cfg::kScaleBase + row * (Cfg::kDwords * 4) + h * KS;
    if constexpr (KS == 4) return *reinterpret_cast<const uint32_t *>(p);
    else return *reinterpret_cast<const uint16_t *>(p);
  };
  const auto read_first = [&](const uint8_t *st) MX_INLINE {
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      tf[0][f] = chunk(st, t_row + f * 32, 0);
      ts[f] = scale(st, t_row + f * 32);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      wf[f] = chunk(st, w_row + f * 32, 0);
      ws[f] = scale(st, w_row + f * 32);
    }
  };

  f32x16 acc[FN][FM];
  const auto clear = [&]() MX_INLINE {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  };

  // ---- a finished tile (!TRANS: exactly kStores stores)
  constexpr int NF = SWIGLU ? FN / 2 : FN;  // 32-column fragments of the result
  constexpr int ESZ = OUT_F32 ? 4 : 2;
  constexpr int kStores = FM * NF * 16;
  const auto finish = [&](const MxJob &j) MX_INLINE {
    const int ncols = (int)(GROUP == NV4_GROUP_K ? g.b_rows : g.N);
    const int col_w = j.nt * (SWIGLU ? BN / 2 : BN) + wn * NF * 32;  // this wave's first column
    const int64_t row_w = (int64_t)j.m0 + wm * FM * 32;
    const int rows = (int)std::min<int64_t>(std::max<int64_t>(j.m_end - row_w, 0), FM * 32);
    const int ldc = (int)g.ldc;
    char *cb = static_cast<char *>(g.C) + ((GROUP == NV4_GROUP_K ? (int64_t)j.e * g.a_rows : 0) + row_w) * g.ldc * ESZ;
    if constexpr (!TRANS) {
      // lane = column l32 of a fragment; registers: rows 8 (r / 4) + 4 h + r % 4
      uint32_t voff[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const int col = col_w + f * 32 + l32;
        voff[f] = col < ncols ? (uint32_t)((h * 4 * ldc + col) * ESZ) : kNoStore;
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // rows r0 (lane half 0) and r0 + 4: a store behind the valid rows falls behind the
            // buffer
            const int r0 = i * 32 + g4 * 8 + q;
            const uint32_t nb = r0 + 4 < rows ? (uint32_t)(5 * ldc * ESZ) : r0 < rows ? (uint32_t)(ldc * ESZ) : 0u;
            void *rb = mx_uniform_ptr(cb + (int64_t)r0 * ldc * ESZ);
#pragma unroll
            for (int f = 0; f < NF; ++f) {
              float x = acc[f][i][g4 * 4 + q];
              if constexpr (SWIGLU) x = mx_swiglu(x, acc[f + NF][i][g4 * 4 + q]);
              if constexpr (OUT_F32) mx_store4(rb, nb, voff[f], __float_as_uint(x));
              else mx_store2(rb, nb, voff[f], __builtin_bit_cast(uint16_t, (__bf16)x));
            }
          }
        }
      }
    } else {
      // lane = token l32 of a fragment; registers: columns 16 h + r
      const int qld = ncols / 2, qsld = (int)((ncols / kMxBlock + 3) / 4 * 4);
      void *qc = mx_uniform_ptr(g.q_codes + row_w * qld), *qs = mx_uniform_ptr(g.q_scales + row_w * qsld);
      const uint32_t qcb = (uint32_t)(rows * qld), qsb = (uint32_t)(rows * qsld);
      void *cu = mx_uniform_ptr(cb);
      const uint32_t cub = g.C ? (uint32_t)(rows * ldc * ESZ) : 0u;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int rw = i * 32 + l32;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          float x[16];
          uint32_t m = 0;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            x[r] = mx_swiglu(acc[f][i][r], acc[f + NF][i][r]);
            m = max(m, __float_as_uint(x[r]) & 0x7FFFFFFFu);
          }
          const auto sm = __builtin_amdgcn_permlane32_swap(m, m, false, false);
          const uint32_t byte = mx_scale_byte(max(sm[0], sm[1]), g.ceil_rule);
          const float s = mx_scale_value(byte);
          uint32_t c[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            c[q] = mx_pack_f32<0>(c[q], x[8 * q], x[8 * q + 1], s);
            c[q] = mx_pack_f32<1>(c[q], x[8 * q + 2], x[8 * q + 3], s);
            c[q] = mx_pack_f32<2>(c[q], x[8 * q + 4], x[8 * q + 5], s);
            c[q] = mx_pack_f32<3>(c[q], x[8 * q + 6], x[8 * q + 7], s);
            if (byte == kMxNan) c[q] = 0;
          }
          const int col = col_w + f * 32;
          const bool live = rw < rows && col < ncols;  // N is a whole number of blocks here
          mx_store8(qc, qcb, live ? (uint32_t)(rw * qld + col / 2 + h * 8) : kNoStore, c[0], c[1]);
          mx_store1(qs, qsb, h == 0 && live ? (uint32_t)(rw * qsld + col / kMxBlock) : kNoStore, byte);
          if (col < ncols && col + kMxBlock >= ncols) {  // the last block: zeros up to the stride
            for (int b = col / kMxBlock + 1; b < qsld; ++b)
              mx_store1(qs, qsb, h == 0 && rw < rows ? (uint32_t)(rw * qsld + b) : kNoStore, 0u);
          }
          // 4-byte pieces: any row stride of C
          const uint32_t v = live ? (uint32_t)(rw * ldc + col + h * 16) * ESZ : kNoStore;
#pragma unroll
          for (int q = 0; q < 4 * ESZ; ++q) {
            if constexpr (OUT_F32) mx_store4(cu, cub, v + q * 4, __float_as_uint(x[q]));
            else
              mx_store4(cu, cub, v + q * 4,
                        __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[2 * q], (__bf16)x[2 * q + 1]}));
          }
        }
      }
    }
  };

  // ---- products
  // the products of weight fragment i in a step
  const auto multiply = [&](auto STEP, int i) MX_INLINE {
    constexpr int step = decltype(STEP)::value, p = step & 1;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      if (TRANS)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            mx_operand(wf[i]), mx_operand(tf[p][j]), acc[i][j], 4, 4, step, (int)ws[i], step, (int)ts[j]);
      else
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            mx_operand(tf[p][j]), mx_operand(wf[i]), acc[i][j], 4, 4, step, (int)ts[j], step, (int)ws[i]);
    }
    // Products stay where they are written.  (They touch no memory, so nothing else keeps the
    // compiler from reading every step's fragments first, for which the registers do not last.)
#pragma unroll
    for (int j = 0; j < FM; ++j) asm volatile("" : "+v"(acc[i][j]));
  };
  // A wave without rows of the tile only loads and keeps the barriers
  const auto idle = [&](auto P, int st, int p_st, bool live, bool of_next) MX_INLINE {
    constexpr int N = decltype(P)::value;
    if (st + 1 >= S) mx_wait_vm<(S - 2) * Cfg::kDma>();
    mx_barrier();
    load_stage(N == 0 ? ring0 : N == 1 ? ring1 : N == 2 ? ring2 : ring3, p_st, live, of_next);
  };
  // stage st of the tile; refills its slot with stage p_st of the loading tile
  const auto stage = [&](auto P, int st, int p_st, bool live, bool of_next) MX_INLINE {
    constexpr int N = decltype(P)::value;
    uint8_t *cur = N == 0 ? ring0 : N == 1 ? ring1 : N == 2 ? ring2 : ring3;
    constexpr int M = (N + 1) % S;
    const uint8_t *next = M == 0 ? ring0 : M == 1 ? ring1 : M == 2 ? ring2 : ring3;
    const auto step = [&](auto STEP) MX_INLINE {
      constexpr int s = decltype(STEP)::value;
#pragma unroll
      for (int f = 0; f < FM; ++f) tf[(s + 1) & 1][f] = chunk(cur, t_row + f * 32, s + 1);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        multiply(STEP, i);
        wf[i] = chunk(cur, w_row + i * 32, s + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    step(std::integral_constant<int, 0>{});
    if constexpr (KS == 4) {
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
    }
    // The last step: half of its products, then the stage is read, and the next one must have
    // landed for every wave.  The tile's first S stages have; behind them, S - 2 later stages'
    // loads may be under way.
    constexpr std::integral_constant<int, KS - 1> last{};
    constexpr int half = (FN + 1) / 2;
#pragma unroll
    for (int i = 0; i < half; ++i) multiply(last, i);
    mx_wait_lds();
    if (st + 1 >= S) mx_wait_vm<(S - 2) * Cfg::kDma>();
    mx_barrier();
    load_stage(cur, p_st, live, of_next);
#pragma unroll
    for (int f = 0; f < FM; ++f) tf[0][f] = chunk(next, t_row + f * 32, 0);
    uint32_t nw[FN], nt[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) nt[f] = scale(next, t_row + f * 32);
#pragma unroll
    for (int f = 0; f < FN; ++f) nw[f] = scale(next, w_row + f * 32);
#pragma unroll
    for (int i = 0; i < half; ++i) wf[i] = chunk(next, w_row + i * 32, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = half; i < FN; ++i) {
      multiply(last, i);
      wf[i] = chunk(next, w_row + i * 32, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) ts[f] = nt[f];
#pragma unroll
    for (int f = 0; f < FN; ++f) ws[f] = nw[f];
  };
#pragma unroll 1
  for (int it = 0; tiles.has(it); ++it) {
    cj = pj;
    clear();
    if (cj.nst > 0) {
      // the tile's first stages land: for this wave (behind them only the last tile's stores
      // may be under way; TRANS stores adjacent pieces, which the compiler may merge), then for
      // all
      if (it > 0 && !TRANS) mx_wait_vm<(kStores < 63 ? kStores : 63)>();
      else mx_wait_vm<0>();
      mx_barrier();
      p_next(it + 1);
      if (gather && p_live) load_index(pj);
      // An expert's last tile costs its rows rounded up to a wave's, not to a tile: the waves behind
      // them leave the matrix cores to the others (128 experts of 1024 rows, gate and up: 305 us if
      // they multiply too, 295 so).
      const auto run = [&](auto ACTIVE) MX_INLINE {
        // stages that refill their slot from this tile, then those that fill it from the next
        const int own = std::max(cj.nst - S, 0);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const int lo = part ? own : 0, hi = part ? cj.nst : own;
          if (part && p_live) {
            if (gather) {  // behind the indices: the loads of `own` stages
              if (own >= S - 1) mx_wait_vm<(S - 1) * Cfg::kDma>();
              else mx_wait_vm<0>();
            }
            p_setup();
          }
#pragma unroll 1
          for (int st = lo / S * S; st < hi; st += S) {
            const auto one = [&](auto P) MX_INLINE {
              constexpr int N = decltype(P)::value;
              const int s = st + N;
              if (N < S && s >= lo && s < hi) {
                const bool live = part == 0 || (p_live && N < pj.nst);
                if constexpr (decltype(ACTIVE)::value) stage(P, s, part ? N : s + S, live, part);
                else idle(P, s, part ? N : s + S, live, part);
              }
            };
            one(std::integral_constant<int, 0>{});
            one(std::integral_constant<int, 1>{});
            if constexpr (S > 2) one(std::integral_constant<int, 2>{});
            if constexpr (S > 3) one(std::integral_constant<int, 3>{});
          }
        }
      };
      if (GROUP == NV4_GROUP_K || cj.m0 + wm * FM * 32 < cj.m_end) {
        read_first(ring0);
        run(std::true_type{});
      } else {
        run(std::false_type{});
      }
      // a short tile did not use every slot
      if (cj.nst < S) {
        if (cj.nst <= 1) load_stage(ring1, 1, p_live && 1 < pj.nst, 1);
        if (S > 2 && cj.nst <= 2) load_stage(ring2, 2, p_live && 2 < pj.nst, 1);
        if (S > 3) load_stage(ring3, 3, p_live && 3 < pj.nst, 1);
      }
    } else {
      p_next(it + 1);
    }
    finish(cj);
  }
  mx_wait_vm<0>();  // loads into this workgroup's LDS end before it does
}

// persistent grid: whole multiples of the XCDs
template <class Cfg, int GROUP, int EPI>
hipError_t mx_launch(const MxGemmArgs &g, hipStream_t stream) {
  constexpr int cols = EPI == NV4_EPI_SWIGLU ? Cfg::BN / 2 : Cfg::BN;
  int64_t tiles;
  if (GROUP == NV4_GROUP_M) {
    if (g.M_cap == 0) return hipSuccess;
    tiles = (g.M_cap / Cfg::BM + std::min<int64_t>(g.E, g.M_cap)) * ((g.N + cols - 1) / cols);
  } else {
    tiles = (int64_t)g.E * ((g.a_rows + Cfg::BM - 1) / Cfg::BM) * ((g.b_rows + Cfg::BN - 1) / Cfg::BN);
    if (tiles == 0) return hipSuccess;
  }
  const int lds = Cfg::kStages * Cfg::kStageBytes + (kMxMaxExperts + 1) * 8 + Cfg::NW * 512;
  const int per_cu = std::max(1, std::min(160 * 1024 / lds, Cfg::kWavesPerSimd * 4 / Cfg::NW));
  const int64_t most = (int64_t)device_cu_count() * per_cu;
  const unsigned grid = (unsigned)std::min<int64_t>((tiles + kMxXcds - 1) / kMxXcds * kMxXcds, most);
  if constexpr (EPI == NV4_EPI_SWIGLU) {
    if (g.q_codes) {
      if (g.c_is_f32) k_mx_gemm<Cfg, GROUP, EPI, true, true><<<grid, Cfg::NT, 0, stream>>>(g);
      else k_mx_gemm<Cfg, GROUP, EPI, false, true><<<grid, Cfg::NT, 0, stream>>>(g);
      return hipGetLastError();
    }
  }
  if (g.c_is_f32) k_mx_gemm<Cfg, GROUP, EPI, true, false><<<grid, Cfg::NT, 0, stream>>>(g);
  else k_mx_gemm<Cfg, GROUP, EPI, false, false><<<grid, Cfg::NT, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace
}  // namespace nv4
