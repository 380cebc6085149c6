// Grouped FP8 x FP8 GEMM for gfx950: the kernel template and its launcher.
//
//   C[r][n] = sum over blocks b of Ga[r][b] Gb[n][b] * sum_i qa[r][b,i] qb[n][b,i]
//
// The matrix unit gives the inner sum of a 32 x 32 fragment over one block of 128, and sixteen FP32
// multiply-adds a lane scale and collect it.  The weights are the instruction's first operand: a lane
// holds 16 columns of one token, whose scale is then the lane's, and the weights' scale (one for 128 x
// 128) the whole wave's.  Weight row n of a fragment sits at the operand row that makes a lane's columns
// consecutive (frag_row).
//
// Two ways to the inner sum, by the type that the result leaves in:
//   BF16 and FP8 results: v_mfma_f32_32x32x64_f8f6f4 on the codes as they are.  It adds products in groups of
//     eight, aligned to the largest of them and cut off 13 bits below its exponent, and the groups in FP32
//     (measured: a product 2^-13 of its group's largest counts, one of 2^-14 does not, and in another group any
//     does).  The error is 1.5e-5 of the result's norm on normal inputs and at most 7 * 2^-13 of the sum of
//     |products|: a hundredth of BF16's rounding, and less beside that of the codes.
//   FP32 results: v_mfma_f32_32x32x16_f16 on the codes converted to FP16, which holds E4M3 exactly: exact
//     products and FP32 sums, at half the rate.
#pragma once

#include <algorithm>
#include <type_traits>

#include "f8_device.h"
#include "f8_internal.h"
#include "grouped_tiles.h"
#include "nv4_internal.h"
#include "../../include/nv4moe.h"

namespace nv4 {
namespace {

// WAVES_M x WAVES_N waves of FM x FN 32 x 32 fragments, stages of one block (K = 128)
template <int WAVES_M, int WAVES_N, int FM, int FN>
struct F8Tile {
  static constexpr int kWavesM = WAVES_M, kWavesN = WAVES_N, kFM = FM, kFN = FN;
  static constexpr int NW = WAVES_M * WAVES_N, NT = NW * 64;
  static constexpr int BM = WAVES_M * FM * 32;  // rows of A (tokens)
  static constexpr int BN = WAVES_N * FN * 32;  // rows of B (weights)
  static constexpr int BK = 128;
  static constexpr int kRows = BM + BN;
  static constexpr int kCodeDma = kRows / 8 / NW;  // 1 KB each: 8 rows of 128 bytes
  static constexpr int kScaleDma = (kRows / 64 + NW - 1) / NW;
  static constexpr int kStageBytes = kRows * 128;
  static_assert(kRows % (8 * NW) == 0 && BN % 64 == 0 && BM % 64 == 0, "DMA blocks of one operand");
};

// ring position of 16-byte chunk q of tile row r: the rows of one LDS read pass cover all banks
__device__ __forceinline__ int f8_swz(int q, int r) { return q ^ ((r >> 1) & 7); }

// A lane's 64 codes of one row and block, as the instruction's operands.  (The order of K is the same for both
// operands, whatever it is.)
template <bool WIDE>
struct F8Frag {
  i32x8 v[2];
  __device__ __forceinline__ void set(int4 a, int4 b, int4 c, int4 d) {
    v[0] = i32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    v[1] = i32x8{c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
  }
};
__device__ __forceinline__ f16x8 f8_to_f16(int lo, int hi) {
  const f16x2 a = e4m3x2_to_f16(lo), b = e4m3x2_to_f16<true>(lo), c = e4m3x2_to_f16(hi), d = e4m3x2_to_f16<true>(hi);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
template <>
struct F8Frag<true> {
  f16x8 v[8];
  __device__ __forceinline__ void set(int4 a, int4 b, int4 c, int4 d) {
    v[0] = f8_to_f16(a.x, a.y), v[1] = f8_to_f16(a.z, a.w), v[2] = f8_to_f16(b.x, b.y), v[3] = f8_to_f16(b.z, b.w);
    v[4] = f8_to_f16(c.x, c.y), v[5] = f8_to_f16(c.z, c.w), v[6] = f8_to_f16(d.x, d.y), v[7] = f8_to_f16(d.z, d.w);
  }
};
__device__ __forceinline__ f32x16 f8_product(const F8Frag<false> &w, const F8Frag<false> &t) {
  f32x16 p = {};
  p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w.v[0], t.v[0], p, 0, 0, 0, 0, 0, 0);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w.v[1], t.v[1], p, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16 f8_product(const F8Frag<true> &w, const F8Frag<true> &t) {
  f32x16 p = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) p = __builtin_amdgcn_mfma_f32_32x32x16_f16(w.v[i], t.v[i], p, 0, 0, 0);
  return p;
}

template <class Cfg, int GROUP, int EPI, bool OUT_F32, bool QUANT>
__global__ __launch_bounds__(Cfg::NT) void k_f8_gemm(F8GemmArgs g) {
  constexpr int BM = Cfg::BM, BN = Cfg::BN, FM = Cfg::kFM, FN = Cfg::kFN, NT = Cfg::NT;
  constexpr bool SWIGLU = EPI == NV4_EPI_SWIGLU;
  constexpr bool K_GROUPS = GROUP == NV4_GROUP_K;
  constexpr int NF = SWIGLU ? FN / 2 : FN;  // 32-column fragments of the result
  constexpr int ESZ = OUT_F32 ? 4 : 2;
  static_assert(!QUANT || (SWIGLU && BN == 256), "a quantised block is the tile's 128 result columns");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[Cfg::kStageBytes];
  __shared__ __attribute__((aligned(256))) float ring_s[Cfg::NW * Cfg::kScaleDma * 64];
  __shared__ int tab[kMxMaxExperts + 1];
  __shared__ int off[kMxMaxExperts + 1];
  __shared__ uint32_t s_max[QUANT ? Cfg::kWavesN : 1][QUANT ? BM : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Cfg::kWavesN, wn = wave % Cfg::kWavesN;
  const int h = lane >> 5, l32 = lane & 31;
  const int64_t kb = (g.K + 127) / 128;
  const uint32_t ld = (uint32_t)g.K, sld = (uint32_t)kb * 4;
  // B is addressed from the tile's expert, so that only one expert's part must stay below 4 GiB
  const int64_t b_rows = K_GROUPS ? g.b_rows : (SWIGLU ? 2 : 1) * g.N;
  const int64_t b_srows = K_GROUPS ? g.b_rows : (b_rows + 127) / 128;
  const uint32_t a_bytes = (uint32_t)(g.a_rows * g.K), a_sbytes = (uint32_t)(g.a_rows * sld);
  const uint32_t b_bytes = (uint32_t)(b_rows * g.K), b_sbytes = (uint32_t)(b_srows * sld);

  // ---- tile space (offsets below zero or decreasing are outside the contract: taken as empty)
  for (int e = tid; e <= g.E; e += NT) off[e] = std::max(g.offsets[e], 0);
  __syncthreads();
  MxTiles<Cfg, GROUP, EPI, F8GemmArgs> tiles{g, off, tab, 0, 0, 0, 0, 0, 0};
  tiles_setup(g, off, tab, reinterpret_cast<int *>(ring), tiles);

#pragma unroll 1
  for (int it = 0; tiles.has(it); ++it) {
    MxJob j = tiles.get(it);
    if (K_GROUPS && j.k_len > 0) {  // whole blocks
      const int hi = j.k_lo + j.k_len;
      j.k_lo &= ~127;
      j.nst = (hi - j.k_lo + 127) / 128;
    }
    const int64_t first = K_GROUPS ? 0 : (int64_t)j.e * b_rows;
    const uint8_t *b_codes = g.b_codes + first * g.K;
    const float *b_scales = g.b_scales + (K_GROUPS ? 0 : (int64_t)j.e * b_srows * kb);
    const auto a_row = [&](int r) MX_INLINE -> int {  // A row of tile row r (behind the weights), or -1
      int row = j.m0 + r - BN;
      if (row >= j.m_end) return -1;
      if (!K_GROUPS && g.a_rows_index) row = min(max(g.a_rows_index[row], 0), (int)g.a_rows - 1);
      return row;
    };
    uint32_t off_c[Cfg::kCodeDma], off_s[Cfg::kScaleDma];
#pragma unroll
    for (int i = 0; i < Cfg::kCodeDma; ++i) {
      const int r = (wave * Cfg::kCodeDma + i) * 8 + (lane >> 3);
      const int row = r < BN ? mx_b_row<Cfg, GROUP, EPI, true>(g, j, r) : a_row(r);
      off_c[i] = row < 0 ? kNoRow : (uint32_t)row * ld + (uint32_t)(f8_swz(lane & 7, r) * 16);
    }
#pragma unroll
    for (int i = 0; i < Cfg::kScaleDma; ++i) {
      const int r = (wave * Cfg::kScaleDma + i) * 64 + lane;
      int row = r < BN ? mx_b_row<Cfg, GROUP, EPI, true>(g, j, r) : r < BN + BM ? a_row(r) : -1;
      if (!K_GROUPS && r < BN && row >= 0) row >>= 7;
      off_s[i] = row < 0 ? kNoRow : (uint32_t)row * sld;
    }
    f32x16 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][f][r] = 0.0f;
    for (int st = 0; st < j.nst; ++st) {
      const uint32_t k0 = (uint32_t)(j.k_lo + st * 128);
      __syncthreads();  // the last stage has been read
#pragma unroll
      for (int i = 0; i < Cfg::kCodeDma; ++i) {
        const int b = wave * Cfg::kCodeDma + i;
        const bool in_k = k0 + f8_swz(lane & 7, b * 8 + (lane >> 3)) * 16 < (uint32_t)g.K;
        const uint32_t v = in_k ? __builtin_elementwise_add_sat(off_c[i], k0) : kNoRow;
        if (b * 8 < BN) mx_dma16(b_codes, b_bytes, ring + b * 1024, v);
        else mx_dma16(g.a_codes, a_bytes, ring + b * 1024, v);
      }
#pragma unroll
      for (int i = 0; i < Cfg::kScaleDma; ++i) {
        const int b = wave * Cfg::kScaleDma + i;
        const uint32_t v = __builtin_elementwise_add_sat(off_s[i], k0 / 128 * 4);
        if (b * 64 < BN) mx_dma4(b_scales, b_sbytes, reinterpret_cast<uint8_t *>(ring_s + b * 64), v);
        else mx_dma4(g.a_scales, a_sbytes, reinterpret_cast<uint8_t *>(ring_s + b * 64), v);
      }
      mx_wait_vm<0>();
      __syncthreads();
      const auto operand = [&](int row) MX_INLINE {
        const auto chunk = [&](int q) MX_INLINE {
          return *reinterpret_cast<const int4 *>(ring + row * 128 + f8_swz(h * 4 + q, row) * 16);
        };
        F8Frag<OUT_F32> f;
        f.set(chunk(0), chunk(1), chunk(2), chunk(3));
        return f;
      };
      F8Frag<OUT_F32> tf[FM];
      float sa[FM];
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const int row = BN + (wm * FM + f) * 32 + l32;
        tf[f] = operand(row);
        sa[f] = ring_s[row];
      }
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int row0 = (wn * FN + i) * 32;
        const F8Frag<OUT_F32> w = operand(row0 + l32);
#pragma unroll
        for (int f = 0; f < FM; ++f) {
          const f32x16 p = f8_product(w, tf[f]);
          const float s = sa[f] * ring_s[row0];
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            // register r: weight row 8 (r / 4) + 4 h + r % 4 of the operand, column 16 h + r of the result
            const float sr = K_GROUPS ? sa[f] * ring_s[row0 + 8 * (r / 4) + 4 * h + r % 4] : s;
            acc[i][f][r] = __builtin_fmaf(p[r], sr, acc[i][f][r]);
          }
        }
      }
    }

    // ---- epilogue: lane = row l32 of a fragment, registers = columns 16 h + r
    const int ncols = (int)(K_GROUPS ? g.b_rows : g.N);
    const int col_w = j.nt * (SWIGLU ? BN / 2 : BN) + wn * NF * 32;
    const int64_t row_w = (int64_t)j.m0 + wm * FM * 32;
    const int rows = (int)std::min<int64_t>(std::max<int64_t>(j.m_end - row_w, 0), FM * 32);
    if constexpr (SWIGLU) {
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][f][r] = mx_swiglu(acc[i][f][r], acc[i + NF][f][r]);
    }
    if (!QUANT || g.C) {
      char *cb = static_cast<char *>(g.C) + ((K_GROUPS ? (int64_t)j.e * g.a_rows : 0) + row_w) * g.ldc * ESZ;
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const int rw = f * 32 + l32;
        if (rw >= rows) continue;
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          const int col = col_w + i * 32 + h * 16;
          char *p = cb + ((int64_t)rw * g.ldc + col) * ESZ;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            if (col + r >= ncols) continue;
            if constexpr (OUT_F32) reinterpret_cast<float *>(p)[r] = acc[i][f][r];
            else reinterpret_cast<__bf16 *>(p)[r] = (__bf16)acc[i][f][r];
          }
        }
      }
    }
    if constexpr (QUANT) {
      // a row's block is the tile's 128 columns: NF * 32 of them in each of the waves beside this one
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            m = max(m, col_w + i * 32 < ncols ? __float_as_uint(acc[i][f][r]) & 0x7FFFFFFFu : 0u);
        const auto sm = __builtin_amdgcn_permlane32_swap(m, m, false, false);
        if (h == 0) s_max[wn][(wm * FM + f) * 32 + l32] = max(sm[0], sm[1]);
      }
      __syncthreads();
      const int64_t qkb = (ncols + 127) / 128;
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const int rw = f * 32 + l32;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < Cfg::kWavesN; ++w) m = max(m, s_max[w][(wm * FM + f) * 32 + l32]);
        const F8Scale s = f8_scale(m, g.q_pow2);
        if (rw < rows) {
#pragma unroll
          for (int i = 0; i < NF; ++i) {
            const int col = col_w + i * 32 + h * 16;
            uint32_t c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              c[q] = s.bad ? 0u : f8_pack4(acc[i][f][4 * q], acc[i][f][4 * q + 1], acc[i][f][4 * q + 2], acc[i][f][4 * q + 3], s.S);
            if (col < ncols)
              *reinterpret_cast<uint4 *>(g.q_codes + (row_w + rw) * ncols + col) = make_uint4(c[0], c[1], c[2], c[3]);
          }
          if (wn == 0 && h == 0) g.q_scales[(row_w + rw) * qkb + j.nt] = s.G;
        }
      }
    }
  }
}

// persistent grid: whole multiples of the XCDs
template <class Cfg, int GROUP, int EPI>
hipError_t f8_launch(const F8GemmArgs &g, hipStream_t stream) {
  constexpr int cols = EPI == NV4_EPI_SWIGLU ? Cfg::BN / 2 : Cfg::BN;
  int64_t tiles;
  if (GROUP == NV4_GROUP_M) {
    if (g.M_cap == 0) return hipSuccess;
    tiles = (g.M_cap / Cfg::BM + std::min<int64_t>(g.E, g.M_cap)) * ((g.N + cols - 1) / cols);
  } else {
    tiles = (int64_t)g.E * ((g.a_rows + Cfg::BM - 1) / Cfg::BM) * ((g.b_rows + Cfg::BN - 1) / Cfg::BN);
    if (tiles == 0) return hipSuccess;
  }
  const int64_t most = (int64_t)device_cu_count() * 2;
  const unsigned grid = (unsigned)std::min<int64_t>((tiles + kMxXcds - 1) / kMxXcds * kMxXcds, most);
  if constexpr (EPI == NV4_EPI_SWIGLU && Cfg::BN == 256) {
    if (g.q_codes) {
      if (g.c_is_f32) k_f8_gemm<Cfg, GROUP, EPI, true, true><<<grid, Cfg::NT, 0, stream>>>(g);
      else k_f8_gemm<Cfg, GROUP, EPI, false, true><<<grid, Cfg::NT, 0, stream>>>(g);
      return hipGetLastError();
    }
  }
  if (g.c_is_f32) k_f8_gemm<Cfg, GROUP, EPI, true, false><<<grid, Cfg::NT, 0, stream>>>(g);
  else k_f8_gemm<Cfg, GROUP, EPI, false, false><<<grid, Cfg::NT, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace
}  // namespace nv4
