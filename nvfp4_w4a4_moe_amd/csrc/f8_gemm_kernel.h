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
//
// Power-of-two scales on both operands go into the scaled instruction (v_mfma_scale_f32_32x32x64_f8f6f4 takes an
// exponent byte for each row), which then adds onto the accumulators itself.
//
// Pipeline.  Codes and scales come to LDS by DMA, in stages of one block, into a ring of kStages slots.  The
// stages of all of a workgroup's tiles are one sequence: the loads run kStages ahead of the products, across
// tile ends and under the epilogue.  A wave takes a stage's token fragments into registers and then
// one weight fragment after the other, the next one's LDS reads under way.  Before the last weight
// fragment's products every wave waits for its own loads of the next stage, the workgroup meets, and the
// slot just read is refilled.  Every stage issues the same number of loads (a load with nothing to fetch has
// an offset behind the buffer), so a wait counts exactly what may still be under way.
//
// 8192^3: 550 us or 1990 TFLOP/s, power-of-two scales 2090, FP32 results 1170.  Gate and up of 131072 rows with SwiGLU
// (128 experts, K 2048, 768 columns): 444 to 454 us, 1830 TFLOP/s.  What bounds it: MFMA is
// busy 44 % of the cycles, the VALU (the sums' multiply-adds, addresses) 45 %, hardly both at once, and LDS reads 24
// KB for 16 MFMA of a wave, as long as they take.
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

// WAVES_M x WAVES_N waves of FM x FN 32 x 32 fragments; a ring of STAGES stages of one block (K = 128).  ANY_ROWS: made
// for rows of C that start between lines too, which takes registers.
template <int WAVES_M, int WAVES_N, int FM, int FN, int STAGES, int WAVES_PER_SIMD, bool ANY_ROWS = (FM * FN < 8)>
struct F8Tile {
  static constexpr int kWavesM = WAVES_M, kWavesN = WAVES_N, kFM = FM, kFN = FN;
  static constexpr int kStages = STAGES, kWavesPerSimd = WAVES_PER_SIMD;
  static constexpr bool kAnyRows = ANY_ROWS;
  static constexpr int NW = WAVES_M * WAVES_N, NT = NW * 64;
  static constexpr int BM = WAVES_M * FM * 32;  // rows of A (tokens)
  static constexpr int BN = WAVES_N * FN * 32;  // rows of B (weights)
  static constexpr int BK = 128;
  static constexpr int kRows = BM + BN;
  static constexpr int kCodeDma = kRows / 8 / NW;                // per wave, 1 KB each: 8 rows of 128 bytes
  static constexpr int kScaleDma = (kRows + 64 * NW - 1) / (64 * NW);  // per wave, 64 rows of 4 bytes each
  static constexpr int kDma = kCodeDma + kScaleDma;              // the same for every wave
  static constexpr int kScaleBase = kRows * 128;
  static constexpr int kStageBytes = kScaleBase + NW * kScaleDma * 256;
  static constexpr int kDmaB = BN / 8 / NW;  // the first of a wave's code DMAs, which fetch weights
  static constexpr int kLook = (kCodeDma * 8 + 63) / 64;  // rows of its code DMAs that a lane looks up
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BN % 64 == 0, "DMAs of one operand");
  // The smallest tile is for a few rows per expert in the mean: hardly another tile reads its part of B, which
  // is streamed past the caches.
  static constexpr bool kStreamB = BM <= 64;
};

// LDS DMA as mx_dma16 and mx_dma4, in assembly: a builtin's load into the ring makes the compiler wait for every load
// in flight before the next LDS read that it cannot tell apart from it, which is most of them (the waits and
// barriers here are placed by hand).  lds: the wave's LDS byte address.  No register is written but m0, which
// nothing else in these kernels uses (the compiler takes it for its own: it can't be named as clobbered).
// A buffer load may read a scalar register five wait states after a vector instruction has written it, and the
// operands here often come straight from a lane read, where scalars are kept: the compiler puts such waits before loads
// of its own only, so m0's move and the nop are five (8192 x 2048 x 768 22.1 -> 22.9 us, 131072 rows of gate and up 436 ->
// 444).
__device__ __forceinline__ i32x4 f8_buffer(const void *base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return i32x4{(int)p, (int)(p >> 32) & 0xFFFF, (int)bytes, 0x00020000};
}
template <bool STREAM>
__device__ __forceinline__ void f8_dma16(i32x4 buffer, uint32_t lds, uint32_t voff, uint32_t soff) {
  if (STREAM)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(lds), "v"(voff),
                 "s"(buffer), "s"(soff)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                 "s"(buffer), "s"(soff)
                 : "memory");
}
__device__ __forceinline__ void f8_dma4(i32x4 buffer, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
               "s"(buffer), "s"(soff)
               : "memory");
}
__device__ __forceinline__ uint32_t f8_lds(const void *p) {
  return __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)static_cast<const uint8_t *>(p));
}

template <class T>
__device__ __forceinline__ const __attribute__((address_space(3))) T *f8_lds_ptr(uint32_t at) {
  return (const __attribute__((address_space(3))) T *)(uintptr_t)at;
}

constexpr int kQueue = 8;  // tiles between the loads and the products, and the one being multiplied

// ring position of 16-byte chunk q of tile row r: the rows of one LDS read pass cover all banks
__device__ __forceinline__ int f8_swz(int q, int r) { return q ^ ((r >> 1) & 7); }

// a lane's 64 codes of one row and block
struct F8Raw {
  i32x4 c[4];
};
// They as the instruction's operands.  (The order of K is the same for both
// operands, whatever it is.)
template <bool WIDE>
struct F8Frag {
  i32x8 v[2];
  __device__ __forceinline__ void set(const F8Raw &r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const i32x4 a = r.c[2 * i], b = r.c[2 * i + 1];
      v[i] = i32x8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
  }
};
template <>
struct F8Frag<true> {
  f16x8 v[8];
  __device__ __forceinline__ void set(const F8Raw &r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = f8_to_f16(r.c[i].x, r.c[i].y);
      v[2 * i + 1] = f8_to_f16(r.c[i].z, r.c[i].w);
    }
  }
};
typedef uint32_t f8_u32x4 __attribute__((ext_vector_type(4)));
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

// Transposes 16-byte pieces in groups of G lanes: piece k of lane i becomes piece i of lane k.
template <int G>
__device__ __forceinline__ void f8_exchange(f8_u32x4 (&c)[G], int lane) {
#pragma unroll
  for (int bit = 1; bit < G; bit *= 2) {
    const bool odd = lane & bit;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      if (k & bit) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t x = c[k][r], y = c[k + bit][r];
        // the neighbour's: lane ^ 1 (quad_perm [1,0,3,2]) or lane ^ 2 ([2,3,0,1])
        const uint32_t nx = (uint32_t)(bit == 1 ? __builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false)
                                                : __builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false));
        const uint32_t ny = (uint32_t)(bit == 1 ? __builtin_amdgcn_mov_dpp((int)y, 0xB1, 0xF, 0xF, false)
                                                : __builtin_amdgcn_mov_dpp((int)y, 0x4E, 0xF, 0xF, false));
        c[k][r] = odd ? ny : x;
        c[k + bit][r] = odd ? y : nx;
      }
    }
  }
}

template <class Cfg, int GROUP, int EPI, bool OUT_F32, bool QUANT, bool POW2>
__global__ __launch_bounds__(Cfg::NT) __attribute__((amdgpu_waves_per_eu(Cfg::kWavesPerSimd)))
void k_f8_gemm(F8GemmArgs g) {
  constexpr int BM = Cfg::BM, BN = Cfg::BN, FM = Cfg::kFM, FN = Cfg::kFN, NT = Cfg::NT, S = Cfg::kStages;
  constexpr bool SWIGLU = EPI == NV4_EPI_SWIGLU, K_GROUPS = GROUP == NV4_GROUP_K;
  constexpr int NF = SWIGLU ? FN / 2 : FN;  // 32-column fragments of the result
  constexpr int ESZ = OUT_F32 ? 4 : 2;
  static_assert(!QUANT || (SWIGLU && BN == 256), "a quantised block is the tile's 128 result columns");
  static_assert(!SWIGLU || FN % 2 == 0, "a wave's gate fragments and their up fragments");
  static_assert(!POW2 || !OUT_F32, "FP32 results take the converted codes");
  static_assert(S >= 2 && S < kQueue && (S - 1) * Cfg::kDma < 64, "ring of a few slots");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[S * Cfg::kStageBytes];
  __shared__ int tab[kMxMaxExperts + 1];
  __shared__ int off[kMxMaxExperts + 1];
  __shared__ int rows_c[Cfg::NW][Cfg::kLook * 64], rows_s[Cfg::NW][Cfg::kScaleDma * 64];
  __shared__ int4 jobs[Cfg::NW][kQueue];
  __shared__ uint32_t s_max[QUANT ? Cfg::kWavesN : 1][QUANT ? BM : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Cfg::kWavesN, wn = wave % Cfg::kWavesN;
  const int h = lane >> 5, l32 = lane & 31;
  const int64_t kb = (g.K + 127) / 128;
  const uint32_t ld = (uint32_t)g.K, sld = (uint32_t)kb * 4;
  const uint32_t a_bytes = (uint32_t)(g.a_rows * g.K), a_sbytes = (uint32_t)(g.a_rows * sld);
  // B is addressed from the tile's expert, so that only one expert's part must stay below 4 GiB
  const int64_t b_rows = K_GROUPS ? g.b_rows : (SWIGLU ? 2 : 1) * g.N;
  const int64_t b_srows = K_GROUPS ? g.b_rows : (b_rows + 127) / 128;
  const uint32_t b_bytes = (uint32_t)(b_rows * g.K), b_sbytes = (uint32_t)(b_srows * sld);

  // ---- tile space (offsets below zero or decreasing are outside the contract: taken as empty; behind the last row: as
  // that)
  const int most = K_GROUPS ? (int)g.K : (int)g.M_cap;
  for (int e = tid; e <= g.E; e += NT) off[e] = std::min(std::max(g.offsets[e], 0), most);
  __syncthreads();
  MxTiles<Cfg, GROUP, EPI, F8GemmArgs> tiles{g, off, tab, 0, 0, 0, 0, 0, 0};
  tiles_setup(g, off, tab, reinterpret_cast<int *>(ring), tiles);
  // ---- loads: this lane's byte offsets of the loading tile's rows (K offset not included).  Without a tile there are none.
  uint32_t off_c[Cfg::kCodeDma], off_s[Cfg::kScaleDma];
#pragma unroll
  for (int i = 0; i < Cfg::kCodeDma; ++i) off_c[i] = kNoRow;
#pragma unroll
  for (int l = 0; l < Cfg::kScaleDma; ++l) off_s[l] = kNoRow;
  const int qrow = lane >> 3, qpos = lane & 7;  // row and ring position in a code DMA
  static_assert(Cfg::NW % 2 == 0, "the chunk there is the same in all of a wave's");
  const int chunk = f8_swz(qpos, wave * 8 + qrow);
  MxJob pj{};     // the loading tile (the loads are up to kStages tiles ahead of the products, and leave them here)
  int4(&queue)[kQueue] = jobs[wave];
  int p_it = -1;  // its number in this workgroup's sequence
  int p_st = 0;   // its next stage
  bool p_live = true;  // there is one
  bool primed = false;
  const bool gather = !K_GROUPS && g.a_rows_index != nullptr;
  // Block b of eight tile rows is wave b % NW's code DMA b / NW; 64 rows' scales are one DMA.  The rows that this lane
  // looks up, 64 at a time (the last ones may lie behind the tile):
  const auto code_row = [&](int l) MX_INLINE { return ((l * 8 + qrow) * Cfg::NW + wave) * 8 + qpos; };
  const auto scale_row = [&](int l) MX_INLINE { return (wave * Cfg::kScaleDma + l) * 64 + lane; };
  // Row indices of a tile come through LDS as well: each wave loads its lanes' own (a row of B
  // or none has the offset behind the buffer) well before they are needed.
  const auto load_index = [&](const MxJob &j) MX_INLINE {
    const auto one = [&](int r, int *dst) MX_INLINE {
      const int row = j.m0 + (r - BN);
      f8_dma4(f8_buffer(g.a_rows_index, (uint32_t)g.M_cap * 4u), f8_lds(dst),
              r >= BN && r < BN + BM && row < j.m_end ? (uint32_t)row * 4u : kNoRow, 0);
    };
#pragma unroll
    for (int l = 0; l < Cfg::kLook; ++l) one(code_row(l), rows_c[wave] + l * 64);
#pragma unroll
    for (int l = 0; l < Cfg::kScaleDma; ++l) one(scale_row(l), rows_s[wave] + l * 64);
  };
  // operand row of tile row r, or -1; idx: what load_index brought
  const auto p_row = [&](int r, const int *idx) MX_INLINE -> int {
    int row = pj.m0 + (r - BN);
    row = r < BN + BM && row < pj.m_end ? row : -1;
    if (gather && row >= 0) row = min(max(mx_table(idx + lane), 0), (int)g.a_rows - 1);
    if (r < BN) row = mx_b_row<Cfg, GROUP, EPI, true>(g, pj, r);
    return row;
  };
  const uint8_t *b_codes = g.b_codes;  // the expert's
  const float *b_scales = g.b_scales;
  const auto p_setup = [&]() MX_INLINE {
    if (!K_GROUPS) {
      b_codes = g.b_codes + (int64_t)pj.e * b_rows * g.K;
      b_scales = g.b_scales + (int64_t)pj.e * b_srows * kb;
    }
    int mc[Cfg::kLook], ms[Cfg::kScaleDma];
#pragma unroll
    for (int l = 0; l < Cfg::kLook; ++l) mc[l] = p_row(code_row(l), rows_c[wave] + l * 64);
#pragma unroll
    for (int l = 0; l < Cfg::kScaleDma; ++l) ms[l] = p_row(scale_row(l), rows_s[wave] + l * 64);
#pragma unroll
    for (int i = 0; i < Cfg::kCodeDma; ++i) {
      const int row = __shfl(mc[i / 8], (i * 8 + qrow) & 63, 64);
      off_c[i] = row < 0 ? kNoRow : (uint32_t)row * ld + (uint32_t)(chunk * 16);
    }
#pragma unroll
    for (int l = 0; l < Cfg::kScaleDma; ++l) {
      const bool of_b = scale_row(l) < BN;
      off_s[l] = ms[l] < 0 ? kNoRow : (uint32_t)(!K_GROUPS && of_b ? ms[l] >> 7 : ms[l]) * sld;
    }
  };
  // The loads go on to the next tile, as long as there is one with a stage (GROUP_K's empty ones come last).  Its
  // row indices were fetched when the tile before was begun: S - 2 stages' loads later they have landed with what
  // every stage waits for; before the first stage (primed) and behind a shorter tile they are waited for.
  const auto next_tile = [&]() MX_INLINE {
    const int before = pj.nst;
    p_live = tiles.has(++p_it);
    if (p_live) {
      pj = tiles.get(p_it);
      if (K_GROUPS && pj.k_len > 0) {  // whole blocks
        const int hi = pj.k_lo + pj.k_len;
        pj.k_lo &= ~127;
        pj.nst = (hi - pj.k_lo + 127) / 128;
      }
      p_live = pj.nst > 0;
      if (p_live && lane == 0) queue[p_it % kQueue] = make_int4(pj.e | pj.nt << 10, pj.m0, pj.m_end, pj.nst);
    }
    p_st = 0;
    if (!p_live) return;
    if (gather && (!primed || before < S - 2)) {
      if (p_it == 0) load_index(pj);
      mx_wait_vm<0>();
    }
    p_setup();
    if (gather && tiles.has(p_it + 1)) {
      mx_wait_lds();  // (this tile's indices have been read)
      load_index(tiles.get(p_it + 1));
    }
  };
  // the sequence's next stage into the slot at LDS address dst, in PARTS parts
  uint32_t l_k0 = 0;
  int l_left = 0;
  const auto load_part = [&](uint32_t dst, int part, int parts) MX_INLINE {
    if (part == 0) {
      if (p_live && (p_it < 0 || p_st == pj.nst)) next_tile();
      l_k0 = p_live ? (uint32_t)(pj.k_lo + p_st * 128) : 0u;
      l_left = (int)g.K - (int)l_k0;  // elements behind k0 (may exceed the block)
      ++p_st;
    }
    // (With nothing to load, buffers of no bytes and l_k0 = 0: the range check takes the scalar offset off the buffer's
    // size, which may not fall below it.  An absent row's offset is behind the buffer under any l_k0, and so are the
    // chunks behind K.)
    const uint32_t some = p_live ? ~0u : 0u;
    const i32x4 buffer_a = f8_buffer(g.a_codes, a_bytes & some), buffer_b = f8_buffer(b_codes, b_bytes & some);
    const bool in_k = chunk * 16 < l_left;
#pragma unroll
    for (int i = 0; i < Cfg::kCodeDma; ++i) {
      if (i * parts / Cfg::kCodeDma != part) continue;
      const int b = i * Cfg::NW + wave;
      const uint32_t v = in_k ? off_c[i] : kNoRow;
      if (i >= Cfg::kDmaB) f8_dma16<false>(buffer_a, dst + b * 1024, v, l_k0);
      else f8_dma16<Cfg::kStreamB>(buffer_b, dst + b * 1024, v, l_k0);
    }
    if (part == parts - 1) {
#pragma unroll
      for (int l = 0; l < Cfg::kScaleDma; ++l) {
        const int b = wave * Cfg::kScaleDma + l;
        const bool of_b = b * 64 < BN;
        f8_dma4(f8_buffer(of_b ? b_scales : g.a_scales, (of_b ? b_sbytes : a_sbytes) & some),
                dst + Cfg::kScaleBase + b * 256, off_s[l], l_k0 / 128 * 4);
      }
    }
  };
  const auto load_stage = [&](uint32_t dst) MX_INLINE { load_part(dst, 0, 1); };
  const uint32_t ring_at = f8_lds(ring);
#pragma unroll
  for (int s = 0; s < S; ++s) load_stage(ring_at + s * Cfg::kStageBytes);
  primed = true;
  mx_wait_vm<(S - 1) * Cfg::kDma>();
  mx_barrier();

  // ---- fragments of one stage: lane half h takes chunks 4 h .. 4 h + 3 of a row
  constexpr bool MANY = K_GROUPS && !POW2;  // a scale for each weight row
  F8Raw tr[FM], wr;
  F8Frag<OUT_F32> tf[FM], wf;
  float sa[FM], sb[MANY ? 16 : 1], nb[MANY ? 16 : 1];
  const int w_row = wn * FN * 32, t_row = BN + wm * FM * 32;
  // LDS addresses are integers: slots, fragments and rows differ by multiples of 128, the chunks of a row by the low
  // bits that the swizzle permutes.  at[q]: chunk q of this lane's row of the wave's first weight fragment, in the slot
  // being read.
  uint32_t at[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) at[q] = ring_at + (uint32_t)((w_row + l32) * 128 + (f8_swz(h * 4, l32) ^ q) * 16);
  const auto read_tokens = [&](int f) MX_INLINE {
#pragma unroll
    for (int q = 0; q < 4; ++q) tr[f].c[q] = *f8_lds_ptr<i32x4>(at[q] + (uint32_t)(t_row - w_row) * 128 + f * 4096);
  };
  const auto read_scales = [&](uint32_t st) MX_INLINE {
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = *f8_lds_ptr<float>(st + Cfg::kScaleBase + (t_row + f * 32 + l32) * 4);
  };
  // weight fragment i and its scales (into nb)
  const auto read_weights = [&](uint32_t st, int i) MX_INLINE {
#pragma unroll
    for (int q = 0; q < 4; ++q) wr.c[q] = *f8_lds_ptr<i32x4>(at[q] + i * 4096);
    const uint32_t sc = st + Cfg::kScaleBase + (w_row + i * 32) * 4;
    if constexpr (POW2) {
      nb[0] = *f8_lds_ptr<float>(sc + l32 * 4);
    } else if constexpr (K_GROUPS) {
      // register r: operand row 8 (r / 4) + 4 h + r % 4
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 t = *f8_lds_ptr<f32x4>(sc + 8 * q * 4 + 4 * h * 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) nb[4 * q + r] = t[r];
      }
    } else {
      nb[0] = *f8_lds_ptr<float>(sc);  // a fragment's 32 rows lie in one block of 128
    }
  };

  f32x16 acc[FN][FM];
  const auto clear = [&]() MX_INLINE {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][f][r] = 0.0f;
  };

  // ---- a finished tile: lane = row l32 of a fragment, registers = columns 16 h + r.  (A 16-byte store may start at
  // any dword.)
  const auto finish = [&](const MxJob &j) MX_INLINE {
    const int ncols = (int)(K_GROUPS ? g.b_rows : g.N);
    const int col_w = j.nt * (SWIGLU ? BN / 2 : BN) + wn * NF * 32;  // this wave's first column
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
      const int ldc = (int)g.ldc;
      char *cb = static_cast<char *>(g.C) + ((K_GROUPS ? (int64_t)j.e * g.a_rows : 0) + row_w) * g.ldc * ESZ;
      // rows behind the valid ones fall behind the buffer
      const auto dst = __builtin_amdgcn_make_buffer_rsrc(mx_uniform_ptr(cb), (short)0, rows * ldc * ESZ, 0x00020000);
      // A lane's 16-byte pieces of its row, G at a time (one FP32 fragment's, two BF16 fragments'), change places in its
      // group of G lanes: each store then writes whole lines, G pieces side by side.
      constexpr int PER = 16 / ESZ, G = OUT_F32 || NF > 1 ? 4 : 2, FRAGS = G / ESZ;
      const int gl = lane & (G - 1);
      const int col_g = col_w + (gl / ESZ) * 32 + h * 16 + (gl % ESZ) * PER;  // this lane's piece of a group's first fragment
      // Rows that start between lines: the parts of a line are put together in L2 and not streamed (8 x 2500 rows of
      // 2047 FP32 columns, K = 720: 122 -> 85 us).  BF16 rows that start between dwords are no buffer's to store.
      // Tiles that are not made for such rows, and SwiGLU's, whose columns are a multiple of 32, stream them or store
      // them one value at a time.
      constexpr bool ANY = !SWIGLU && Cfg::kAnyRows;
      const int64_t starts = (int64_t)reinterpret_cast<uintptr_t>(g.C) | g.ldc * ESZ;
      const bool lines = !ANY || starts % 64 == 0, dwords = OUT_F32 || starts % 4 == 0;
      const bool ragged = (!ANY && !dwords) || (ncols % PER != 0 && col_w + NF * 32 > ncols);
#pragma unroll
      for (int f = 0; f < FM; ++f) {
#pragma unroll
        for (int i = 0; i < NF; i += FRAGS) {
          f8_u32x4 c[G];
#pragma unroll
          for (int q = 0; q < G; ++q) {
            const f32x16 &x = acc[i + q / ESZ][f];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if constexpr (OUT_F32) c[q][r] = __float_as_uint(x[4 * q + r]);
              else
                c[q][r] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x[8 * (q % 2) + 2 * r], (__bf16)x[8 * (q % 2) + 2 * r + 1]});
            }
          }
          f8_exchange<G>(c, lane);
          const int col = col_g + i * 32;
#pragma unroll
          for (int k = 0; k < G; ++k) {
            const uint32_t at = (uint32_t)((f * 32 + (l32 & ~(G - 1)) + k) * ldc + col) * ESZ;
            const bool piece = (ANY || dwords) && col + PER <= ncols;
            if (lines) {
              __builtin_amdgcn_raw_buffer_store_b128(c[k], dst, piece ? at : kNoStore, 0, kStream);
            } else if (dwords) {
              __builtin_amdgcn_raw_buffer_store_b128(c[k], dst, piece ? at : kNoStore, 0, 0);
            } else if (piece && f * 32 + (l32 & ~(G - 1)) + k < rows) {
              typedef f8_u32x4 Anywhere __attribute__((aligned(2)));
              *reinterpret_cast<Anywhere *>(cb + at) = c[k];
            }
            if (ragged) {  // one by one
#pragma unroll
              for (int r = 0; r < PER; ++r) {
                const uint32_t v = !piece && col + r < ncols ? at + r * ESZ : kNoStore;
                if constexpr (OUT_F32) __builtin_amdgcn_raw_buffer_store_b32(c[k][r], dst, v, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(c[k][r / 2] >> (16 * (r & 1))), dst, v, 0, 0);
              }
            }
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
      mx_wait_lds();
      mx_barrier();
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
              c[q] = s.bad ? 0u
                           : f8_pack4(acc[i][f][4 * q], acc[i][f][4 * q + 1], acc[i][f][4 * q + 2], acc[i][f][4 * q + 3], s.S);
            if (col < ncols)
              *reinterpret_cast<uint4 *>(g.q_codes + (row_w + rw) * ncols + col) = make_uint4(c[0], c[1], c[2], c[3]);
          }
          if (wn == 0 && h == 0) g.q_scales[(row_w + rw) * qkb + j.nt] = s.G;
        }
      }
    }
  };

  // ---- products
  // A fragment pair's sum over the block goes onto the accumulators under the block's scales: while the
  // SIMD's other wave multiplies, or, for FP32 results of up to four pairs, whose products take twice as long, from one of
  // two buffers under its own next pair's products as well (8192^3 with FP32 results 997 -> 940 us).
  constexpr int NP = OUT_F32 && !MANY && FM * FN <= 4 ? 2 : 1;
  f32x16 p[NP];
  float ps = 0.0f;  // the waiting sum's scale
  const auto multiply = [&](int i, int f) MX_INLINE {
    p[(i * FM + f) % NP] = f8_product(wf, tf[f]);
    // (products stay where they are written: they touch no memory, so nothing else keeps the compiler
    // from moving them past the reads, for which the registers do not last)
    if constexpr (NP == 2) asm volatile("" : "+v"(p[(i * FM + f) % NP]));
  };
  const auto collect = [&](int i, int f) MX_INLINE {
    const float s = NP == 2 ? ps : MANY ? sa[f] : sa[f] * sb[0];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      acc[i][f][r] = __builtin_fmaf(p[(i * FM + f) % NP][r], MANY ? s * sb[MANY ? r : 0] : s, acc[i][f][r]);
    }
    asm volatile("" : "+v"(acc[i][f]));
  };
  // Power-of-two scales: straight onto the accumulators, a fragment's tokens in turn (no product waits for the one
  // before).  The scales are the exponent bytes of both rows' (a NaN's is 255, which is NaN there too).
  const auto scaled_products = [&](int i) MX_INLINE {
    if constexpr (POW2) {
      const int ws = (int)(__float_as_uint(sb[0]) >> 23);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int f = 0; f < FM; ++f)
          acc[i][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf.v[s], tf[f].v[s], acc[i][f], 0, 0, 0, ws, 0,
                                                                       (int)(__float_as_uint(sa[f]) >> 23));
#pragma unroll
      for (int f = 0; f < FM; ++f) asm volatile("" : "+v"(acc[i][f]));
    }
  };
  const auto products = [&](int i, int f) MX_INLINE {
    multiply(i, f);
    if constexpr (NP == 2) {
      // the pair before, in the stage before's last fragment if this is the first
      const int n = (i * FM + f + FN * FM - 1) % (FN * FM);
      collect(n / FM, n % FM);
      ps = sa[f] * sb[0];
    } else {
      collect(i, f);
    }
  };
  // A slot is refilled in parts, behind the products of its last weight fragment and, where a wave has four, of
  // the next stage's first: DMAs issued at once keep the wave from its products (gate and up of 131072 rows
  // 486 us, in two parts 472, in four 459; in six 472).
  constexpr int SPREAD = FN >= 4 ? 1 : 0, PARTS = (1 + SPREAD) * FM;
  int slot = 0, next_slot = Cfg::kStageBytes;
  // the stage has been read by this wave: wait for its own loads of the next one, meet, and refill
  const auto meet = [&]() MX_INLINE {
    mx_wait_lds();
    mx_wait_vm<(S - 2) * Cfg::kDma>();
    mx_barrier();
  };
  const auto turn = [&]() MX_INLINE {
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] += (uint32_t)(next_slot - slot);
    slot = next_slot;
    next_slot = next_slot == (S - 1) * Cfg::kStageBytes ? 0 : next_slot + Cfg::kStageBytes;
  };
#pragma unroll 1
  for (int it = 0; tiles.has(it); ++it) {
    MxJob cj;
    if (p_live || it < p_it) {
      const int *q = reinterpret_cast<const int *>(&queue[it % kQueue]);
      const int x = __builtin_amdgcn_readfirstlane(q[0]);
      cj.e = x & 1023;
      cj.nt = x >> 10;
      cj.m0 = __builtin_amdgcn_readfirstlane(q[1]);
      cj.m_end = __builtin_amdgcn_readfirstlane(q[2]);
      cj.nst = __builtin_amdgcn_readfirstlane(q[3]);
    } else {  // behind the last tile that has been loaded
      cj = tiles.get(it);
      cj.nst = 0;
    }
    clear();
    // (the waves behind an expert's last row leave the matrix cores to the others)
    if (K_GROUPS || cj.m0 + wm * FM * 32 < cj.m_end) {
      if (cj.nst > 0) {
        read_weights(ring_at + slot, 0);
#pragma unroll
        for (int f = 0; f < FM; ++f) read_tokens(f);
        read_scales(ring_at + slot);
      }
      if constexpr (NP == 2) {  // nothing waits yet
        ps = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) p[1][r] = 0.0f;
      }
      uint32_t done = 0;  // the slot being refilled
#pragma unroll 1
      for (int st = 0; st < cj.nst; ++st) {
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          wf.set(wr);
#pragma unroll
          for (int r = 0; r < (MANY ? 16 : 1); ++r) sb[r] = nb[r];
          if (i == FN - 1) {
            meet();
            done = ring_at + slot;
            turn();
          }
          read_weights(ring_at + slot, i < FN - 1 ? i + 1 : 0);
          if (POW2) {
#pragma unroll
            for (int f = 0; f < FM; ++f)
              if (i == 0) tf[f].set(tr[f]);
            scaled_products(i);
          }
#pragma unroll
          for (int f = 0; f < FM; ++f) {
            if (!POW2) {
              if (i == 0) tf[f].set(tr[f]);
              products(i, f);
            }
            if (i < SPREAD && st > 0) load_part(done, (i + 1) * FM + f, PARTS);
            if (i == FN - 1) {
              load_part(done, f, PARTS);
              read_tokens(f);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        read_scales(ring_at + slot);
      }
      if (cj.nst > 0) {
#pragma unroll
        for (int n = FM; n < PARTS; ++n) load_part(done, n, PARTS);
      }
      if constexpr (NP == 2) collect(FN - 1, FM - 1);
    } else {
#pragma unroll 1
      for (int st = 0; st < cj.nst; ++st) {
        meet();
        load_stage(ring_at + slot);
        turn();
      }
    }
    finish(cj);
  }
  mx_wait_vm<0>();  // loads into this workgroup's LDS end before it does
}

// persistent grid: whole multiples of the XCDs
template <class Cfg, int GROUP, int EPI, bool OUT_F32, bool QUANT = false>
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
  const int lds = Cfg::kStages * Cfg::kStageBytes + (kMxMaxExperts + 1) * 8 +
                  Cfg::NW * ((Cfg::kLook * 64 + Cfg::kScaleDma * 64) * 4 + kQueue * 16) + (QUANT ? Cfg::kWavesN * Cfg::BM * 4 : 0);
  const int per_cu = std::max(1, std::min(160 * 1024 / lds, Cfg::kWavesPerSimd * 4 / Cfg::NW));
  const int64_t most = (int64_t)device_cu_count() * per_cu;
  const unsigned grid = (unsigned)std::min<int64_t>((tiles + kMxXcds - 1) / kMxXcds * kMxXcds, most);
  if constexpr (!OUT_F32) {
    if (g.pow2) {
      k_f8_gemm<Cfg, GROUP, EPI, OUT_F32, QUANT, true><<<grid, Cfg::NT, 0, stream>>>(g);
      return hipGetLastError();
    }
  }
  k_f8_gemm<Cfg, GROUP, EPI, OUT_F32, QUANT, false><<<grid, Cfg::NT, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace
}  // namespace nv4
