// What the grouped GEMMs of the 4- and 8-bit formats share: the order of a workgroup's tiles, the rows
// of B in a tile, SwiGLU, and the loads, stores and waits of their pipelines.
#pragma once

#include "mx_device.h"
#include "../../include/nv4moe.h"

// (lambdas that hold the accumulators by reference must be inlined for them to stay in registers)
#define MX_INLINE __attribute__((always_inline))

namespace nv4 {
namespace {

constexpr int kMxMaxExperts = 1024;
constexpr int kMxXcds = 8;
constexpr uint32_t kNoRow = 0xFFFFFF00u;  // a byte offset behind every buffer: loads return zeros

// workgroup barrier without a memory fence (which would drain the prefetches)
__device__ __forceinline__ void mx_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Branch-free stores into [base, base + bytes) at byte offset voff; an offset of kNoStore is
// dropped.  base is the same for the whole wave.
constexpr uint32_t kNoStore = 0x80000000u;
__device__ __forceinline__ void *mx_uniform_ptr(const void *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<void *>(((uint64_t)hi << 32) | lo);
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void mx_store8(void *base, uint32_t bytes, uint32_t voff, uint32_t a, uint32_t b) {
  __builtin_amdgcn_raw_buffer_store_b64(
      u32x2{a, b},
      __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000), voff,
      0, 0);
}
// Outputs are stored as streamed (non-temporal): the kernel does not read them again, and lines that
// would stay in L2 push out the codes that neighbouring tiles share.  dW of 64 experts (768 x 2048,
// FP32, 32768 rows): 139 -> 105 us; dX in FP32 85 -> 66; BF16 rows 67 -> 63 with 128 x 128
// tiles, unchanged with 256 x 256.  Codes and scale bytes are part lines and stay cached.
__device__ __forceinline__ void mx_store4(void *base, uint32_t bytes, uint32_t voff, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b32(
      v, __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000), voff,
      0, kStream);
}
__device__ __forceinline__ void mx_store2(void *base, uint32_t bytes, uint32_t voff, uint16_t v) {
  __builtin_amdgcn_raw_buffer_store_b16(
      v, __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000), voff,
      0, kStream);
}
__device__ __forceinline__ void mx_store1(void *base, uint32_t bytes, uint32_t voff, uint32_t b) {
  __builtin_amdgcn_raw_buffer_store_b8(
      (uint8_t)b,
      __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000), voff,
      0, 0);
}

__device__ __forceinline__ int64_t mx_uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// An LDS dword that no load in flight can change, read without the compiler's wait for those
// loads (it cannot tell the tables from the ring); the wait for the value is in the block.
__device__ __forceinline__ int mx_table(const int *p) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(v)
               : "v"((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) int *)p)
               : "memory");
  return v;
}

// TRANS: weight row (within its 32-row fragment) at operand row i.  Accumulator register r of
// lane half h holds operand row 8 (r / 4) + 4 h + r % 4; it shall be column 16 h + r.
__device__ __forceinline__ int frag_row(int i) { return ((i >> 2) & 1) * 16 + (i >> 3) * 4 + (i & 3); }

// gate / (1 + exp(-gate)) * up in FP32, with the hardware's exp2 and reciprocal.  The exponent
// -gate log2(e) is rounded to FP32 before exp2, so the relative error grows with the gate:
// (1.25 |gate| + 8) 2^-24 at most, 6e-6 at -80.  A more exact exponent would take a second product
// and an addition per value, for a result that leaves as BF16 or FP4 (half a step: 2^-8 and 2^-2).
// Below -87.3, where the reciprocal is under FP32's smallest normal number, the result may be 0.
__device__ __forceinline__ float mx_swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

struct MxJob {
  int e, nt;
  int m0, m_end;   // rows of A / C
  int k_lo, nst;   // contraction: start and stages
  int k_len;
};

// The workgroup's sequence of tiles.  GROUP_M: logical tiles in XCD order (workgroup i runs on
// XCD i % 8): the workgroups of one XCD take consecutive tiles, which share A rows and an
// expert's weights in its L2.  GROUP_K: experts by decreasing length and the tiles dealt out in
// turn, forwards then backwards, so that every workgroup gets long and short ones; the empty
// ones come last.
// Finding a tile takes a search, so a wave finds 64 at a time, one per lane, and each is then a
// few lane reads away.
template <class Cfg, int GROUP, int EPI, class Args>
struct MxTiles {
  const Args &g;
  const int *off;  // the expert offsets
  const int *tab;  // GROUP_M: first M tile of each expert; GROUP_K: experts by length
  int total;
  int ntn;
  int en, m, lo, hi;  // this lane's tile: expert | column tile << 10, first row, and row end or K range
  __device__ __forceinline__ int index(int it) const {  // grows with it
    const int G = gridDim.x, b = blockIdx.x;
    if (GROUP == NV4_GROUP_K) return it * G + ((it & 1) ? G - 1 - b : b);
    const int per = G / kMxXcds;
    return it * G + (b < per * kMxXcds ? (b % kMxXcds) * per + b / kMxXcds : b);
  }
  __device__ __forceinline__ bool has(int it) const { return index(it) < total; }
  __device__ __forceinline__ void find(int it) {
    const int L = index(it + (int)(threadIdx.x & 63));
    en = m = lo = hi = 0;
    if (L >= total) return;
    if (GROUP == NV4_GROUP_M) {
      const int mt = L / ntn;
      int e = 0, top = g.E - 1;  // last expert with tab[e] <= mt (it owns at least one tile)
      while (e < top) {
        const int mid = (e + top + 1) >> 1;
        if (tab[mid] <= mt) e = mid; else top = mid - 1;
      }
      en = e | (L - mt * ntn) << 10;
      m = off[e] + (mt - tab[e]) * Cfg::BM;
      hi = min(off[e + 1], (int)g.M_cap);
    } else {
      const int tn = (int)((g.a_rows + Cfg::BM - 1) / Cfg::BM), per_e = tn * ntn;
      const int rank = L / per_e, r = L - rank * per_e, e = tab[rank];
      en = e | (r % ntn) << 10;
      m = r / ntn * Cfg::BM;
      lo = min(off[e], (int)g.K);
      hi = max(min(off[e + 1], (int)g.K), lo);
    }
  }
  // tile `it`, called with it = 0, 1, 2, ..
  __device__ __forceinline__ MxJob get(int it) {
    const int l = it & 63;
    if (l == 0) find(it);
    const int x = __builtin_amdgcn_readlane(en, l), h = __builtin_amdgcn_readlane(hi, l);
    MxJob j;
    j.e = x & 1023;
    j.nt = x >> 10;
    j.m0 = __builtin_amdgcn_readlane(m, l);
    j.m_end = GROUP == NV4_GROUP_M ? h : (int)g.a_rows;
    j.k_lo = GROUP == NV4_GROUP_M ? 0 : __builtin_amdgcn_readlane(lo, l);
    j.k_len = GROUP == NV4_GROUP_M ? (int)g.K : h - j.k_lo;
    j.nst = (j.k_len + Cfg::BK - 1) / Cfg::BK;
    return j;
  }
};

// Row of B (of the tile's expert's part of it) for tile row r, or -1 behind the matrix.  SwiGLU: a
// wave's fragments are FN/2 of gate rows, then the up rows of the same columns.
template <class Cfg, int GROUP, int EPI, bool TRANS, class Args>
__device__ __forceinline__ int mx_b_row(const Args &g, const MxJob &j, int r) {
  const int in = TRANS ? (r & ~31) | frag_row(r & 31) : r;
  if (GROUP == NV4_GROUP_K) {
    const int64_t col = (int64_t)j.nt * Cfg::BN + in;
    return col < g.b_rows ? (int)col : -1;
  }
  if (EPI == NV4_EPI_SWIGLU) {
    constexpr int half = Cfg::kFN / 2;
    const int wv = in / (Cfg::kFN * 32), f = (in / 32) % Cfg::kFN;
    const int64_t col = (int64_t)j.nt * (Cfg::BN / 2) + wv * (half * 32) + (f % half) * 32 + (in & 31);
    return col < g.N ? (int)((f >= half ? g.N : 0) + col) : -1;
  }
  const int64_t col = (int64_t)j.nt * Cfg::BN + in;
  return col < g.N ? (int)col : -1;
}

// The tables behind MxTiles, by the whole workgroup: the first M tile of every expert (GROUP_M) or the
// experts by decreasing length (GROUP_K), from the offsets in LDS; scratch: an int for each wave.
template <class Cfg, int GROUP, int EPI, class Args>
__device__ __forceinline__ void tiles_setup(const Args &g, const int *off, int *tab, int *scratch,
                                            MxTiles<Cfg, GROUP, EPI, Args> &tiles) {
  constexpr int BM = Cfg::BM, BN = Cfg::BN, NT = Cfg::NT;
  const int tid = threadIdx.x, lane = tid & 63;
  if (GROUP == NV4_GROUP_M) {
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = (g.E + NT - 1) / NT;
    int own = 0;
    for (int i = 0; i < per; ++i) {
      const int e = tid * per + i;
      if (e < g.E) own += (max(off[e + 1] - off[e], 0) + BM - 1) / BM;
    }
    int run = own;  // inclusive sum over the wave, then the waves before
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(run, o, 64);
      if (lane >= o) run += x;
    }
    if (lane == 63) scratch[wave] = run;
    __syncthreads();
    for (int w = 0; w < wave; ++w) run += scratch[w];
    run -= own;
    for (int i = 0; i < per; ++i) {
      const int e = tid * per + i;
      if (e < g.E) {
        tab[e] = run;
        run += (max(off[e + 1] - off[e], 0) + BM - 1) / BM;
      }
    }
    if (tid == NT - 1) tab[g.E] = run;
    __syncthreads();
    constexpr int cols = EPI == NV4_EPI_SWIGLU ? BN / 2 : BN;
    tiles.ntn = (int)((g.N + cols - 1) / cols);
    tiles.total = __builtin_amdgcn_readfirstlane(tab[g.E] * tiles.ntn);
  } else {
    for (int e = tid; e < g.E; e += NT) {
      const int n = off[e + 1] - off[e];
      int rank = 0;
      for (int f = 0; f < g.E; ++f) {
        const int m = off[f + 1] - off[f];
        rank += (m > n) || (m == n && f < e);
      }
      tab[rank] = e;
    }
    __syncthreads();
    tiles.ntn = (int)((g.b_rows + BN - 1) / BN);
    tiles.total = (int)(g.E * ((g.a_rows + BM - 1) / BM) * tiles.ntn);
  }
}

}  // namespace
}  // namespace nv4
