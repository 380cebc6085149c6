// FP8 quantisation, its inverse and the transposition of quantised weights for gfx950 (E4M3 codes with an
// FP32 scale for each block of 128 values).
//
// A block's scale depends on its own values only, so one pass over the input is enough: read
// 2 (BF16) or 4 bytes per element, write 1.03 per direction.  The kernels are bound by that traffic: 131072 x 1536
// BF16 both ways, 163 us, 5.0 TB/s of what has to move; values of as many codes as FP32, 200 us, 5.0 TB/s.
//
// Rows: 16 lanes take one block, 8 elements each, so that a wave reads 1 KB (BF16) or 2 KB
// contiguous and writes 512 bytes of codes.
// Tokens (the transpose by segments): a workgroup holds a tile of 128 rows x 128 columns in LDS, which
// is a block of every one of its columns, and of every row too: the form that writes both directions
// reads the input once.
// Weights: a workgroup takes a 128 x 128 block in registers.
#include <algorithm>

#include "f8_device.h"
#include "f8_internal.h"
#include "many_groups.h"
#include "nv4_internal.h"
#include "segment_tile.h"
#include "../../include/nv4moe.h"

namespace nv4 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr uint32_t kXcds = 8;
constexpr uint32_t kNoLoad = 0x80000000u;  // behind every tile (128 rows of at most 16 MiB)

__device__ __forceinline__ uint32_t f8_clamp_row(const F8QuantArgs &a, int32_t i) {
  return (uint32_t)min(max(i, 0), (int)(a.x_rows - 1));
}

// One row-direction block (16 lanes, 8 elements each, zeros behind K): codes and scale of `row`.
template <bool F32>
__device__ __forceinline__ bool f8_row_block(const uint4 (&v)[F32 ? 2 : 1], int l16, int pow2, uint2 &codes, float &G) {
  uint32_t m;
  if constexpr (F32) m = max(f8_amax<true>(v[0]), f8_amax<true>(v[1]));
  else m = f8_amax<false>(v[0]);
  const F8Scale s = f8_scale(row16_umax(m), pow2);
  if constexpr (F32) codes = make_uint2(f8_pack_f32(v[0], s.S), f8_pack_f32(v[1], s.S));
  else codes = f8_pack_bf16(v[0], s.S);
  if (s.bad) codes = make_uint2(0u, 0u);
  G = s.G;
  return s.bad;
}

// U blocks per 16-lane group; kb: blocks of a row
template <bool F32, int U>
__global__ __launch_bounds__(256) void k_f8_rows(F8QuantArgs a, uint32_t units, uint32_t kb) {
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const uint32_t first = (group_index() * 4 + (threadIdx.x >> 6)) * (4 * U) + (lane >> 4);
  uint4 v[U][F32 ? 2 : 1];
  uint32_t row[U], blk[U], src[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t unit = first + u * 4;
    row[u] = unit / kb;
    blk[u] = unit - row[u] * kb;
    src[u] = row[u];
  }
  if (a.row_index) {  // all of them before the first dependent load: loads return in order
#pragma unroll
    for (int u = 0; u < U; ++u) src[u] = f8_clamp_row(a, a.row_index[min(row[u], (uint32_t)a.rows - 1)]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t col = (int64_t)blk[u] * kF8Block + l16 * 8;
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[u][i] = make_uint4(0, 0, 0, 0);
    if (first + u * 4 < units && col < a.K) {
      const int64_t at = (int64_t)src[u] * a.ldx + col;
      const uint4 *p = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(a.x) + at)
                           : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at);
#pragma unroll
      for (int i = 0; i < (F32 ? 2 : 1); ++i) v[u][i] = p[i];
    }
  }
  bool bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint2 c;
    float G;
    bad |= f8_row_block<F32>(v[u], l16, a.pow2, c, G);
    const int64_t col = (int64_t)blk[u] * kF8Block + l16 * 8;
    if (first + u * 4 < units) {
      if (col < a.K) *reinterpret_cast<uint2 *>(a.codes + (int64_t)row[u] * a.K + col) = c;
      if (l16 == 0) a.scales[(int64_t)row[u] * kb + blk[u]] = G;
    }
  }
  if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
}

// One tile: 128 rows of one segment x 128 columns.  A padded segment starts at a multiple of 128, so a
// tile lies in one segment.  LDS row r keeps dword p of the tile at p ^ (16 * (r / 32 % 4)): the four
// 32-row parts of a column, which neighbouring lanes read at once, then fall into different banks.
template <bool F32, bool ROWS>
__global__ __launch_bounds__(F32 ? 512 : 256) void k_f8_cols(F8QuantArgs a, int chunks, uint32_t n) {
  constexpr int NT = F32 ? 512 : 256, ES = F32 ? 4 : 2;
  constexpr int LPR = F32 ? 32 : 16;       // lanes of a row, 16 bytes each
  constexpr int W = LPR * 4;               // dwords of a tile row
  __shared__ uint32_t tile[128 * W];
  __shared__ SegmentOf s_seg;
  const int tid = threadIdx.x, lr = tid % LPR;
  // Each XCD (workgroup i runs on XCD i % 8) takes a contiguous share of the tiles, column tile by
  // column tile, so that with gathered rows it reads few columns of x.
  const uint32_t b0 = group_index(), per = n / kXcds, full = per * kXcds;
  if (b0 >= n) return;  // uniform
  const uint32_t L = b0 < full ? (b0 % kXcds) * per + b0 / kXcds : b0;
  const uint32_t ct = L / (uint32_t)chunks, ch = L - ct * (uint32_t)chunks;
  const int64_t p0 = (int64_t)ch * 128;
  if (p0 >= a.seg_padded_offsets[a.nseg]) return;  // uniform
  find_segment<NT>(a.seg_offsets, a.seg_padded_offsets, a.nseg, p0, &s_seg);
  const int64_t row0 = s_seg.first_row + (p0 - s_seg.start);
  int64_t valid = std::min<int64_t>(s_seg.end_row, a.rows) - row0;
  if (row0 < 0) valid = 0;
  const int64_t col0 = (int64_t)ct * 128;
  const int64_t mycol = col0 + lr * (16 / ES);
  uint4 v[8];
  if (!a.row_index) {
    // rows of one matrix: 32-bit offsets into the tile, whose range check gives the zeros
    const uint32_t ld = (uint32_t)a.ldx * ES;
    const auto src = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(static_cast<const char *>(a.x)) + row0 * a.ldx * ES, (short)0,
        (int)(uint32_t)(std::max<int64_t>(std::min<int64_t>(valid, 128), 0) * ld), 0x00020000);
    uint32_t at = (tid / LPR) * ld + (uint32_t)mycol * ES;
#pragma unroll
    for (int i = 0; i < 8; ++i, at += 16 * ld) {
      const auto t = __builtin_amdgcn_raw_buffer_load_b128(src, mycol < a.K ? at : kNoLoad, 0, 0);
      v[i] = make_uint4(t[0], t[1], t[2], t[3]);
    }
  } else {
    int32_t idx[8];  // all of them before the first dependent load: loads return in order
#pragma unroll
    for (int i = 0; i < 8; ++i)
      idx[i] = a.row_index[std::min<int64_t>(std::max<int64_t>(row0 + i * 16 + tid / LPR, 0), a.rows - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (i * 16 + tid / LPR < valid && mycol < a.K)
        v[i] = *reinterpret_cast<const uint4 *>(static_cast<const char *>(a.x) +
                                                ((int64_t)f8_clamp_row(a, idx[i]) * a.ldx + mycol) * ES);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 16 + tid / LPR;
    *reinterpret_cast<uint4 *>(&tile[r * W + ((lr * 4) ^ (16 * ((r >> 5) & 3)))]) = v[i];
  }
  bool bad = false;
  if (ROWS) {
    const int64_t kb = (a.K + kF8Block - 1) / kF8Block;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 16 + tid / LPR;
      const uint32_t m = f8_amax<F32>(v[i]);
      const F8Scale s = f8_scale(F32 ? half_umax(m) : row16_umax(m), a.pow2);
      if (r < valid) {
        uint8_t *p = a.codes2 + (row0 + r) * a.K + mycol;
        if (mycol < a.K) {
          if constexpr (F32) *reinterpret_cast<uint32_t *>(p) = s.bad ? 0u : f8_pack_f32(v[i], s.S);
          else *reinterpret_cast<uint2 *>(p) = s.bad ? make_uint2(0u, 0u) : f8_pack_bf16(v[i], s.S);
        }
        if (lr == 0) a.scales2[(row0 + r) * kb + ct] = s.G;
      }
    }
  }
  __syncthreads();
  // thread = dword column w (two BF16 columns, or one FP32), 32-row part b: a column's four parts are a quad
  const int b = tid & 3, w = tid >> 2;
  uint32_t q[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) q[i] = tile[(b * 32 + i) * W + (w ^ (16 * b))];
  constexpr int NC = F32 ? 1 : 2;
  uint32_t amax[NC];
  uint32_t mx = 0;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) mx = max(mx, q[i] & 0x7FFFFFFFu);
    amax[0] = mx;
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) mx = pk_umax16(mx, q[i] & 0x7FFF7FFFu);
    amax[0] = mx << 16;
    amax[1] = mx & 0xFFFF0000u;
  }
  const int64_t okb = a.out_K / kF8Block;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = col0 + w * NC + c;
    const F8Scale s = f8_scale(quad_umax(amax[c]), a.pow2);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = F32 ? __uint_as_float(q[4 * j + i]) : c == 0 ? bf16_lo(q[4 * j + i]) : bf16_hi(q[4 * j + i]);
      o[j] = s.bad ? 0u : f8_pack4(f[0], f[1], f[2], f[3], s.S);
    }
    bad |= s.bad;
    if (col < a.K) {
      uint4 *p = reinterpret_cast<uint4 *>(a.codes + col * a.out_K + p0 + b * 32);
      p[0] = make_uint4(o[0], o[1], o[2], o[3]);
      p[1] = make_uint4(o[4], o[5], o[6], o[7]);
      if (b == 0) a.scales[col * okb + ch] = s.G;
    }
  }
  if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
}

// One 128 x 128 block of a matrix of m rows
template <bool F32>
__global__ __launch_bounds__(F32 ? 512 : 256) void k_f8_tiles(F8QuantArgs a, uint32_t mb, uint32_t kb, int64_t m, uint32_t n) {
  constexpr int NT = F32 ? 512 : 256, ES = F32 ? 4 : 2, LPR = F32 ? 32 : 16;
  __shared__ uint32_t s_max[NT / 64];
  const int tid = threadIdx.x, lr = tid % LPR;
  const uint32_t block = group_index();
  if (block >= n) return;  // uniform
  const uint32_t ct = block % kb, rb = block / kb;  // rb: block row over all matrices
  const uint32_t s = rb / mb;
  const int64_t in0 = (int64_t)(rb - s * mb) * 128, row0 = (int64_t)s * m + in0;
  const int64_t valid = m - in0, mycol = (int64_t)ct * 128 + lr * (16 / ES);
  uint4 v[8];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 16 + tid / LPR;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < valid && mycol < a.K)
      v[i] = *reinterpret_cast<const uint4 *>(static_cast<const char *>(a.x) + ((row0 + r) * a.ldx + mycol) * ES);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max(mx, f8_amax<F32>(v[i]));
  mx = wave_reduce_u32(mx, [](uint32_t x, uint32_t y) { return max(x, y); });
  if ((tid & 63) == 0) s_max[tid >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) mx = max(mx, s_max[i]);
  const F8Scale sc = f8_scale(mx, a.pow2);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 16 + tid / LPR;
    if (r < valid && mycol < a.K) {
      uint8_t *p = a.codes + (row0 + r) * a.K + mycol;
      if constexpr (F32) *reinterpret_cast<uint32_t *>(p) = sc.bad ? 0u : f8_pack_f32(v[i], sc.S);
      else *reinterpret_cast<uint2 *>(p) = sc.bad ? make_uint2(0u, 0u) : f8_pack_bf16(v[i], sc.S);
    }
  }
  if (tid == 0) {
    a.scales[block] = sc.G;
    if (sc.bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
  }
}

// Values of U blocks, 16 lanes each.  BF16: a lane takes 8 codes of a block, one 16-byte store; FP32: 4 codes
// of either half, so that both of its stores are contiguous over the lanes.  The output is stored as
// streamed: nothing reads it here.  m: rows of a matrix and mb its block rows (blocks of 128 x 128), or 0.
template <bool F32, int U>
__global__ __launch_bounds__(256) void k_f8_dequant(F8DequantArgs a, uint32_t units, uint32_t kb, uint32_t m, uint32_t mb) {
  constexpr int H = F32 ? 2 : 1, W = 8 / H;  // accesses per block, codes each
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const uint32_t first = (group_index() * 4 + (threadIdx.x >> 6)) * (4 * U) + (lane >> 4);
  uint32_t c[U][2], row[U];
  float G[U];
  int64_t col[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t unit = first + u * 4;
    row[u] = unit / kb;
    const uint32_t blk = unit - row[u] * kb;
    col[u] = unit < units ? (int64_t)blk * kF8Block + l16 * W : a.K;
    uint32_t srow = row[u];
    if (m) {
      const uint32_t s = row[u] / m;
      srow = s * mb + (row[u] - s * m) / 128u;
    }
    G[u] = unit < units ? a.scales[(int64_t)srow * kb + blk] : 0.0f;
    c[u][0] = c[u][1] = 0;
    const uint8_t *p = a.codes + (int64_t)row[u] * a.K + col[u];
    if constexpr (F32) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (col[u] + h * 64 < a.K) c[u][h] = *reinterpret_cast<const uint32_t *>(p + h * 64);
    } else if (col[u] < a.K) {
      const uint2 t = *reinterpret_cast<const uint2 *>(p);
      c[u][0] = t.x;
      c[u][1] = t.y;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float f[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(c[u][h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(c[u][h], true);
      f[4 * h] = lo[0] * G[u], f[4 * h + 1] = lo[1] * G[u], f[4 * h + 2] = hi[0] * G[u], f[4 * h + 3] = hi[1] * G[u];
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (col[u] + h * 64 >= a.K) continue;
      const int64_t at = (int64_t)row[u] * a.ldo + col[u] + h * 64;
      if constexpr (F32) {
        __builtin_nontemporal_store(f32x4{f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]},
                                    reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at));
      } else {
        u32x4 t;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
        __builtin_nontemporal_store(t, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + at));
      }
    }
  }
}

// One 128 x 128 block of a matrix [m][K] to its place in [K][m].  Rows of 33 dwords in LDS: 16 rows x 8
// dword columns, which a wave reads at once, fall into different banks.
__global__ __launch_bounds__(256) void k_f8_transpose(F8TransposeArgs a, uint32_t mb, uint32_t kb, uint32_t n) {
  __shared__ uint32_t tile[128 * 33];
  const int tid = threadIdx.x;
  const uint32_t block = group_index();
  if (block >= n) return;  // uniform
  const uint32_t rest = block / kb, ct = block - rest * kb, s = rest / mb, rb = rest - s * mb;
  const int64_t r0 = (int64_t)rb * 128, c0 = (int64_t)ct * 128;
  const uint8_t *src = a.codes + ((int64_t)s * a.m + r0) * a.K + c0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (tid >> 3), c = (tid & 7) * 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r0 + r < a.m && c0 + c < a.K) v = *reinterpret_cast<const uint4 *>(src + (int64_t)r * a.K + c);
    uint32_t *t = &tile[r * 33 + c / 4];
    t[0] = v.x, t[1] = v.y, t[2] = v.z, t[3] = v.w;
  }
  __syncthreads();
  // 16 rows of one dword column: 16 bytes of each of its four columns
  const int rg = tid & 7, w = tid >> 3;
  uint32_t o[4][4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = tile[(rg * 16 + g * 4 + i) * 33 + w];
    // four bytes of four rows, transposed
    const uint32_t a01 = __builtin_amdgcn_perm(q[1], q[0], 0x05010400u), b01 = __builtin_amdgcn_perm(q[1], q[0], 0x07030602u);
    const uint32_t a23 = __builtin_amdgcn_perm(q[3], q[2], 0x05010400u), b23 = __builtin_amdgcn_perm(q[3], q[2], 0x07030602u);
    o[0][g] = __builtin_amdgcn_perm(a23, a01, 0x05040100u);
    o[1][g] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
    o[2][g] = __builtin_amdgcn_perm(b23, b01, 0x05040100u);
    o[3][g] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
  }
  uint8_t *dst = a.out_codes + ((int64_t)s * a.K + c0 + w * 4) * a.m + r0 + rg * 16;
  if (r0 + rg * 16 < a.m) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + w * 4 + j < a.K)
        *reinterpret_cast<uint4 *>(dst + (int64_t)j * a.m) = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
  }
  if (tid == 0) a.out_scales[((int64_t)s * kb + ct) * mb + rb] = a.scales[((int64_t)s * mb + rb) * kb + ct];
}

// blocks per 16-lane group: few where the problem would not fill the chip
int f8_units_per_group(int64_t units) { return units > (int64_t)device_cu_count() * 16 * 64 ? 4 : units > 4096 ? 2 : 1; }

template <bool F32>
hipError_t launch_rows(const F8QuantArgs &a, hipStream_t stream) {
  const int64_t kb = f8_blocks(a.K), units = a.rows * kb;
  const int u = f8_units_per_group(units);
  const dim3 grid = many_groups((units + 16 * u - 1) / (16 * u));
  if (u == 4) k_f8_rows<F32, 4><<<grid, 256, 0, stream>>>(a, (uint32_t)units, (uint32_t)kb);
  else if (u == 2) k_f8_rows<F32, 2><<<grid, 256, 0, stream>>>(a, (uint32_t)units, (uint32_t)kb);
  else k_f8_rows<F32, 1><<<grid, 256, 0, stream>>>(a, (uint32_t)units, (uint32_t)kb);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f8_quantize(const F8QuantArgs &a, hipStream_t stream) {
  if (a.layout == NV4_ROWS) return a.x_is_f32 ? launch_rows<true>(a, stream) : launch_rows<false>(a, stream);
  const int64_t kb = f8_blocks(a.K);
  if (a.layout == NV4_F8_TILES) {
    const int64_t m = a.rows / a.nseg, mb = f8_blocks(m);
    const uint32_t n = (uint32_t)(a.nseg * mb * kb);
    const dim3 grid = many_groups(n);
    if (a.x_is_f32) k_f8_tiles<true><<<grid, 512, 0, stream>>>(a, (uint32_t)mb, (uint32_t)kb, m, n);
    else k_f8_tiles<false><<<grid, 256, 0, stream>>>(a, (uint32_t)mb, (uint32_t)kb, m, n);
    return hipGetLastError();
  }
  // no more chunks than the rows can fill: every segment may have a ragged last one
  const int chunks = (int)std::min<int64_t>(a.out_K / 128, f8_blocks(a.rows) + a.nseg);
  const uint32_t n = (uint32_t)(chunks * kb);
  const dim3 grid = many_groups(n);
  const bool both = a.layout == NV4_ROWS_AND_COLS;
  if (a.x_is_f32) {
    if (both) k_f8_cols<true, true><<<grid, 512, 0, stream>>>(a, chunks, n);
    else k_f8_cols<true, false><<<grid, 512, 0, stream>>>(a, chunks, n);
  } else {
    if (both) k_f8_cols<false, true><<<grid, 256, 0, stream>>>(a, chunks, n);
    else k_f8_cols<false, false><<<grid, 256, 0, stream>>>(a, chunks, n);
  }
  return hipGetLastError();
}

hipError_t launch_f8_dequantize(const F8DequantArgs &a, hipStream_t stream) {
  const int64_t kb = f8_blocks(a.K), units = a.rows * kb;
  const int64_t m = a.nseg ? a.rows / a.nseg : 0, mb = f8_blocks(m);
  const int u = f8_units_per_group(units);
  const dim3 grid = many_groups((units + 16 * u - 1) / (16 * u));
  const auto go = [&](auto f32, auto n) {
    k_f8_dequant<decltype(f32)::value, decltype(n)::value>
        <<<grid, 256, 0, stream>>>(a, (uint32_t)units, (uint32_t)kb, (uint32_t)m, (uint32_t)mb);
  };
  const auto by_u = [&](auto f32) {
    if (u == 4) go(f32, std::integral_constant<int, 4>{});
    else if (u == 2) go(f32, std::integral_constant<int, 2>{});
    else go(f32, std::integral_constant<int, 1>{});
  };
  if (a.out_is_f32) by_u(std::true_type{});
  else by_u(std::false_type{});
  return hipGetLastError();
}

hipError_t launch_f8_transpose(const F8TransposeArgs &a, hipStream_t stream) {
  const int64_t mb = f8_blocks(a.m), kb = f8_blocks(a.K);
  const int64_t n = a.nseg * mb * kb;
  k_f8_transpose<<<many_groups(n), 256, 0, stream>>>(a, (uint32_t)mb, (uint32_t)kb, (uint32_t)n);
  return hipGetLastError();
}

}  // namespace nv4
