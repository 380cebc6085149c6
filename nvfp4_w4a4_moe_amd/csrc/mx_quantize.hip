// MXFP4 quantisation and its inverse for gfx950 (OCP Microscaling v1.0: 32 E2M1 codes
// under one power-of-two E8M0 scale).
//
// A block's scale depends on its own 32 values only, so one pass over the input is enough:
// read 2 (BF16) or 4 bytes per element, write 0.53.  The kernels are bound by that traffic;
// what is left is to keep every load and store wide and the instructions per element few (the
// converter takes BF16 pairs as they are and divides by the scale itself).
//
// Rows: a lane takes 8 elements (mx_rows.h), so a wave reads 1 KB (BF16) or 2 KB contiguous and
// writes 256 B of codes.
// Columns: a workgroup holds a tile of 128 rows x 256 bytes in LDS, each thread then takes
// a 32-row block of one dword column (two BF16 columns or one FP32).
//
// Measured, 131072 x 2048 BF16 (537 MB in, 143 MB out per direction): rows 114 us (6.0 TB/s), columns
// 140 (4.9), both from one read 178 (4.6), values back 95 (7.1).  The column form is bound by its
// pieces: 256 bytes of a row in, 64 bytes of a column and its scale bytes out (tiles of 256 rows x
// 128 bytes, whole lines out, were no faster).
// Columns of rows gathered from 16384 tokens: 104 us for the same tokens again, 113 to 122 for others
// each time; 65536 rows from 8192 tokens 51.  By counters about 240 MB are fetched and 150 written
// (65536 rows: 43 and 80, the columns of x that are in use staying in L2): 3.3 (2.4) TB/s, so
// memory does not bound it.  A wave waits for 60 % of its cycles: a tile is one chain of dependent
// loads (padded total, segment, row index, row), which four workgroups per CU (33 KB of LDS each)
// do not hide.
#include <algorithm>

#include "many_groups.h"
#include "mx_device.h"
#include "mx_internal.h"
#include "mx_rows.h"
#include "nv4_internal.h"
#include "../../include/nv4moe.h"

namespace nv4 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kXcds = 8;
constexpr uint32_t kNoLoad = 0x80000000u;  // behind every tile (128 rows of at most 16 MiB)

// a row index clamped into x
__device__ __forceinline__ uint32_t clamp_row(const MxQuantArgs &a, int32_t i) {
  return (uint32_t)min(max(i, 0), (int)(a.x_rows - 1));
}

// U units (mx_rows.h) per 16-lane group
template <bool F32, int U>
__global__ __launch_bounds__(256) void k_mx_rows(MxQuantArgs a, uint32_t units, uint32_t spr) {
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const uint32_t wave = group_index() * 4 + (threadIdx.x >> 6);
  const uint32_t first = wave * (4 * U) + (lane >> 4);
  uint4 v[U][F32 ? 2 : 1];
  uint32_t row[U], seg[U], src[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t unit = first + u * 4;
    row[u] = unit / spr;
    seg[u] = unit - row[u] * spr;
    src[u] = row[u];
  }
  if (a.row_index) {  // all of them before the first dependent load: loads return in order
#pragma unroll
    for (int u = 0; u < U; ++u) src[u] = clamp_row(a, a.row_index[min(row[u], (uint32_t)a.rows - 1)]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t unit = first + u * 4;
    const int64_t col = (int64_t)seg[u] * 128 + l16 * 8;
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[u][i] = make_uint4(0, 0, 0, 0);
    if (unit < units && col < a.K) {
      const int64_t at = (int64_t)src[u] * a.ldx + col;
      const uint4 *p = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(a.x) + at)
                           : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at);
#pragma unroll
      for (int i = 0; i < (F32 ? 2 : 1); ++i) v[u][i] = p[i];
    }
  }
  bool bad = false;
  const int64_t sld = (a.K / kMxBlock + 3) / 4 * 4;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t c, d;
    bad |= mx_unit<F32>(v[u], l16, a.ceil_rule, c, d);
    const int64_t col = (int64_t)seg[u] * 128 + l16 * 8;
    if (first + u * 4 < units) {
      if (col < a.K) *reinterpret_cast<uint32_t *>(a.codes + (int64_t)row[u] * (a.K / 2) + col / 2) = c;
      if (l16 == 0) *reinterpret_cast<uint32_t *>(a.scales + (int64_t)row[u] * sld + seg[u] * 4) = d;
    }
  }
  if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
}

// One tile: 128 positions of one segment x TC columns (256 bytes of a row).  BATCHED: the
// segments are the nseg equal matrices; otherwise their padded starts are multiples of 128,
// so a tile lies in one segment.  LDS row r keeps dword p of the tile at p ^ (16 * (r / 32 % 4)):
// the four 32-row blocks that a wave's lanes read at once then fall into different banks.
template <bool F32, bool BATCHED, bool ROWS>
__global__ __launch_bounds__(256) void k_mx_cols(MxQuantArgs a, int chunks, int64_t m, uint32_t n) {
  constexpr int TC = F32 ? 64 : 128;
  __shared__ uint32_t tile[128 * 64];
  __shared__ int32_t s_seg[4];  // segment, its padded start, its rows
  const int tid = threadIdx.x, l16 = tid & 15;
  // Each XCD (workgroup i runs on XCD i % 8) takes a contiguous share of the tiles, so that the
  // pieces of an output line that several tiles write meet in one L2.  Chunk by chunk down a
  // column tile for the column output (its 64-byte pieces); with gathered rows an XCD then reads
  // few columns of x, which its L2 keeps between the k copies of a token.  ROWS: two (FP32: four)
  // column tiles side by side, 128 bytes of a row's codes: 131072 x 2048 BF16 230 -> 203 us.
  const uint32_t b0 = group_index(), per = n / kXcds, full = per * kXcds;
  if (b0 >= n) return;  // uniform
  const uint32_t L = b0 < full ? (b0 % kXcds) * per + b0 / kXcds : b0;
  constexpr uint32_t G = ROWS ? 256 / TC : 1;
  const uint32_t g0 = L / (G * chunks) * G, gw = min(G, n / chunks - g0), in = L - g0 * chunks;
  const uint32_t ch = in / gw, ct = g0 + in - ch * gw;
  int64_t row0, valid, p0, out_row0;
  if (BATCHED) {
    const uint32_t cpm = (uint32_t)((m + 127) / 128);
    const uint32_t s = ch / cpm;
    p0 = (int64_t)(ch - s * cpm) * 128;
    row0 = (int64_t)s * m + p0;
    valid = m - p0;
    out_row0 = (int64_t)s * a.K;
  } else {
    p0 = (int64_t)ch * 128;
    if (p0 >= a.seg_padded_offsets[a.nseg]) return;  // uniform
    // the last segment whose padded start is <= p0, every thread a candidate: one round trip for
    // up to 256 segments where a binary search takes eight (with the loads below: 131072 x 2048
    // BF16 159 -> 139 us, gathered from 16384 rows 130 -> 91)
    if (tid < 4) s_seg[tid] = 0;  // (starts that do not begin at 0 leave an empty segment)
    __syncthreads();
    for (int lo = 0, n = a.nseg;;) {
      const int step = (n + 255) / 256, at = lo + tid * step;
      if (tid * step < n) {
        const int32_t start = a.seg_padded_offsets[at], r0 = a.seg_offsets[at], r1 = a.seg_offsets[at + 1];
        const bool last = (tid + 1) * step >= n || a.seg_padded_offsets[at + step] > p0;
        if (start <= p0 && last) s_seg[0] = at, s_seg[1] = start, s_seg[2] = r0, s_seg[3] = r1;
      }
      __syncthreads();
      if (step == 1) break;
      n = min(step, n - (s_seg[0] - lo));
      lo = s_seg[0];
      __syncthreads();
    }
    row0 = s_seg[2] + (p0 - s_seg[1]);
    valid = min((int64_t)s_seg[3], a.rows) - row0;
    if (row0 < 0) valid = 0;
    out_row0 = 0;
  }
  const int64_t col0 = (int64_t)ct * TC;
  const int64_t mycol = col0 + l16 * (F32 ? 4 : 8);
  uint4 v[8];
  constexpr int ES = F32 ? 4 : 2;
  if (!a.row_index) {
    // rows of one matrix: 32-bit offsets into the tile, whose range check gives the zeros
    const uint32_t ld = (uint32_t)a.ldx * ES;
    const auto src = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(static_cast<const char *>(a.x)) + row0 * a.ldx * ES, (short)0,
        (int)(uint32_t)(max(min(valid, (int64_t)128), (int64_t)0) * ld), 0x00020000);
    uint32_t at = (tid >> 4) * ld + (uint32_t)mycol * ES;
#pragma unroll
    for (int i = 0; i < 8; ++i, at += 16 * ld) {
      const auto t = __builtin_amdgcn_raw_buffer_load_b128(src, mycol < a.K ? at : kNoLoad, 0, 0);
      v[i] = make_uint4(t[0], t[1], t[2], t[3]);
    }
  } else {
    int32_t idx[8];  // all of them before the first dependent load: loads return in order
#pragma unroll
    for (int i = 0; i < 8; ++i)
      idx[i] = a.row_index[min(max(row0 + i * 16 + (tid >> 4), (int64_t)0), a.rows - 1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (i * 16 + (tid >> 4) < valid && mycol < a.K)
        v[i] = *reinterpret_cast<const uint4 *>(static_cast<const char *>(a.x) +
                                                ((int64_t)clamp_row(a, idx[i]) * a.ldx + mycol) * ES);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 16 + (tid >> 4);
    *reinterpret_cast<uint4 *>(&tile[r * 64 + ((l16 * 4) ^ (16 * ((r >> 5) & 3)))]) = v[i];
  }
  bool bad = false;
  if (ROWS) {
    const int64_t sld = (a.K / kMxBlock + 3) / 4 * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 16 + (tid >> 4);
      uint32_t mx, byte, c, d;
      if constexpr (F32) {
        mx = oct_umax(mx_amax4_f32(v[i]));
        byte = mx_scale_byte(mx, a.ceil_rule);
        c = mx_pack4_f32(v[i], mx_scale_value(byte));
        d = byte << (8 * (l16 >> 3));
        d |= (uint32_t)__builtin_amdgcn_mov_dpp((int)d, 0x128, 0xF, 0xF, false);  // row_ror:8
      } else {
        mx = quad_umax(mx_amax8_bf16(v[i]));
        byte = mx_scale_byte(mx, a.ceil_rule);
        c = mx_pack8_bf16(v[i], mx_scale_value(byte));
        d = byte << (8 * (l16 >> 2));
        d |= (uint32_t)__builtin_amdgcn_mov_dpp((int)d, 0x124, 0xF, 0xF, false);  // row_ror:4
        d |= (uint32_t)__builtin_amdgcn_mov_dpp((int)d, 0x128, 0xF, 0xF, false);  // row_ror:8
      }
      if (byte == kMxNan) c = 0u;  // the column pass below raises the flag
      if (r < valid) {
        if (mycol < a.K) {
          uint8_t *p = a.codes2 + (row0 + i * 16) * (a.K / 2) + ((tid >> 4) * (uint32_t)(a.K / 2) + (uint32_t)(mycol / 2));
          if constexpr (F32) *reinterpret_cast<uint16_t *>(p) = (uint16_t)c;
          else *reinterpret_cast<uint32_t *>(p) = c;
        }
        if (l16 == 0) {
          uint8_t *p = a.scales2 + (row0 + i * 16) * sld + ((tid >> 4) * (uint32_t)sld + (uint32_t)(col0 / kMxBlock));
          if constexpr (F32) *reinterpret_cast<uint16_t *>(p) = (uint16_t)d;
          else *reinterpret_cast<uint32_t *>(p) = d;
        }
      }
    }
  }
  __syncthreads();
  // thread = dword column w, 32-row block b (the four blocks of a column in a quad)
  const int b = tid & 3, w = tid >> 2;
  uint32_t q[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) q[i] = tile[(b * 32 + i) * 64 + (w ^ (16 * b))];
  const int64_t oK = a.out_K, osld = (oK / kMxBlock + 3) / 4 * 4;
  const bool whole = p0 + b * 32 < oK;  // BATCHED: blocks behind the matrix's rows do not exist
  constexpr int NC = F32 ? 1 : 2;
  uint32_t amax[NC];
  if constexpr (F32) {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) mx = max(mx, q[i] & 0x7FFFFFFFu);
    amax[0] = mx;
  } else {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) mx = pk_umax16(mx, q[i] & 0x7FFF7FFFu);
    amax[0] = mx << 16;
    amax[1] = mx & 0xFFFF0000u;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint32_t wc = w * NC + c;
    const int64_t col = col0 + wc;
    const uint32_t byte = mx_scale_byte(amax[c], a.ceil_rule);
    const float s = mx_scale_value(byte);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t acc = 0;
      if constexpr (F32) {
        acc = mx_pack_f32<0>(acc, __uint_as_float(q[8 * j]), __uint_as_float(q[8 * j + 1]), s);
        acc = mx_pack_f32<1>(acc, __uint_as_float(q[8 * j + 2]), __uint_as_float(q[8 * j + 3]), s);
        acc = mx_pack_f32<2>(acc, __uint_as_float(q[8 * j + 4]), __uint_as_float(q[8 * j + 5]), s);
        acc = mx_pack_f32<3>(acc, __uint_as_float(q[8 * j + 6]), __uint_as_float(q[8 * j + 7]), s);
      } else {
        // the two rows' values of this column as one pair: low halves (column 0) or high halves
        const uint32_t sel = c == 0 ? 0x05040100u : 0x07060302u;
        acc = mx_pack_bf16<0>(acc, __builtin_amdgcn_perm(q[8 * j + 1], q[8 * j], sel), s);
        acc = mx_pack_bf16<1>(acc, __builtin_amdgcn_perm(q[8 * j + 3], q[8 * j + 2], sel), s);
        acc = mx_pack_bf16<2>(acc, __builtin_amdgcn_perm(q[8 * j + 5], q[8 * j + 4], sel), s);
        acc = mx_pack_bf16<3>(acc, __builtin_amdgcn_perm(q[8 * j + 7], q[8 * j + 6], sel), s);
      }
      o[j] = byte == kMxNan ? 0u : acc;
    }
    bad |= byte == kMxNan;
    const uint32_t d = quad_or(byte << (8 * b));
    if (col < a.K) {
      if (whole)
        *reinterpret_cast<uint4 *>(a.codes + (out_row0 + col0) * (oK / 2) + p0 / 2 +
                                   ((uint64_t)wc * (uint32_t)(oK / 2) + (uint32_t)(b * 16))) =
            make_uint4(o[0], o[1], o[2], o[3]);
      if (b == 0) 
        *reinterpret_cast<uint32_t *>(a.scales + (out_row0 + col0) * osld + p0 / kMxBlock +
                                      (uint64_t)wc * (uint32_t)osld) = d;
    }
  }
  if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
}

// Values of U units.  BF16: a lane takes 8 codes of a unit, one 16-byte store; FP32: 4 codes of
// either half, so that both of its stores are contiguous over the lanes.  The output is stored as
// streamed (non-temporal): nothing reads it here.  131072 x 2048 BF16 129 -> 93 us.
template <bool F32, int U>
__global__ __launch_bounds__(256) void k_mx_dequant(MxDequantArgs a, uint32_t units, uint32_t spr) {
  constexpr int H = F32 ? 2 : 1, W = 8 / H;  // accesses per unit, codes each
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const uint32_t first = (group_index() * 4 + (threadIdx.x >> 6)) * (4 * U) + (lane >> 4);
  const int64_t sld = (a.K / kMxBlock + 3) / 4 * 4;
  uint32_t c[U][H], row[U], d[U];
  int64_t col[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t unit = first + u * 4;
    row[u] = unit / spr;
    const uint32_t seg = unit - row[u] * spr;
    col[u] = unit < units ? (int64_t)seg * 128 + l16 * W : a.K;
    d[u] = 0;
    if (unit < units) d[u] = *reinterpret_cast<const uint32_t *>(a.scales + (int64_t)row[u] * sld + seg * 4);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      c[u][h] = 0;
      if (col[u] + h * 64 < a.K) {
        const uint8_t *p = a.codes + (int64_t)row[u] * (a.K / 2) + (col[u] + h * 64) / 2;
        if constexpr (F32) c[u][h] = *reinterpret_cast<const uint16_t *>(p);
        else c[u][h] = *reinterpret_cast<const uint32_t *>(p);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (col[u] + h * 64 >= a.K) continue;
      const uint32_t byte = (d[u] >> (8 * (F32 ? 2 * h + (l16 >> 3) : l16 >> 2))) & 255u;
      const float s = mx_scale_value(byte);
      const int64_t at = (int64_t)row[u] * a.ldo + col[u] + h * 64;
      if constexpr (F32) {
        const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u][h], s, 0);
        const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u][h], s, 1);
        const float nan = __builtin_nanf("");
        __builtin_nontemporal_store(
            byte == kMxNan ? f32x4{nan, nan, nan, nan} : f32x4{lo[0], lo[1], hi[0], hi[1]},
            reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at));
      } else {
        u32x4 t;
        t[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u][h], s, 0));
        t[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u][h], s, 1));
        t[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u][h], s, 2));
        t[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[u][h], s, 3));
        if (byte == kMxNan) t = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        __builtin_nontemporal_store(t, reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + at));
      }
    }
  }
}

// padded[s] = exclusive prefix sum of the lengths rounded up to 128 (nseg <= 1024): within the
// waves by shuffles, then over the waves before
__global__ __launch_bounds__(1024) void k_mx_padded_offsets(const int32_t *offsets, int nseg, int32_t *padded) {
  __shared__ int total[16];
  const int s = threadIdx.x, lane = s & 63, wave = s >> 6;
  const int len = s < nseg ? offsets[s + 1] - offsets[s] : 0;
  const int own = (len + kMxSegment - 1) / kMxSegment * kMxSegment;
  int sum = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(sum, o, 64);
    if (lane >= o) sum += x;
  }
  if (lane == 63) total[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) sum += total[w];
  if (s < nseg) padded[s] = sum - own;
  if (s == nseg - 1) padded[nseg] = sum;
}

template <bool F32>
void launch_rows(const MxQuantArgs &a, hipStream_t stream) {
  const int64_t spr = (a.K + 127) / 128, units = a.rows * spr;
  // Two units per lane keep two loads in flight (65536 x 2048 BF16: 56 us; four: 63); with few
  // units one each spreads them wider.
  const bool many = units >= (int64_t)device_cu_count() * 64;
  const unsigned per = many ? 32 : 16;
  const dim3 grid = many_groups((units + per - 1) / per);
  if (many) k_mx_rows<F32, 2><<<grid, 256, 0, stream>>>(a, (uint32_t)units, (uint32_t)spr);
  else k_mx_rows<F32, 1><<<grid, 256, 0, stream>>>(a, (uint32_t)units, (uint32_t)spr);
}

template <bool F32>
void launch_cols(const MxQuantArgs &a, hipStream_t stream) {
  constexpr int TC = F32 ? 64 : 128;
  // whole 128-column units, so that the padding of the row-direction scales is written
  const int64_t ctiles = (a.K + 127) / 128 * (128 / TC);
  if (a.layout == NV4_COLS_BATCHED) {
    const int64_t m = a.rows / a.nseg, chunks = a.nseg * ((m + 127) / 128);
    const int64_t n = ctiles * chunks;
    k_mx_cols<F32, true, false><<<many_groups(n), 256, 0, stream>>>(a, (int)chunks, m, (uint32_t)n);
    return;
  }
  // every segment ends at most 127 columns of padding behind its rows
  const int64_t chunks = std::min(a.out_K / 128, (a.rows + 127 * (int64_t)a.nseg) / 128);
  if (chunks == 0) return;
  const uint32_t n = (uint32_t)(ctiles * chunks);
  const dim3 grid = many_groups(n);
  if (a.layout == NV4_COLS) k_mx_cols<F32, false, false><<<grid, 256, 0, stream>>>(a, (int)chunks, 0, n);
  else k_mx_cols<F32, false, true><<<grid, 256, 0, stream>>>(a, (int)chunks, 0, n);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs &a, hipStream_t stream) {
  if (a.rows == 0 || a.K == 0) return hipSuccess;
  if (a.layout == NV4_ROWS) {
    if (a.x_is_f32) launch_rows<true>(a, stream); else launch_rows<false>(a, stream);
  } else {
    if (a.x_is_f32) launch_cols<true>(a, stream); else launch_cols<false>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxDequantArgs &a, hipStream_t stream) {
  if (a.rows == 0 || a.K == 0) return hipSuccess;
  const int64_t spr = (a.K + 127) / 128, units = a.rows * spr;
  const bool many = units >= (int64_t)device_cu_count() * 64;
  const unsigned per = many ? 32 : 16;
  const dim3 grid = many_groups((units + per - 1) / per);
  const uint32_t n = (uint32_t)units, s = (uint32_t)spr;
  if (a.out_is_f32) {
    if (many) k_mx_dequant<true, 2><<<grid, 256, 0, stream>>>(a, n, s);
    else k_mx_dequant<true, 1><<<grid, 256, 0, stream>>>(a, n, s);
  } else {
    if (many) k_mx_dequant<false, 2><<<grid, 256, 0, stream>>>(a, n, s);
    else k_mx_dequant<false, 1><<<grid, 256, 0, stream>>>(a, n, s);
  }
  return hipGetLastError();
}

hipError_t launch_mx_padded_offsets(const int32_t *offsets, int nseg, int32_t *padded, hipStream_t stream) {
  k_mx_padded_offsets<<<1, (unsigned)(nseg + 63) / 64 * 64, 0, stream>>>(offsets, nseg, padded);
  return hipGetLastError();
}

}  // namespace nv4
