// The microscaled 4-bit copy of a W12 record for the Q pass (SpecPilot, arXiv 2611.02501, summary
// page, Main Findings: the RTX PRO 6000 port reads a separate low-bit copy in the Q pass; the pages
// give no quantiser).  It is block floating point with 4-bit elements, the element and block sizes
// of the OCP microscaling formats:
//   a block is 32 columns of a row; e = the largest exponent field among the block's in-window
//   weights (the window bottom for a block with none), scale 2^(e - 127 - 2);
//   an in-window weight becomes the E2M1 code (sign, 2 exponent bits, 1 mantissa bit: magnitudes 0,
//   0.5, 1, 1.5, 2, 3, 4, 6) nearest to weight / scale, ties to the even code, saturating at 6;
//   escaped slots hold code 0 and stay exact through the record's escape list.
// The scale is stored as the exponent field the decoded weight w' = w / 2^(base - 112) needs
// (w12_device.hpp), s = e - 2 - base + 112 in 110..125, so decoding never leaves the normal range
// and the GEMMs finish a row with the same 2^(base - 112) as the exact pass.
//
// Storage: one tile record of 1088 bytes per 16 rows x 128 columns, row-tile-major.  Lane
// l = r + 16 g of a wave owns row r, columns 32 g .. 32 g + 31 -- one block: its 32 codes are the 16
// bytes at 16 l (column 2 i in the low nibble of byte i), its scale the byte at 1024 + l.
#include "mx4_device.hpp"
#include "w12_launch.hpp"

namespace w12 {

// The escapes of row `row` from column c on: the index of the first (every lane its own row and c).
__device__ __forceinline__ uint32_t first_escape(const uint32_t* __restrict__ esc_col, uint32_t lo, uint32_t hi,
                                                 uint32_t c) {
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (esc_col[mid] < c) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// One wave's part of the copy's list of escapes that are not zero: tile row `tr`'s escapes in order, 64
// at a time, packed from the place of its first escape in the record's list.  (The product reads
// only those, since a zero contributes what its code does.)
__device__ __forceinline__ void nonzero_escapes(const Planes& p, int64_t tr, int64_t n, uint32_t* __restrict__ nz_ptr,
                                                uint32_t* __restrict__ nz_end, uint32_t* __restrict__ nz_col,
                                                uint16_t* __restrict__ nz_val, int lane) {
  const int64_t row0 = tr * kTileRows;
  // lane r <= 16: where row row0 + r starts (rows past n: the end)
  const int64_t rr = row0 + (lane < kTileRows ? lane : kTileRows);
  const uint32_t start = p.esc_ptr[rr < n ? rr : n];
  const uint32_t t0 = __builtin_amdgcn_readfirstlane(start);
  const uint32_t t1 = (uint32_t)__builtin_amdgcn_readlane(start, kTileRows);
  uint32_t kept = t0, mine = t0;                   // kept so far; kept ahead of this lane's row
  for (uint32_t e0 = t0; e0 < t1; e0 += 64) {
    const uint32_t e = e0 + (uint32_t)lane;
    const uint32_t col = e < t1 ? p.esc_col[e] : 0u;
    const uint16_t val = e < t1 ? p.esc_val[e] : (uint16_t)0;
    const bool keep = (val & 0x7FFFu) != 0;
    const uint64_t b = __ballot(keep);
    if (keep) {
      const uint32_t at = kept + (uint32_t)__popcll(b & ((1ull << lane) - 1));
      nz_col[at] = col;
      nz_val[at] = val;
    }
    if (start >= e0 && start < e0 + 64) mine = kept + (uint32_t)__popcll(b & ((1ull << (start - e0)) - 1));
    kept += (uint32_t)__popcll(b);
  }
  if (start >= t1 && t1 > t0) mine = kept;         // rows that start at the list's end
  const uint32_t next = (uint32_t)__shfl_down((int)mine, 1);
  if (lane < kTileRows && row0 + lane < n) {
    nz_ptr[row0 + lane] = mine;
    nz_end[row0 + lane] = lane == kTileRows - 1 ? kept : next;
    if (row0 + lane == n - 1) nz_ptr[n] = kept;
  }
}

// One wave per tile: lane l decodes its block's 32 window values, takes their largest exponent
// (an escaped slot's placeholder has the window's lowest, so it never raises it and stands for a
// block without weights), and converts.  Rows past n get zeros.  The placeholder's code is 0
// already, as an escaped slot's has to be, unless the block's own exponent is within 3 of the window
// bottom (2^-2 of the scale ties to 0): only such a block looks its escapes up.
// The last list_blocks workgroups write the list of escapes that are not zero, a wave per tile row
// (as a launch of its own, and one more for the escaped slots, [5120, 5120] built and read back in
// 33 us instead of 27).  Bound by memory, 1.5 bytes read and 17/32 written per weight:
// [5120, 5120] 11.6 us (4.6 TB/s), [34816, 5120] 58 us (6.2 TB/s).
__global__ __launch_bounds__(kBlock) void k_mx4_build(Planes p, int64_t n, int64_t k, uint8_t* __restrict__ q,
                                                      uint32_t* __restrict__ nz_ptr, uint32_t* __restrict__ nz_end,
                                                      uint32_t* __restrict__ nz_col, uint16_t* __restrict__ nz_val,
                                                      int list_blocks) {
  const int lane = threadIdx.x & 63;
  const int64_t ktiles = k / kTileCols;
  const int64_t trows = (n + kTileRows - 1) / kTileRows, tiles = trows * ktiles;
  const int64_t tile_blocks = (int64_t)gridDim.x - list_blocks;
  if ((int64_t)blockIdx.x >= tile_blocks) {
    const int64_t nw = (int64_t)list_blocks * (kBlock / 64);
    for (int64_t tr = (blockIdx.x - tile_blocks) * (kBlock / 64) + (threadIdx.x >> 6); tr < trows; tr += nw)
      nonzero_escapes(p, tr, n, nz_ptr, nz_end, nz_col, nz_val, lane);
    return;
  }
  const uint32_t e112 = exp112_pair();
  const int64_t step = tile_blocks * (kBlock / 64);
  for (int64_t t = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6); t < tiles; t += step) {
    const int64_t tr = t / ktiles, row = tr * kTileRows + (lane & 15);
    const bool live = row < n;
    const u32x4 a0 = load_nt(reinterpret_cast<const u32x4*>(p.ae + t * kTileAE + 16 * lane));
    const u32x4 a1 = load_nt(reinterpret_cast<const u32x4*>(p.ae + t * kTileAE + 1024 + 16 * lane));
    const u32x4 b = load_nt(reinterpret_cast<const u32x4*>(p.lo + t * kTileLO + 16 * lane));
    uint32_t w[16];
    window_group8(a0.x, a0.y, b.x, e112, w);
    window_group8(a0.z, a0.w, b.y, e112, w + 4);
    window_group8(a1.x, a1.y, b.z, e112, w + 8);
    window_group8(a1.z, a1.w, b.w, e112, w + 12);
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t l16 = w[i] & 0x7F80u, h16 = (w[i] >> 16) & 0x7F80u;
      big = big > l16 ? big : l16;
      big = big > h16 ? big : h16;
    }
    const uint32_t s = (big >> 7) - 2u;
    const float scale = __uint_as_float(s << 23);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mx4_encode8(w + 4 * i, scale);
    if (live && s <= kMXLowest + 3) {
      const uint32_t c0 = (uint32_t)(t - tr * ktiles) * kTileCols + 32u * (lane >> 4);
      const uint32_t e1 = p.esc_ptr[row + 1];
      for (uint32_t e = first_escape(p.esc_col, p.esc_ptr[row], e1, c0); e < e1; ++e) {
        const uint32_t j = p.esc_col[e] - c0;      // column within the block: nibble j
        if (j >= 32) break;
        const uint32_t m = ~(0xFu << (4 * (j % 8)));
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] &= j / 8 == (uint32_t)i ? m : 0xFFFFFFFFu;
      }
    }
    if (!live) o = (u32x4){0u, 0u, 0u, 0u};
    uint8_t* dst = q + t * kTileMX;
    *reinterpret_cast<u32x4*>(dst + 16 * lane) = o;
    dst[1024 + lane] = live ? (uint8_t)s : (uint8_t)0;
  }
}

// The bfloat16 matrix the Q pass multiplies.  One wave per tile; w' times 2^(base - 112) is exact in
// bfloat16 (at the lowest windows as a subnormal), so the high half of the float product is the
// value.  A lane's 32 columns are 64 bytes of its row, but stored as they lie each store would touch
// 16 bytes of 64 pieces; so the tile turns in LDS and leaves as whole 256-byte row pieces (16 lanes
// each, rotated by the row against bank conflicts): gate+up [34816, 5120] 136.1 -> 86 us; and past
// the caches, which nothing of it would stay in: 73 us.  The escapes go over their slots there: each
// lane finds those of its own block in its row's list.  Bound by memory, 17/32 bytes read and 2
// written per weight: those 73 us are 6.2 TB/s, [5120, 5120] takes 14.2 us (4.7 TB/s).
__global__ __launch_bounds__(kBlock) void k_mx4_decode(Planes pl, int64_t n, int64_t k, uint16_t* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) u32x4 s_t[kBlock / 64][256];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  u32x4* const st = s_t[threadIdx.x >> 6];
  const int64_t ktiles = k / kTileCols;
  const int64_t tiles = (n + kTileRows - 1) / kTileRows * ktiles;
  const int64_t step = (int64_t)gridDim.x * (kBlock / 64);
  for (int64_t t = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6); t < tiles; t += step) {
    const int64_t tr = t / ktiles, row = tr * kTileRows + r;
    const u32x4 v = load_nt(reinterpret_cast<const u32x4*>(pl.mx4 + t * kTileMX + 16 * lane));
    const uint32_t s = pl.mx4[t * kTileMX + 1024 + lane];
    const uint32_t c0 = (uint32_t)(t - tr * ktiles) * kTileCols + 32u * g;
    uint32_t e = 0, e1 = 0;
    if (row < n) {
      e1 = pl.esc_ptr[row + 1];
      e = first_escape(pl.esc_col, pl.esc_ptr[row], e1, c0);
    }
    const float rs = window_scale(row < n ? pl.base[row] : 112u);
    uint32_t p[16];
    mx4_pairs(v, s, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = p[4 * i + j];
        const uint32_t f0 = __float_as_uint(bf16_to_float(w & 0xFFFFu) * rs);
        const uint32_t f1 = __float_as_uint(__uint_as_float(w & 0xFFFF0000u) * rs);
        o[j] = __builtin_amdgcn_perm(f1, f0, 0x07060302u);
      }
      st[16 * r + ((4 * g + i + r) & 15)] = o;     // piece 4 g + i of row r
    }
    for (; e < e1; ++e) {
      const uint32_t j = pl.esc_col[e] - c0;
      if (j >= 32) break;
      reinterpret_cast<uint16_t*>(&st[16 * r + ((4 * g + (int)(j / 8) + r) & 15)])[j % 8] = pl.esc_val[e];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rr = 4 * i + g;                    // 16 lanes a row
      const u32x4 o = st[16 * rr + ((r + rr) & 15)];
      if (tr * kTileRows + rr < n)
        __builtin_nontemporal_store(
            o, reinterpret_cast<u32x4*>(out + (tr * kTileRows + rr) * k + (t - tr * ktiles) * kTileCols + 8 * r));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

static unsigned mx4_grid(const DevInfo& di, int64_t waves) {
  const int64_t blocks = (waves + 3) / 4, cap = (int64_t)di.cus * 32;
  return (unsigned)(blocks < cap ? blocks : cap);
}

hipError_t launch_mx4_build(const Planes& p, int64_t n, int64_t k, uint8_t* q, uint32_t* nz_ptr, uint32_t* nz_end,
                            uint32_t* nz_col, uint16_t* nz_val, hipStream_t s) {
  DevInfo di;
  hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  const int64_t trows = (n + kTileRows - 1) / kTileRows;
  const unsigned lists = mx4_grid(di, trows);
  hipLaunchKernelGGL(k_mx4_build, dim3(mx4_grid(di, trows * (k / kTileCols)) + lists), dim3(kBlock), 0, s, p, n, k, q,
                     nz_ptr, nz_end, nz_col, nz_val, (int)lists);
  return hipGetLastError();
}

hipError_t launch_mx4_decode(const Planes& p, int64_t n, int64_t k, uint16_t* out, hipStream_t s) {
  DevInfo di;
  hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  const int64_t tiles = (n + kTileRows - 1) / kTileRows * (k / kTileCols);
  hipLaunchKernelGGL(k_mx4_decode, dim3(mx4_grid(di, tiles)), dim3(kBlock), 0, s, p, n, k, out);
  return hipGetLastError();
}

}  // namespace w12
