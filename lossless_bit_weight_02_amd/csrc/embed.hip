// Embedding lookup from a W12 record: out[j][c] = scale * W[ids[j]][c].
//
// A model whose embedding table is its LM head (tied weights) then keeps one record for both ends
// of a step, instead of a second, dense copy for the lookup.
//
// Work split.  A wave takes 1024 columns of one looked-up row: lane l decodes the 16 columns
// 16 (l % 8) .. +15 of the wave's 128-column block l / 8 (one 16-byte load of the AE plane, one
// 8-byte load of the B plane), so one id of a 5120-column table already spreads over five waves.
// The decoded row piece goes to LDS, the row's escapes inside the piece overwrite their slots
// there, and the piece leaves in 16-byte stores.
//
// Decode: the window trick's w' (w12_device.hpp) has the exponent field 112 + E, the weight
// base + E, so adding base - 112 to the exponent field gives the exact bfloat16 bits.  Scaling is one
// product in float; bfloat16 outputs round it once, to nearest even (half a step, 2^-8 relative).
//
// What bounds it: the record's tile order, made for the GEMMs.  A row's bytes lie in it as 16-byte
// pieces 256 bytes apart, each fetched as 64, so 4096 rows of 5120 columns read 128 MB (counted)
// for their 31 MB, and write 42 MB: 49 us back to back, 3.5 TB/s (52 as one call among others; float
// rows, 84 MB written, 57.5).  (The dense gather with its scaling, reading 42 MB: 79.6 us as elementary
// operations.)  16 rows: 3.4 us, a launch's latency.
#include "w12_device.hpp"
#include "w12_launch.hpp"

namespace w12 {

constexpr int kEmbCols = 1024;                  // columns of a row one wave takes

// Between LDS accesses of one wave's lanes to each other's slots: orders them for the compiler (the
// hardware keeps a wave's LDS accesses in order).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <bool PAST, class T>
__device__ __forceinline__ void put(void* at, const T& v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, static_cast<T*>(at));
  else *static_cast<T*>(at) = v;
}

// PAST: stores go past the caches.  ids: int32 or (ids64) int64.  An id outside 0 .. n-1 reads nothing and gives a row of zeros.
// OUT16: bfloat16 outputs, else float.  RAW (with OUT16): scale is 1, the weight's own bits.
template <bool OUT16, bool RAW, bool PAST>
__global__ __launch_bounds__(kBlock) void k_embed(const void* __restrict__ ids, int ids64, int64_t cnt,
                                                  Planes p, int64_t n, int64_t k, float scale,
                                                  void* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint16_t s_w[kBlock / 64][kEmbCols];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint16_t* const sw = s_w[w];
  const uint32_t e112 = exp112_pair();
  const int64_t chunks = (k + kEmbCols - 1) / kEmbCols;
  const int64_t ktiles = k / kTileCols;
  const int64_t items = cnt * chunks, step = (int64_t)gridDim.x * (kBlock / 64);
  for (int64_t it = (int64_t)blockIdx.x * (kBlock / 64) + w; it < items; it += step) {
    const int64_t j = it / chunks, ch = it - j * chunks;
    const int64_t id = ids64 ? static_cast<const int64_t*>(ids)[j] : (int64_t)static_cast<const int32_t*>(ids)[j];
    const bool real = id >= 0 && id < n;
    const int64_t row = real ? id : 0;
    const int64_t kb = ch * (kEmbCols / kTileCols) + (lane >> 3);
    const bool have = real && kb < ktiles;
    const int g = (lane & 7) >> 1, h = lane & 1, r = (int)(row & 15);
    u32x4 a = {0u, 0u, 0u, 0u};
    u32x2 b = {0u, 0u};
    uint32_t e0 = 0, e1 = 0, bs = 112;
    if (have) {
      const int64_t t = (row >> 4) * ktiles + kb;
      a = *reinterpret_cast<const u32x4*>(p.ae + t * kTileAE + 1024 * h + 16 * (r + 16 * g));
      b = *reinterpret_cast<const u32x2*>(p.lo + t * kTileLO + 16 * (r + 16 * g) + 8 * h);
    }
    if (real) {
      e0 = p.esc_ptr[row];
      e1 = p.esc_ptr[row + 1];
      bs = p.base[row];
    }
    uint32_t v[8];
    window_group8(a.x, a.y, b.x, e112, v);
    window_group8(a.z, a.w, b.y, e112, v + 4);
    const short d = (short)(((int)bs - 112) * 128);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const short2v s = __builtin_bit_cast(short2v, v[i]) + (short2v){d, d};
      v[i] = have ? __builtin_bit_cast(uint32_t, s) : 0u;
    }
    // columns 16 l .. +15 of the piece
    u32x4* dst = reinterpret_cast<u32x4*>(sw + 16 * lane);
    dst[0] = (u32x4){v[0], v[1], v[2], v[3]};
    dst[1] = (u32x4){v[4], v[5], v[6], v[7]};
    wave_fence();
    // the escapes of the piece (columns ascend within the row: the first one at or past the piece
    // by bisection, which every lane does alike)
    const int64_t c0 = ch * kEmbCols;
    if (e1 > e0) {
      uint32_t lo = e0, hi = e1;
      if (e1 - e0 > 64)
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if ((int64_t)p.esc_col[mid] < c0) lo = mid + 1;
          else hi = mid;
        }
      for (uint32_t eb = lo; eb < e1; eb += 64) {
        const uint32_t e = eb + (uint32_t)lane;
        const int64_t c = e < e1 ? (int64_t)p.esc_col[e] - c0 : (int64_t)kEmbCols;
        if (c >= 0 && c < kEmbCols) sw[c] = p.esc_val[e];
        if (__ballot(c >= kEmbCols) != 0) break;   // past the piece
      }
    }
    wave_fence();
    // 8 columns per lane and store
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = 512 * q + 8 * lane;
      const u32x4 x = *reinterpret_cast<const u32x4*>(sw + c);
      if (c0 + c >= k) continue;                 // (k is a multiple of 128: whole stores)
      const int64_t at = j * k + c0 + c;
      if constexpr (RAW) {
        put<PAST>(static_cast<uint16_t*>(out) + at, x);
      } else {
        float f[8];
        const float sc = real || fabsf(scale) < INFINITY ? scale : 0.0f;   // (padding: zeros at any scale)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16_to_float(x[i] & 0xFFFFu) * sc;
          f[2 * i + 1] = bf16_to_float(x[i] >> 16) * sc;
        }
        if constexpr (OUT16) {
          u32x4 o;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = (uint32_t)float_to_bf16_rne(f[2 * i]) | (uint32_t)float_to_bf16_rne(f[2 * i + 1]) << 16;
          put<PAST>(static_cast<uint16_t*>(out) + at, o);
        } else {
          put<PAST>(static_cast<float*>(out) + at, (floatx4){f[0], f[1], f[2], f[3]});
          put<PAST>(static_cast<float*>(out) + at + 4, (floatx4){f[4], f[5], f[6], f[7]});
        }
      }
    }
    wave_fence();                                // the next piece overwrites the slots
  }
}

hipError_t launch_embed(const void* ids, bool ids64, int64_t cnt, const Planes& p, int64_t n, int64_t k,
                        float scale, void* out, bool out16, hipStream_t s) {
  const int64_t items = cnt * ((k + kEmbCols - 1) / kEmbCols);
  int64_t blocks = (items + 3) / 4;
  if (blocks > (1 << 20)) blocks = 1 << 20;
  const dim3 grid((unsigned)blocks), block(kBlock);
  const int i64 = ids64 ? 1 : 0;
  // Outputs of more than an L2's 4 MiB go past the caches, which hold the sectors of the table meanwhile
  // (5120 columns, scaled: 4096 rows 53.7 -> 49.0 us, 1024 rows 16.9 -> 15.2; 256 rows 7.2 and 6.8, 16
  // rows 3.4 and 3.4: small ones are left to the caches for whoever reads them next).
  const bool past = cnt * k * (out16 ? 2 : 4) > (int64_t(4) << 20);
  typedef void (*Kernel)(const void*, int, int64_t, Planes, int64_t, int64_t, float, void*);
  const Kernel f = !out16          ? (past ? k_embed<false, false, true> : k_embed<false, false, false>)
                   : scale == 1.0f ? (past ? k_embed<true, true, true> : k_embed<true, true, false>)
                                   : (past ? k_embed<true, false, true> : k_embed<true, false, false>);
  hipLaunchKernelGGL(f, grid, block, 0, s, ids, i64, cnt, p, n, k, scale, out);
  return hipGetLastError();
}

}  // namespace w12
