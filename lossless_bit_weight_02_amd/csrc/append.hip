// Rows of the stacked q/k/v product into a decoding step's cache: q and k rotated by position, k and v
// into the pages.
//
// The pair (x_a, x_b) of a head turns by its position's angle, (x_a cos - x_b sin, x_b cos + x_a sin),
// all in float; cosines and sines come from the caller's table, which was made once in as many bits
// as far positions need.
//
// Work split.  A unit is 16 columns of a head whose pairs are complete in it: a rotated half's 8 columns and
// their 8 partners half a rotation away (or 16 side by side where pairs are), or 16 columns of a head
// that does not turn.  A thread takes a unit: every access is 16 bytes or more, the columns of a row that
// neighbouring lanes hold lie side by side, and one token of 64 heads already spreads over two
// workgroups.  A workgroup stays in one row, so its place, page and position are looked up once for all.
// A unit of q is written by the thread that has read it, so q_out may be q.
//
// What bounds it: memory for prompts (5 of 1024 .. 4096 tokens of 48 + 2 * 8 heads of 128 columns from float,
// 595 MB in 106 us, 5.6 TB/s; a plain copy on this card 4.95), the launch for single tokens (the kernel
// 3.2 us, the call 8.4), the lookups' chain of loads and the division by the scale for drafts (64 sequences
// of 16 into e4m3, 25 MB in 8.4 us).
#include "kv_device.hpp"

namespace w12 {

struct Vec8 {
  float v[8];
};

template <bool F32>
__device__ __forceinline__ Vec8 load8(const void* p, int64_t at) {
  Vec8 r;
  if constexpr (F32) {
    const floatx4* f = reinterpret_cast<const floatx4*>(static_cast<const float*>(p) + at);
    const floatx4 a = f[0], b = f[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[i] = a[i];
      r.v[4 + i] = b[i];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = __uint_as_float(w[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  return r;
}

__device__ __forceinline__ u32x4 pack_bf16(const Vec8& x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)float_to_bf16_rne(x.v[2 * i]) | (uint32_t)float_to_bf16_rne(x.v[2 * i + 1]) << 16;
  return w;
}

// value / scale as e4m3, to nearest even after the clamp (a NaN passes it)
__device__ __forceinline__ u32x2 pack_e4m3(const Vec8& x, float scale) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = x.v[4 * i + j] / scale;
      q[j] = t != t ? t : fminf(fmaxf(t, -448.0f), 448.0f);
    }
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], r, true);
    w[i] = (uint32_t)r;
  }
  return w;
}

template <bool F32, bool PAIRS, bool E4M3>
__global__ __launch_bounds__(kBlock) void k_append(AppendArgs a, KvArgs kv, BatchArgs b, int chunks, int64_t first) {
  const int64_t row = first + blockIdx.x / chunks;
  const int units = (int)kv.dim / 16;                       // of a head
  const int unit = (int)(blockIdx.x % chunks) * kBlock + threadIdx.x;
  const int64_t s = find_seq(b, row);
  if (s < 0) return;
  const SeqRows sr = seq_rows(b, s);
  if (row >= sr.first + sr.count) return;
  const int64_t place = sr.len - sr.count + (row - sr.first);
  const int64_t pos = b.positions ? b.positions[row] : place;
  const bool turns = a.rot == 0 || (pos >= 0 && pos < a.rope_rows);
  const int64_t page = turns ? page_of(kv, b, s, place) : -1;
  const int64_t head = unit / units;
  if (head >= a.hq + 2 * kv.heads) return;
  const int in = unit % units;
  const bool is_q = head < a.hq, is_v = head >= a.hq + kv.heads;
  if (!is_q && page < 0) return;
  const int64_t h = is_q ? head : is_v ? head - a.hq - kv.heads : head - a.hq;
  // the unit's two runs of 8 columns, and whether they turn
  const int rot = (int)a.rot;
  const bool turn = !is_v && in * 16 < rot;
  const int ca = turn && !PAIRS ? 8 * in : 16 * in;
  const int cb = turn && !PAIRS ? rot / 2 + 8 * in : 16 * in + 8;
  const void* src = is_q ? a.q : is_v ? a.v : a.k;
  const int64_t at = row * (is_q ? a.ldq : is_v ? a.ldv : a.ldk) + h * kv.dim;
  Vec8 x = load8<F32>(src, at + ca), z = load8<F32>(src, at + cb);
  if (turn) {
    const int64_t p = turns ? pos : 0;
    const Vec8 c = load8<true>(a.rope, p * rot + 8 * in), sn = load8<true>(a.rope, p * rot + rot / 2 + 8 * in);
    if constexpr (PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = x.v[2 * i], x1 = x.v[2 * i + 1], z0 = z.v[2 * i], z1 = z.v[2 * i + 1];
        x.v[2 * i] = x0 * c.v[i] - x1 * sn.v[i];
        x.v[2 * i + 1] = x1 * c.v[i] + x0 * sn.v[i];
        z.v[2 * i] = z0 * c.v[4 + i] - z1 * sn.v[4 + i];
        z.v[2 * i + 1] = z1 * c.v[4 + i] + z0 * sn.v[4 + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x0 = x.v[i], z0 = z.v[i];
        x.v[i] = x0 * c.v[i] - z0 * sn.v[i];
        z.v[i] = z0 * c.v[i] + x0 * sn.v[i];
      }
    }
  }
  if (is_q) {
    uint16_t* const o = a.q_out + (row * a.hq + h) * kv.dim;
    const u32x4 zero = {0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(o + ca) = turns ? pack_bf16(x) : zero;
    *reinterpret_cast<u32x4*>(o + cb) = turns ? pack_bf16(z) : zero;
    return;
  }
  const int64_t to = page * kv.page_stride + h * kv.head_stride + (int64_t)((uint32_t)place % (uint32_t)kv.page) * kv.token_stride;
  if constexpr (E4M3) {
    const float* const sp = is_v ? kv.v_scale : kv.k_scale;
    const float sc = sp ? sp[h] : 1.0f;
    uint8_t* const o = static_cast<uint8_t*>(is_v ? kv.v : kv.k) + to;
    *reinterpret_cast<u32x2*>(o + ca) = pack_e4m3(x, sc);
    *reinterpret_cast<u32x2*>(o + cb) = pack_e4m3(z, sc);
  } else {
    uint16_t* const o = static_cast<uint16_t*>(is_v ? kv.v : kv.k) + to;
    *reinterpret_cast<u32x4*>(o + ca) = pack_bf16(x);
    *reinterpret_cast<u32x4*>(o + cb) = pack_bf16(z);
  }
}

template <bool F32, bool PAIRS>
static void append_go(const AppendArgs& a, const KvArgs& kv, const BatchArgs& b, int chunks, int64_t first,
                      dim3 grid, hipStream_t s) {
  if (kv.e4m3) hipLaunchKernelGGL((k_append<F32, PAIRS, true>), grid, dim3(kBlock), 0, s, a, kv, b, chunks, first);
  else hipLaunchKernelGGL((k_append<F32, PAIRS, false>), grid, dim3(kBlock), 0, s, a, kv, b, chunks, first);
}

hipError_t launch_kv_append(const AppendArgs& a, const KvArgs& kv, const BatchArgs& b, hipStream_t s) {
  const int64_t units = (a.hq + 2 * kv.heads) * (kv.dim / 16);
  const int chunks = (int)((units + kBlock - 1) / kBlock);
  // a launch holds fewer than 2^32 work items
  const int64_t rows = ((int64_t(1) << 31) / kBlock) / chunks;
  for (int64_t r0 = 0; r0 < a.m; r0 += rows) {
    const int64_t cnt = a.m - r0 < rows ? a.m - r0 : rows;
    const dim3 grid((unsigned)(cnt * chunks));
    if (a.f32 && a.pairs) append_go<true, true>(a, kv, b, chunks, r0, grid, s);
    else if (a.f32) append_go<true, false>(a, kv, b, chunks, r0, grid, s);
    else if (a.pairs) append_go<false, true>(a, kv, b, chunks, r0, grid, s);
    else append_go<false, false>(a, kv, b, chunks, r0, grid, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace w12
