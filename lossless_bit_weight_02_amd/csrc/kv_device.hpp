// The paged cache and the batch of new tokens as the kernels see them (w12_kv, w12_kv_batch of
// w12.h), and a row's way from its number to its place.
#pragma once

#include "w12_device.hpp"
#include "w12_launch.hpp"

namespace w12 {

// Inclusive sum over the wave's lanes up to each, by DPP.
__device__ __forceinline__ int lane_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15, 31
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The same of 64-bit values.
template <int CTRL, int ROWS, class V>
__device__ __forceinline__ V lane_step(V v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
}
template <class V>
__device__ __forceinline__ V lane_scan(V v) {
  static_assert(sizeof(V) == 8);
  v = lane_step<0x111, 0xF>(v);
  v = lane_step<0x112, 0xF>(v);
  v = lane_step<0x114, 0xF>(v);
  v = lane_step<0x118, 0xF>(v);
  v = lane_step<0x142, 0xA>(v);
  return lane_step<0x143, 0xC>(v);
}
__device__ __forceinline__ int last_lane(int v) { return __builtin_amdgcn_readlane(v, 63); }
template <class V>
__device__ __forceinline__ V last_lane(V v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63);
  return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
}

// A sequence's rows and lengths.
struct SeqRows {
  int64_t first;      // its first new token's row
  int64_t count;      // T, 0 for an empty or senseless one (their rows from m on do not exist)
  int64_t len;        // places it has, new ones included
};

__device__ __forceinline__ SeqRows seq_rows(const BatchArgs& b, int64_t s) {
  SeqRows r;
  r.len = b.lens[s];
  if (b.q_start == nullptr) {
    r.first = s;
    r.count = 1;
    return r;
  }
  r.first = b.q_start[s];
  const int64_t end = b.q_start[s + 1];
  r.count = r.first >= 0 && end > r.first ? end - r.first : 0;
  return r;
}

// The sequence that row i belongs to, -1 for none: the last s with q_start[s] <= i, by all lanes of a
// wave at once, a 64th of the range each step.  Every index stays in 0 .. seqs whatever the values.
__device__ __forceinline__ int64_t find_seq(const BatchArgs& b, int64_t i) {
  if (b.q_start == nullptr) return i < b.seqs ? i : -1;
  const int lane = threadIdx.x & 63;
  int64_t cur = 0, len = b.seqs + 1;
  while (len > 1) {
    const int64_t step = (len + 63) / 64;
    const int64_t at = lane * step;
    const uint64_t bl = __ballot(at < len && b.q_start[cur + (at < len ? at : 0)] <= i);
    if (bl == 0) return -1;
    const int64_t last = (__popcll(bl) - 1) * step;
    cur += last;
    len = len - last < step ? len - last : step;
  }
  return cur < b.seqs ? cur : -1;
}

// The page that holds place c of sequence s, -1 where the place does not exist.
__device__ __forceinline__ int64_t page_of(const KvArgs& kv, const BatchArgs& b, int64_t s, int64_t c) {
  if (c < 0 || c >= b.cols * kv.page) return -1;
  const int32_t p = b.table[s * b.table_stride + (uint32_t)c / (uint32_t)kv.page];
  return p >= 0 && p < kv.pages ? p : -1;
}

}  // namespace w12
