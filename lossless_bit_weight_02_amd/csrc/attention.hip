// Attention of a step's new tokens over the paged cache.
//
// The rows of one sequence that read the same keys are its T new tokens times the G = hq / heads query heads
// of a key head; 16 of them are a column block of the matrix instruction.  A wave takes 32 places at a
// time and keeps all of it in registers:
//   S^T = K Q^T    K is the A operand as it lies in the cache: lane (r, g) = (lane % 16, lane / 16) holds
//                  place r's columns 8 g .. +7 of each 32, so a load is a piece of a row.  The result
//                  has the row of q in lane % 16 and places 4 g .. 4 g + 3 of either 16 in its registers.
//   softmax        per row of q the running maximum (in units of log 2) is the same in its four lanes, each
//                  of which sums its own places.  A probability may pass 1 by 2^8 before the maximum
//                  moves, so nearly every step needs neither a reduction over lanes nor a rescaling.
//   O^T += V^T P^T the eight probabilities a lane has are its B operand as they are, if the eight places
//                  of V^T's operand are those same ones: lane (r, g) loads `kRun` columns (r kRun ..) of
//                  them, eight rows, and turns the eight rows of 16-bit values in its registers (one byte
//                  permute per pair).  No value passes between lanes, and nothing goes through LDS.
// Probabilities meet V as two bfloat16 terms (the leading 8 bits and the rest, 16 bits together): one would
// be off by as much again as the output's own rounding.
//
// Split.  The work of the whole batch is a line of units of 128 places (of one sequence, key head and
// block of rows); every workgroup takes an equal run of it, found from the lengths on the device, so
// uneven batches fill the chip alike and a captured graph follows its lengths.  A workgroup's four
// waves take 32 of the 128 places each (kWr = 1), or 64 by pairs (2) or all of them (4) for as many blocks
// of 16 rows more, and join through LDS.  A run that ends inside a sequence leaves
// a partial (sum, maximum, unnormalised output) in the scratch; whoever counts itself last joins them.
#include "kv_device.hpp"

namespace w12 {

constexpr int kAtUnit = 128;                      // places of a unit
constexpr float kAtLog2e = 1.44269504088896340736f;
constexpr float kAtSlack = 8.0f;                  // powers of two a probability may pass 1 by
constexpr int kAuxAgent = 16;                     // sc1: stores and loads that every die of the device sees

struct AttnArgs {
  const uint16_t* q;
  int64_t ldq;
  int m, hq, group;       // group: query heads of a key head
  KvArgs kv;
  BatchArgs b;
  int cap;                // places of the table
  int page_tiles;         // 16-place tiles of a page
  uint32_t page_magic;    // ceil(2^32 / page_tiles)
  float scale;            // of the scores, times log2 e
  uint16_t* y;
  int wgs;
  uint32_t* count;        // [wgs], zero between calls
  float* part;            // [2 wgs] partials: [rows][dim] sums, [rows] maxima, [rows] sums of probabilities
};

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// eight e4m3 values as bfloat16
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, bool high) {
  return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                           : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ u32x4 e4m3_run(uint32_t a, uint32_t b) {
  return u32x4{e4m3_pair(a, false), e4m3_pair(a, true), e4m3_pair(b, false), e4m3_pair(b, true)};
}

template <int DIM, bool E4M3>
struct AttnShape {
  static constexpr int kSize = E4M3 ? 1 : 2;
  static constexpr int kFrag = DIM / 32;                     // 32-column pieces of a key row
  static constexpr int kLoads = DIM * kSize / 64;            // 16-byte loads of a lane for 16 key rows
  static constexpr int kSubs = DIM / 16;                     // 16-column blocks of the output
  static constexpr int kRun = kSubs * kSize < 16 ? kSubs : 16 / kSize;   // columns of a lane's load of V
  static constexpr int kRuns = kSubs / kRun;                 // such loads per place
  static constexpr int kRunWords = kRun * kSize / 4;
};

// The keys of 16 places, a lane's pieces of place lane % 16.
template <int DIM, bool E4M3>
struct KeyTile {
  using S = AttnShape<DIM, E4M3>;
  u32x4 w[S::kLoads];
  __device__ __forceinline__ void load(Rsrc tile, uint32_t off) {
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) w[i] = __builtin_amdgcn_raw_buffer_load_b128(tile, off + 64 * i, 0, 0);
  }
  // piece f as the A operand: columns 32 f + 8 g .. +7 (e4m3: 64 (f / 2) + 16 g + 8 (f % 2) ..)
  __device__ __forceinline__ bf16x8 frag(int f) const {
    if constexpr (E4M3) return as_bf16(e4m3_run(w[f / 2][2 * (f % 2)], w[f / 2][2 * (f % 2) + 1]));
    else return as_bf16(w[f]);
  }
  static __device__ __forceinline__ int column(int f, int g) {
    return E4M3 ? 64 * (f / 2) + 16 * g + 8 * (f % 2) : 32 * f + 8 * g;
  }
};

// The values of 32 places: of places 4 g .. +3 of either 16, columns kRun r .. of each 16 kRun.
template <int DIM, bool E4M3>
struct ValueTile {
  using S = AttnShape<DIM, E4M3>;
  uint32_t w[8][S::kRuns][S::kRunWords];
  __device__ __forceinline__ void load4(int e0, Rsrc tile, uint32_t off, uint32_t row_bytes) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int q = 0; q < S::kRuns; ++q) {
        const uint32_t at = off + 16 * S::kRun * S::kSize * q;
        if constexpr (S::kRunWords == 4) {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(tile, at, e * row_bytes, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[e0 + e][q][i] = v[i];
        } else if constexpr (S::kRunWords == 2) {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(tile, at, e * row_bytes, 0);
          w[e0 + e][q][0] = v[0];
          w[e0 + e][q][1] = v[1];
        } else {
          w[e0 + e][q][0] = __builtin_amdgcn_raw_buffer_load_b32(tile, at, e * row_bytes, 0);
        }
      }
    }
  }
  // block `sub` as the A operand: its rows are the columns kRun r + sub % kRun
  __device__ __forceinline__ u32x4 frag(int sub) const {
    const int q = sub / S::kRun, i = sub % S::kRun;
    u32x4 f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if constexpr (E4M3) {
        // two columns' bytes of two places next to each other, the column's pair converted
        const uint32_t t = __builtin_amdgcn_perm(w[2 * p + 1][q][i / 4], w[2 * p][q][i / 4],
                                                 (i & 2) ? 0x07030602u : 0x05010400u);
        f[p] = e4m3_pair(t, i & 1);
      } else {
        f[p] = __builtin_amdgcn_perm(w[2 * p + 1][q][i / 2], w[2 * p][q][i / 2],
                                     (i & 1) ? 0x07060302u : 0x05040100u);
      }
    }
    return f;
  }
  __device__ __forceinline__ void clear(int e, bool yes) {
#pragma unroll
    for (int q = 0; q < S::kRuns; ++q)
#pragma unroll
      for (int i = 0; i < S::kRunWords; ++i) w[e][q][i] = yes ? 0u : w[e][q][i];
  }
  // whether place e has a NaN or an infinity
  __device__ __forceinline__ bool odd(int e) const {
    bool r = false;
#pragma unroll
    for (int q = 0; q < S::kRuns; ++q)
#pragma unroll
      for (int i = 0; i < S::kRunWords; ++i) {
        const uint32_t v = w[e][q][i];
        if constexpr (E4M3) {
#pragma unroll
          for (int b = 0; b < 4; ++b) r |= (v >> (8 * b) & 0x7Fu) == 0x7Fu;
        } else {
          r |= (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
        }
      }
    return r;
  }
};

__device__ __forceinline__ int lane_get(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// The batch's line of units, its sequences 64 at a time, a lane each.
struct UnitLine {
  const AttnArgs& a;
  int rows;               // rows of q of a block
  int c0 = 0;             // the 64 sequences c0 ..
  int base = 0;           // units before them
  int first = 0, count = 0, len = 0, upto = 0;               // a lane's sequence; units up to and with it
  int total = 0;          // units of the 64
  __device__ __forceinline__ UnitLine(const AttnArgs& a_, int rows_) : a(a_), rows(rows_) {}

  __device__ __forceinline__ int blocks(int count) const {
    return (int)(((uint32_t)count * (uint32_t)a.group + (uint32_t)rows - 1) / (uint32_t)rows);
  }
  __device__ __forceinline__ int seen(int len) const { return len < 0 ? 0 : len < a.cap ? len : a.cap; }
  __device__ __forceinline__ int tiles(int len) const {
    const int n = seen(len);
    return n > 0 ? (n + kAtUnit - 1) / kAtUnit : 1;
  }
  __device__ __forceinline__ int of(int s) {
    count = 0;
    if (s < a.b.seqs) {
      const SeqRows r = seq_rows(a.b, s, a.m);
      first = (int)r.first;
      count = (int)r.count;
      len = (int)r.len;
    }
    return blocks(count) * (int)a.kv.heads * tiles(len);
  }
  __device__ __forceinline__ void fill(int lane) {
    upto = lane_scan(of(c0 + lane));
    total = lane_get(upto, 63);
  }
  // units of the whole batch
  __device__ __forceinline__ int all(int lane) {
    int sum = 0;
    for (int s = lane; s < a.b.seqs; s += 64) sum += of(s);
    return lane_get(lane_scan(sum), 63);
  }
  // the lane that has unit u (calls only ever go up the line)
  __device__ __forceinline__ int find(int u, int lane) {
    while (u >= base + total && c0 + 64 < a.b.seqs) {
      base += total;
      c0 += 64;
      fill(lane);
    }
    const uint64_t bl = __ballot(u < base + upto);
    return bl ? __ffsll((unsigned long long)bl) - 1 : 0;
  }
};

// kNq blocks of 16 rows of q a wave, kWr waves side by side with other rows, 4 / kWr on other places.
template <int DIM, bool E4M3, int NQ, int WR>
__global__ __launch_bounds__(kBlock, (DIM * NQ <= 128 ? 3 : 2)) void k_attention(AttnArgs a) {
  using S = AttnShape<DIM, E4M3>;
  constexpr int kRows = 16 * NQ * WR, kTg = 4 / WR;
  constexpr int kCols = DIM < 128 ? DIM : 128;              // columns joined at a time
  constexpr int kPitch = kCols + 4;
  __shared__ __attribute__((aligned(16))) float s_o[4][16][kPitch];
  __shared__ float s_m[4][16 * NQ], s_l[4][16 * NQ];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w % WR, tg = w / WR;
  const int wg = blockIdx.x;

  UnitLine line(a, kRows);
  int total;
  if (a.b.seqs <= 64) {
    line.fill(lane);
    total = line.total;
  } else {
    total = line.all(lane);
    line.fill(lane);
  }
  const int share = (total + a.wgs - 1) / a.wgs;
  int u = wg * share;
  const int end = u + share < total ? u + share : total;
  const uint32_t row_bytes = (uint32_t)a.kv.token_stride * S::kSize;
  const uint32_t k_off = r * row_bytes + 16 * g;
  const uint32_t v_off = 4 * g * row_bytes + r * S::kRun * S::kSize;

  while (u < end) {
    const int own = line.find(u, lane);
    const int s = line.c0 + own;
    const int first = lane_get(line.first, own), count = lane_get(line.count, own), len = lane_get(line.len, own);
    const int blocks = line.blocks(count), tiles = line.tiles(len), seen = line.seen(len);
    const int start = line.base + lane_get(line.upto, own) - blocks * (int)a.kv.heads * tiles;
    const uint32_t idx = (uint32_t)(u - start) / (uint32_t)tiles;
    const int tile0 = (u - start) - (int)idx * tiles;
    const int tile1 = tiles - tile0 < end - u ? tiles : tile0 + (end - u);
    const int hk = (int)(idx / (uint32_t)blocks), block = (int)(idx - (uint32_t)hk * blocks);
    const int seg = u - tile0;                               // the line's place of the segment's first unit
    u += tile1 - tile0;
    const int base = (len < 0 ? 0 : len) - count;            // (fewer than 2^30 rows)
    const int t_end = tile1 * kAtUnit < seen ? tile1 * kAtUnit : seen;
    const int32_t* const table = a.b.table + (int64_t)s * a.b.table_stride;
    const uint8_t* const kp = static_cast<const uint8_t*>(a.kv.k) + (int64_t)hk * a.kv.head_stride * S::kSize;
    const uint8_t* const vp = static_cast<const uint8_t*>(a.kv.v) + (int64_t)hk * a.kv.head_stride * S::kSize;
    const float scale = a.scale * (a.kv.k_scale ? a.kv.k_scale[hk] : 1.0f);

    // this wave's rows of q
    bf16x8 q[NQ][S::kFrag];
    int new_j[NQ];
    uint64_t tree[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const uint32_t row = block * kRows + (wr * NQ + n) * 16 + r;
      const bool real = row < (uint32_t)count * (uint32_t)a.group;
      const uint32_t j = real ? row / (uint32_t)a.group : 0, h = real ? row - j * a.group : 0;
      new_j[n] = (int)j;
      tree[n] = a.b.tree ? a.b.tree[first + (int)j] : 0;
      const uint16_t* const qr = a.q + (int64_t)(first + (int)j) * a.ldq + ((int64_t)hk * a.group + h) * DIM;
#pragma unroll
      for (int f = 0; f < S::kFrag; ++f) {
        u32x4 v = *reinterpret_cast<const u32x4*>(qr + KeyTile<DIM, E4M3>::column(f, g));
        if (!real) v = u32x4{0, 0, 0, 0};
        q[n][f] = as_bf16(v);
      }
    }

    floatx4 acc[NQ][S::kSubs];
    float m[NQ], l[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int c = 0; c < S::kSubs; ++c) acc[n][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // the pages of this wave's next 32 steps, two tiles of 16 places each: a lane per tile
    int page = -1, in_page = 0;
    const auto pages = [&](int t0) {
      const int t = t0 + (lane >> 1) * (32 * kTg) + (lane & 1) * 16;
      const uint32_t tile = (uint32_t)t / 16u;
      const uint32_t p = a.page_tiles == 1 ? tile : __umulhi(tile, a.page_magic);
      in_page = (int)(tile - p * (uint32_t)a.page_tiles);
      page = -1;
      if (t < t_end) {
        const int v = table[p];
        if (v >= 0 && v < a.kv.pages) page = v;
      }
    };
    // (a tile that does not exist reads page 0, and is masked)
    const auto tile_at = [&](const uint8_t* p, int i) {
      const int pg = lane_get(page, i), in = lane_get(in_page, i);
      const int64_t at = (int64_t)(pg & ~(pg >> 31)) * a.kv.page_stride * S::kSize + (int64_t)in * 16 * row_bytes;
      return make_rsrc(p + at, 0x7FFFFFFF);
    };

    KeyTile<DIM, E4M3> key[2];
    ValueTile<DIM, E4M3> val;
    int t = tile0 * kAtUnit + tg * 32, i = 0;
    if (t < t_end) {
      pages(t);
      key[0].load(tile_at(kp, 0), k_off);
      key[1].load(tile_at(kp, 1), k_off);
      val.load4(0, tile_at(vp, 0), v_off, row_bytes);
      val.load4(4, tile_at(vp, 1), v_off, row_bytes);
    }
    while (t < t_end) {
      const int pg0 = lane_get(page, 2 * i), pg1 = lane_get(page, 2 * i + 1);
      floatx4 sc[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[n][h] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int f = 0; f < S::kFrag; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bf16x8 kf = key[h].frag(f);
#pragma unroll
          for (int n = 0; n < NQ; ++n) sc[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[n][f], sc[n][h], 0, 0, 0);
        }
      // the next step's keys, in flight while this one's values are used
      const int t_next = t + 32 * kTg;
      ++i;
      if (i == 32) {
        pages(t_next);
        i = 0;
      }
      key[0].load(tile_at(kp, 2 * i), k_off);                // (past the end: page 0)
      key[1].load(tile_at(kp, 2 * i + 1), k_off);

      const bool masked = !(t + 32 <= base && pg0 >= 0 && pg1 >= 0);
      uint32_t hide[NQ];                                     // places that a row does not see
#pragma unroll
      for (int n = 0; n < NQ; ++n) hide[n] = 0;
      int tm = t + 4 * g;                                    // (made here: few steps are masked)
      asm volatile("" : "+v"(tm));
      const auto there = [&](int e) { return tm + (e < 4 ? e : 12 + e) < seen && (e < 4 ? pg0 : pg1) >= 0; };
      const auto sees = [&](int n, int bit) {            // place base + bit
        return bit < 0 || (a.b.tree ? bit < count && bit < 64 && (tree[n] >> (bit & 63) & 1) : bit <= new_j[n]);
      };
      if (masked) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int bit = tm + (e < 4 ? e : 12 + e) - base;
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            if (!there(e) || !sees(n, bit)) hide[n] |= 1u << e;
        }
      }

      bf16x8 ph[NQ], pl[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = sc[n][e / 4][e % 4] * scale;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = hide[n] >> e & 1u ? -INFINITY : x[e];
        }
        float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        if (__ballot(top > m[n] + kAtSlack)) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float now = fmaxf(m[n], top);
          const float f = m[n] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[n] - now);
          m[n] = now;
          l[n] *= f;
#pragma unroll
          for (int c = 0; c < S::kSubs; ++c) acc[n][c] *= f;
        }
        const float ref = m[n] == -INFINITY ? 0.0f : m[n];
        uint32_t hi[4], lo[4];
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = __builtin_amdgcn_exp2f(x[e] - ref);
          l[n] += p[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hi[e] = __builtin_amdgcn_perm(__float_as_uint(p[2 * e + 1]), __float_as_uint(p[2 * e]), 0x07060302u);
          const float r0 = p[2 * e] - __uint_as_float(hi[e] << 16);
          const float r1 = p[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u);
          const bf16x2 rr = {(__bf16)r0, (__bf16)r1};
          lo[e] = __builtin_bit_cast(uint32_t, rr);
        }
        ph[n] = as_bf16(u32x4{hi[0], hi[1], hi[2], hi[3]});
        pl[n] = as_bf16(u32x4{lo[0], lo[1], lo[2], lo[3]});
      }

      if (masked) {
        // places of V with a NaN or an infinity, where some rows may not see them: one at a time, for the
        // rows that do; then they and the places that do not exist are nothing
        uint32_t odd = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (there(e) && val.odd(e)) odd |= 1u << e;
        if (__ballot(odd != 0)) {
#pragma unroll 1
          for (int k = 0; k < 32; ++k) {
            const int e = k >> 2, g1 = k & 3;
            if (__ballot(g == g1 && (odd >> e & 1)) == 0) continue;
            const int bit = t + (e < 4 ? 4 * g1 + e : 12 + 4 * g1 + e) - base;
            const uint32_t mine = g == g1 ? (e & 1) ? 0xFFFF0000u : 0x0000FFFFu : 0u;
#pragma unroll
            for (int c = 0; c < S::kSubs; ++c) {
              u32x4 vf = val.frag(c);
#pragma unroll
              for (int p = 0; p < 4; ++p) vf[p] &= p == e >> 1 ? mine : 0u;
#pragma unroll
              for (int n = 0; n < NQ; ++n) {
                floatx4 one = {0.0f, 0.0f, 0.0f, 0.0f};
                one = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(vf), ph[n], one, 0, 0, 0);
                one = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(vf), pl[n], one, 0, 0, 0);
                if (sees(n, bit)) acc[n][c] += one;
              }
              __builtin_amdgcn_sched_barrier(0);             // (one block's registers at a time)
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) val.clear(e, !there(e) || (odd >> e & 1));
      }
#pragma unroll
      for (int c = 0; c < S::kSubs; ++c) {
        const bf16x8 vf = as_bf16(val.frag(c));
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          acc[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, ph[n], acc[n][c], 0, 0, 0);
          acc[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl[n], acc[n][c], 0, 0, 0);
        }
      }
      val.load4(0, tile_at(vp, 2 * i), v_off, row_bytes);
      val.load4(4, tile_at(vp, 2 * i + 1), v_off, row_bytes);
      t = t_next;
    }

    // the waves' sums of the same rows into one (its addresses are made here: no registers kept for them)
    int tj = tid;
    asm volatile("" : "+v"(tj));
    const int r = tj & 15, g = tj >> 4 & 3;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] += __shfl_xor(l[n], 16);
      l[n] += __shfl_xor(l[n], 32);
      if (g == 0) {
        s_m[w][16 * n + r] = m[n];
        s_l[w][16 * n + r] = l[n];
      }
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == tiles;
    // a partial's slot: the workgroup's second if the segment begins here, else its first
    const int slot = 2 * wg + (tile0 == 0 ? 1 : 0);
    constexpr int kPart = kRows * (DIM + 2);
    const uint32_t nrows = (uint32_t)count * (uint32_t)a.group - (uint32_t)(block * kRows);
    const int valid = nrows < (uint32_t)kRows ? (int)nrows : kRows;
    const Rsrc part = make_rsrc(a.part + (size_t)slot * kPart, kPart * 4);
    const float vs = a.kv.v_scale ? a.kv.v_scale[hk] : 1.0f;
#pragma unroll 1
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int blk = 0; blk < DIM / kCols; ++blk) {
        // columns blk kCols .. of the waves' outputs, relative to the rows' common maximum
        if (n > 0 || blk > 0) __syncthreads();
#pragma unroll
        for (int nn = 0; nn < NQ; ++nn) {
          if (nn != n) continue;
          float top = -INFINITY;
#pragma unroll
          for (int v = 0; v < kTg; ++v) top = fmaxf(top, s_m[v * WR + wr][16 * nn + r]);
          const float f = m[nn] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[nn] - top);
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
#pragma unroll
            for (int c = 0; c < S::kSubs; ++c) {
              // column of block c's row 4 g + ii
              const int col0 = c / S::kRun * (16 * S::kRun) + c % S::kRun;
              constexpr int kHalf = S::kRuns > 1 ? 1 : 0;
              const int col = col0 + S::kRun * (4 * g + ii);
              if (kHalf || DIM == kCols) {
                if (c / (kCols / 16) == blk || DIM == kCols) s_o[w][r][col - blk * kCols] = acc[nn][c][ii] * f;
              } else if ((4 * g + ii) / 8 == blk) {
                s_o[w][r][col - blk * kCols] = acc[nn][c][ii] * f;
              }
            }
          }
        }
        __syncthreads();
        // WR blocks of 16 rows x kCols columns, four columns a thread at a time
        constexpr int kItems = WR * 16 * kCols / 4;
        for (int it = tj; it < kItems; it += kBlock) {
          const int c4 = it % (kCols / 4), rr = it / (kCols / 4) % 16, gr = it / (kCols / 4 * 16);
          const int row = (gr * NQ + n) * 16 + rr;
          if (row >= valid) continue;
          float top = -INFINITY;
#pragma unroll
          for (int v = 0; v < kTg; ++v) top = fmaxf(top, s_m[v * WR + gr][16 * n + rr]);
          float sum = 0.0f;
          floatx4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int v = 0; v < kTg; ++v) {
            const float mv = s_m[v * WR + gr][16 * n + rr];
            sum += mv == -INFINITY ? s_l[v * WR + gr][16 * n + rr] : s_l[v * WR + gr][16 * n + rr] * __builtin_amdgcn_exp2f(mv - top);
            o += *reinterpret_cast<const floatx4*>(&s_o[v * WR + gr][rr][4 * c4]);
          }
          const int col = blk * kCols + 4 * c4;
          if (whole) {
            const float f = sum == 0.0f ? 0.0f : vs / sum;
            const uint32_t rq = block * kRows + row, j = rq / (uint32_t)a.group, h = rq - j * a.group;
            uint16_t* const out = a.y + ((int64_t)(first + (int)j) * a.hq + (int64_t)hk * a.group + h) * DIM + col;
            u32x2 v;
            v[0] = (uint32_t)float_to_bf16_rne(o[0] * f) | (uint32_t)float_to_bf16_rne(o[1] * f) << 16;
            v[1] = (uint32_t)float_to_bf16_rne(o[2] * f) | (uint32_t)float_to_bf16_rne(o[3] * f) << 16;
            *reinterpret_cast<u32x2*>(out) = v;
          } else {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), part, (row * DIM + col) * 4, 0, kAuxAgent);
            if (col == 0) {
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(top), part, (kRows * DIM + row) * 4, 0, kAuxAgent);
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sum), part, (kRows * (DIM + 1) + row) * 4, 0, kAuxAgent);
            }
          }
        }
      }
    }
    if (!whole) {
      // the workgroups that share the segment: first to last of those that own its units
      const int from = seg / share, to = (seg + tiles - 1) / share;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tj == 0) {
        const uint32_t old = __hip_atomic_fetch_add(&a.count[from], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = old == (uint32_t)(to - from) ? 1 : 0;
        if (s_last) __hip_atomic_store(&a.count[from], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (s_last) {
        asm volatile("" ::: "memory");
        for (int it = tj; it < valid * (DIM / 4); it += kBlock) {
          const int row = it / (DIM / 4), col = it % (DIM / 4) * 4;
          float top = -INFINITY, sum = 0.0f;
          for (int p = from; p <= to; ++p) {
            const Rsrc b = make_rsrc(a.part + (size_t)(2 * p + (p == from ? 1 : 0)) * kPart, kPart * 4);
            top = fmaxf(top, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (kRows * DIM + row) * 4, 0, kAuxAgent)));
          }
          floatx4 o = {0.0f, 0.0f, 0.0f, 0.0f};
          for (int p = from; p <= to; ++p) {
            const Rsrc b = make_rsrc(a.part + (size_t)(2 * p + (p == from ? 1 : 0)) * kPart, kPart * 4);
            const float mv = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (kRows * DIM + row) * 4, 0, kAuxAgent));
            const float lv = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (kRows * (DIM + 1) + row) * 4, 0, kAuxAgent));
            const floatx4 ov = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(b, (row * DIM + col) * 4, 0, kAuxAgent));
            const float f = mv == -INFINITY ? (lv == lv ? 0.0f : lv) : __builtin_amdgcn_exp2f(mv - top);
            sum += lv * f;
            o += ov * f;
          }
          const float f = sum == 0.0f ? 0.0f : vs / sum;
          const uint32_t rq = block * kRows + row, j = rq / (uint32_t)a.group, h = rq - j * a.group;
          uint16_t* const out = a.y + ((int64_t)(first + (int)j) * a.hq + (int64_t)hk * a.group + h) * DIM + col;
          u32x2 v;
          v[0] = (uint32_t)float_to_bf16_rne(o[0] * f) | (uint32_t)float_to_bf16_rne(o[1] * f) << 16;
          v[1] = (uint32_t)float_to_bf16_rne(o[2] * f) | (uint32_t)float_to_bf16_rne(o[3] * f) << 16;
          *reinterpret_cast<u32x2*>(out) = v;
        }
      }
    }
    __syncthreads();
  }
}

// Rows of q a workgroup takes at once, by the average of a sequence.
struct AttnPlan {
  int nq, wr, rows;
  int wgs;
  bool fits;              // the line of units has fewer than 2^31
};
static AttnPlan attn_plan(const DevInfo& di, int64_t m, int64_t hq, const KvArgs& kv, const BatchArgs& b) {
  const int64_t group = hq / kv.heads, avg = (m * group + b.seqs - 1) / b.seqs;
  AttnPlan p;
  if (kv.dim == 256) {
    p.nq = 1;
    p.wr = avg <= 16 ? 1 : avg <= 32 ? 2 : 4;
  } else {
    p.nq = avg <= 16 ? 1 : 2;
    p.wr = avg <= 32 ? 1 : 2;
  }
  p.rows = 16 * p.nq * p.wr;
  const double most = ((double)m * group / p.rows + (double)b.seqs) * (double)kv.heads *
                      ((double)b.cols * kv.page / kAtUnit + 1.0);
  p.fits = most < 2147483648.0 && m * hq < (int64_t(1) << 30);
  p.wgs = di.cus * 2;
  if (p.fits && most < p.wgs) p.wgs = (int)most + 1;
  return p;
}

constexpr uint64_t kAtCounts = 4096;                         // counts ahead of the partials
static uint64_t attn_part(const AttnPlan& p, int64_t dim) { return (uint64_t)p.rows * (dim + 2) * sizeof(float); }

bool attention_fits(const DevInfo& di, int64_t m, int64_t hq, const KvArgs& kv, const BatchArgs& b) {
  return attn_plan(di, m, hq, kv, b).fits;
}

uint64_t attention_scratch(const DevInfo& di, int64_t m, int64_t hq, const KvArgs& kv, const BatchArgs& b,
                           uint64_t* zero) {
  const AttnPlan p = attn_plan(di, m, hq, kv, b);
  *zero = kAtCounts * sizeof(uint32_t);
  return *zero + 2 * (uint64_t)p.wgs * attn_part(p, kv.dim);
}

template <int DIM, int NQ, int WR>
static void attn_go(const AttnArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.wgs);
  if (a.kv.e4m3) hipLaunchKernelGGL((k_attention<DIM, true, NQ, WR>), grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL((k_attention<DIM, false, NQ, WR>), grid, dim3(kBlock), 0, s, a);
}

hipError_t launch_attention(const uint16_t* q, int64_t ldq, int64_t m, int64_t hq, const KvArgs& kv,
                            const BatchArgs& b, float scale, uint16_t* y, void* scratch, hipStream_t s) {
  DevInfo di;
  const hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  const AttnPlan p = attn_plan(di, m, hq, kv, b);
  if (!p.fits || (uint64_t)p.wgs > kAtCounts) return hipErrorInvalidValue;
  AttnArgs a;
  a.q = q; a.ldq = ldq;
  a.m = (int)m; a.hq = (int)hq; a.group = (int)(hq / kv.heads);
  a.kv = kv; a.b = b;
  a.cap = (int)(b.cols * kv.page);
  a.page_tiles = (int)(kv.page / 16);
  // (exact below 2^26 tiles: the rounding of the reciprocal, under page_tiles <= 64, times that is under 2^32)
  a.page_magic = (uint32_t)(((uint64_t(1) << 32) + a.page_tiles - 1) / a.page_tiles);
  a.scale = scale * kAtLog2e;
  a.y = y;
  a.wgs = p.wgs;
  a.count = static_cast<uint32_t*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + kAtCounts * sizeof(uint32_t));
  if (kv.dim == 64) {
    if (p.wr == 2) attn_go<64, 2, 2>(a, s);
    else if (p.nq == 2) attn_go<64, 2, 1>(a, s);
    else attn_go<64, 1, 1>(a, s);
  } else if (kv.dim == 128) {
    if (p.wr == 2) attn_go<128, 2, 2>(a, s);
    else if (p.nq == 2) attn_go<128, 2, 1>(a, s);
    else attn_go<128, 1, 1>(a, s);
  } else {
    if (p.wr == 4) attn_go<256, 1, 4>(a, s);
    else if (p.wr == 2) attn_go<256, 1, 2>(a, s);
    else attn_go<256, 1, 1>(a, s);
  }
  return hipGetLastError();
}

}  // namespace w12
