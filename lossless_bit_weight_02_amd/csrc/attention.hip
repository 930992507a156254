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
// Probabilities meet bfloat16 values as two bfloat16 terms (the leading 8 bits and the rest, 16 bits
// together): one would be off by as much again as the output's own rounding.  e4m3 values are float16
// exactly, so there float16 terms do (11 bits each), the probabilities brought up to 2^15: those too
// small for it are off by 2^-32 of the largest.  Two terms (22 bits) cost k_attention nothing (64 sequences of one token,
// 6 rows each, 67.2 us with one, 67.9 with two); k_attention_rows, whose products are the most of it, has one (16 trees
// of 256 columns 90 us, with two 120; of 128 columns 93 and 108): there the output is off by 0.9e-3 of
// its size from what float probabilities give, half its own rounding (1.7e-3 in all, as without).
//
// Split.  The work of the whole batch is a line of units of 128 places (of one sequence, key head and
// block of rows); every workgroup takes an equal run of it, found from the lengths on the device, so
// uneven batches fill the chip alike and a captured graph follows its lengths.  A workgroup's four
// waves take 32 of the 128 places each and join through LDS (k_attention: 16 or 32 rows), or its eight waves
// take 16 rows each and all places (k_attention_rows: up to 128).  A run that ends inside a segment leaves a partial
// (unnormalised sum, maximum, sum of probabilities) in the scratch, which a second kernel joins.
//
// What bounds it: few rows read the cache once, and the loads of keys and values (16 bytes a lane, past the
// caches: nothing is read twice; 64 sequences of 60 .. 8192 places, 48 heads over 8 of 128 columns, 88 us
// so, 92 through them) run at 6.4 TB/s in a long sequence (131071 places, 537 MB: 84 us and 10 to join), at 5.4
// where 64 sequences end unevenly (76 + 12 us), at 6.0 over 256 sequences (1.67 GB: 277 + 10 us).  One
// sequence of 517 places is a chain of steps, 11 us for 2 MB.  Trees of 16 drafts and 6 heads over an e4m3
// cache of 256 columns (184 MB) take 79 us and 10 to join: their 1 .. 16 drafts fill 1 .. 6 of a block's eight waves, which
// wait 69 % of their time, the idle ones at the barriers and the others for a step's chain of LDS reads, products
// and softmax with less than one of them a SIMD (LDS is in use 29 % of the time, the vector units 19, the matrix
// cores 10; without loads 61 us, without products 54).
// Prompts are not what this split is for: a block of rows goes through all of its sequence's places, also those behind
// its last row's, and has every step of a whole prompt as a masked one (5 of 1206 .. 3941 tokens, 48 heads: 2.6 ms, the
// products alone 0.33; 2048 tokens behind 32768 places 3.9 ms, 1.4).
#include "kv_device.hpp"

namespace w12 {

constexpr int kAtUnit = 128;                      // places of a unit
// Units of a segment worth a workgroup of their own: with 8, one sequence of 517 places takes 11.5 us and 16
// trees over 1000 .. 16384 places 88, with 4 15.9 and 88, with 16 11.5 and 98.
constexpr int kAtPiece = 8;
// Units that a segment's beginning and end cost: with 2, 64 and 256 sequences take 89 and 289 us, with 0
// 121 and 308, with 4 90 and 299.
constexpr int kAtStart = 2;
constexpr float kAtLog2e = 1.44269504088896340736f;
constexpr float kAtSlack = 8.0f;                  // powers of two a probability may pass 1 by
constexpr int kAtWideRows = 128, kAtWide = 512;   // rows and threads of k_attention_rows

struct Split;

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
  Split* split;           // [wgs]
  float* part;            // [2 wgs] partials: [rows][dim] sums, [rows] maxima, [rows] sums of probabilities
};

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// acc + V^T P^T: e4m3 values and their probabilities as float16, bfloat16 ones in bfloat16
template <bool E4M3>
__device__ __forceinline__ floatx4 mfma_pv(u32x4 v, u32x4 p, floatx4 acc) {
  if constexpr (E4M3)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, v), __builtin_bit_cast(f16x8, p), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(v), as_bf16(p), acc, 0, 0, 0);
}

// a pair of e4m3 values as float16 (exact)
__device__ __forceinline__ uint32_t e4m3_pair16(uint32_t w, bool high) {
  return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}
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

// A lane's share of 32 places' keys or values as they lie in the cache.
//   keys:   of place r of either 16, 16 bytes at 64 i + 16 g of the row
//   values: of places 4 g .. +3 of either 16 (e = 0 .. 3, 4 .. 7), columns kRun r .. of each 16 kRun
// PARTS = 2: of one of the 16s (h = 0 here), of one of the runs of columns.
template <int DIM, bool E4M3, int PARTS = 1>
struct RawTile {
  using S = AttnShape<DIM, E4M3>;
  static constexpr int kRuns = S::kRuns / PARTS;
  uint32_t w[DIM * S::kSize / 8 / PARTS];

  __device__ __forceinline__ void load_keys(int h, const uint8_t* at_tile, uint32_t off) {
    const Rsrc tile = make_rsrc(at_tile, 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) put4(h * S::kLoads + i, __builtin_amdgcn_raw_buffer_load_b128(tile, off, 64 * i, kAuxNT));
  }
  __device__ __forceinline__ void put4(int i, u32x4 v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[4 * i + k] = v[k];
  }
  // keys h as the A operand, piece f: columns key_column(f, g) .. +7 of place r
  __device__ __forceinline__ bf16x8 key(int h, int f) const {
    const uint32_t* const v = &w[h * S::kLoads * 4];
    if constexpr (E4M3) return as_bf16(e4m3_run(v[2 * f], v[2 * f + 1]));
    else return as_bf16(u32x4{v[4 * f], v[4 * f + 1], v[4 * f + 2], v[4 * f + 3]});
  }

  __device__ __forceinline__ void load_values(int h, const uint8_t* at_tile, uint32_t off, uint32_t row_bytes) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const Rsrc tile = make_rsrc(at_tile + (uint64_t)e * row_bytes, 0x7FFFFFFF);
#pragma unroll
      for (int q = 0; q < kRuns; ++q) {
        const int at = 16 * S::kRun * S::kSize * q;
        const int i = ((4 * h + e) * kRuns + q) * S::kRunWords;
        if constexpr (S::kRunWords == 4) {
          put4(i / 4, __builtin_amdgcn_raw_buffer_load_b128(tile, off, at, kAuxNT));
        } else if constexpr (S::kRunWords == 2) {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(tile, off, at, kAuxNT);
          w[i] = v[0];
          w[i + 1] = v[1];
        } else {
          w[i] = __builtin_amdgcn_raw_buffer_load_b32(tile, off, at, kAuxNT);
        }
      }
    }
  }
  __device__ __forceinline__ uint32_t at(int e, int q, int i) const { return w[(e * kRuns + q) * S::kRunWords + i]; }
  // values as the A operand, block c of the output: rows are the columns kRun r + c % kRun of run c / kRun
  __device__ __forceinline__ u32x4 value(int c) const {
    const int q = c / S::kRun, i = c % S::kRun;
    u32x4 f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if constexpr (E4M3) {
        // two columns' bytes of two places next to each other, the column's pair converted
        const uint32_t t = __builtin_amdgcn_perm(at(2 * p + 1, q, i / 4), at(2 * p, q, i / 4), (i & 2) ? 0x07030602u : 0x05010400u);
        f[p] = e4m3_pair16(t, i & 1);
      } else {
        f[p] = __builtin_amdgcn_perm(at(2 * p + 1, q, i / 2), at(2 * p, q, i / 2), (i & 1) ? 0x07060302u : 0x05040100u);
      }
    }
    return f;
  }
  // whether place e's values have a NaN or an infinity
  __device__ __forceinline__ bool odd(int e) const {
    bool r = false;
#pragma unroll
    for (int i = 0; i < kRuns * S::kRunWords; ++i) {
      const uint32_t v = at(e, 0, i);
      if constexpr (E4M3) {
#pragma unroll
        for (int b = 0; b < 4; ++b) r |= (v >> (8 * b) & 0x7Fu) == 0x7Fu;
      } else {
        r |= ((v & 0x7F80u) == 0x7F80u) | ((v & 0x7F800000u) == 0x7F800000u);
      }
    }
    return r;
  }
  __device__ __forceinline__ void clear(int e, bool yes) {
#pragma unroll
    for (int i = 0; i < kRuns * S::kRunWords; ++i) {
      uint32_t& v = w[e * kRuns * S::kRunWords + i];
      v = yes ? 0u : v;
    }
  }
};
// (where key pieces begin: e4m3 loads have two)
template <bool E4M3>
__device__ __forceinline__ int key_column(int f, int g) {
  return E4M3 ? 64 * (f / 2) + 16 * g + 8 * (f % 2) : 32 * f + 8 * g;
}

__device__ __forceinline__ int lane_get(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// The batch as a line that the workgroups share out, its sequences 64 at a time, a lane each.  A segment is
// one key head and block of rows of a sequence.  While the chip has a workgroup for every kAtPiece units
// of each segment, the line is those pieces, one a workgroup; else a segment takes its units and
// kAtStart more, what beginning and ending one costs, so a workgroup with many short ones is not late.
struct UnitLine {
  const AttnArgs& a;
  int rows;               // rows of q of a block
  bool pieces = true;
  int share = 1;          // of a workgroup
  int c0 = 0;             // the 64 sequences c0 ..
  int base = 0;           // the line before them
  int first = 0, count = 0, len = 0, upto = 0;               // a lane's sequence; the line up to and with it
  int total = 0;          // of the 64
  __device__ __forceinline__ UnitLine(const AttnArgs& a_, int rows_) : a(a_), rows(rows_) {}

  __device__ __forceinline__ int blocks(int count) const {
    return (int)(((uint32_t)count * (uint32_t)a.group + (uint32_t)rows - 1) / (uint32_t)rows);
  }
  __device__ __forceinline__ int seen(int len) const { return len < 0 ? 0 : len < a.cap ? len : a.cap; }
  __device__ __forceinline__ int tiles(int len) const {
    const int n = seen(len);
    return n > 0 ? (n + kAtUnit - 1) / kAtUnit : 1;
  }
  __device__ __forceinline__ int length(int tiles) const {
    return pieces ? (tiles + kAtPiece - 1) / kAtPiece : tiles + kAtStart;
  }
  __device__ __forceinline__ void read(int s) {
    count = 0;
    if (s < a.b.seqs) {
      const SeqRows r = seq_rows(a.b, s);
      first = (int)r.first;
      count = (int)r.count;
      len = (int)r.len;
    }
  }
  // of a sequence's new tokens' rows those there are
  __device__ __forceinline__ int exist(int first, int count) const {
    const int most = first >= 0 && first < a.m ? a.m - first : 0;
    return count < most ? count : most;
  }
  __device__ __forceinline__ int mine() const { return blocks(exist(first, count)) * (int)a.kv.heads * length(tiles(len)); }
  __device__ __forceinline__ void scan() {
    upto = lane_scan(mine());
    total = lane_get(upto, 63);
  }
  __device__ __forceinline__ int all(int lane) {
    int sum = 0;
    int64_t rows_n = 0;
    for (int s = lane; s < a.b.seqs; s += 64) {
      read(s);
      sum += mine();
      rows_n += exist(first, count);
    }
    return apart(rows_n) ? lane_get(lane_scan(sum), 63) : 0;
  }
  // whether the sequences' rows can be apart: a q_start that falls may give more of them than there are, and the
  // line's length and the scratch are made for no more (it is left alone then)
  __device__ __forceinline__ bool apart(int64_t rows_n) const {
    return a.b.q_start == nullptr || last_lane(lane_scan(rows_n)) <= a.m;
  }
  // the share of each workgroup; returns the line's length
  __device__ __forceinline__ int start(int lane) {
    if (a.b.seqs <= 64) {
      read(lane);
      if (!apart(exist(first, count))) return 0;
      scan();
      if (total <= a.wgs) return total;
      pieces = false;
      scan();
      share = (total + a.wgs - 1) / a.wgs;
      return total;
    }
    int sum = all(lane);
    if (sum > a.wgs) {
      pieces = false;
      sum = all(lane);
      share = (sum + a.wgs - 1) / a.wgs;
    }
    read(lane);
    scan();
    return sum;
  }
  // the lane that has place u of the line (calls only ever go up it)
  __device__ __forceinline__ int find(int u, int lane) {
    while (u >= base + total && c0 + 64 < a.b.seqs) {
      base += total;
      c0 += 64;
      read(c0 + lane);
      scan();
    }
    const uint64_t bl = __ballot(u < base + upto);
    return bl ? __ffsll((unsigned long long)bl) - 1 : 0;
  }
};

// What a workgroup has of the segment at place u of the line.
struct Segment {
  int first, count, old, seen;                               // its sequence; old: places before its new tokens
  int s, hk, block, tiles;
  int tile0, tile1;                                          // this workgroup's units
  int from, to;                                              // the workgroups that have some
  int next;                                                  // where the line goes on
  bool whole;
  __device__ __forceinline__ Segment(UnitLine& line, int u, int end, int lane) {
    const int own = line.find(u, lane);
    s = line.c0 + own;
    first = lane_get(line.first, own);
    const int all = lane_get(line.count, own), len = lane_get(line.len, own);
    count = line.exist(first, all);
    // (below -2^30 no place is within 2^30, the most rows there are, of the first new token, or in a mask)
    const int64_t before = (int64_t)len - all;
    old = before > -(1 << 30) ? (int)before : -(1 << 30);
    tiles = line.tiles(len);
    seen = line.seen(len);
    const int blocks = line.blocks(count), each = line.length(tiles);
    const int start = line.base + lane_get(line.upto, own) - blocks * (int)line.a.kv.heads * each;
    const uint32_t idx = (uint32_t)(u - start) / (uint32_t)each;
    hk = (int)(idx / (uint32_t)blocks);
    block = (int)(idx - (uint32_t)hk * blocks);
    const int seg = start + (int)idx * each;                 // where the segment begins on the line
    next = seg + each < end ? seg + each : end;
    if (line.pieces) {
      const int per = (tiles + each - 1) / each;
      tile0 = (u - seg) * per;
      tile1 = tile0 + per < tiles ? tile0 + per : tiles;
      from = seg;
    } else {
      tile0 = u - seg - kAtStart > 0 ? u - seg - kAtStart : 0;
      tile1 = next - seg - kAtStart;
      from = (seg + kAtStart) / line.share;
    }
    to = (seg + each - 1) / line.share;
    whole = from == to;
  }
  __device__ __forceinline__ int valid(int group, int rows) const {
    const uint32_t n = (uint32_t)count * (uint32_t)group - (uint32_t)(block * rows);
    return n < (uint32_t)rows ? (int)n : rows;
  }
};

// What a row of q sees of its sequence's new places: those up to `last`, and those of `mask`.  (Arithmetic, not
// branches: the same few instructions for every lane.)
struct SeenBy {
  int last;
  uint64_t mask;
  // the place `bit` after the first new one, one that exists (the places before have bit < 0)
  __device__ __forceinline__ bool operator()(int bit) const {
    return (bit <= last) | ((bit < 64) & (int)(mask >> (bit & 63) & 1));
  }
};

// The row of q at `row` of the segment's block as the B operand of K Q^T, zeros for none.
template <int DIM, bool E4M3>
__device__ __forceinline__ SeenBy load_query(const AttnArgs& a, const Segment& sg, uint32_t row, int g, bf16x8* q) {
  const bool real = row < (uint32_t)sg.count * (uint32_t)a.group;
  const uint32_t j = real ? row / (uint32_t)a.group : 0, h = real ? row - j * a.group : 0;
  const int64_t at = sg.first + (int)j;
  const uint16_t* const qr = a.q + at * a.ldq + ((int64_t)sg.hk * a.group + h) * DIM;
#pragma unroll
  for (int f = 0; f < AttnShape<DIM, E4M3>::kFrag; ++f) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(qr + key_column<E4M3>(f, g));
    q[f] = as_bf16(real ? v : u32x4{0, 0, 0, 0});
  }
  return a.b.tree ? SeenBy{-1, a.b.tree[at]} : SeenBy{(int)j, 0};
}

// Scores of eight places into probabilities relative to the running maximum m (see the top), added to l, as
// B operands, in one term (hi) or TWO.
template <bool E4M3, bool TWO, int SUBS>
__device__ __forceinline__ void soften(const float (&x)[8], float& m, float& l, floatx4 (&acc)[SUBS], u32x4& hi, u32x4& lo) {
  constexpr float kUp = E4M3 ? 7.0f : 0.0f;
  float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
  if (__ballot(top > m + kAtSlack)) {
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float now = fmaxf(m, top);
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - now);
    m = now;
    l *= f;
#pragma unroll
    for (int c = 0; c < SUBS; ++c) acc[c] *= f;
  }
  const float ref = m == -INFINITY ? 0.0f : m - kUp;
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    p[e] = __builtin_amdgcn_exp2f(x[e] - ref);
    l += p[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (E4M3) {
      const f16x2 rr = {(_Float16)p[2 * e], (_Float16)p[2 * e + 1]};
      hi[e] = __builtin_bit_cast(uint32_t, rr);
      if constexpr (TWO) {
        const f16x2 ll = {(_Float16)(p[2 * e] - (float)rr[0]), (_Float16)(p[2 * e + 1] - (float)rr[1])};
        lo[e] = __builtin_bit_cast(uint32_t, ll);
      }
    } else {
      hi[e] = __builtin_amdgcn_perm(__float_as_uint(p[2 * e + 1]), __float_as_uint(p[2 * e]), 0x07060302u);
      const bf16x2 rr = {(__bf16)(p[2 * e] - __uint_as_float(hi[e] << 16)),
                         (__bf16)(p[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u))};
      lo[e] = __builtin_bit_cast(uint32_t, rr);
    }
  }
}

// The pages of a wave's next steps: a lane per 16 places.  A tile that does not exist reads page 0, and is masked.
template <int SIZE>
struct Pages {
  int page = -1, in = 0;
  __device__ __forceinline__ void fill(const AttnArgs& a, const int32_t* table, int t, int t_end) {
    const uint32_t tile = (uint32_t)t / 16u;
    const uint32_t p = a.page_tiles == 1 ? tile : __umulhi(tile, a.page_magic);
    in = (int)(tile - p * (uint32_t)a.page_tiles);
    page = -1;
    if (t < t_end) {
      const int v = table[p];
      if (v >= 0 && v < a.kv.pages) page = v;
    }
  }
  __device__ __forceinline__ const uint8_t* tile(const AttnArgs& a, const uint8_t* p, int i, uint32_t row_bytes) const {
    const int pg = lane_get(page, i), r = lane_get(in, i);
    const int64_t at = (int64_t)(pg & ~(pg >> 31)) * a.kv.page_stride * SIZE + (int64_t)r * 16 * row_bytes;
    return p + at;
  }
};

// Four columns of row `rq` of a sequence's rows for key head hk.  (y may be q: a segment's rows of q are read by the
// workgroups that have some of it, before the one that has all of it, or the join, writes them.)
template <int DIM>
__device__ __forceinline__ void attn_put(const AttnArgs& a, int first, int hk, uint32_t rq, int col, floatx4 o) {
  const uint32_t j = rq / (uint32_t)a.group, h = rq - j * a.group;
  const bf16x2 lo = {(__bf16)o[0], (__bf16)o[1]}, hi = {(__bf16)o[2], (__bf16)o[3]};
  u32x2 v;
  v[0] = __builtin_bit_cast(uint32_t, lo);
  v[1] = __builtin_bit_cast(uint32_t, hi);
  *reinterpret_cast<u32x2*>(a.y + ((int64_t)(first + (int)j) * a.hq + (int64_t)hk * a.group + h) * DIM + col) = v;
}

// A workgroup's part of a segment in the scratch, ROWS x DIM sums in units of four columns (unit u: row and
// column of unit_at), then the rows' maxima and sums of probabilities.  A workgroup's second slot
// is for the segment that begins in it.
template <int DIM, int ROWS>
struct Partial {
  static constexpr int kPart = ROWS * (DIM + 2);
  float* p;
  __device__ __forceinline__ Partial(const AttnArgs& a, int wg, bool begins)
      : p(a.part + (size_t)(2 * wg + (begins ? 1 : 0)) * kPart) {}
  __device__ __forceinline__ void put(int unit, floatx4 o) const { *reinterpret_cast<floatx4*>(p + 4 * unit) = o; }
  __device__ __forceinline__ void put_ml(int row, float m, float l) const {
    p[ROWS * DIM + row] = m;
    p[ROWS * (DIM + 1) + row] = l;
  }
  __device__ __forceinline__ floatx4 get(int unit) const { return *reinterpret_cast<const floatx4*>(p + 4 * unit); }
  __device__ __forceinline__ float m(int row) const { return p[ROWS * DIM + row]; }
  __device__ __forceinline__ float l(int row) const { return p[ROWS * (DIM + 1) + row]; }
};

// Column of register ii of output block c in the lanes g.
template <int DIM, bool E4M3>
__device__ __forceinline__ int out_column(int c, int ii, int g) {
  constexpr int kRun = AttnShape<DIM, E4M3>::kRun;
  return c / kRun * (16 * kRun) + kRun * (4 * g + ii) + c % kRun;
}

// Row and column of a partial's unit: row by row, or (k_attention_rows) as a wave's registers have them, its
// lanes side by side.
template <int DIM, bool E4M3, int ROWS>
__device__ __forceinline__ void unit_at(int unit, int& row, int& col) {
  if constexpr (ROWS < kAtWideRows) {
    row = unit / (DIM / 4);
    col = unit % (DIM / 4) * 4;
  } else {
    constexpr int kSubs = DIM / 16;
    const int lane = unit & 63, q = unit >> 6;
    row = 16 * (q / kSubs) + (lane & 15);
    col = out_column<DIM, E4M3>(q / 4 % (kSubs / 4) * 4, q & 3, lane >> 4);
  }
}

// The segment that begins in a workgroup and goes on in others: how many have some of it (0: none).
struct Split {
  int parts = 0, first = 0, hk = 0, block = 0, valid = 0;
  __device__ __forceinline__ void add(const Segment& sg, int rows) {
    if (sg.whole || blockIdx.x != (uint32_t)sg.from) return;
    parts = sg.to - sg.from + 1;
    first = sg.first;
    hk = sg.hk;
    block = sg.block;
    valid = rows;
  }
};

// Sums the parts of split segments: blockIdx.x the workgroup that one begins in, blockIdx.y some of its units.
// Few rows: four lanes share a unit's parts, eight each in flight (a long sequence of one request has 32 parts
// a head).  Many rows: a lane has four units, four parts of each in flight.
template <int DIM, bool E4M3, int ROWS>
__global__ __launch_bounds__(kBlock) void k_attention_join(AttnArgs a) {
  using P = Partial<DIM, ROWS>;
  constexpr int kShare = ROWS < kAtWideRows ? 4 : 1, kItems = 4 / kShare, kAhead = ROWS < kAtWideRows ? 8 : 4;
  constexpr int kEach = kBlock / kShare;                     // units of a workgroup at a time
  const Split sp = a.split[blockIdx.x];
  if (sp.parts == 0) return;
  const float vs = a.kv.v_scale ? a.kv.v_scale[sp.hk] : 1.0f;
  const int part0 = threadIdx.x % kShare;
  const int units = (sp.valid + 15) / 16 * 16 * (DIM / 4);
  for (int u0 = blockIdx.y * kEach * kItems + threadIdx.x / kShare; u0 < units; u0 += gridDim.y * kEach * kItems) {
    int unit[kItems], row[kItems], col[kItems];
    float top[kItems], sum[kItems];
    floatx4 o[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      unit[i] = u0 + i * kEach;
      unit_at<DIM, E4M3, ROWS>(unit[i], row[i], col[i]);
      if (unit[i] >= units || row[i] >= sp.valid) unit[i] = -1;
      if (unit[i] < 0) row[i] = 0;
      top[i] = -INFINITY;
      sum[i] = 0.0f;
      o[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const auto add = [&](int i, float m, float l, floatx4 v) {   // (a part that saw nothing has the sum 0, or NaN)
      const float now = fmaxf(top[i], m);
      const float fa = top[i] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(top[i] - now);
      const float fb = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - now);
      sum[i] = sum[i] * fa + l * fb;
      o[i] = o[i] * fa + v * fb;
      top[i] = now;
    };
    for (int p = part0; p < sp.parts; p += kShare * kAhead) {
      float mv[kAhead][kItems], lv[kAhead][kItems];
      floatx4 ov[kAhead][kItems];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int at = p + kShare * k < sp.parts ? p + kShare * k : p;   // (again, for nothing)
        const P part(a, blockIdx.x + at, at == 0);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          mv[k][i] = part.m(row[i]);
          lv[k][i] = part.l(row[i]);
          ov[k][i] = part.get(unit[i] < 0 ? 0 : unit[i]);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const bool on = p + kShare * k < sp.parts;
#pragma unroll
        for (int i = 0; i < kItems; ++i) add(i, on ? mv[k][i] : -INFINITY, on ? lv[k][i] : 0.0f, on ? ov[k][i] : floatx4{0.0f, 0.0f, 0.0f, 0.0f});
      }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
#pragma unroll
      for (int d = 1; d < kShare; d <<= 1) {
        const float m = __shfl_xor(top[i], d), l = __shfl_xor(sum[i], d);
        const floatx4 v = {__shfl_xor(o[i][0], d), __shfl_xor(o[i][1], d), __shfl_xor(o[i][2], d), __shfl_xor(o[i][3], d)};
        add(i, m, l, v);
      }
      if (unit[i] >= 0 && part0 == 0)
        attn_put<DIM>(a, sp.first, sp.hk, sp.block * ROWS + row[i], col[i], o[i] * (sum[i] == 0.0f ? 0.0f : vs / sum[i]));
    }
  }
}

// Up to 16 NQ rows of q: each wave all of them on places of its own.
template <int DIM, bool E4M3, int NQ>
__global__ __launch_bounds__(kBlock, 1) void k_attention(AttnArgs a) {
  using S = AttnShape<DIM, E4M3>;
  constexpr int kRows = 16 * NQ;
  constexpr int kCols = DIM < 128 ? DIM : 128;              // columns joined at a time
  constexpr int kPitch = kCols + 4;
  __shared__ __attribute__((aligned(16))) float s_o[4][16][kPitch];
  __shared__ float s_m[4][kRows], s_l[4][kRows];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

  UnitLine line(a, kRows);
  const int total = line.start(lane);
  Split split;
  int u = blockIdx.x * line.share;
  const int end = u + line.share < total ? u + line.share : total;
  const uint32_t row_bytes = (uint32_t)a.kv.token_stride * S::kSize;
  const uint32_t k_off = r * row_bytes + 16 * g;
  const uint32_t v_off = 4 * g * row_bytes + r * S::kRun * S::kSize;

  while (u < end) {
    const Segment sg(line, u, end, lane);
    u = sg.next;
    if (sg.tile1 <= sg.tile0) continue;
    const int base = sg.old;
    const int t_end = sg.tile1 * kAtUnit < sg.seen ? sg.tile1 * kAtUnit : sg.seen;
    const int32_t* const table = a.b.table + (int64_t)sg.s * a.b.table_stride;
    const uint8_t* const kp = static_cast<const uint8_t*>(a.kv.k) + (int64_t)sg.hk * a.kv.head_stride * S::kSize;
    const uint8_t* const vp = static_cast<const uint8_t*>(a.kv.v) + (int64_t)sg.hk * a.kv.head_stride * S::kSize;
    const float scale = a.scale * (a.kv.k_scale ? a.kv.k_scale[sg.hk] : 1.0f);

    // the first step's keys and values, then q
    Pages<S::kSize> pages;                                   // of 32 steps, two a step
    RawTile<DIM, E4M3> key, val;
    int t = sg.tile0 * kAtUnit + w * 32, i = 0;
    pages.fill(a, table, t + (lane >> 1) * 128 + (lane & 1) * 16, t_end);
#pragma unroll
    for (int h = 0; h < 2; ++h) key.load_keys(h, pages.tile(a, kp, h, row_bytes), k_off);
#pragma unroll
    for (int h = 0; h < 2; ++h) val.load_values(h, pages.tile(a, vp, h, row_bytes), v_off, row_bytes);
    bf16x8 q[NQ][S::kFrag];
    SeenBy sees[NQ];
    floatx4 acc[NQ][S::kSubs];
    float m[NQ], l[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      sees[n] = load_query<DIM, E4M3>(a, sg, sg.block * kRows + 16 * n + r, g, q[n]);
      m[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int c = 0; c < S::kSubs; ++c) acc[n][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    while (t < t_end) {
      const int pg0 = lane_get(pages.page, 2 * i), pg1 = lane_get(pages.page, 2 * i + 1);
      floatx4 sc[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[n][h] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int f = 0; f < S::kFrag; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bf16x8 kf = key.key(h, f);
#pragma unroll
          for (int n = 0; n < NQ; ++n) sc[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[n][f], sc[n][h], 0, 0, 0);
        }
      // the next step's keys, in flight while this one's values are used
      const int t_next = t + 128;
      if (++i == 32) {
        pages.fill(a, table, t_next + (lane >> 1) * 128 + (lane & 1) * 16, t_end);
        i = 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) key.load_keys(h, pages.tile(a, kp, 2 * i + h, row_bytes), k_off);

      const bool masked = !(t + 32 <= base && pg0 >= 0 && pg1 >= 0);
      int tm = t + 4 * g;                                    // (made here: few steps are masked)
      asm volatile("" : "+v"(tm));
      const auto there = [&](int e) { return (tm + (e < 4 ? e : 12 + e) < sg.seen) & ((e < 4 ? pg0 : pg1) >= 0); };
      u32x4 ph[NQ], pl[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = sc[n][e / 4][e % 4] * scale;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = (there(e) & sees[n](tm + (e < 4 ? e : 12 + e) - base)) ? x[e] : -INFINITY;
        }
        soften<E4M3, true>(x, m[n], l[n], acc[n], ph[n], pl[n]);
      }
      if (masked) {
        // places of V with a NaN or an infinity, where some rows may not see them: one at a time, for the
        // rows that do; then they and the places that do not exist are nothing
        uint32_t odd = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          odd |= (there(e) & val.odd(e)) ? 1u << e : 0u;
        if (__ballot(odd != 0)) {
          // (a place's columns are in 16 lanes, one of which may have it: all 16 take it out)
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) odd |= __shfl_xor(odd, d);
          int go = g;
          asm volatile("" : "+v"(go));
#pragma unroll 1
          for (int k = 0; k < 32; ++k) {
            const int e = k >> 2, g1 = k & 3;
            if (__ballot((go == g1) & (odd >> e & 1)) == 0) continue;
            const int bit = t + (e < 4 ? 4 * g1 + e : 12 + 4 * g1 + e) - base;
            const uint32_t mine = go == g1 ? (e & 1) ? 0xFFFF0000u : 0x0000FFFFu : 0u;
#pragma unroll
            for (int c = 0; c < S::kSubs; ++c) {
              u32x4 vf = val.value(c);
#pragma unroll
              for (int p = 0; p < 4; ++p) vf[p] &= p == e >> 1 ? mine : 0u;
#pragma unroll
              for (int n = 0; n < NQ; ++n) {
                floatx4 one = {0.0f, 0.0f, 0.0f, 0.0f};
                one = mfma_pv<E4M3>(vf, ph[n], one);
                one = mfma_pv<E4M3>(vf, pl[n], one);
                acc[n][c] = sees[n](bit) ? acc[n][c] + one : acc[n][c];
              }
              __builtin_amdgcn_sched_barrier(0);             // (one block's registers at a time)
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) val.clear(e, !there(e) | (odd >> e & 1));
      }
#pragma unroll
      for (int c = 0; c < S::kSubs; ++c) {
        const u32x4 vf = val.value(c);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          acc[n][c] = mfma_pv<E4M3>(vf, ph[n], acc[n][c]);
          acc[n][c] = mfma_pv<E4M3>(vf, pl[n], acc[n][c]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) val.load_values(h, pages.tile(a, vp, 2 * i + h, row_bytes), v_off, row_bytes);
      t = t_next;
    }

    // the waves' sums of the same rows into one (its addresses are made here: no registers kept for them)
    int tj = tid;
    asm volatile("" : "+v"(tj));
    const int rj = tj & 15, gj = tj >> 4 & 3;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] += __shfl_xor(l[n], 16);
      l[n] += __shfl_xor(l[n], 32);
      if (gj == 0) {
        s_m[w][16 * n + rj] = m[n];
        s_l[w][16 * n + rj] = l[n];
      }
    }
    __syncthreads();
    const int valid = sg.valid(a.group, kRows);
    const Partial<DIM, kRows> part(a, blockIdx.x, blockIdx.x == (uint32_t)sg.from);
    const float vs = a.kv.v_scale ? a.kv.v_scale[sg.hk] : 1.0f;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int blk = 0; blk < DIM / kCols; ++blk) {
        // columns blk kCols .. of the waves' outputs, relative to the rows' common maximum
        if (n > 0 || blk > 0) __syncthreads();
        const float top = fmaxf(fmaxf(s_m[0][16 * n + rj], s_m[1][16 * n + rj]), fmaxf(s_m[2][16 * n + rj], s_m[3][16 * n + rj]));
        const float f = m[n] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[n] - top);
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int c = 0; c < S::kSubs; ++c) {
            // column of block c's row 4 g + ii
            const int col = out_column<DIM, E4M3>(c, ii, gj);
            if (col >= blk * kCols && col < (blk + 1) * kCols) s_o[w][rj][col - blk * kCols] = acc[n][c][ii] * f;
          }
        __syncthreads();
        // 16 rows x kCols columns, four columns a thread at a time
        for (int it = tj; it < 16 * kCols / 4; it += kBlock) {
          const int c4 = it % (kCols / 4), rr = 16 * n + it / (kCols / 4);
          if (rr >= valid) continue;
          const float tp = fmaxf(fmaxf(s_m[0][rr], s_m[1][rr]), fmaxf(s_m[2][rr], s_m[3][rr]));
          float sum = 0.0f;
          floatx4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float mv = s_m[v][rr];
            sum += mv == -INFINITY ? s_l[v][rr] : s_l[v][rr] * __builtin_amdgcn_exp2f(mv - tp);
            o += *reinterpret_cast<const floatx4*>(&s_o[v][rr - 16 * n][4 * c4]);
          }
          const int col = blk * kCols + 4 * c4;
          if (sg.whole) {
            attn_put<DIM>(a, sg.first, sg.hk, sg.block * kRows + rr, col, o * (sum == 0.0f ? 0.0f : vs / sum));
          } else {
            part.put((rr * DIM + col) / 4, o);
            if (col == 0) part.put_ml(rr, tp, sum);
          }
        }
      }
    }
    split.add(sg, valid);
    __syncthreads();
  }
  if (tid == 0) a.split[blockIdx.x] = split;
}

// Up to 128 rows of q, 16 a wave, all waves on the same 128 (or 64) places: a wave loads the keys or the values of 32
// of them (waves 0 .. 3 and 4 .. 7), turns them into operands once and leaves those in LDS for all.
// Without that every wave would convert and turn everything, which takes longer than to load it; with 64 rows
// a workgroup, sequences of more would be read again.
template <int DIM, bool E4M3>
__global__ __launch_bounds__(kAtWide, 2) void k_attention_rows(AttnArgs a) {
  using S = AttnShape<DIM, E4M3>;
  constexpr int kRows = kAtWideRows;
  constexpr bool kTwo = !E4M3;                               // terms of a probability
  // two waves share 32 places where one's would take too many registers: steps are of 64 then
  constexpr int kParts = DIM * S::kSize > 256 ? 2 : 1, kSlices = 4 / kParts, kStep = 32 * kSlices;
  __shared__ u32x4 s_kv[kSlices][2 * S::kSubs][64];          // per 32 places: keys (two 16s), then values
  __shared__ uint32_t s_odd[kSlices][kParts];                // per 32 places: those with a NaN or an infinity
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), mine = (w & 3) / kParts, sub = (w & 3) % kParts;
  const bool keys = w < 4;

  UnitLine line(a, kRows);
  const int total = line.start(lane);
  Split split;
  int u = blockIdx.x * line.share;
  const int end = u + line.share < total ? u + line.share : total;
  const uint32_t row_bytes = (uint32_t)a.kv.token_stride * S::kSize;
  const uint32_t k_off = r * row_bytes + 16 * g;
  const uint32_t v_off = 4 * g * row_bytes + (16 * sub + r) * S::kRun * S::kSize;

  while (u < end) {
    const Segment sg(line, u, end, lane);
    u = sg.next;
    if (sg.tile1 <= sg.tile0) continue;
    const int base = sg.old;
    const int t_end = sg.tile1 * kAtUnit < sg.seen ? sg.tile1 * kAtUnit : sg.seen;
    const int32_t* const table = a.b.table + (int64_t)sg.s * a.b.table_stride;
    const uint8_t* const src = static_cast<const uint8_t*>(keys ? a.kv.k : a.kv.v) + (int64_t)sg.hk * a.kv.head_stride * S::kSize;
    const float scale = a.scale * (a.kv.k_scale ? a.kv.k_scale[sg.hk] : 1.0f);
    const int valid = sg.valid(a.group, kRows);

    Pages<S::kSize> pages;                                   // of 32 / kSlices steps
    RawTile<DIM, E4M3, kParts> raw;
    const auto load = [&](int i) {
      const int at = 2 * (kSlices * i + mine);
      if (keys) {
#pragma unroll
        for (int h = 0; h < 2 / kParts; ++h) raw.load_keys(h, pages.tile(a, src, at + h + sub, row_bytes), k_off);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) raw.load_values(h, pages.tile(a, src, at + h, row_bytes), v_off, row_bytes);
      }
    };
    int t = sg.tile0 * kAtUnit, i = 0;
    pages.fill(a, table, t + lane * 16, t_end);
    load(0);
    bf16x8 q[S::kFrag];
    const SeenBy sees = load_query<DIM, E4M3>(a, sg, sg.block * kRows + 16 * w + r, g, q);
    floatx4 acc[S::kSubs];
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int c = 0; c < S::kSubs; ++c) acc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    while (t < t_end) {
      // which of the step's tiles of 16 exist
      const uint32_t have = (uint32_t)(__ballot(pages.page >= 0) >> (2 * kSlices * i));
      // operands into LDS (a few at a time: their registers are many)
      if (keys) {
#pragma unroll
        for (int h = 0; h < 2 / kParts; ++h)
#pragma unroll
          for (int f = 0; f < S::kFrag; ++f) {
            s_kv[mine][(h + sub) * S::kFrag + f][lane] = __builtin_bit_cast(u32x4, raw.key(h, f));
            if (f & 1) __builtin_amdgcn_sched_barrier(0);
          }
      } else {
        const int t0 = t + 32 * mine;
        const uint32_t two = have >> (2 * mine) & 3u;
        uint32_t odd = 0;
        if (!(t0 + 32 <= base && two == 3u)) {
          int tm = t0 + 4 * g;
          asm volatile("" : "+v"(tm));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool there = (tm + (e < 4 ? e : 12 + e) < sg.seen) & (two >> (e / 4) & 1u);
            const uint64_t bl = __ballot(there & raw.odd(e));
#pragma unroll
            for (int g1 = 0; g1 < 4; ++g1) odd |= (bl >> (16 * g1) & 0xFFFFu) != 0 ? 1u << (4 * e + g1) : 0u;
            raw.clear(e, !there);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        if (lane == 0) s_odd[mine][sub] = odd;
#pragma unroll
        for (int c = 0; c < S::kSubs / kParts; ++c) {
          s_kv[mine][S::kSubs + sub * (S::kSubs / kParts) + c][lane] = raw.value(c);
          if (c & 1) __builtin_amdgcn_sched_barrier(0);
        }
      }
      // the next step's, in flight
      const int t_next = t + kStep;
      if (++i == 32 / kSlices) {
        pages.fill(a, table, t_next + lane * 16, t_end);
        i = 0;
      }
      load(i);
      lds_barrier();

      if (16 * w < valid) {
#pragma unroll 1
        for (int k = 0; k < kSlices; ++k) {
          const int t0 = t + 32 * k;
          if (t0 >= t_end) break;
          // operands four at a time, the next four on their way from LDS
          u32x4 op[2][4];
          const auto fetch = [&](int n, u32x4 (&to)[4]) {    // the slice's operands n .. n + 3
#pragma unroll
            for (int z = 0; z < 4; ++z) to[z] = s_kv[k][n + z][lane];
            __builtin_amdgcn_sched_barrier(0);
          };
          floatx4 sc[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) sc[h] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
          fetch(0, op[0]);
#pragma unroll
          for (int n = 0; n < S::kSubs; n += 4) {
            fetch(n + 4, op[(n / 4 + 1) & 1]);
#pragma unroll
            for (int z = 0; z < 4; ++z)
              sc[(n + z) / S::kFrag] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(op[(n / 4) & 1][z]), q[(n + z) % S::kFrag],
                                                                              sc[(n + z) / S::kFrag], 0, 0, 0);
          }
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = sc[e / 4][e % 4] * scale;
          const uint32_t two = have >> (2 * k) & 3u;
          if (!(t0 + 32 <= base && two == 3u)) {
            int tm = t0 + 4 * g;                             // (made here: few steps are masked)
            asm volatile("" : "+v"(tm));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int at = tm + (e < 4 ? e : 12 + e);
              x[e] = ((at < sg.seen) & (two >> (e / 4) & 1u) & sees(at - base)) ? x[e] : -INFINITY;
            }
          }
          u32x4 ph, pl;
          soften<E4M3, kTwo>(x, m, l, acc, ph, pl);
          const uint32_t odd = __builtin_amdgcn_readfirstlane(s_odd[k][0] | s_odd[k][kParts - 1]);
          if (odd == 0) {
#pragma unroll
            for (int c = 0; c < S::kSubs; c += 4) {
              const int now = ((S::kSubs + c) / 4) & 1;
              if (c + 4 < S::kSubs) fetch(S::kSubs + c + 4, op[now ^ 1]);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                acc[c + z] = mfma_pv<E4M3>(op[now][z], ph, acc[c + z]);
                if constexpr (kTwo) acc[c + z] = mfma_pv<E4M3>(op[now][z], pl, acc[c + z]);
              }
            }
          } else {
            // places with a NaN or an infinity, which some rows may not see: the others first, then one at
            // a time, for the rows that do
            int go = g;                                      // (made here, too)
            asm volatile("" : "+v"(go));
#pragma unroll 1
            for (int z = -1; z < 32; ++z) {
              if (z >= 0 && !(odd >> z & 1)) continue;
              u32x4 part = {0, 0, 0, 0};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const bool on = z < 0 ? !(odd >> (4 * e + go) & 1) : 4 * e + go == z;
                part[e / 2] |= on ? (e & 1) ? 0xFFFF0000u : 0x0000FFFFu : 0u;
              }
              const int e = z >> 2, bit = t0 + 4 * (z & 3) + (e < 4 ? e : 12 + e) - base;
              const bool seen = (z < 0) | sees(bit);
#pragma unroll
              for (int c = 0; c < S::kSubs; ++c) {
                const u32x4 vf = s_kv[k][S::kSubs + c][lane] & part;
                floatx4 one = {0.0f, 0.0f, 0.0f, 0.0f};
                one = mfma_pv<E4M3>(vf, ph, one);
                if constexpr (kTwo) one = mfma_pv<E4M3>(vf, pl, one);
                acc[c] = seen ? acc[c] + one : acc[c];
                __builtin_amdgcn_sched_barrier(0);
              }
            }
          }
        }
      }
      lds_barrier();
      t = t_next;
    }

    int tj = tid;                                            // (made here: no registers kept for it)
    asm volatile("" : "+v"(tj));
    const int lj = tj & 63, rj = lj & 15, gj = lj >> 4;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    const float vs = a.kv.v_scale ? a.kv.v_scale[sg.hk] : 1.0f;
    const int row = 16 * w + rj;
    if (row < valid) {
      const Partial<DIM, kRows> part(a, blockIdx.x, blockIdx.x == (uint32_t)sg.from);
      const float f = sg.whole ? l == 0.0f ? 0.0f : vs / l : 1.0f;
#pragma unroll
      for (int ii = 0; ii < 4; ++ii)
#pragma unroll
        for (int c = 0; c < S::kSubs; c += 4) {
          const floatx4 o = floatx4{acc[c][ii], acc[c + 1][ii], acc[c + 2][ii], acc[c + 3][ii]} * f;
          if (sg.whole) attn_put<DIM>(a, sg.first, sg.hk, sg.block * kRows + row, out_column<DIM, E4M3>(c, ii, gj), o);
          else part.put(((w * (S::kSubs / 4) + c / 4) * 4 + ii) * 64 + lj, o);   // (a wave's lanes side by side)
        }
      if (!sg.whole && gj == 0) part.put_ml(row, m, l);
    }
    split.add(sg, valid);
    __syncthreads();
  }
  if (tid == 0) a.split[blockIdx.x] = split;
}

// Rows of q a workgroup takes at once, by the average of a sequence (which is all the host knows): 16 up to 16,
// since 32 hold registers that loads in flight need (64 sequences of one token, 6 rows each: 89 us, with 32
// 103; of 1 or 2 tokens, 56 and 59); 32 up to 32 where they fit, else 128 (16 sequences of 3000 .. 5000 places and
// 1 .. 8 tokens, 27 rows on average: 77 us, with 128 83); 128 beyond (54 rows on average: 96, with
// 32, the sequence read again for each 32, 99).  A batch of both kinds has one of them: 63 single tokens of 2048 places
// and a chunk of 2048 tokens take 760 us together, 88 and 547 apart; 255 and a chunk of 100 452, 339 and 56.
struct AttnPlan {
  int rows;               // 16, 32: k_attention, 128: k_attention_rows
  int wgs;
  bool fits;              // the line of units has fewer than 2^31
};
static AttnPlan attn_plan(const DevInfo& di, int64_t m, int64_t hq, const KvArgs& kv, const BatchArgs& b) {
  const int64_t group = hq / kv.heads, avg = (m * group + b.seqs - 1) / b.seqs;
  AttnPlan p;
  p.rows = avg <= 16 ? 16 : avg <= 32 && kv.dim <= 128 ? 32 : kAtWideRows;
  const double most = ((double)m * group / p.rows + (double)b.seqs) * (double)kv.heads *
                      ((double)b.cols * kv.page / kAtUnit + 1.0 + kAtStart);
  p.fits = most < 1073741824.0 && m * hq < (int64_t(1) << 30);
  p.wgs = di.cus;
  return p;
}

static uint64_t attn_part(const AttnPlan& p, int64_t dim) { return (uint64_t)p.rows * (dim + 2) * sizeof(float); }

bool attention_fits(const DevInfo& di, int64_t m, int64_t hq, const KvArgs& kv, const BatchArgs& b) {
  return attn_plan(di, m, hq, kv, b).fits;
}

// No segment is split where each has a workgroup and the table holds no more than a piece.
static bool attn_splits(const AttnPlan& p, int64_t m, int64_t hq, const KvArgs& kv, const BatchArgs& b) {
  const int64_t segments = ((m * (hq / kv.heads) + p.rows - 1) / p.rows + b.seqs) * kv.heads;
  return b.cols * kv.page > (int64_t)kAtPiece * kAtUnit || segments > p.wgs;
}

uint64_t attention_scratch(const DevInfo& di, int64_t m, int64_t hq, const KvArgs& kv, const BatchArgs& b) {
  const AttnPlan p = attn_plan(di, m, hq, kv, b);
  return p.wgs * sizeof(Split) + 16 + (attn_splits(p, m, hq, kv, b) ? 2 * p.wgs * attn_part(p, kv.dim) : 0);
}

template <int DIM, bool E4M3, int ROWS>
static void attn_go(const AttnArgs& a, bool splits, hipStream_t s) {
  const dim3 grid((unsigned)a.wgs);
  if constexpr (ROWS == kAtWideRows) hipLaunchKernelGGL((k_attention_rows<DIM, E4M3>), grid, dim3(kAtWide), 0, s, a);
  else hipLaunchKernelGGL((k_attention<DIM, E4M3, ROWS / 16>), grid, dim3(kBlock), 0, s, a);
  const dim3 join((unsigned)a.wgs, 8);
  if (splits) hipLaunchKernelGGL((k_attention_join<DIM, E4M3, ROWS>), join, dim3(kBlock), 0, s, a);
}
template <int DIM, bool E4M3>
static void attn_go(const AttnPlan& p, const AttnArgs& a, bool splits, hipStream_t s) {
  if (p.rows == kAtWideRows) attn_go<DIM, E4M3, kAtWideRows>(a, splits, s);
  else if constexpr (DIM == 256) attn_go<DIM, E4M3, 16>(a, splits, s);
  else if (p.rows == 32) attn_go<DIM, E4M3, 32>(a, splits, s);
  else attn_go<DIM, E4M3, 16>(a, splits, s);
}

hipError_t launch_attention(const uint16_t* q, int64_t ldq, int64_t m, int64_t hq, const KvArgs& kv,
                            const BatchArgs& b, float scale, uint16_t* y, void* scratch, hipStream_t s) {
  DevInfo di;
  const hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  const AttnPlan p = attn_plan(di, m, hq, kv, b);
  if (!p.fits) return hipErrorInvalidValue;
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
  a.split = static_cast<Split*>(scratch);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + (p.wgs * sizeof(Split) + 15) / 16 * 16);
  const bool splits = attn_splits(p, m, hq, kv, b);
  if (kv.dim == 64) kv.e4m3 ? attn_go<64, true>(p, a, splits, s) : attn_go<64, false>(p, a, splits, s);
  else if (kv.dim == 128) kv.e4m3 ? attn_go<128, true>(p, a, splits, s) : attn_go<128, false>(p, a, splits, s);
  else kv.e4m3 ? attn_go<256, true>(p, a, splits, s) : attn_go<256, false>(p, a, splits, s);
  return hipGetLastError();
}

}  // namespace w12
