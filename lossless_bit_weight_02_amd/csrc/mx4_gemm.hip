// Skinny GEMM on the microscaled 4-bit copy (mx4.hip) on the matrix cores, several weight tiles per wave:
// y[m][n] = 2^(base_n - 112) sum_k x[m][k] w'[n][k] + sum over the escapes that are not zero of x v.
//
// A block of 16 weight rows x 128 columns is 1088 bytes, half of the 8-bit view's, and decodes in 16
// instructions (a scaled conversion yields two bfloat16), so what bounds the other formats' kernels
// here is no longer the weight stream but what a wave does per block: its loop, the reads of x from
// LDS (16 KiB per block at 64 rows) and, with many tiles, every workgroup's passes over x in L2.  So
// a wave takes TP tiles at a time: each x fragment it reads from LDS multiplies TP decoded blocks,
// and the loop's instructions, a round's start and its reads of x are spread over them.
//
// Measured (us; weights alone at the rate of a large read, 6.4 TB/s, in parentheses): 64 rows,
// [34816, 5120] 37 to 39 (16.3; k_mfma_wide's loop 54.2), [152064, 5120] 139 to 147 (71), [5120, 17408]
// 31.6 (8.0), [5120, 5120] 18.2 (2.5); 16 rows, [152064, 5120] 81.3 (66.4; one tile per wave 95.3); 32
// rows 93.2 (67.9; 111.2).  More than 64 rows run as passes of 64 that each read the copy again ([34816,
// 5120], 128 rows: 73.6).  At 64 rows the weights, the matrix cores (the fullest SIMD's) and the LDS
// reads take about 15 us each of the 39, the start and the end of the kernel 7: what is missing is
// their overlap in two waves per SIMD.
//
// Work split.  One workgroup of 8 waves per CU, in two halves: four waves take the even and four the odd
// blocks of the same tiles (two waves a SIMD, so one multiplies while the other decodes, yet only
// four read each block of x), and their sums meet in LDS at the end.  The tiles are dealt
// round-robin over the workgroups and a workgroup's over its four wave pairs, TP each and round at
// most, as evenly as that allows.  Shapes with few tiles split k into ranges of whole chunks, whose
// partial sums a second kernel adds in range order.  Two blocks of each tile are in flight per wave:
// with four, [152064, 5120] at 16 rows took 97.7 us instead of 88.4.
//
// x: chunks of S blocks (128 S columns) of all rows in LDS, double buffered, loaded straight from
// memory (global-to-LDS) while the chunk before is multiplied, rows rotated against bank conflicts as
// in k_mfma (mfma.hip).  Rows past m and columns past the range read zeros.  The weights run through
// a ring of D blocks per tile in registers.
//
// Escapes: few remain (the zeros are gone), so a tile's are not walked chunk by chunk but added from
// memory when its sums are done.
#include "mfma_common.hpp"

namespace w12 {

constexpr int kMxWaves = 8;

struct Mx4Args {
  const uint16_t* x;             // x[m][k]
  int m;
  const uint8_t* base;
  const uint8_t* q;
  const uint32_t* esc_ptr;
  const uint32_t* esc_end;
  const uint32_t* esc_col;
  const uint16_t* esc_val;
  float* y;                      // y[m][ldy]; with splits > 1, range j writes y + j * ysplit
  uint16_t* y16;                 // one range: bfloat16 outputs here instead
  int64_t ldy;
  int64_t n, k;
  int rounds, tpr;               // rounds, and tiles of a workgroup per round (<= 4 TP)
  int splits;                    // k ranges: workgroup b takes range b % splits
  int cps;                       // x chunks per range
  int64_t ysplit;
  int yvec;                      // 4 outputs of a row as one store (aligned, ldy % 4 == 0)
};

// PAST: past the caches
template <bool PAST, class T>
__device__ __forceinline__ void mx_put(void* at, const T& v) {
  if constexpr (PAST) __builtin_nontemporal_store(v, static_cast<T*>(at));
  else *static_cast<T*>(at) = v;
}

template <int N>
__device__ __forceinline__ void mx_wait_le() {
  constexpr int M = N < 63 ? N : 63;
  __builtin_amdgcn_s_waitcnt((M & 15) | ((M >> 4) << 14) | 0x70 | 0xF00);
}

// NT: 16-row activation tiles; TP: weight tiles per wave; S: blocks per x chunk, of which a wave takes S / 2.
// PAST: y is final (one k range) and goes past the caches ([152064, 5120], 16 rows 94.3 -> 87.7 us
// through a y kept from call to call; also where log probabilities read it next: 16 rows, both
// together, 100.5 -> 95.9, 64 rows 162.4 -> 162.7; [34816, 5120], 64 rows 50.8 -> 48.8; [17408, 5120]
// 38.1 -> 37.9); partial sums are read again at once.
template <int NT, int TP, int S, bool PAST>
__global__ __launch_bounds__(64 * kMxWaves) __attribute__((amdgpu_waves_per_eu(2)))
void k_mx4_gemm(Mx4Args a) {
  constexpr int W = kMxWaves;
  constexpr int D = 2;                             // blocks in flight per wave and tile
  constexpr int F = 4 * NT * S;                    // 1 KiB x pieces per chunk
  constexpr int FW = F / W;
  static_assert(F % W == 0 && S % (2 * D) == 0, "whole rings and 256-column pieces per chunk");
  static_assert(4 * TP * NT * 2 <= 2 * F, "the odd blocks' sums and the escapes' products fit the x buffers");
  constexpr int kLoads = 2 * TP;                   // loads per step
  __shared__ __attribute__((aligned(16))) u32x4 s_x[2][F * 64];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t half = (uint32_t)w >> 2, sub = (uint32_t)w & 3u;
  const uint32_t KB = (uint32_t)(a.k / kTileCols);
  const int64_t tiles = (a.n + kTileRows - 1) / kTileRows;
  const int sp = (int)(blockIdx.x % (uint32_t)a.splits);
  const int64_t grp = blockIdx.x / (uint32_t)a.splits, n_grp = gridDim.x / (uint32_t)a.splits;
  const uint32_t kb0 = (uint32_t)(sp * a.cps) * S;
  const uint32_t nkb = KB - kb0 < (uint32_t)a.cps * S ? KB - kb0 : (uint32_t)a.cps * S;
  const uint32_t n_chunks = (nkb + S - 1) / S;
  const uint32_t col0 = 128u * kb0, col1 = 128u * (kb0 + nkb);
  float* const yout = a.y + sp * a.ysplit;
  const uint32_t kx = (uint32_t)a.k;
  const Rsrc rx = make_rsrc(a.x, (uint32_t)a.m * kx * 2u);

  // Workgroups walk the chunks in the same cyclic order from different starts (workgroup b runs on die
  // b % 8): all of them reading the same chunk of x at the same time waits for the few cache channels
  // its rows lie in.
  const uint32_t first = (uint32_t)((grp >> 3) % n_chunks);
  const auto chunk_at = [&](uint32_t pos) { return pos + first < n_chunks ? pos + first : pos + first - n_chunks; };

  // x pieces and their LDS layout as in k_mfma: piece P of a chunk holds rows 2 q and 2 q + 1
  // (q = P % 8 NT) of its 256-column half P / 8 NT, 512 bytes a row, slot (c16 + row) % 32 the row's
  // 16-byte column slot c16; wave w loads pieces w + 8 i.
  const uint32_t prow = (uint32_t)lane >> 5, pslot = (uint32_t)lane & 31u;
  uint32_t xoff[FW];                               // the lane's bytes of a piece in the first chunk
#pragma unroll
  for (int i = 0; i < FW; ++i) {
    const uint32_t P = (uint32_t)(w + W * i), q = P % (8u * NT), hb = P / (8u * NT);
    const uint32_t row = 2u * q + prow, c16 = (pslot - row) & 31u;
    xoff[i] = (int)row < a.m ? 2u * (row * kx + col0 + 256u * hb + 8u * c16) : kOOB;
  }
  // (pos: the chunk's place in the workgroup's order; n_chunks and past it: nothing, as zeros -- the
  // load pattern stays fixed, so the compiler's wait counts stay exact)
  const auto x_fetch = [&](uint32_t pos, uint32_t buf) {
    const uint32_t c = chunk_at(pos), at = 128u * S * c;   // columns from the range's start
    const bool whole = pos < n_chunks && at + 128u * S <= col1 - col0;
#pragma unroll
    for (int i = 0; i < FW; ++i) {
      const uint32_t P = (uint32_t)(w + W * i), q = P % (8u * NT), hb = P / (8u * NT);
      const uint32_t c16 = (pslot - (2u * q + prow)) & 31u;
      const bool ok = whole || (pos < n_chunks && at + 256u * hb + 8u * c16 < col1 - col0);
      const uint32_t off = ok && xoff[i] != kOOB ? xoff[i] + 2u * at : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (__attribute__((address_space(3))) void*)&s_x[buf][P * 64u], 16, off,
                                               0, 0, 0);
    }
  };
  // operand reads: block 2 s + half, k-group t, activation tile cc at 512 NT s + 512 cc +
  // xo[cc % 2][t] (see k_mfma: the slot's bit 16 is the parity of block and tile)
  uint32_t xo[2][4];
#pragma unroll
  for (int par = 0; par < 2; ++par)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      xo[par][t] = 32u * (uint32_t)r16 + ((4u * (uint32_t)g + (uint32_t)r16 + (uint32_t)t) ^ (16u * (par ^ half)));
      asm volatile("" : "+v"(xo[par][t]));
    }

  const int64_t mine = grp < tiles ? (tiles - grp + n_grp - 1) / n_grp : 0;   // tiles of this workgroup
  for (int round = 0; round < a.rounds; ++round) {
    const int64_t lo = (int64_t)round * a.tpr;
    if (lo >= mine) break;                         // (alike in every wave)
    const int64_t cnt = mine - lo < a.tpr ? mine - lo : a.tpr;
    // the wave's tiles: sub, sub + 4, ... of the round's
    int64_t row0[TP];
    bool have[TP];
    Rsrc rq[TP];
#pragma unroll
    for (int j = 0; j < TP; ++j) {
      const int64_t i = sub + 4 * j;
      have[j] = i < cnt;
      const int64_t tile = have[j] ? grp + (lo + i) * n_grp : 0;
      row0[j] = tile * kTileRows;
      rq[j] = make_rsrc(a.q + (tile * KB + kb0) * kTileMX, have[j] ? nkb * (uint32_t)kTileMX : 0u);
    }
    u32x4 bv[D][TP];
    uint32_t bs[D][TP];
    const auto load = [&](uint32_t kb, int d) {
#pragma unroll
      for (int j = 0; j < TP; ++j) {
        const uint32_t off = kb < nkb ? kb * kTileMX : kOOB;
        bv[d][j] = __builtin_amdgcn_raw_buffer_load_b128(rq[j], off + 16u * lane, 0, kAuxNT);
        bs[d][j] = __builtin_amdgcn_raw_buffer_load_b8(rq[j], off + 1024u + lane, 0, kAuxNT);
      }
    };
    __builtin_amdgcn_sched_barrier(0);
    x_fetch(0, 0u);
    __builtin_amdgcn_sched_barrier(0);
    // escape lists of the round's tiles: wave w looks after tiles w, w + 8, ...: where the list lies
    // and how long it is, and (first k range) its first 64 entries, a lane each; row r's start in lane
    // r of lstart, from which the sums below find an entry's row by its place
    constexpr int EL = (4 * TP + W - 1) / W;
    uint32_t lt0[EL], lcnt[EL], lstart[EL];
#pragma unroll
    for (int q = 0; q < EL; ++q) {
      const int64_t i = w + W * q;
      const bool in = i < cnt && sp == 0;
      const int64_t r0 = in ? (grp + (lo + i) * n_grp) * kTileRows : 0, rr = r0 + r16;
      lstart[q] = in ? (rr < a.n ? a.esc_ptr[rr] : a.esc_ptr[a.n]) : 0u;
      const uint32_t end = in ? (rr < a.n ? a.esc_end[rr] : a.esc_ptr[a.n]) : 0u;
      lt0[q] = lstart[q];
      lcnt[q] = end;
    }
    uint32_t bases[TP];
#pragma unroll
    for (int j = 0; j < TP; ++j) {
      const Rsrc rb = make_rsrc(a.base, (uint32_t)a.n);
      bases[j] = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        bases[j] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rb, (uint32_t)(row0[j] + 4 * g + r), 0, 0) << (8 * r);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < D; ++d) load(S * first + 2u * d + half, d);
    __builtin_amdgcn_sched_barrier(0);
    mx_wait_le<D * kLoads>();                      // the first chunk of x is in LDS
    lds_barrier();
    uint32_t lent[EL], lval[EL];                   // entry: column, bfloat16 bits
#pragma unroll
    for (int q = 0; q < EL; ++q) {
      lt0[q] = __builtin_amdgcn_readfirstlane(lt0[q]);
      lcnt[q] = (uint32_t)__builtin_amdgcn_readlane(lcnt[q], 15) - lt0[q];
      lent[q] = 0;
      lval[q] = 0;
      if ((uint32_t)lane < lcnt[q]) {
        lent[q] = a.esc_col[lt0[q] + lane];
        lval[q] = a.esc_val[lt0[q] + lane];
      }
    }
    const int xm = lane & (16 * NT - 1);
    const bool xlive = lane < 16 * NT && xm < a.m;
    const auto gather = [&](uint32_t ent, uint32_t cntl, uint32_t i0, uint32_t (&xe)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t col = (uint32_t)__builtin_amdgcn_readlane(ent, i0 + i);
        xe[i] = __builtin_amdgcn_raw_buffer_load_b16(rx, xlive && i0 + i < cntl ? 2u * (xm * kx + col) : kOOB, 0, 0);
      }
    };

    floatx4 acc[TP][NT];
#pragma unroll
    for (int j = 0; j < TP; ++j)
#pragma unroll
      for (int cc = 0; cc < NT; ++cc) acc[j][cc] = (floatx4){0.f, 0.f, 0.f, 0.f};

    for (uint32_t c = 0; c < n_chunks; ++c) {
      const uint32_t b = c & 1u;
      const uint32_t kb_here = S * chunk_at(c), kb_next = c + 1 < n_chunks ? S * chunk_at(c + 1) : nkb;
      // Stage i = 4 s + t multiplies k-group t of block 2 s + half; meanwhile the next stage's x fragments
      // are read and its quarter of the block decodes, in the shadow of the products.
      constexpr int kStages = 2 * S;
      u32x4 xv[2][NT], p[2][TP];
      const u32x4* const xb = &s_x[b][0];
      const auto fetch = [&](int i, u32x4 (&x)[NT], u32x4 (&pq)[TP]) {
        const int s = i >> 2, t = i & 3;
#pragma unroll
        for (int cc = 0; cc < NT; ++cc) x[cc] = xb[s * 512 * NT + 512 * cc + xo[cc & 1][t]];
#pragma unroll
        for (int j = 0; j < TP; ++j) pq[j] = mx4_quarter(bv[s % D][j][t], bs[s % D][j]);
      };
      fetch(0, xv[0], p[0]);
      __builtin_amdgcn_sched_barrier(0);
      x_fetch(c + 1, b ^ 1u);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        const int s = i >> 2;
        if (i + 1 < kStages) fetch(i + 1, xv[(i + 1) & 1], p[(i + 1) & 1]);
        // the block's last quarter has just been decoded: its slot takes the block D steps on
        if ((i & 3) == 2)
          load((s + D < S / 2 ? kb_here + 2u * (s + D) : kb_next + 2u * (s + D - S / 2)) + half, s % D);
#pragma unroll
        for (int cc = 0; cc < NT; ++cc)
#pragma unroll
          for (int j = 0; j < TP; ++j)
            acc[j][cc] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p[i & 1][j]),
                                                                 __builtin_bit_cast(bf16x8, xv[i & 1][cc]), acc[j][cc],
                                                                 0, 0, 0);
        // the reads first, then products and conversions in turn
        __builtin_amdgcn_sched_group_barrier(0x100, NT, 0);
#pragma unroll
        for (int g2 = 0; g2 < NT * TP; ++g2) {
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x2, NT == 1 ? 5 : NT == 2 ? 3 : 2, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // the next chunk is in LDS: its loads went out before this chunk's refills
      mx_wait_le<S / 2 * kLoads>();
      lds_barrier();
    }

    // Into the x buffers, which nothing reads any more: each half's sums of the tiles the other half
    // finishes (the even ones the first half, the odd ones the second); and behind them, per tile, the
    // escapes' products, [16 rows][16 NT x rows]: lane m adds x row m's, entry by entry in order (a
    // row's entries follow each other, so its sum is stored once).
    u32x4* const part = &s_x[0][0] + sub * (TP * NT * 64) + lane;
#pragma unroll
    for (int j = 0; j < TP; ++j)
      if ((j & 1) != (int)half) {
#pragma unroll
        for (int cc = 0; cc < NT; ++cc) part[(j * NT + cc) * 64] = __builtin_bit_cast(u32x4, acc[j][cc]);
      }
    float* const s_q = reinterpret_cast<float*>(&s_x[0][0] + 4 * TP * NT * 64);   // [4 TP][16][16 NT]
#pragma unroll
    for (int q = 0; q < EL; ++q) {
      if (w + W * q >= cnt || sp != 0) continue;
      float* const tq = s_q + (w + W * q) * (256 * NT);
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) tq[64 * i + lane] = 0.0f;
      uint32_t row = 0;
      float sum = 0.0f;
      for (uint32_t e0 = 0; e0 < lcnt[q]; e0 += 64) {
        if (e0 > 0) {                              // past the first 64: from memory
          const bool in = e0 + lane < lcnt[q];
          lent[q] = in ? a.esc_col[lt0[q] + e0 + lane] : 0u;
          lval[q] = in ? a.esc_val[lt0[q] + e0 + lane] : 0u;
        }
        // the entry's row: the last whose list starts at or before it
        uint32_t er = 0;
#pragma unroll
        for (int i = 1; i < 16; ++i)
          er += lt0[q] + e0 + lane >= (uint32_t)__builtin_amdgcn_readlane(lstart[q], i) ? 1u : 0u;
        const uint32_t here = lcnt[q] - e0 < 64u ? lcnt[q] - e0 : 64u;
        for (uint32_t i0 = 0; i0 < here; i0 += 8) {
          uint32_t xe[8];                          // lane m's: x row m's value at each entry
          gather(lent[q], here, i0, xe);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i0 + i >= here) break;
            const uint32_t r = (uint32_t)__builtin_amdgcn_readlane(er, i0 + i);
            const float v = bf16_to_float((uint32_t)__builtin_amdgcn_readlane(lval[q], i0 + i));
            if (r != row) {
              if (xlive) tq[row * (16 * NT) + xm] = sum;
              row = r;
              sum = 0.0f;
            }
            sum = fmaf(bf16_to_float(xe[i]), v, sum);
          }
        }
      }
      if (xlive) tq[row * (16 * NT) + xm] = sum;   // (without entries: zeros over zeros)
    }
    lds_barrier();
    // sums, scale and store: lane (g, r16) holds rows 4 g .. 4 g + 3 of x row 16 cc + r16
#pragma unroll
    for (int j = 0; j < TP; ++j) {
      if ((j & 1) != (int)half || !have[j]) continue;
      float qv[NT][4];
#pragma unroll
      for (int cc = 0; cc < NT; ++cc) {
        acc[j][cc] += __builtin_bit_cast(floatx4, part[(j * NT + cc) * 64]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          qv[cc][r] = sp == 0 ? s_q[(sub + 4 * j) * (256 * NT) + (4 * g + r) * (16 * NT) + 16 * cc + r16] : 0.0f;
      }
#pragma unroll
      for (int cc = 0; cc < NT; ++cc) {
        const int64_t row = 16 * cc + r16;
        if (row >= a.m) continue;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r] = fmaf(window_scale((bases[j] >> (8 * r)) & 0xFFu), acc[j][cc][r], qv[cc][r]);
        const int64_t col = row0[j] + 4 * g, at = row * a.ldy + col;
        if (a.y16) {
          if (a.yvec && col + 3 < a.n) {
            mx_put<PAST>(a.y16 + at,
                         (u32x2){(uint32_t)float_to_bf16_rne(v[0]) | (uint32_t)float_to_bf16_rne(v[1]) << 16,
                                 (uint32_t)float_to_bf16_rne(v[2]) | (uint32_t)float_to_bf16_rne(v[3]) << 16});
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (col + r < a.n) a.y16[at + r] = float_to_bf16_rne(v[r]);
          }
        } else if (a.yvec && col + 3 < a.n) {
          mx_put<PAST>(yout + at, (floatx4){v[0], v[1], v[2], v[3]});
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (col + r < a.n) yout[at + r] = v[r];
        }
      }
    }
    if (round + 1 < a.rounds) lds_barrier();       // before the next round's x
  }
}

// ---------------------------------------------------------------------------------------------
// launcher
// ---------------------------------------------------------------------------------------------
typedef void (*Mx4Kernel)(Mx4Args);
struct Mx4Shape {
  int tiles, chunk;              // tiles per wave and round at most, blocks per x chunk
};
static Mx4Shape mx4_shape(int nt) { return nt <= 2 ? Mx4Shape{5, 8} : Mx4Shape{3, 4}; }
// tp: tiles per wave.  Passes of at most 32 rows come here with at least 13 tiles per workgroup and
// round (launch_mx4_gemm), so with four or five per wave.
static Mx4Kernel mx4_pick(int nt, int tp, bool split) {
  if (nt == 1) return tp <= 4 ? k_mx4_gemm<1, 4, 8, true> : k_mx4_gemm<1, 5, 8, true>;
  if (nt == 2) return tp <= 4 ? k_mx4_gemm<2, 4, 8, true> : k_mx4_gemm<2, 5, 8, true>;
  if (split) return tp == 1 ? k_mx4_gemm<4, 1, 4, false> : k_mx4_gemm<4, 2, 4, false>;   // at most eight tiles
  return tp == 1 ? k_mx4_gemm<4, 1, 4, true> : tp == 2 ? k_mx4_gemm<4, 2, 4, true> : k_mx4_gemm<4, 3, 4, true>;
}

hipError_t launch_mx4_gemm(const uint16_t* x, int64_t m, const Planes& p, int64_t n, int64_t k, YOut y,
                           hipStream_t s, const Scratch& sc) {
  DevInfo di;
  hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  const int64_t tiles = (n + kTileRows - 1) / kTileRows, kb = k / kTileCols;
  for (int64_t m0 = 0; m0 < m; m0 += 64) {
    const int mb = (int)(m - m0 < 64 ? m - m0 : 64);
    // At most 32 rows: k_mfma (mfma.hip), which deals one tile per wave and round, unless its last round
    // would be so empty that it runs as a launch of its own ([152064, 5120], 16 and 32 rows: 95.3 and
    // 111.2 us there, 81.3 and 93.2 here; [65536, 5120] 52.2 and 65.2, 36.7 and 44.2; with full rounds,
    // [49152, 5120], 28.2 and 34.1 there, 29.0 and 36.3 here, [98304, 5120] 56.3 and 66.4, 55.4 and 65.8).
    if (mb <= 32 && mfma_tail_row(di, mb, tiles) == 0)
      return launch_mfma(kFmtMX4, x + m0 * k, mb, p, n, k, y + m0 * n, s, sc);
    const int nt = (mb + 15) / 16;
    const Mx4Shape sh = mx4_shape(nt);
    const int64_t chunks = (kb + sh.chunk - 1) / sh.chunk;
    const int64_t slots = di.cus;
    // k ranges: as many as give every wave pair of the chip a tile, of at least one chunk
    int64_t ranges = slots * (kMxWaves / 2) / tiles;
    if (ranges > chunks) ranges = chunks;
    if ((uint64_t)ranges * mb * n * sizeof(float) > sc.bytes)
      ranges = (int64_t)(sc.bytes / ((uint64_t)mb * n * sizeof(float)));
    if (ranges < 2) ranges = 1;
    const int64_t cps = (chunks + ranges - 1) / ranges;
    ranges = (chunks + cps - 1) / cps;
    float* ws = nullptr;
    if (ranges > 1) {
      err = sc.get(&ws);
      if (err != hipSuccess) return err;
    }
    int64_t groups = slots / ranges;
    if (groups > tiles) groups = tiles;
    if (groups < 1) groups = 1;
    const int64_t most = (tiles + groups - 1) / groups;             // tiles of the busiest workgroup
    const int64_t rounds = (most + kMxWaves / 2 * sh.tiles - 1) / (kMxWaves / 2 * sh.tiles);
    const YOut yp = y + m0 * n;
    Mx4Args a;
    a.x = x + m0 * k;
    a.m = mb;
    a.base = p.base; a.q = p.mx4;
    a.esc_ptr = p.esc_ptr; a.esc_end = p.esc_end; a.esc_col = p.esc_col; a.esc_val = p.esc_val;
    a.y = ws ? ws : yp.f;
    a.y16 = ws ? nullptr : yp.h;
    a.ldy = n;
    a.n = n; a.k = k;
    a.rounds = (int)rounds;
    a.tpr = (int)((most + rounds - 1) / rounds);
    a.splits = (int)ranges;
    a.cps = (int)cps;
    a.ysplit = (int64_t)mb * n;
    a.yvec = a.y16 ? (reinterpret_cast<uintptr_t>(a.y16) & 7u) == 0 && n % 4 == 0
                   : (reinterpret_cast<uintptr_t>(a.y) & 15u) == 0 && n % 4 == 0;
    hipLaunchKernelGGL(mx4_pick(nt, (a.tpr + kMxWaves / 2 - 1) / (kMxWaves / 2), ws != nullptr), dim3((unsigned)(groups * ranges)),
                       dim3(64 * kMxWaves), 0, s, a);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (ws) {
      err = launch_split_reduce(ws, (int)ranges, mb, n, yp, n, s);
      if (err != hipSuccess) return err;
    }
  }
  return hipSuccess;
}

}  // namespace w12
