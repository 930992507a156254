// Log probabilities of given tokens, entropy and the top alternatives of rows of logits, in one pass
// over the logits.
//
// With M the row's largest logit, s = sum e^(x - M) over all logits but one that equals M, and
// T = sum e^(x - M) (x - M):
//   log p(t) = (x_t - M) - log1p(s)          H = log1p(s) - T / (1 + s)
// Leaving one maximum out of s keeps the small probabilities of a confident row (its maximum's own
// log probability is -log1p(s), not the difference of two numbers near zero), and T <= 0, so
// neither formula cancels.  Everything is held in float; bfloat16 logits widen exactly.
//
// Two runs (M, s, T) of a row join into one with the larger M: with f = e^(M_b - M_a), d = M_b - M_a,
//   s = s_a + f (1 + s_b),   T = T_a + f (T_b + (1 + s_b) d).
//
// Two kernels share the rest.  Rows that fill the chip by themselves are streamed (k_logprobs): a
// workgroup of 4 waves takes a row (or a few parts of one), each wave batch after batch of 64 lanes
// x 16 logits in 16-byte loads with the next batch in flight; the running maximum is the wave's (one
// compare per batch finds the rare batch that raises it), sums are each lane's own.  Fewer rows are
// cut into parts of 4096 logits that a workgroup holds in registers (k_logprobs_part): the maximum
// comes first, so nothing is put right afterwards, and the whole part shares one bound for its
// candidates below.  The parts of a row go to the caller's scratch, each workgroup counts itself
// off, and the row's last one joins them in part order, lane by part, so the result does not depend
// on which came last, and there is no second launch.  At one row what a launch costs is latency: the
// code runs once, so every line of it is fetched for the occasion, and short code beats few
// instructions.
//
// Top alternatives.  A candidate is a 64-bit key: the logit's order (NaN above +Inf, -0 as +0), then
// the complement of its index, so equal logits go by the lower index and every order is total.
// The K-th largest of the lanes' own maxima is a bound that K logits already reach; logits at or
// above it are the candidates (about 1.2 K of them for a part, and about 1.35 K / i of a streaming
// wave's i-th batch, whose other logits cost one compare per batch).  They are collected in an LDS
// list; its K best are picked by rank, the number of larger keys.
//
// Measured (152064 float logits a row unless said, calls back to back): 1024 rows 109.5 us (5.7 TB/s;
// bfloat16 63.0, 4.9 TB/s), with 8 alternatives 118.4 (92.5): bound by memory, and in bfloat16 by the
// instructions per logit.  64 rows 14.7 us, with 16 alternatives 23.4: six of the 15 are the read at
// 6.4 TB/s, the rest is what one part waits for in turn -- its logits, the maximum, the bound, the
// candidates, the last part's join (5.0 us at one row, 9.9 with 8 alternatives) -- little of which
// other parts fill.
#include "w12_device.hpp"
#include "w12_launch.hpp"

namespace w12 {

constexpr int kLpCap = 256;                      // keys of a wave's candidate list
constexpr int kLpWaves = 4;
constexpr int kLpElems = 16;                     // logits of a lane per batch
constexpr int kLpBatch = 64 * kLpElems;          // logits of a wave per batch
constexpr uint32_t kLpMasked = 0x007FFFFFu;      // the order of -Inf
constexpr int kLpCountStep = 32;                 // rows' counts 128 bytes apart: counts of one line wait for each other
constexpr int kLpAhead = 4;                      // keys of a part loaded together when parts join
constexpr float kLog2e = 1.44269504088896340736f;

typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

struct LpPart {
  float M, s, T, pad;
};

struct LpArgs {
  const void* y;          // logits [m][ldy], float or bfloat16
  int64_t m, n, ldy;
  const void* tokens;     // [m][nt] int32 or int64
  int tok64, nt, top;
  float* logp;            // [m][nt]
  float* ent;             // [m]
  int32_t* tidx;          // [m][top]
  float* tlogp;           // [m][top]
  int splits;             // workgroups per row
  int64_t part;           // logits per workgroup (a multiple of a workgroup's batch)
  // splits > 1: a count per row (zero between calls), then [m][splits] LpPart, [m][splits][top] keys
  uint32_t* count;
  LpPart* parts;
  uint64_t* keys;
};

__device__ __forceinline__ void lp_wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Stores and loads that every die of the device sees at once, and the wait for this wave's stores.
template <typename T>
__device__ __forceinline__ void dev_store(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T dev_load(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void stores_done() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// e^d for d <= 0 (or NaN)
__device__ __forceinline__ float lp_exp(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

__device__ __forceinline__ uint32_t lp_order(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);    // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float lp_value(uint32_t ord) {
  if (ord == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}

__device__ __forceinline__ uint64_t lp_key(float x, int64_t column) {
  return (uint64_t)lp_order(x) << 32 | (0xFFFFFFFFu - (uint32_t)column);
}

// Reductions over the wave's 64 lanes by DPP (row shifts within 16 lanes, then the two row
// broadcasts); every lane gets the result.  (As shuffles through LDS each cost about 600 cycles.)
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_f(float identity, float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(identity), __float_as_uint(v), CTRL, ROWS,
                                                     0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
  const float lo = -INFINITY;
  v = fmaxf(v, dpp_f<0x111, 0xF>(lo, v));          // row_shr:1
  v = fmaxf(v, dpp_f<0x112, 0xF>(lo, v));
  v = fmaxf(v, dpp_f<0x114, 0xF>(lo, v));
  v = fmaxf(v, dpp_f<0x118, 0xF>(lo, v));
  v = fmaxf(v, dpp_f<0x142, 0xA>(lo, v));          // row_bcast:15 into rows 1, 3
  v = fmaxf(v, dpp_f<0x143, 0xC>(lo, v));          // row_bcast:31 into rows 2, 3
  return last_lane(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<0x111, 0xF>(0.0f, v);
  v += dpp_f<0x112, 0xF>(0.0f, v);
  v += dpp_f<0x114, 0xF>(0.0f, v);
  v += dpp_f<0x118, 0xF>(0.0f, v);
  v += dpp_f<0x142, 0xA>(0.0f, v);
  v += dpp_f<0x143, 0xC>(0.0f, v);
  return last_lane(v);
}

// Inclusive sum over the lanes up to each.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The lanes' runs (M, s, T) into one (see the top), the same in every lane; M = -Inf: a run without
// any logit above -Inf (its s is 0, or NaN if it has a NaN).
__device__ __forceinline__ void lp_join(float& M, float& s, float& T) {
  const float Mx = wave_max(M);
  const uint64_t own = __ballot(M == Mx);
  const int owner = own ? __ffsll((unsigned long long)own) - 1 : 0;
  const float d = M - Mx, f = lp_exp(d), g = 1.0f + s;
  float s2 = s, T2 = T;
  if (M == -INFINITY) {
    s2 = s != s ? s : 0.0f;
    T2 = 0.0f;
  } else if ((int)(threadIdx.x & 63) != owner) {
    s2 = f * g;
    T2 = f > 0.0f ? f * (T + g * d) : f != f ? f : 0.0f;   // (g d may overflow where f is 0)
  }
  M = Mx;
  s = wave_sum(s2);
  T = wave_sum(T2);
}

// A wave's candidates for the K best keys: a list in LDS, and a bound.
struct LpTop {
  uint64_t* list;         // [kLpCap], this wave's
  int K;
  int cnt = 0;            // keys in the list (uniform)
  uint32_t seen = 0;      // K logits have been seen at or above this order (uniform)

  // the list cut back to its K largest keys, in descending order; with K keys left, nothing below
  // the last can enter
  __device__ __forceinline__ void cut(int lane) {
    lp_wave_fence();
    uint64_t key[kLpCap / 64];
    int rank[kLpCap / 64];
#pragma unroll
    for (int q = 0; q < kLpCap / 64; ++q) {
      const int i = lane + 64 * q;
      key[q] = i < cnt ? list[i] : 0;
      rank[q] = 0;
    }
    if (cnt <= 64) {
      const uint32_t lo = (uint32_t)key[0], hi = (uint32_t)(key[0] >> 32);
      for (int i = 0; i < cnt; ++i) {
        const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, i) << 32 |
                           (uint32_t)__builtin_amdgcn_readlane(lo, i);
        rank[0] += o > key[0] ? 1 : 0;
      }
    } else if (cnt <= 128) {
#pragma unroll 8
      for (int i = 0; i < cnt; ++i) {
        const uint64_t o = list[i];
        rank[0] += o > key[0] ? 1 : 0;
        rank[1] += o > key[1] ? 1 : 0;
      }
    } else {
#pragma unroll 4
      for (int i = 0; i < cnt; ++i) {
        const uint64_t o = list[i];
#pragma unroll
        for (int q = 0; q < kLpCap / 64; ++q) rank[q] += o > key[q] ? 1 : 0;
      }
    }
    lp_wave_fence();
#pragma unroll
    for (int q = 0; q < kLpCap / 64; ++q)
      if (lane + 64 * q < cnt && rank[q] < K) list[rank[q]] = key[q];
    lp_wave_fence();
    if (cnt >= K) {
      cnt = K;
      const uint32_t last = __builtin_amdgcn_readfirstlane((uint32_t)(list[K - 1] >> 32));
      if (last > seen) seen = last;
    }
  }

  // whether the keys of the lanes with `in` fit the list
  __device__ __forceinline__ bool fits(uint64_t ballot) const { return cnt + __popcll(ballot) <= kLpCap; }
  __device__ __forceinline__ void put(bool in, uint64_t ballot, uint64_t key, int lane) {
    if (in) list[cnt + __popcll(ballot & ((1ull << lane) - 1))] = key;
    cnt += __popcll(ballot);
  }
};

// A bound that at least K of the lanes' values (N a lane) reach, and that is at most their K-th
// largest: found bit by bit, from the leading bits of `hi` (at or above every value) where K values
// share them, down to 16 bits where that leaves at most 4 values more (a bound a little low costs a
// candidate or two, the other 16 steps as much as ten), else to all 32.
template <int N>
__device__ __forceinline__ uint32_t lp_kth(const uint32_t (&v)[N], int K, uint32_t hi) {
  const auto reach = [&](uint32_t c) {
    int k = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) k += __popcll(__ballot(v[i] >= c));
    return k;
  };
  // 22 low bits of a float's order: a half of a binade; 25: four binades
  uint32_t t = 0;
  int b = 31;
  if (reach(hi >> 22 << 22) >= K) {
    t = hi >> 22 << 22;
    b = 21;
  } else if (reach(hi >> 25 << 25) >= K) {
    t = hi >> 25 << 25;
    b = 24;
  }
  // (rolled: this runs once or twice in a short launch, where each line of code is fetched anew)
#pragma unroll 1
  for (; b >= 0; --b) {
    const uint32_t c = t | (1u << b);
    if (reach(c) >= K) t = c;
    if (b == 16 && K <= 64 * N - 8 && reach(t) <= K + 4) break;
  }
  return t;
}

// Element e of a lane's batch at column c of the row: column c + 64 V (e / V) + V lane + e % V, with V
// the logits of a 16-byte load.  Past c1 the batch reads -Inf.
template <bool BF>
struct LpBatch {
  static constexpr int V = BF ? 8 : 4, Q = kLpElems / V;
  u32x4 raw[Q];
  static __device__ __forceinline__ int64_t column(int64_t c, int e, int lane) {
    return c + 64 * V * (e / V) + V * lane + e % V;
  }
  __device__ __forceinline__ void load(const uint8_t* yr, int64_t c, int64_t c1, int lane) {
    if (c + kLpBatch <= c1) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint8_t* src = yr + (c + 64 * V * q + V * lane) * (BF ? 2 : 4);
        if constexpr (BF) raw[q] = *reinterpret_cast<const u32x4_a2*>(src);
        else raw[q] = *reinterpret_cast<const u32x4_a4*>(src);
      }
    } else {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t cc = c + 64 * V * q + V * lane + (V / 4) * i;
          if constexpr (BF) {
            const uint16_t* src = reinterpret_cast<const uint16_t*>(yr);
            const uint32_t lo = cc < c1 ? src[cc] : 0xFF80u, hi = cc + 1 < c1 ? src[cc + 1] : 0xFF80u;
            raw[q][i] = lo | hi << 16;
          } else {
            raw[q][i] = cc < c1 ? reinterpret_cast<const uint32_t*>(yr)[cc] : 0xFF800000u;
          }
        }
    }
  }
  __device__ __forceinline__ void values(float (&x)[kLpElems]) const {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF) {
          x[8 * q + 2 * i] = bf16_to_float(raw[q][i] & 0xFFFFu);
          x[8 * q + 2 * i + 1] = __uint_as_float(raw[q][i] & 0xFFFF0000u);
        } else {
          x[4 * q + i] = __uint_as_float(raw[q][i]);
        }
      }
  }
};

// Sums of a lane's batch under the maximum M; `leave`: but for one logit equal to M.  x - M comes first:
// it rounds once, relative to itself, at any magnitude.  (x log2 e - M log2 e as one operation carries
// the rounding of M log2 e, which grows with M, and is no faster: 1024 rows of 152064 112.4 us
// against 109.5, 64 rows, 16 alternatives 23.2 against 23.4.)
__device__ __forceinline__ void lp_sums(const float (&x)[kLpElems], float M, bool leave, float& s, float& T) {
#pragma unroll
  for (int e = 0; e < kLpElems; ++e) {
    const float d = x[e] - M;
    float p = lp_exp(d);
    if (leave && x[e] == M) {
      p = 0.0f;
      leave = false;
    }
    s += p;
    T = fmaf(p, fmaxf(d, -200.0f), T);             // (a masked logit: 0 times a finite number)
  }
}

// The candidates (at or above lowf, or NaN) of a wave's batch at column c, elements from..15, into the
// wave's list when they may be more than it holds, or the batch passes the part's end: of those
// equal to the bound (a masked row: all of them) only the K of the lowest indices can stay.
template <bool BF>
__device__ __forceinline__ void lp_enter(LpTop& top, const float (&x)[kLpElems], float lowf, int from, int64_t c,
                                         int64_t c1, int lane) {
  constexpr int V = LpBatch<BF>::V, Q = LpBatch<BF>::Q, E = kLpElems;
  uint32_t in = 0, eq = 0;                         // a bit per element
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const bool ok = e >= from && !(x[e] < lowf) && LpBatch<BF>::column(c, e, lane) < c1;
    in |= (ok ? 1u : 0u) << e;
    eq |= (ok && x[e] == lowf ? 1u : 0u) << e;
  }
  int before = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    uint32_t g = eq & (((1u << V) - 1u) << (V * q));
    const int mine = __popc(g);
    int pre = before;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint64_t bl = __ballot((mine >> b) & 1);
      pre += __popcll(bl & ((1ull << lane) - 1)) << b;
      before += __popcll(bl) << b;
    }
    int drop = mine - (top.K - pre > 0 ? top.K - pre : 0);
    while (drop-- > 0) {
      const uint32_t high = 1u << (31 - __clz(g));
      g ^= high;
      in ^= high;
    }
  }
  while (from < E) {
    int full = E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool ok = (in >> e) & 1u;
      const uint64_t bl = __ballot(ok);
      if (bl == 0 || e < from || full < E) continue;
      if (!top.fits(bl)) {
        full = e;
        continue;
      }
      top.put(ok, bl, lp_key(x[e], LpBatch<BF>::column(c, e, lane)), lane);
    }
    from = full;
    if (full < E) top.cut(lane);
  }
}

// The four waves' lists into `best` (wave 0), its K largest keys in descending order: above one
// bound, the highest of the waves' own, or where the lists are long the K-th largest of the 256
// lanes' maxima.
__device__ __forceinline__ void lp_merge(LpTop& top, uint64_t* best, const uint64_t (*lists)[kLpCap], const int* cnt,
                                         const uint32_t* seen, const float (*lmax)[64], float M, int lane) {
  top.list = best;
  top.cnt = 0;
  int all = 0;
  for (int v = 0; v < kLpWaves; ++v) {
    top.seen = seen[v] > top.seen ? seen[v] : top.seen;
    all += cnt[v];
  }
  if (all > 64) {
    uint32_t lm[kLpWaves];
#pragma unroll
    for (int v = 0; v < kLpWaves; ++v) lm[v] = lp_order(lmax[v][lane]);
    const uint32_t kth = lp_kth<kLpWaves>(lm, top.K, lp_order(M));
    top.seen = kth > top.seen ? kth : top.seen;
  }
  top.seen = __builtin_amdgcn_readfirstlane(top.seen);
  for (int v = 0; v < kLpWaves; ++v) {
    const int cv = __builtin_amdgcn_readfirstlane(cnt[v]);
    for (int i = 0; i < cv; i += 64) {
      const uint64_t key = i + lane < cv ? lists[v][i + lane] : 0;
      const bool ok = i + lane < cv && (uint32_t)(key >> 32) >= top.seen;
      const uint64_t bl = __ballot(ok);
      if (!top.fits(bl)) top.cut(lane);
      top.put(ok, bl, key, lane);
    }
  }
  top.cut(lane);
}

struct LpToken {
  float x;
  bool real;
};
// The logit of token j of the row.
template <bool BF>
__device__ __forceinline__ LpToken lp_token(const LpArgs& a, int64_t row, int j) {
  const int64_t at = row * a.nt + j;
  const int64_t t = a.tok64 ? static_cast<const int64_t*>(a.tokens)[at]
                            : (int64_t)static_cast<const int32_t*>(a.tokens)[at];
  LpToken r = {0.0f, t >= 0 && t < a.n};
  if (r.real) {
    const int64_t o = row * a.ldy + t;
    r.x = BF ? bf16_to_float(static_cast<const uint16_t*>(a.y)[o]) : static_cast<const float*>(a.y)[o];
  }
  return r;
}

// Outputs of a row from its joined sums and (top > 0) its K best keys in descending order.
// tok: token `lane` of the row, loaded ahead.
template <bool BF>
__device__ __forceinline__ void lp_finish(const LpArgs& a, int64_t row, float M, float s, float T,
                                          const uint64_t* best, LpToken tok, int lane) {
  // a row of -Inf alone has no distribution: log probabilities -Inf, entropy 0; one with +Inf or
  // NaN: all NaN
  const bool none = M == -INFINITY && s == s;
  const bool bad = s != s || M == INFINITY || T != T;
  const float nan = __uint_as_float(0x7FC00000u);
  const float ls = log1pf(s);
  const auto lp = [&](float x) { return bad ? nan : none ? -INFINITY : (x - M) - ls; };
  for (int j = lane; j < a.nt; j += 64) {
    if (j >= 64) tok = lp_token<BF>(a, row, j);
    // (a token outside the vocabulary has probability 0)
    a.logp[row * a.nt + j] = tok.real ? lp(tok.x) : -INFINITY;
  }
  if (lane == 0) a.ent[row] = bad ? nan : none ? 0.0f : ls - T / (1.0f + s);
  for (int j = lane; j < a.top; j += 64) {
    const uint64_t key = best[j];
    a.tidx[row * a.top + j] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
    a.tlogp[row * a.top + j] = lp(lp_value((uint32_t)(key >> 32)));
  }
}

// One wave, the end of a workgroup: the outputs of a row in one part; or this part to the scratch,
// and if it is the row's last, the parts joined.  Parts move by device-scope atomic stores and
// loads, which other dies' caches see as they are, so no cache needs writing back or invalidating
// (a device-scope fence per workgroup cost 64 rows of 152064 36.6 us in all against 19.2); the wait
// orders the part before the count.
template <bool BF>
__device__ __forceinline__ void lp_end(const LpArgs& a, int64_t row, int sp, float M, float s, float T, LpTop& top,
                                       LpToken tok, int lane) {
  if (a.splits > 1) {
    const int64_t at = row * a.splits + sp;
    if (lane < 3)
      dev_store(reinterpret_cast<uint32_t*>(a.parts + at) + lane, __float_as_uint(lane == 0 ? M : lane == 1 ? s : T));
    if (lane < a.top) dev_store(a.keys + at * a.top + lane, lane < top.cnt ? top.list[lane] : (uint64_t)0);
    stores_done();
    uint32_t done = 0;
    if (lane == 0)
      done = __hip_atomic_fetch_add(a.count + row * kLpCountStep, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    done = __builtin_amdgcn_readfirstlane(done);
    if (done + 1 != (uint32_t)a.splits) return;
    asm volatile("" ::: "memory");
    if (lane == 0) dev_store(a.count + row * kLpCountStep, 0u);   // zero again for the next call
    M = -INFINITY;
    s = T = 0.0f;
    const bool mine = lane < a.splits;
    if (mine) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.parts + row * a.splits + lane);
      M = __uint_as_float(dev_load(p));
      s = __uint_as_float(dev_load(p + 1));
      T = __uint_as_float(dev_load(p + 2));
    }
    const uint64_t* keys = a.keys + (row * a.splits + lane) * a.top;
    uint64_t key[kLpAhead];
#pragma unroll
    for (int r = 0; r < kLpAhead; ++r) key[r] = mine && r < a.top ? dev_load(keys + r) : 0;
    lp_join(M, s, T);
    if (a.top > 0) {
      // each part's keys descend: the K-th of their first four each bounds the rest, and a part whose
      // next key is below the bound is done
      top.cnt = 0;
      uint32_t heads[kLpAhead];
#pragma unroll
      for (int r = 0; r < kLpAhead; ++r) heads[r] = (uint32_t)(key[r] >> 32);
      // (the largest: the row's maximum, or a NaN)
      top.seen = lp_kth<kLpAhead>(heads, a.top, __ballot(heads[0] == 0xFFFFFFFFu) ? 0xFFFFFFFFu : lp_order(M));
      bool more = true;
      for (int r0 = 0; r0 < a.top && more; r0 += kLpAhead) {
        if (r0 > 0) {
#pragma unroll
          for (int r = 0; r < kLpAhead; ++r) key[r] = mine && r0 + r < a.top ? dev_load(keys + r0 + r) : 0;
        }
#pragma unroll
        for (int r = 0; r < kLpAhead; ++r) {
          // (of the masked logits, those of the first part alone: its K keys come before the others')
          const uint32_t ord = (uint32_t)(key[r] >> 32);
          const bool ok = key[r] != 0 && ord >= top.seen && (ord != kLpMasked || lane == 0);
          const uint64_t bl = __ballot(ok);
          if (bl == 0) more = false;
          if (!more) continue;
          if (!top.fits(bl)) top.cut(lane);
          top.put(ok, bl, key[r], lane);
        }
      }
      top.cut(lane);
    }
  }
  lp_finish<BF>(a, row, M, s, T, top.list, tok, lane);
}

template <bool BF>
__global__ __launch_bounds__(64 * kLpWaves) __attribute__((amdgpu_waves_per_eu(4)))
void k_logprobs(LpArgs a) {
  constexpr int E = kLpElems;
  __shared__ uint64_t s_list[kLpWaves][kLpCap];
  __shared__ uint64_t s_best[kLpCap];
  __shared__ float s_max[kLpWaves][64];
  __shared__ float s_run[kLpWaves][4];
  __shared__ int s_cnt[kLpWaves];
  __shared__ uint32_t s_seen[kLpWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = blockIdx.x / a.splits;
  const int sp = (int)(blockIdx.x - row * a.splits);
  const int64_t c0 = sp * a.part;
  const int64_t c1 = c0 + a.part < a.n ? c0 + a.part : a.n;
  const uint8_t* const yr = static_cast<const uint8_t*>(a.y) + row * a.ldy * (BF ? 2 : 4);

  float M = -INFINITY, s = 0.0f, T = 0.0f;         // M uniform; s, T the lane's
  int owner = 0;                                   // the lane that left the maximum out
  LpTop top;
  top.list = s_list[w];
  top.K = a.top;
  float lmax = -INFINITY;                          // the lane's largest logit so far (NaN passed over)
  float thrf = -INFINITY;                          // a logit below this cannot enter the list
  int batch = 0;
  bool anynan = false, closed = a.top == 0;        // closed: nothing can enter any more

  int64_t c = c0 + (int64_t)w * kLpBatch;
  constexpr int64_t kStep = (int64_t)kLpWaves * kLpBatch;
  LpBatch<BF> bt;
  if (c < c1) bt.load(yr, c, c1, lane);
  LpToken tok = {0.0f, false};
  if (w == 0 && lane < a.nt) tok = lp_token<BF>(a, row, lane);
  for (; c < c1; c += kStep) {
    float x[E];
    bt.values(x);
    if (c + kStep < c1) bt.load(yr, c + kStep, c1, lane);   // the next batch, in flight meanwhile
    float mx = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) mx = fmaxf(mx, x[e]);   // (a NaN is passed over)
    if (__ballot(mx > M)) {
      // a new maximum: the sums so far relative to it, and one logit that equals it left out
      const float mn = wave_max(mx);
      if (M > -INFINITY) {
        const float d = M - mn, f = lp_exp(d);
        if (lane == owner) s += 1.0f;
        T = f > 0.0f ? f * (T + s * d) : s != s ? s : 0.0f;   // (s d may overflow where f is 0)
        s *= f;
      }
      M = mn;
      owner = __ffsll((unsigned long long)__ballot(mx == M)) - 1;
      lp_sums(x, M, lane == owner, s, T);
    } else if (M > -INFINITY) {
      lp_sums(x, M, false, s, T);
    } else {
      bool bad = false;
#pragma unroll
      for (int e = 0; e < E; ++e) bad |= x[e] != x[e];
      if (bad) s = __uint_as_float(0x7FC00000u);
    }
    ++batch;
    if (!closed) {
      anynan = anynan || __ballot(s != s) != 0;
      if (anynan || __ballot(mx >= thrf)) {
        lmax = fmaxf(lmax, mx);
        // the bound again at the batches 1, 2, 4, 8, ...: a bound twice as old lets through about
        // twice as many logits, each cheaper than the bound itself
        float lowf = thrf;
        const auto bound = [&]() {
          const uint32_t hi = lp_order(M);
          const uint32_t kth = a.top == 1 ? hi : lp_kth<1>({lp_order(lmax)}, a.top, hi);
          if (kth > top.seen) top.seen = kth;
          // earlier batches have lower indices: of the logits equal to a bound they reached none
          // can enter (thrf), of those equal to one that this batch reached the first can
          lowf = lp_value(top.seen);               // (NaN: the comparisons below let all through)
          if (lowf < thrf) lowf = thrf;
        };
        if (a.top == 1 || (batch & (batch - 1)) == 0) bound();
        int from = c + kLpBatch > c1 ? 0 : E;
        if (from == E) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const bool ok = !(x[e] < lowf);        // (NaN enters)
            const uint64_t bl = __ballot(ok);
            if (bl == 0 || from < E) continue;
            if (!top.fits(bl)) {
              from = e;
              continue;
            }
            top.put(ok, bl, lp_key(x[e], LpBatch<BF>::column(c, e, lane)), lane);
          }
        }
        if (from < E) {                            // more than the list holds, or the part's end
          bound();
          lp_enter<BF>(top, x, lowf, from, c, c1, lane);
        }
        // later batches: only above the bound (its order's successor; nothing is above a NaN, and the
        // order of -Inf is the lowest a logit has)
        if (top.seen == 0xFFFFFFFFu) closed = true;
        else if (top.seen >= 0xFF800000u) thrf = INFINITY;
        else if (top.seen >= 0x007FFFFFu) thrf = lp_value(top.seen + 1);
      }
    }
  }

  // the lanes' sums (relative to the same M) in a fixed order, then the waves'
  s = wave_sum(s);
  T = wave_sum(T);
  if (lane == 0) {
    s_run[w][0] = M;
    s_run[w][1] = s;
    s_run[w][2] = T;
    s_cnt[w] = top.cnt;
    s_seen[w] = top.seen;
  }
  if (a.top > 0) s_max[w][lane] = lmax;
  __syncthreads();
  if (w != 0) return;
  M = lane < kLpWaves ? s_run[lane][0] : -INFINITY;
  s = lane < kLpWaves ? s_run[lane][1] : 0.0f;
  T = lane < kLpWaves ? s_run[lane][2] : 0.0f;
  lp_join(M, s, T);
  top.list = s_best;
  if (a.top > 0) lp_merge(top, s_best, s_list, s_cnt, s_seen, s_max, M, lane);
  lp_end<BF>(a, row, sp, M, s, T, top, tok, lane);
}

// A part of at most kLpWaves kLpBatch logits, held in the workgroup's registers.  (Six waves per SIMD, 80
// registers: 64 rows of 152064, 8 alternatives, 22.6 us; as the compiler leaves it, 83 and five,
// 23.3; held to 64 registers, 23.4.)
template <bool BF>
__global__ __launch_bounds__(64 * kLpWaves) __attribute__((amdgpu_waves_per_eu(6)))
void k_logprobs_part(LpArgs a) {
  constexpr int E = kLpElems;
  __shared__ uint64_t s_list[kLpWaves][kLpCap];    // each wave's list, where the shared one overflows
  __shared__ uint64_t s_best[kLpCap];
  __shared__ float s_max[kLpWaves][64];
  __shared__ float s_run[kLpWaves][4];
  __shared__ int s_cnt[kLpWaves];                  // keys in each wave's own list
  __shared__ int s_masked[kLpWaves];               // (apart from s_cnt: a slow wave may still read it when a fast one counts)
  __shared__ uint32_t s_seen[kLpWaves];
  __shared__ int s_total;                          // keys offered to the shared list
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = blockIdx.x / a.splits;
  const int sp = (int)(blockIdx.x - row * a.splits);
  const int64_t c0 = sp * a.part;
  const int64_t c1 = c0 + a.part < a.n ? c0 + a.part : a.n;
  const uint8_t* const yr = static_cast<const uint8_t*>(a.y) + row * a.ldy * (BF ? 2 : 4);
  const int64_t c = c0 + (int64_t)w * kLpBatch;
  LpBatch<BF> bt;
  bt.load(yr, c, c1, lane);
  LpToken tok = {0.0f, false};
  if (w == 0 && lane < a.nt) tok = lp_token<BF>(a, row, lane);
  if (tid == 0) s_total = 0;
  float x[E];
  bt.values(x);
  float mx = x[0];
#pragma unroll
  for (int e = 1; e < E; ++e) mx = fmaxf(mx, x[e]);   // (a NaN is passed over)
  s_max[w][lane] = mx;
  const float wm = wave_max(mx);
  if (lane == 0) s_run[w][0] = wm;
  __syncthreads();

  // the part's maximum; the first lane of the first wave that has it leaves one out
  float M = -INFINITY;
  int wo = 0;
#pragma unroll
  for (int v = kLpWaves - 1; v >= 0; --v) {
    const float mv = s_run[v][0];
    if (mv >= M) {
      M = mv;
      wo = v;
    }
  }
  M = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(M)));
  wo = __builtin_amdgcn_readfirstlane(wo);
  float s = 0.0f, T = 0.0f;
  if (M == -INFINITY) {
    bool bad = false;
#pragma unroll
    for (int e = 0; e < E; ++e) bad |= x[e] != x[e];
    if (bad) s = __uint_as_float(0x7FC00000u);
  } else {
    const int owner = __ffsll((unsigned long long)__ballot(mx == M)) - 1;
    lp_sums(x, M, w == wo && lane == owner, s, T);
  }
  s = wave_sum(s);
  T = wave_sum(T);
  if (lane == 0) {
    s_run[w][1] = s;
    s_run[w][2] = T;
  }
  LpTop top;
  top.K = a.top;
  top.list = s_best;
  float lowf = 0.0f;
  // nothing but masked logits: the first columns
  const bool masked = M == -INFINITY && __ballot(s != s) == 0;
  if (lane == 0) s_masked[w] = masked ? 1 : 0;
  if (a.top > 0 && !masked) {
    const uint32_t hi = lp_order(M);
    if (a.top == 1) {
      top.seen = hi;
    } else {
      uint32_t lm[kLpWaves];
#pragma unroll
      for (int v = 0; v < kLpWaves; ++v) lm[v] = lp_order(s_max[v][lane]);
      top.seen = lp_kth<kLpWaves>(lm, a.top, hi);
    }
    lowf = lp_value(top.seen);                     // (NaN: the comparisons let all through)
    uint32_t in = 0;                               // a bit per candidate of the lane
#pragma unroll
    for (int e = 0; e < E; ++e) in |= (!(x[e] < lowf) ? 1u : 0u) << e;
    if (c + kLpBatch > c1) {                       // the row's end
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (LpBatch<BF>::column(c, e, lane) >= c1) in &= ~(1u << e);
    }
    if (__ballot(in != 0)) {
      const int mine = __popc(in), upto = wave_scan(mine);
      const int tot = __builtin_amdgcn_readlane(upto, 63);
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_total, tot);
      at = __builtin_amdgcn_readfirstlane(at);
      if (at + tot <= kLpCap) {
        at += upto - mine;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((in >> e) & 1u) s_best[at++] = lp_key(x[e], LpBatch<BF>::column(c, e, lane));
      }
    }
  }
  __syncthreads();
  const bool none = __builtin_amdgcn_readfirstlane(s_masked[0] + s_masked[1] + s_masked[2] + s_masked[3]) == kLpWaves;
  int total = a.top > 0 ? __builtin_amdgcn_readfirstlane(s_total) : 0;
  if (a.top > 0 && M == -INFINITY && !none) {      // masked logits and a NaN: the long way
    lowf = -INFINITY;
    top.seen = 0;
    total = kLpCap + 1;
  }
  if (a.top > 0 && none) {
    if (w == 0 && lane < a.top && c0 + lane < c1) s_best[lane] = (uint64_t)kLpMasked << 32 | (0xFFFFFFFFu - (uint32_t)(c0 + lane));
  }
  if (total > kLpCap) {
    // more candidates than the shared list holds (many equal to the bound): by each wave's own
    top.list = s_list[w];
    lp_enter<BF>(top, x, lowf, 0, c, c1, lane);
    if (lane == 0) {
      s_cnt[w] = top.cnt;
      s_seen[w] = top.seen;
    }
    __syncthreads();
  }
  if (w != 0) return;
  // (the waves' sums are relative to the same maximum)
  s = ((s_run[0][1] + s_run[1][1]) + s_run[2][1]) + s_run[3][1];
  T = ((s_run[0][2] + s_run[1][2]) + s_run[2][2]) + s_run[3][2];
  if (total > kLpCap) {
    lp_merge(top, s_best, s_list, s_cnt, s_seen, s_max, M, lane);
  } else if (a.top > 0 && none) {
    lp_wave_fence();
    top.cnt = c1 - c0 < a.top ? (int)(c1 - c0) : a.top;   // (already in order)
  } else if (a.top > 0) {
    top.cnt = total;
    top.cut(lane);
  }
  lp_end<BF>(a, row, sp, M, s, T, top, tok, lane);
}

// Parts in registers while they are few for the chip; else whole rows, or if those are still fewer
// than it runs at once, as many streamed parts as fill it.  (Rows of 152064 float logits, parts in
// registers against streamed: 32 rows, 8 alternatives 15.3 vs 20.3 us, 64 rows, 16 alternatives 23.3
// vs 26.4, without any 14.7 vs 13.4; 128 rows, 8 alternatives 33.0 vs 32.0, 256 rows 54.8 vs 45.6.)
constexpr int kLpParts = 16;                     // workgroups per CU up to which rows are cut into register parts
constexpr int kLpPerCu = 4;                      // streaming workgroups per CU
constexpr int64_t kLpUnit = (int64_t)kLpWaves * kLpBatch;
struct LpPlan {
  bool regs;              // k_logprobs_part
  int splits;
  int64_t part;
};
static LpPlan lp_plan(const DevInfo& di, int64_t m, int64_t n) {
  const int64_t units = (n + kLpUnit - 1) / kLpUnit;
  LpPlan p;
  p.regs = units <= 64 && m * units <= (int64_t)di.cus * kLpParts;
  int64_t want = p.regs ? units : (int64_t)di.cus * kLpPerCu / m;
  if (want < 1) want = 1;
  if (want > 64) want = 64;
  if (want > units) want = units;
  const int64_t per = (units + want - 1) / want;
  p.part = per * kLpUnit;
  p.splits = (int)((units + per - 1) / per);
  return p;
}

// The counts of the rows, ahead of the parts: as many rows as either rule cuts in two or more.
static uint64_t lp_counts(const DevInfo& di) {
  static_assert(kLpPerCu <= kLpParts, "register parts are the rule for more rows");
  return (uint64_t)di.cus * (kLpParts / 2) * kLpCountStep * sizeof(uint32_t);
}

uint64_t logprobs_scratch(const DevInfo& di, int64_t m, int64_t n, int top) {
  const LpPlan p = lp_plan(di, m, n);
  if (p.splits == 1) return 0;
  return lp_counts(di) + (uint64_t)m * p.splits * (sizeof(LpPart) + 8ull * top);
}

hipError_t launch_logprobs(const void* y, bool bf, int64_t m, int64_t n, int64_t ldy, const void* tokens,
                           bool tok64, int nt, int top, float* logp, float* ent, int32_t* tidx,
                           float* tlogp, void* scratch, hipStream_t s) {
  DevInfo di;
  hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  const LpPlan p = lp_plan(di, m, n);
  LpArgs a;
  a.y = y; a.m = m; a.n = n; a.ldy = ldy;
  a.tokens = tokens; a.tok64 = tok64; a.nt = nt; a.top = top;
  a.logp = logp; a.ent = ent; a.tidx = tidx; a.tlogp = tlogp;
  a.splits = p.splits;
  a.part = p.part;
  a.count = static_cast<uint32_t*>(scratch);
  a.parts = reinterpret_cast<LpPart*>(static_cast<uint8_t*>(scratch) + lp_counts(di));
  a.keys = reinterpret_cast<uint64_t*>(a.parts + m * a.splits);
  // a launch holds fewer than 2^32 work items: more rows (whole ones, then) in several
  constexpr int64_t kRows = int64_t(1) << 23;
  static_assert(kRows * 64 * kLpWaves < (int64_t(1) << 32), "work items of a launch");
  for (int64_t r0 = 0; r0 < m; r0 += kRows) {
    a.m = m - r0 < kRows ? m - r0 : kRows;
    const dim3 grid((unsigned)(a.m * a.splits)), block(64 * kLpWaves);
    if (p.regs && bf) hipLaunchKernelGGL(k_logprobs_part<true>, grid, block, 0, s, a);
    else if (p.regs) hipLaunchKernelGGL(k_logprobs_part<false>, grid, block, 0, s, a);
    else if (bf) hipLaunchKernelGGL(k_logprobs<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_logprobs<false>, grid, block, 0, s, a);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    a.y = static_cast<const uint8_t*>(a.y) + kRows * ldy * (bf ? 2 : 4);
    if (nt > 0) {
      a.tokens = static_cast<const uint8_t*>(a.tokens) + kRows * nt * (tok64 ? 8 : 4);
      a.logp += kRows * nt;
    }
    a.ent += kRows;
    if (top > 0) {
      a.tidx += kRows * top;
      a.tlogp += kRows * top;
    }
  }
  return hipSuccess;
}

}  // namespace w12
