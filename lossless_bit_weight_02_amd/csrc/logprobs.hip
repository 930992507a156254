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
// Work split.  A row's logits are split over S workgroups of 4 waves (S = 1 when the rows alone
// fill the chip), a workgroup's part over its waves batch by batch: 64 lanes x 16 floats (32
// bfloat16) per batch, four 16-byte loads a lane, the next batch in flight.  The running maximum
// is the wave's (a scalar compare per batch finds the rare batch that raises it), sums are each
// lane's own and join at the end in a fixed order.  With S > 1 the parts go to the caller's
// scratch and a second kernel of one wave per row joins them, lane by part.
//
// Top alternatives.  A candidate is a 64-bit key: the logit's order (NaN above +Inf, -0 as +0), then
// the complement of its index, so equal logits go by the lower index and every order is total.
// Each lane keeps the largest order it has seen; the K-th largest of the 64 lanes' is a bound that
// K logits already reach, so a batch without a logit above it needs one compare in all.  Otherwise
// the batch's logits at or above the new bound are appended to the wave's list in LDS, and a full
// list is cut back to its K best (each key's rank is the number of larger keys).
#include "w12_device.hpp"
#include "w12_launch.hpp"

namespace w12 {

constexpr int kLpCap = 256;                      // keys of a wave's candidate list
constexpr int kLpWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f;

typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

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
  uint8_t* scratch;       // splits > 1: [m][splits] LpPart, then [m][splits][top] keys
};

struct LpPart {
  float M, s, T, pad;
};

__device__ __forceinline__ void lp_wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
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

// (M, s, T) of two runs into one (see the top); -Inf: a run without any logit above -Inf.
__device__ __forceinline__ void lp_join(float& M, float& s, float& T, float Mb, float sb, float Tb) {
  const bool sw = Mb > M;
  const float Mh = sw ? Mb : M, sh = sw ? sb : s, Th = sw ? Tb : T;
  const float Ml = sw ? M : Mb, sl = sw ? s : sb, Tl = sw ? T : Tb;
  M = Mh;
  if (Ml == -INFINITY) {
    s = sl != sl ? sl : sh;                        // (a NaN among the run's logits stays)
    T = Th;
    return;
  }
  const float d = Ml - Mh, f = lp_exp(d);
  s = sh + f * (1.0f + sl);
  T = f > 0.0f ? Th + f * (Tl + (1.0f + sl) * d) : (f != f ? f : Th);
}

// A wave's candidates for the K best keys: a list in LDS, and a bound.
struct LpTop {
  uint64_t* list;         // [kLpCap], this wave's
  int K;
  int cnt = 0;            // keys in the list (uniform)
  uint32_t thr = 0;       // orders below this are out (uniform)

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
#pragma unroll 8
      for (int i = 0; i < cnt; ++i) rank[0] += list[i] > key[0] ? 1 : 0;
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
      if (last > thr) thr = last;
    }
  }

  // whether the keys of the lanes with `in` fit the list
  __device__ __forceinline__ bool fits(uint64_t ballot) const { return cnt + __popcll(ballot) <= kLpCap; }
  __device__ __forceinline__ void put(bool in, uint64_t ballot, uint64_t key, int lane) {
    if (in) list[cnt + __popcll(ballot & ((1ull << lane) - 1))] = key;
    cnt += __popcll(ballot);
  }
};

// the K-th largest of the 64 lanes' values
__device__ __forceinline__ uint32_t lp_kth(uint32_t v, int K) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 0; --b) {
    const uint32_t c = t | (1u << b);
    if (__popcll(__ballot(v >= c)) >= K) t = c;
  }
  return t;
}

// Outputs of a row from its joined sums and (top > 0) its K best keys in descending order.
template <bool BF>
__device__ __forceinline__ void lp_finish(const LpArgs& a, int64_t row, float M, float s, float T,
                                          const uint64_t* best, int lane) {
  // a row of -Inf alone has no distribution: log probabilities -Inf, entropy 0; one with +Inf or
  // NaN: all NaN
  const bool none = M == -INFINITY && s == s;
  const bool bad = s != s || M == INFINITY || T != T;
  const float nan = __uint_as_float(0x7FC00000u);
  const float ls = log1pf(s);
  const auto lp = [&](float x) { return bad ? nan : none ? -INFINITY : (x - M) - ls; };
  for (int j = lane; j < a.nt; j += 64) {
    const int64_t at = row * a.nt + j;
    const int64_t t = a.tok64 ? static_cast<const int64_t*>(a.tokens)[at]
                              : (int64_t)static_cast<const int32_t*>(a.tokens)[at];
    float v = -INFINITY;                           // a token outside the vocabulary: probability 0
    if (t >= 0 && t < a.n) {
      const int64_t o = row * a.ldy + t;
      v = BF ? bf16_to_float(static_cast<const uint16_t*>(a.y)[o]) : static_cast<const float*>(a.y)[o];
      v = lp(v);
    }
    a.logp[at] = v;
  }
  if (lane == 0) a.ent[row] = bad ? nan : none ? 0.0f : ls - T / (1.0f + s);
  for (int j = lane; j < a.top; j += 64) {
    const uint64_t key = best[j];
    a.tidx[row * a.top + j] = (int32_t)(0xFFFFFFFFu - (uint32_t)key);
    a.tlogp[row * a.top + j] = lp(lp_value((uint32_t)(key >> 32)));
  }
}

template <bool BF>
__global__ __launch_bounds__(64 * kLpWaves) void k_logprobs(LpArgs a) {
  constexpr int V = BF ? 8 : 4;                    // logits per 16-byte load
  constexpr int E = 4 * V;                         // logits of a lane per batch
  constexpr int B = 64 * E;                        // logits of a wave per batch
  __shared__ uint64_t s_list[kLpWaves][kLpCap];
  __shared__ float s_run[kLpWaves][4];
  __shared__ int s_cnt[kLpWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = blockIdx.x / a.splits;
  const int sp = (int)(blockIdx.x - row * a.splits);
  const int64_t c0 = sp * a.part;
  const int64_t c1 = c0 + a.part < a.n ? c0 + a.part : a.n;
  const uint8_t* const yr = static_cast<const uint8_t*>(a.y) + row * a.ldy * (BF ? 2 : 4);

  // element e of the lane's batch at column c: c + 64 V (e / V) + V lane + e % V
  const auto load = [&](int64_t c, u32x4 v[4]) {
    if (c + B <= c1) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint8_t* src = yr + (c + 64 * V * q + V * lane) * (BF ? 2 : 4);
        if constexpr (BF) v[q] = *reinterpret_cast<const u32x4_a2*>(src);
        else v[q] = *reinterpret_cast<const u32x4_a4*>(src);
      }
    } else {                                       // the part's end: -Inf past it
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t cc = c + 64 * V * q + V * lane + (V / 4) * i;
          if constexpr (BF) {
            const uint16_t* src = reinterpret_cast<const uint16_t*>(yr);
            const uint32_t lo = cc < c1 ? src[cc] : 0xFF80u, hi = cc + 1 < c1 ? src[cc + 1] : 0xFF80u;
            v[q][i] = lo | hi << 16;
          } else {
            v[q][i] = cc < c1 ? reinterpret_cast<const uint32_t*>(yr)[cc] : 0xFF800000u;
          }
        }
    }
  };

  float M = -INFINITY, s = 0.0f, T = 0.0f;         // M uniform; s, T the lane's
  int owner = 0;                                   // the lane that left the maximum out
  LpTop top;
  top.list = s_list[w];
  top.K = a.top;
  uint32_t lmax = 0;                               // the lane's largest order so far
  float thrf = -INFINITY;                          // a logit below this cannot enter the list
  bool anynan = false;

  int64_t c = c0 + (int64_t)w * B;
  u32x4 cur[4], nxt[4];
  if (c < c1) load(c, cur);
  for (; c < c1; c += (int64_t)kLpWaves * B) {
    const int64_t cn = c + (int64_t)kLpWaves * B;
    if (cn < c1) load(cn, nxt);
    float x[E];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF) {
          x[8 * q + 2 * i] = bf16_to_float(cur[q][i] & 0xFFFFu);
          x[8 * q + 2 * i + 1] = __uint_as_float(cur[q][i] & 0xFFFF0000u);
        } else {
          x[4 * q + i] = __uint_as_float(cur[q][i]);
        }
      }
    float mx = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) mx = fmaxf(mx, x[e]);   // (a NaN is passed over)
    bool leave = false;                            // the lane leaves one maximum out of this batch
    if (__ballot(mx > M)) {
      float mn = mx;
#pragma unroll
      for (int sh = 32; sh >= 1; sh /= 2) mn = fmaxf(mn, __shfl_xor(mn, sh));
      if (M > -INFINITY) {
        const float d = M - mn, f = lp_exp(d);
        if (lane == owner) s += 1.0f;
        T = f > 0.0f ? f * (T + s * d) : s != s ? s : 0.0f;   // (s d may overflow where f is 0)
        s *= f;
      }
      M = mn;
      owner = __ffsll((unsigned long long)__ballot(mx == M)) - 1;
      leave = lane == owner;
    }
    if (M > -INFINITY) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = x[e] - M;
        float p = lp_exp(d);
        if (leave && x[e] == M) {
          p = 0.0f;
          leave = false;
        }
        s += p;
        T = fmaf(p, fmaxf(d, -200.0f), T);         // (a masked logit: 0 times a finite number)
      }
    } else {
      bool bad = false;
#pragma unroll
      for (int e = 0; e < E; ++e) bad |= x[e] != x[e];
      if (bad) s = __uint_as_float(0x7FC00000u);
    }
    if (a.top > 0) {
      anynan = anynan || __ballot(s != s) != 0;
      if (anynan || __ballot(mx >= thrf)) {
        uint32_t ord[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          ord[e] = lp_order(x[e]);
          lmax = ord[e] > lmax ? ord[e] : lmax;
        }
        const uint32_t kth = lp_kth(lmax, a.top);
        if (kth > top.thr) top.thr = kth;
        // the lane's logits that enter, a bit each
        uint32_t in = 0;
        int tot = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int64_t cc = c + 64 * V * (e / V) + V * lane + e % V;
          const bool ok = ord[e] >= top.thr && cc < c1;
          in |= (ok ? 1u : 0u) << e;
          tot += __popcll(__ballot(ok));
        }
        if (tot > 64) {
          // many: of those equal to the bound (a masked row: all of them) only the K of the lowest
          // indices can stay
          uint32_t eq = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) eq |= (ord[e] == top.thr ? 1u : 0u) << e;
          eq &= in;
          int before = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t g = eq & (((1u << V) - 1u) << (V * q));
            const int mine = __popc(g);
            int pre = before;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint64_t bl = __ballot((mine >> b) & 1);
              pre += __popcll(bl & ((1ull << lane) - 1)) << b;
              before += __popcll(bl) << b;
            }
            int drop = mine - (a.top - pre > 0 ? a.top - pre : 0);
            while (drop-- > 0) {
              const uint32_t high = 1u << (31 - __clz(g));
              g ^= high;
              in ^= high;
            }
          }
        }
        int from = 0;
        while (from < E) {
          int full = E;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (e < from || full < E) continue;
            const bool ok = ((in >> e) & 1u) && ord[e] >= top.thr;
            const uint64_t bl = __ballot(ok);
            if (bl == 0) continue;
            if (!top.fits(bl)) {
              full = e;
              continue;
            }
            const int64_t cc = c + 64 * V * (e / V) + V * lane + e % V;
            top.put(ok, bl, (uint64_t)ord[e] << 32 | (0xFFFFFFFFu - (uint32_t)cc), lane);
          }
          from = full;
          if (full < E) top.cut(lane);
        }
        // later batches have higher indices: only a larger logit can still enter
        if (kth >= top.thr && kth != 0xFFFFFFFFu && kth > 0) top.thr = kth + 1;
        thrf = top.thr <= 0x007FFFFFu ? -INFINITY : lp_value(top.thr);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) cur[q] = nxt[q];
  }

  // the lanes' sums (relative to the same M) in a fixed order
#pragma unroll
  for (int sh = 32; sh >= 1; sh /= 2) {
    s += __shfl_xor(s, sh);
    T += __shfl_xor(T, sh);
  }
  if (a.top > 0) top.cut(lane);
  if (lane == 0) {
    s_run[w][0] = M;
    s_run[w][1] = s;
    s_run[w][2] = T;
    s_cnt[w] = top.cnt;
  }
  __syncthreads();
  if (w != 0) return;
  for (int v = 1; v < kLpWaves; ++v) lp_join(M, s, T, s_run[v][0], s_run[v][1], s_run[v][2]);
  if (a.top > 0) {
    // (at most 64 keys from each wave: they fit the first wave's list)
    for (int v = 1; v < kLpWaves; ++v) {
      const int cv = s_cnt[v];
      if (lane < cv) top.list[top.cnt + lane] = s_list[v][lane];
      top.cnt += cv;
    }
    top.cut(lane);
  }
  if (a.splits == 1) {
    lp_finish<BF>(a, row, M, s, T, top.list, lane);
    return;
  }
  const int64_t at = row * a.splits + sp;
  if (lane == 0) reinterpret_cast<LpPart*>(a.scratch)[at] = LpPart{M, s, T, 0.0f};
  uint64_t* keys = reinterpret_cast<uint64_t*>(a.scratch + a.m * a.splits * sizeof(LpPart));
  if (lane < a.top) keys[at * a.top + lane] = lane < top.cnt ? top.list[lane] : 0;
}

// The parts of each row joined: one wave per row, lane l takes part l (splits <= 64).
template <bool BF>
__global__ __launch_bounds__(64) void k_logprobs_join(LpArgs a) {
  __shared__ uint64_t s_list[kLpCap];
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const LpPart* parts = reinterpret_cast<const LpPart*>(a.scratch) + row * a.splits;
  const uint64_t* keys = reinterpret_cast<const uint64_t*>(a.scratch + a.m * a.splits * sizeof(LpPart)) +
                         row * a.splits * a.top;
  float M = -INFINITY, s = 0.0f, T = 0.0f;
  if (lane < a.splits) {
    const LpPart p = parts[lane];
    M = p.M;
    s = p.s;
    T = p.T;
  }
#pragma unroll
  for (int sh = 1; sh < 64; sh *= 2) {
    const float Mb = __shfl_xor(M, sh), sb = __shfl_xor(s, sh), Tb = __shfl_xor(T, sh);
    // the lower lane's run first on both sides, so all lanes hold the same bits
    float M2 = (lane & sh) ? Mb : M, s2 = (lane & sh) ? sb : s, T2 = (lane & sh) ? Tb : T;
    lp_join(M2, s2, T2, (lane & sh) ? M : Mb, (lane & sh) ? s : sb, (lane & sh) ? T : Tb);
    M = M2;
    s = s2;
    T = T2;
  }
  LpTop top;
  top.list = s_list;
  top.K = a.top;
  if (a.top > 0) {
    // each part's keys descend: its first bounds the rest, and a part whose next key is below the
    // bound is done
    uint64_t key = lane < a.splits ? keys[(int64_t)lane * a.top] : 0;
    top.thr = lp_kth((uint32_t)(key >> 32), a.top);
    for (int r = 0; r < a.top; ++r) {
      const bool in = key != 0 && (uint32_t)(key >> 32) >= top.thr;
      const uint64_t bl = __ballot(in);
      if (bl == 0) break;
      if (!top.fits(bl)) top.cut(lane);
      top.put(in, bl, key, lane);
      key = in && r + 1 < a.top ? keys[(int64_t)lane * a.top + r + 1] : 0;
    }
    top.cut(lane);
  }
  lp_finish<BF>(a, row, M, s, T, top.list, lane);
}

// Workgroups per row: the whole row in one where the rows fill the chip, otherwise as many parts
// as give it about eight workgroups per CU, of at least one batch per wave, and at most 64.
static void lp_plan(const DevInfo& di, int64_t m, int64_t n, bool bf, int* splits, int64_t* part) {
  const int64_t unit = (bf ? 2048 : 1024) * kLpWaves;
  const int64_t units = (n + unit - 1) / unit;
  int64_t want = ((int64_t)di.cus * 8 + m - 1) / m;
  if (want > units) want = units;
  if (want > 64) want = 64;
  const int64_t per = (units + want - 1) / want;
  *part = per * unit;
  *splits = (int)((units + per - 1) / per);
}

uint64_t logprobs_scratch(const DevInfo& di, int64_t m, int64_t n, int top, bool bf) {
  int splits;
  int64_t part;
  lp_plan(di, m, n, bf, &splits, &part);
  if (splits == 1) return 0;
  return (uint64_t)m * splits * (sizeof(LpPart) + 8ull * top);
}

hipError_t launch_logprobs(const void* y, bool bf, int64_t m, int64_t n, int64_t ldy, const void* tokens,
                           bool tok64, int nt, int top, float* logp, float* ent, int32_t* tidx,
                           float* tlogp, void* scratch, hipStream_t s) {
  DevInfo di;
  hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  LpArgs a;
  a.y = y; a.m = m; a.n = n; a.ldy = ldy;
  a.tokens = tokens; a.tok64 = tok64; a.nt = nt; a.top = top;
  a.logp = logp; a.ent = ent; a.tidx = tidx; a.tlogp = tlogp;
  a.scratch = static_cast<uint8_t*>(scratch);
  lp_plan(di, m, n, bf, &a.splits, &a.part);
  const dim3 grid((unsigned)(m * a.splits)), block(64 * kLpWaves);
  if (bf) hipLaunchKernelGGL(k_logprobs<true>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(k_logprobs<false>, grid, block, 0, s, a);
  err = hipGetLastError();
  if (err != hipSuccess || a.splits == 1) return err;
  if (bf) hipLaunchKernelGGL(k_logprobs_join<true>, dim3((unsigned)m), dim3(64), 0, s, a);
  else hipLaunchKernelGGL(k_logprobs_join<false>, dim3((unsigned)m), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace w12
