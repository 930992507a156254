// A token for each row of logits from temperature, top-k, top-p, min-p and a given random number.
//
// With M the row's largest logit and w = e^((x - M) / T), all three filters keep a prefix of the tokens'
// order (descending logit, equal ones by the lower column), so what is kept is known by its last token.
// The token drawn is the first kept one in column order at which the mass passes u * (mass of all kept).
//
// A row is cut into parts of 16 logits a thread, which a workgroup holds in registers (k_sample).  It leaves
// the part's maximum, its mass, a histogram (of counts with top-k, else of masses, of bins of a 16th of a power of
// two of w, from the part's maximum down) and, in column order, the part's largest logits as far as whole bins of
// them fit a short list.  A workgroup a row joins the parts (k_sample_join): the histogram says how far down
// what is kept can reach, and then
//   one      a row that keeps one token (temperature 0, top-k 1, min-p above 1) needs the first column of the
//            largest logit alone, which is in the first part that has it;
//   lists    where everything down to there is in the lists, their logits are sorted, cut and drawn from;
//   no cut   without filters the parts' masses say which part the token is in, and that part is scanned;
//   cut bin  else (thousands kept) two more kernels, which have nothing to do for other rows, look again: the
//            parts (k_sample_cut) sum the masses above the bin that the cut falls in and list the bin's logits,
//            the rows (k_sample_cut_join) select the last one kept of those and go on as without a cut;
//   radix    if even one bin holds too many (thousands of equal logits), or top-p cuts what a top-k of
//            thousands leaves, one workgroup reads the row, 8 bits of the logits' order a time.
//
// What bounds it: the chain of a row's join for few rows (1 row of 152064: 6 us for the parts, 13 for the
// join, 3 for two kernels that find nothing to do; 22 in all), instructions for many: the parts of 64 rows take
// 27 us (39 MB) for 77 vector instructions a logit (18 of them in double, 6 conversions, 9 of integers), whose issue
// is busy 71 % of the time; of 256 rows of bfloat16 60 (78 MB).  Those need 81 and 126 us in all: the rest is joins
// (25 and 27 us) and the second pair of kernels (9 + 16 and 19 + 25 us) for rows that keep thousands.  Greedy rows take
// 14 us (1 row), 17 (64), 41 (256 of bfloat16).  The radix reads a row up to 11 times, its parts one after the other:
// 520 us for one row with a top-k of 5000 and top-p, 620 for 64.
//
// A border between two tokens has to fall as it does in the formula: where each border were off by 1e-7, as
// sums of 152064 floats are, one draw in a hundred from a flat row would be a neighbour's.  So weights
// that decide are e^(..) in double (their own 2^f by a polynomial: |f ln 2| < 0.35, 12 terms,
// 1e-14), those below 2^-24 of the maximum in float times an exact power of two (1e-7 of 2^-24), and sums are doubles in a
// fixed order or integers of 2^-61 of what can be kept.  The histogram's masses, which only choose
// where to look, are floats rounded to 2^-30.
#include "kv_device.hpp"

namespace w12 {

constexpr int kSmElems = 16;                      // logits of a part's thread
constexpr int kSmJoin = 1024;                     // threads of a row's join
constexpr int kSmBins = 512;
constexpr float kSmPerOctave = 16.0f;             // bins of a power of two of w
constexpr double kSmPerUnit = 16.0;               // of a logit's 1.0 at most with top-k, whose last one may have any w
constexpr int kSmParts = 64;                      // parts of a row at most
constexpr int kSmSort = 2048;                     // logits that a row's join can sort
constexpr int kSmAll = 2100000000;                // a cut's bin below every logit's
constexpr int kSmRows = 4096;                     // rows of a launch
constexpr uint32_t kSmMasked = 0x007FFFFFu;       // the order of -Inf
constexpr double kSmNear = 1048576.0;             // 2^20 grains (SmOf): what the roundings of 2^20 logits come to

template <int T>
struct SmShape {
  static constexpr int kPart = T * kSmElems;
  // Entries of a part's list: all are read by the row's join, and where a row's do not reach down to its cut the
  // second pair of kernels runs.  128 instead of 64 save that for rows that a mask leaves few of (64 rows, 97 % masked,
  // of 8, 16, 17, 24 and 38 parts: 38, 44, 49, 52, 78 us with 128, 52, 61, 61, 68, 79 with 64) and cost others up to
  // a tenth (top-p 0.95: 40, 63, 64, 71, 83 us with 128, 45, 60, 59, 68, 82 with 64; top-k 20 as much either way).
  // Vocabularies up to 65536 (16 parts), of which a mask leaves more parts with few, have 128.
  static constexpr int kList = 128;
  static __device__ __forceinline__ int list_bits(int parts) { return T == 256 && parts > 16 ? 6 : 7; }
  static constexpr int kHead = 4;                  // a part's record, in 64-bit words
  static constexpr int kCutList = 512;             // entries of the cut's list, which takes the place of both
  static constexpr int kRec = kHead + kCutList;
  static_assert(kList + kSmBins / 2 <= kCutList);
  static constexpr int kBpt = (kSmBins + T - 1) / T;   // bins of a thread
  static constexpr int kNone = (1 << 28) - 1;          // a word behind every record: reads as 0
};

__device__ __forceinline__ uint32_t sm_order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);    // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float sm_value(uint32_t ord) {
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}

// (of a row's records, `i` in words of 64, 32 bits; behind them 0)
__device__ __forceinline__ uint64_t sm_load(Rsrc rec, int i) {
  return __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(rec, 8 * i, 0, 0));
}
__device__ __forceinline__ uint32_t sm_load32(Rsrc rec, int i) { return __builtin_amdgcn_raw_buffer_load_b32(rec, 4 * i, 0, 0); }

// E logits of each of T threads: loads of 16 bytes (8 for 4 of bfloat16), the threads side by side in each.
// Columns from n on are -Inf.
template <bool BF, int T, int E>
struct SmLoad {
  static constexpr int kPer = BF && E >= 8 ? 8 : 4, kLoads = E / kPer, kWords = BF ? kPer / 2 : kPer;
  typedef uint32_t words __attribute__((ext_vector_type(kWords), aligned(BF ? 2 : 4)));
  static __device__ __forceinline__ int column(int e, int tid) { return (e / kPer * T + tid) * kPer + e % kPer; }
  static __device__ __forceinline__ void load(const uint8_t* row, int64_t c0, int64_t n, int tid, float (&x)[E]) {
    if (c0 + T * E <= n) {
#pragma unroll
      for (int v = 0; v < kLoads; ++v) {
        const words w = *reinterpret_cast<const words*>(row + (c0 + (int64_t)(v * T + tid) * kPer) * (BF ? 2 : 4));
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          if constexpr (BF) {
            x[kPer * v + 2 * i] = __uint_as_float(w[i] << 16);
            x[kPer * v + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          } else {
            x[kPer * v + i] = __uint_as_float(w[i]);
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int64_t c = c0 + column(e, tid);
        x[e] = -INFINITY;
        if (c < n) x[e] = BF ? bf16_to_float(reinterpret_cast<const uint16_t*>(row)[c]) : reinterpret_cast<const float*>(row)[c];
      }
    }
  }
};

// (a constant in scalar registers: in vector ones a multiply-add takes two moves first)
__device__ __forceinline__ double sm_scalar(double c) {
  asm("" : "+s"(c));
  return c;
}
// 2^t for t <= 0 (below 2^-1000: 0)
__device__ __forceinline__ double sm_exp2(double t) {
  t = t > -1000.0 ? t : -1000.0;
  const double n = __builtin_rint(t);
  const double f = (t - n) * 0.693147180559945309417;
  double p = 1.0 / 479001600.0;
  p = __builtin_fma(p, f, sm_scalar(1.0 / 39916800.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 3628800.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 362880.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 40320.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 5040.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 720.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 120.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 24.0));
  p = __builtin_fma(p, f, sm_scalar(1.0 / 6.0));
  p = __builtin_fma(p, f, 0.5);
  p = __builtin_fma(p, f, 1.0);
  p = __builtin_fma(p, f, 1.0);
  return n > -1000.0 ? __builtin_ldexp(p, (int)n) : 0.0;
}

// What a row asks for.
struct SmRow {
  double c;               // log2 e / temperature
  float bins;             // bins of a logit's 1.0
  int64_t k;              // n: off; 1: the first token alone
  double p;               // 1 or more: off
  double min_p;           // 0: off
  __device__ __forceinline__ SmRow(const SampleArgs& a, int64_t row, float temp) {
    const bool hard = temp <= 0.0f;
    c = hard ? 1.4426950408889634 : 1.4426950408889634 / (double)temp;
    const int32_t kk = a.top_k ? a.top_k[row] : 0;
    const float pp = a.top_p ? a.top_p[row] : 1.0f, mp = a.min_p ? a.min_p[row] : 0.0f;
    const bool one = hard || mp > 1.0f;
    k = one ? 1 : kk > 0 && kk < a.n ? kk : a.n;
    p = !one && pp < 1.0f ? (pp > 0.0f ? (double)pp : 0.0) : 1.0;
    min_p = !one && mp > 0.0f ? (double)mp : 0.0;
    const double per = c * kSmPerOctave, most = k < a.n ? kSmPerUnit : 1e30;
    bins = (float)(per < most ? per : most);
  }
  // bin of a logit above -Inf: never falls as x rises
  __device__ __forceinline__ int bin(float x) const {
    return (int)floorf(fminf(fmaxf(x * bins, -1e9f), 1e9f));
  }
};

// The lane ahead's value, 0 in the first.
template <class V>
__device__ __forceinline__ V sm_ahead(V v) {
  const V up = __shfl_up(v, 1);
  return (threadIdx.x & 63) != 0 ? up : V(0);
}

// Sums over the workgroup's threads, in a fixed order.  N at once, one wait for all.
template <int T, int N, class V>
__device__ __forceinline__ void sm_scans(const V (&v)[N], V (*s_w)[N], V (&before)[N], V (&tot)[N]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  V in[N];
#pragma unroll
  for (int z = 0; z < N; ++z) in[z] = lane_scan(v[z]);
  __syncthreads();
  if (lane == 63) {
#pragma unroll
    for (int z = 0; z < N; ++z) s_w[w][z] = in[z];
  }
  __syncthreads();
#pragma unroll
  for (int z = 0; z < N; ++z) {
    V pre = 0;
    tot[z] = 0;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) {
      if (i == w) pre = tot[z];
      tot[z] += s_w[i][z];
    }
    before[z] = pre + sm_ahead(in[z]);             // (not a difference, which a double would round)
  }
}
template <int T, class V>
__device__ __forceinline__ V sm_scan(V v, V* s_w, V* before) {   // *before: of the threads ahead
  const V vs[1] = {v};
  V b[1], t[1];
  sm_scans<T, 1>(vs, reinterpret_cast<V(*)[1]>(s_w), b, t);
  *before = b[0];
  return t[0];
}
template <int T>
__device__ __forceinline__ unsigned long long sm_most(unsigned long long v, unsigned long long* s_w) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const unsigned long long other = __shfl_xor(v, o);
    v = other > v ? other : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < T / 64; ++i) v = s_w[i] > v ? s_w[i] : v;
  return v;
}
template <int T, class V>
__device__ __forceinline__ V sm_sum(V v, V* s_w) {
  v = last_lane(lane_scan(v));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = v;
  __syncthreads();
  V tot = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) tot += s_w[i];
  return tot;
}

// The end of what is kept: a logit's order and a column; tokens of a higher order, and of the same up to the
// column, are in.
struct SmCut {
  uint32_t key;
  uint32_t col;
  __device__ __forceinline__ bool in(uint32_t key_, uint32_t col_) const { return key_ > key || (key_ == key && col_ <= col); }
};

// What a row's first join leaves for the second kernel.
struct SmPlanned {
  int state;              // 0: done, 1: cut in a bin, 2: by radix
  int bin, big;           // the cut's bin (kSmAll: no cut but min-p), the largest logit's bin
  float M;
  double W;               // the row's mass (top-k off)
};

// A row.
template <bool BF>
struct SmOf {
  const SampleArgs& a;
  const int tid;
  const int64_t row;
  const uint8_t* const y;
  const int parts;
  const float temp;
  const SmRow r;
  double M = 0.0;                                  // the row's largest logit
  uint32_t top = 0;                                // its order

  __device__ __forceinline__ SmOf(const SampleArgs& args, int64_t row_, int parts_)
      : a(args), tid((int)threadIdx.x), row(row_), y(static_cast<const uint8_t*>(args.y) + row_ * args.ldy * (BF ? 2 : 4)),
        parts(parts_), temp(args.temperature ? args.temperature[row_] : 1.0f), r(args, row_, temp) {}
  __device__ __forceinline__ void is_top(float x) {
    M = (double)x;
    top = sm_order(x);
  }
  __device__ __forceinline__ double weight(float x) const { return sm_exp2(((double)x - M) * r.c); }
  __device__ __forceinline__ bool passes(double w, uint32_t key) const { return w >= r.min_p || key == top; }
};

// The parts' kernels.
template <bool BF, int T>
struct SmPart : SmOf<BF> {
  using S = SmShape<T>;
  using L = SmLoad<BF, T, kSmElems>;
  using Of = SmOf<BF>;
  using Of::a, Of::tid, Of::y, Of::temp, Of::r, Of::weight, Of::passes;

  struct Shared {
    unsigned long long hist[kSmBins];              // count << 48 | mass in 2^-30
    double wd[T / 64];
    unsigned long long wu[T / 64];
    float wf[T / 64];
    int bad, n;
  };
  Shared& s;
  __device__ __forceinline__ SmPart(const SampleArgs& args, int64_t row_, int parts_, Shared& sh) : Of(args, row_, parts_), s(sh) {}

  // A part: its record into rec.
  __device__ __forceinline__ void part(int p, uint64_t* rec) {
    const bool cuts = r.k < a.n || r.p < 1.0 || r.min_p > 0.0, masses = !(r.k < a.n);
    const int64_t c0 = (int64_t)p * S::kPart;
    float x[kSmElems];
    L::load(y, c0, a.n, tid, x);
    if (tid == 0) s.bad = temp != temp ? 1 : 0;
    if (cuts)
      for (int b = tid; b < kSmBins; b += T) s.hist[b] = 0;
    float mx = x[0];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kSmElems; ++e) {
      bad |= !(x[e] < INFINITY);
      mx = fmaxf(mx, x[e]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    if ((tid & 63) == 0) s.wf[tid >> 6] = mx;
    __syncthreads();
    if (bad) s.bad = 1;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) mx = fmaxf(mx, s.wf[i]);
    const int big = mx > -INFINITY ? r.bin(mx) : -1000000000;
    double tot = 0.0;
    int rel[kSmElems];
#pragma unroll
    for (int e = 0; e < kSmElems; ++e) {
      const bool live = x[e] > -INFINITY && mx < INFINITY;
      float wf = 0.0f;
      if (masses) {
        const double t = live ? ((double)x[e] - (double)mx) * r.c : -1e4;
        double w;
        if (__ballot(t > -24.0)) {
          w = sm_exp2(t);
        } else {
          const double n = __builtin_rint(t > -1000.0 ? t : -1000.0);
          w = __builtin_ldexp((double)__builtin_amdgcn_exp2f((float)((t > -1000.0 ? t : -1000.0) - n)), (int)n);
        }
        w = live ? w : 0.0;
        tot += w;
        wf = (float)w;
      }
      __builtin_amdgcn_sched_barrier(0);           // (else all 16 are in flight, in more registers than there are)
      rel[e] = kSmBins;
      if (cuts && live) {
        const int d = big - r.bin(x[e]);
        rel[e] = d < kSmBins ? d : kSmBins - 1;
        atomicAdd(&s.hist[rel[e]], 1ull << 48 | (uint32_t)(wf * 1073741824.0f + 0.5f));
      }
    }
    if (masses) tot = sm_sum<T>(tot, s.wd);
    else __syncthreads();
    int bound = -1, listed = 0, live = 0;
    if (!cuts) {
#pragma unroll
      for (int e = 0; e < kSmElems; ++e) live += x[e] > -INFINITY ? 1 : 0;
      live = sm_sum<T>(live, reinterpret_cast<int*>(s.wf));
    }
    if (cuts) {
      // whole bins from the top while they fit the list
      int mine = 0, own[S::kBpt];
#pragma unroll
      for (int i = 0; i < S::kBpt; ++i) {
        const int b = tid * S::kBpt + i;
        own[i] = 0;
        if (b < kSmBins) {
          const unsigned long long h = s.hist[b];
          own[i] = (int)(h >> 48);
          reinterpret_cast<uint32_t*>(rec + S::kHead + S::kList)[b] =
              masses ? __float_as_uint((float)(h & 0xFFFFFFFFFFFFull) * (1.0f / 1073741824.0f)) : (uint32_t)own[i];
        }
        mine += own[i];
      }
      int before;
      sm_scan<T>(mine, reinterpret_cast<int*>(s.wf), &before);
      int fit = 0;
#pragma unroll
      for (int i = 0; i < S::kBpt; ++i) {
        before += own[i];
        fit += tid * S::kBpt + i < kSmBins && before <= 1 << S::list_bits(this->parts) ? 1 : 0;
      }
      bound = sm_sum<T>(fit, reinterpret_cast<int*>(s.wf)) - 1;
      // (the counts of a load's logits, 16 bits each, in one sum)
      unsigned long long cnt = 0;
#pragma unroll
      for (int e = 0; e < kSmElems; ++e) cnt += rel[e] <= bound ? 1ull << (16 * (e / L::kPer)) : 0ull;
      unsigned long long ahead;
      const unsigned long long all = sm_scan<T>(cnt, s.wu, &ahead);
      int base = 0;
#pragma unroll
      for (int v = 0; v < L::kLoads; ++v) {
        int at = base + (int)(ahead >> (16 * v) & 0xFFFFu);
#pragma unroll
        for (int i = 0; i < L::kPer; ++i) {
          const int e = v * L::kPer + i;
          if (rel[e] <= bound) rec[S::kHead + at++] = (uint64_t)sm_order(x[e]) << 32 | (uint32_t)(c0 + L::column(e, tid));
        }
        base += (int)(all >> (16 * v) & 0xFFFFu);
      }
      listed = base;
    }
    if (tid == 0) {
      rec[0] = (uint64_t)__float_as_uint(mx) << 32 | (uint32_t)s.bad;
      rec[1] = (uint64_t)(uint32_t)big << 32 | (uint32_t)(bound + 1);
      rec[2] = (uint64_t)(uint32_t)live << 32 | (uint32_t)listed;
      rec[3] = (uint64_t)__double_as_longlong(tot);
    }
  }

  // The second kernel's part of a row with a plan: masses and counts of what lies above the cut's bin (also of
  // those that min-p leaves), and the bin's logits, into the record.
  __device__ __forceinline__ void cut_part(int p, const SmPlanned& plan, uint64_t* rec) {
    const int64_t c0 = (int64_t)p * S::kPart;
    float x[kSmElems];
    L::load(y, c0, a.n, tid, x);
    if (tid == 0) s.n = 0;
    __syncthreads();
    double mass = 0.0, left = 0.0;
    unsigned long long counts = 0;                 // above, and of those the ones min-p leaves << 32
#pragma unroll
    for (int e = 0; e < kSmElems; ++e) {
      const int d = x[e] > -INFINITY ? plan.big - r.bin(x[e]) : 0x7FFFFFFF;
      if (d < plan.bin) {
        const double w = weight(x[e]);
        mass += w;
        const bool in = passes(w, sm_order(x[e]));
        left += in ? w : 0.0;
        counts += in ? 1ull << 32 | 1 : 1;
      }
      if (d == plan.bin) {
        const int at = atomicAdd(&s.n, 1);
        if (at < S::kCutList) rec[S::kHead + at] = (uint64_t)sm_order(x[e]) << 32 | (uint32_t)~(uint32_t)(c0 + L::column(e, tid));
      }
    }
    mass = sm_sum<T>(mass, s.wd);
    left = sm_sum<T>(left, s.wd);
    counts = sm_sum<T>(counts, s.wu);
    if (tid == 0) {
      rec[0] = (uint64_t)__double_as_longlong(mass);
      rec[1] = (uint64_t)__double_as_longlong(left);
      rec[2] = counts;
      rec[3] = (uint64_t)s.n;
    }
  }
};

// The rows' kernels: a workgroup a row.
template <bool BF, int P>
struct SmJoin : SmOf<BF> {
  static constexpr int T = kSmJoin;
  using S = SmShape<P>;
  static constexpr int kElems = S::kPart / T;
  using L = SmLoad<BF, T, kElems>;
  using Of = SmOf<BF>;
  using Of::a, Of::tid, Of::row, Of::y, Of::parts, Of::r, Of::M, Of::top, Of::weight, Of::passes;

  struct Shared {
    union {
      struct {
        unsigned long long sorting[kSmSort];       // order, then the column's complement
        unsigned long long cand[kSmSort];          // order, column; in column order
      };
      unsigned long long all[2 * kSmSort];         // the cut's bin: order, then the column's complement
      struct {
        double ms[kSmJoin - kSmBins];
        int cnt[kSmJoin - kSmBins];
      };
    };
    unsigned long long mass8[256];
    uint32_t cnt8[256];
    double wd[T / 64];
    unsigned long long wu[T / 64], wv[T / 64][L::kLoads];
    float wf[T / 64];
    // the parts
    double scale[kSmParts];
    unsigned long long mass[kSmParts];             // of what is kept, in grains
    uint32_t ties[kSmParts];
    int shift[kSmParts], list[kSmParts];
    int found;
    int place[256];
    int at;
    unsigned long long ahead, last;                // a selection's: ahead of its bin, what it selects
    double val;
  };
  Shared& s;
  double grain = 0.0;                              // masses that are added in any order are integers of 1 / grain
  __device__ __forceinline__ SmJoin(const SampleArgs& args, int64_t row_, int parts_, Shared& sh) : Of(args, row_, parts_), s(sh) {}

  // What is kept, of a mass up to `most`, is less than 2^62 grains.  (With a grain for all rows, 2^-42 of the largest
  // weight, 150000 logits 22.5 below one that stands alone were cut, and drawn from, some places off.)
  __device__ __forceinline__ void set_grain(double most) {
    grain = __builtin_ldexp(1.0, 61 - ((int)(__double_as_longlong(most) >> 52) - 1023));
  }
  __device__ __forceinline__ unsigned long long fine(double w) const { return (unsigned long long)(w * grain + 0.5); }

  __device__ __forceinline__ void put(int64_t token, double logp, int64_t kept) const {
    if (a.token) a.token[row] = (int32_t)token;
    if (a.logp) a.logp[row] = (float)logp;
    if (a.kept) a.kept[row] = (int32_t)kept;
  }

  // s.sorting's first `size` (a power of two, 64 or more) descending.  A wave has 128 of them to itself while the
  // steps are short.
  __device__ __forceinline__ void sort(int size) {
    for (int len = 2; len <= size; len <<= 1)
      for (int step = len >> 1; step > 0; step >>= 1) {
        if (step >= 64) {
          __syncthreads();
        } else {
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
        for (int z = tid; z < size / 2; z += T) {
          const int i = (z & ~(step - 1)) * 2 + (z & (step - 1)), j = i + step;
          const unsigned long long u = s.sorting[i], v = s.sorting[j];
          if ((u < v) == ((i & len) == 0)) {
            s.sorting[i] = v;
            s.sorting[j] = u;
          }
        }
      }
    __syncthreads();
  }

  // The weight of a logit where it is kept, else 0.
  __device__ __forceinline__ double kept_weight(SmCut cut, float x, uint32_t col) const {
    const uint32_t key = sm_order(x);
    const double w = weight(x > -INFINITY ? x : (float)M);
    return key > kSmMasked && cut.in(key, col) && passes(w, key) ? w : 0.0;
  }
  // (s.found and s.val, the token and its logit, are written; sum: of all kept, in grains)
  __device__ __forceinline__ void put_drawn(unsigned long long sum, int64_t kept) const {
    if (tid == 0) put(s.found, 0.6931471805599453 * (s.val - log2((double)sum / grain)), kept);
  }

  // The token, where `cut` is known and s.mass holds the kept mass of every part (in grains): the part, then in it.
  __device__ __forceinline__ void draw(SmCut cut, int64_t kept) {
    // (a lane a part, every wave alike)
    const int lane = tid & 63;
    const unsigned long long own = lane < parts ? s.mass[lane] : 0;
    const unsigned long long upto = lane_scan(own), sum = last_lane(upto);
    const float u = a.u[row];
    const double target = u > 0.0f ? (double)u * (double)sum : 0.0;
    bool last = u >= 1.0f;
    int64_t stop = a.n;
    if (!last && target >= kSmNear) {
      unsigned long long want = (unsigned long long)target;
      if (want >= sum) want = sum - 1;
      const int p = __popcll(__ballot(lane < parts - 1 && upto <= want));
      const int64_t c0 = (int64_t)p * S::kPart;
      if (draw_part(cut, c0, want - __shfl(upto - own, p))) {
        put_drawn(sum, kept);
        return;
      }
      // the part's mass was more than its weights' by their roundings: its last one
      last = true;
      stop = c0 + S::kPart < a.n ? c0 + S::kPart : a.n;
    }
    draw_end(cut, stop, last, target / grain);
    put_drawn(sum, kept);
  }

  // In the part from column c0 on the token at which the mass passes `left`, into s.found; false if it never does.
  __device__ __forceinline__ bool draw_part(SmCut cut, int64_t c0, unsigned long long left) {
    float x[kElems];
    L::load(y, c0, a.n, tid, x);
    unsigned long long m[kElems], mine[L::kLoads], before[L::kLoads], tot[L::kLoads];
    if (tid == 0) s.found = -1;
#pragma unroll
    for (int v = 0; v < L::kLoads; ++v) {
      mine[v] = 0;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int e = v * L::kPer + i;
        m[e] = fine(kept_weight(cut, x[e], (uint32_t)(c0 + L::column(e, tid))));
        mine[v] += m[e];
      }
    }
    sm_scans<T, L::kLoads>(mine, s.wv, before, tot);
    unsigned long long sofar = 0;
#pragma unroll
    for (int v = 0; v < L::kLoads; ++v) {
      unsigned long long at = sofar + before[v];
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int e = v * L::kPer + i;
        if (at <= left && left < at + m[e]) {
          s.found = (int)(c0 + L::column(e, tid));
          s.val = ((double)x[e] - M) * r.c;
        }
        at += m[e];
      }
      sofar += tot[v];
    }
    __syncthreads();
    const int found = s.found;
    __syncthreads();                               // (all have read it before some write it again)
    return found >= 0;
  }

  // The same at u's ends, where the roundings to grains could decide: of the columns before `stop` the last kept one of
  // any mass, or the first at which the mass passes target, in doubles, 4 logits a thread at a time from that end.
  __device__ __forceinline__ void draw_end(SmCut cut, int64_t stop, bool last, double target) {
    using Q = SmLoad<BF, T, 4>;
    constexpr int kRun = 4 * T, kNone = 0x7FFFFFFF;
    const int runs = (int)((stop + kRun - 1) / kRun);
    double sofar = 0.0;
    for (int i = 0; i < runs; ++i) {
      const int64_t c0 = (int64_t)(last ? runs - 1 - i : i) * kRun;
      float x[4];
      Q::load(y, c0, stop, tid, x);
      if (tid == 0) s.found = last ? -1 : kNone;
      double w[4], mine = 0.0, before;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = kept_weight(cut, x[e], (uint32_t)(c0 + Q::column(e, tid)));
        mine += w[e];
      }
      const double all = sm_scan<T>(mine, s.wd, &before);
      double end = sofar + before;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        end += w[e];
        if (!(w[e] > 0.0)) continue;
        if (last) atomicMax(&s.found, (int)(c0 + Q::column(e, tid)));
        else if (end > target) atomicMin(&s.found, (int)(c0 + Q::column(e, tid)));
      }
      sofar += all;
      __syncthreads();
      const int found = s.found;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((int)(c0 + Q::column(e, tid)) == found) s.val = ((double)x[e] - M) * r.c;
      __syncthreads();                             // (and all have read s.found before the next run's)
      if (last ? found >= 0 : found != kNone) return;
    }
  }

  // Every logit of the row, a part at a time: f(x, key, column, part).
  template <class F, class G>
  __device__ __forceinline__ void each(const F& f, const G& end) {
    for (int p = 0; p < parts; ++p) {
      const int64_t c0 = (int64_t)p * S::kPart;
      float x[kElems];
      L::load(y, c0, a.n, tid, x);
#pragma unroll
      for (int e = 0; e < kElems; ++e)
        if (x[e] > -INFINITY) f(x[e], sm_order(x[e]), (uint32_t)(c0 + L::column(e, tid)));
      end(p);
    }
  }

  // The kept mass of every part into s.mass; returns the number kept.
  __device__ __forceinline__ int64_t part_masses(SmCut cut) {
    unsigned long long mine = 0, cnt = 0, kept = 0;
    each([&](float x, uint32_t key, uint32_t col) {
      if (!cut.in(key, col)) return;
      const double w = weight(x);
      if (!passes(w, key)) return;
      mine += fine(w);
      ++cnt;
    }, [&](int p) {
      const unsigned long long m = sm_sum<T>(mine, s.wu);
      if (tid == 0) s.mass[p] = m;
      kept += sm_sum<T>(cnt, s.wu);
      mine = cnt = 0;
    });
    __syncthreads();
    return (int64_t)kept;
  }

  // The first token in order at which `want` tokens (by_mass: that mass, in grains) have come, the last one there
  // is where they never do, by 8 bits of the order at a time.
  __device__ SmCut radix(unsigned long long want, bool by_mass, SmCut within) {
    uint32_t key = 0, mask = 0;
    unsigned long long had = 0, ties = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int b = tid; b < 256; b += T) {
        s.cnt8[b] = 0;
        s.mass8[b] = 0;
      }
      __syncthreads();
      each([&](float x, uint32_t k, uint32_t col) {
        if ((k & mask) != key || !within.in(k, col)) return;
        atomicAdd(&s.cnt8[k >> shift & 255u], 1u);
        if (by_mass) atomicAdd(&s.mass8[k >> shift & 255u], fine(weight(x)));
      }, [](int) {});
      __syncthreads();
      int bin = 0;
      unsigned long long upto = had;
      for (int b = 255; b >= 0; --b) {               // (all threads alike)
        const uint32_t c = s.cnt8[b];
        if (c == 0) continue;
        bin = b;
        had = upto;
        upto += by_mass ? s.mass8[b] : c;
        if (upto >= want) break;
      }
      ties = s.cnt8[bin];
      key |= (uint32_t)bin << shift;
      mask |= 255u << shift;
    }
    // of the equal ones, as many as it takes: the column of the last of them
    unsigned long long need = 1;
    const unsigned long long step = by_mass ? fine(weight(sm_value(key))) : 1;
    if (want > had && step > 0) need = (want - had + step - 1) / step;
    if (need > ties) need = ties;
    unsigned long long cnt = 0, seen = 0;
    each([&](float, uint32_t k, uint32_t) { cnt += k == key ? 1 : 0; }, [&](int p) {
      const unsigned long long t = sm_sum<T>(cnt, s.wu);
      if (tid == 0) s.ties[p] = (uint32_t)t;
      cnt = 0;
    });
    __syncthreads();
    int p = 0;
    while (p < parts - 1 && seen + s.ties[p] < need) seen += s.ties[p++];
    const int64_t c0 = (int64_t)p * S::kPart;
    float x[kElems];
    L::load(y, c0, a.n, tid, x);
    if (tid == 0) s.found = 0;
#pragma unroll
    for (int v = 0; v < L::kLoads; ++v) {
      unsigned long long n = 0, before;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) n += sm_order(x[v * L::kPer + i]) == key ? 1 : 0;
      const unsigned long long tot = sm_scan<T>(n, s.wu, &before);
      before += seen;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int e = v * L::kPer + i;
        if (sm_order(x[e]) != key) continue;
        if (++before == need) s.found = (int)(c0 + L::column(e, tid));
      }
      seen += tot;
    }
    __syncthreads();
    const SmCut cut = {key, (uint32_t)s.found};
    __syncthreads();
    return cut;
  }

  // The cuts by k and p over the row itself.
  __device__ __forceinline__ void whole_row(SmCut& cut, int64_t& kept) {
    const SmCut all = {kSmMasked + 1, 0xFFFFFFFFu};
    cut = all;
    if (r.k < a.n) cut = radix((unsigned long long)r.k, false, all);
    double mine = 0.0;
    each([&](float x, uint32_t key, uint32_t col) { mine += cut.in(key, col) ? weight(x) : 0.0; }, [](int) {});
    const double mass = sm_sum<T>(mine, s.wd);
    set_grain(mass);
    if (r.p < 1.0) cut = radix((unsigned long long)ceil(r.p * mass * grain), true, cut);
    kept = part_masses(cut);
  }

  // The first column of the row's largest logit, in part p.
  __device__ __forceinline__ void first_of(float mx, int p) {
    const int64_t c0 = (int64_t)p * S::kPart;
    float x[kElems];
    L::load(y, c0, a.n, tid, x);
    int first = 0x7FFFFFFF;
#pragma unroll
    for (int e = kElems - 1; e >= 0; --e)
      if (x[e] == mx) first = (int)c0 + L::column(e, tid);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const int other = __shfl_xor(first, o);
      first = other < first ? other : first;
    }
    if ((tid & 63) == 0) s.list[tid >> 6] = first;
    __syncthreads();
    if (tid != 0) return;
#pragma unroll
    for (int i = 1; i < T / 64; ++i) first = s.list[i] < first ? s.list[i] : first;
    put(first, 0.0, 1);
  }

  // The row, from its parts' records.
  __device__ __forceinline__ void join(const uint64_t* rec0, SmPlanned* plan) {
    const bool cuts = r.k < a.n || r.p < 1.0 || r.min_p > 0.0;
    const Rsrc recs = make_rsrc(rec0, (uint32_t)(parts * S::kRec * 8));
    if (tid == 0) plan->state = 0;
    // a lane a part, every wave alike
    const int lane = tid & 63;
    float tops = -INFINITY;
    bool bads = false;
    int bigs = -1000000000, bounds = kSmBins - 1, lists_n = 0, lives = 0;
    double totals = 0.0;
    if (lane < parts) {
      const int at = lane * S::kRec;
      const uint64_t h0 = sm_load(recs, at), h1 = sm_load(recs, at + 1), h2 = sm_load(recs, at + 2), h3 = sm_load(recs, at + 3);
      tops = __uint_as_float((uint32_t)(h0 >> 32));
      bads = (uint32_t)h0 != 0;
      bigs = (int)(uint32_t)(h1 >> 32);
      bounds = (int)(uint32_t)h1 - 1;
      lists_n = (int)(uint32_t)h2;
      lives = (int)(h2 >> 32);
      totals = __longlong_as_double((long long)h3);
    }
    float mx = tops;
    int big = bigs;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      mx = fmaxf(mx, __shfl_xor(mx, o));
      const int ob = __shfl_xor(big, o);
      big = ob > big ? ob : big;
    }
    const bool bad = __ballot(bads) != 0;
    if (bad || mx == -INFINITY) {
      if (tid == 0) put(-1, bad ? (double)__uint_as_float(0x7FC00000u) : -(double)INFINITY, 0);
      return;
    }
    if (r.k == 1) {
      first_of(mx, __ffsll((unsigned long long)__ballot(lane < parts && tops == mx)) - 1);
      return;
    }
    this->is_top(mx);
    const double scale = tops > -INFINITY ? sm_exp2(((double)tops - M) * r.c) : 0.0;
    const int shifts = big - bigs;
    double W = totals * scale;                     // (top-k off: the row's mass)
    __syncthreads();
    if (tid < parts) {
      s.scale[tid] = scale;
      s.shift[tid] = shifts;
      s.list[tid] = lists_n;
    }
    const double own = W;
    W = last_lane(lane_scan(W));
    set_grain(W);
    if (tid < parts) s.mass[tid] = fine(own);
    __syncthreads();
    if (!cuts) {
      draw({kSmMasked + 1, 0xFFFFFFFFu}, last_lane(lane_scan(lives)));
      return;
    }

    // the row's histogram (with top-k of counts, else of masses), a run of bins a thread, and how far down what
    // is kept can reach
    const bool counted = r.k < a.n;
    constexpr int kGroups = T / kSmBins, kAhead = 16;    // groups of parts, a group's parts in flight
    const int mine = tid % kSmBins, group = tid / kSmBins;
    int cnt = 0;
    double ms = 0.0;
    for (int p0 = group; p0 < parts; p0 += kAhead * kGroups) {
      uint32_t v[kAhead];
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        // (the last bin takes what lies below in its part, too)
        const int p = p0 + z * kGroups, b = mine - s.shift[p < parts ? p : 0];
        v[z] = sm_load32(recs, p < parts && mine < kSmBins - 1 && b >= 0 ? (p * S::kRec + S::kHead + S::kList) * 2 + b : S::kNone);
      }
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        const int p = p0 + z * kGroups;
        if (counted) cnt += (int)v[z];
        else ms += s.scale[p < parts ? p : 0] * (double)__uint_as_float(v[z]);
      }
    }
    if (group > 0) {
      s.cnt[tid - kSmBins] = cnt;
      s.ms[tid - kSmBins] = ms;
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 0; g < kGroups - 1; ++g) {
        cnt += s.cnt[g * kSmBins + mine];
        ms += s.ms[g * kSmBins + mine];
      }
    } else {
      cnt = 0;
      ms = 0.0;
    }
    int bin = kSmBins - 1;
    if (tid == 0) s.at = kSmBins - 1;
    if (counted) {
      int c;
      sm_scan<T>(cnt, reinterpret_cast<int*>(s.wf), &c);
      if (c < r.k && c + cnt >= r.k && mine < kSmBins - 1) s.at = mine;
      __syncthreads();
      bin = s.at;
    } else if (r.p < 1.0) {
      double m;
      sm_scan<T>(ms, s.wd, &m);
      const double want = r.p * W;
      if (m < want && m + ms >= want && mine < kSmBins - 1) s.at = mine;
      __syncthreads();
      bin = want > 0.0 ? s.at : 0;
    }
    int need = bin;
    // (top-k and top-p together: the mass of all k is asked for)
    bool by_min = false;
    if (r.min_p > 0.0 && !(r.k < a.n && r.p < 1.0)) {
      const double f = r.min_p < 1.0 ? -log2(r.min_p) / r.c * (double)r.bins + 3.0 : 3.0;
      if (f < (double)need) {
        need = (int)f;
        by_min = true;
      }
    }
    // how far down every list reaches (its last bin: all of a part)
    int reach = bounds == kSmBins - 1 ? kSmAll : bounds + shifts;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const int other = __shfl_xor(reach, o);
      reach = other < reach ? other : reach;
    }
    const bool lists = need < kSmBins - 1 ? need <= reach : reach == kSmAll;
    // top-p may end well before the last one of top-k, whose mass then hardly counts
    const bool partly = !lists && counted && r.p < 1.0 && reach >= 0;
    if (partly) need = reach < kSmBins - 2 ? reach : kSmBins - 2;
    if ((lists || partly) && from_lists(recs, need, by_min, partly, big, W)) return;
    if (tid != 0) return;
    bin = counted || r.p < 1.0 ? bin : kSmAll;
    plan->state = (counted && r.p < 1.0) || bin == kSmBins - 1 ? 2 : 1;
    plan->bin = bin;
    plan->big = big;
    plan->M = mx;
    plan->W = W;
  }

  // A row with a plan: its cut, and the token.
  __device__ __forceinline__ void cut_join(const SmPlanned& plan, const uint64_t* rec0) {
    SmCut cut = {kSmMasked + 1, 0xFFFFFFFFu};
    int64_t kept = 0;
    if (plan.state == 2 || !cut_bin(plan, rec0, cut, kept)) whole_row(cut, kept);
    draw(cut, kept);
  }
  // The cut from the second records: the bin's logits, selected from; false if it is not in them.
  __device__ __forceinline__ bool cut_bin(const SmPlanned& plan, const uint64_t* rec0, SmCut& cut, int64_t& all) {
    const Rsrc recs = make_rsrc(rec0, (uint32_t)(parts * S::kRec * 8));
    const int lane = tid & 63;
    double above = 0.0, left = 0.0;
    int count = 0, kept = 0, mine_n = 0;
    if (lane < parts) {
      const int at = lane * S::kRec;
      above = __longlong_as_double((long long)sm_load(recs, at));
      left = __longlong_as_double((long long)sm_load(recs, at + 1));
      const uint64_t c = sm_load(recs, at + 2);
      count = (int)(uint32_t)c;
      kept = (int)(c >> 32);
      mine_n = (int)sm_load(recs, at + 3);
    }
    const bool fits = __ballot(mine_n > S::kCutList) == 0;
    above = last_lane(lane_scan(above));
    count = last_lane(lane_scan(count));
    kept = last_lane(lane_scan(kept));
    const int upto_n = lane_scan(mine_n), n = last_lane(upto_n);
    if (!fits || n > 2 * kSmSort) return false;
    double most = last_lane(lane_scan(left));
    if (plan.bin < kSmBins) {
      if (tid < parts) s.list[tid] = upto_n - mine_n;
      __syncthreads();
      // the bin's logits, a wave a part
      for (int p = tid >> 6; p < parts; p += T / 64) {
        const int at = s.list[p], size = (p + 1 < parts ? s.list[p + 1] : n) - at;
        for (int e = lane; e < size; e += 64) s.all[at + e] = sm_load(recs, p * S::kRec + S::kHead + e);
      }
      __syncthreads();
      const double want = r.k < a.n ? (double)(r.k - count) : r.p * plan.W - above;
      unsigned long long last;
      // (the histogram's masses may be off by a bin)
      if (!(want > 0.0 || count == 0) || !select(n, !(r.k < a.n), want, plan.bin, &last)) return false;
      cut = {(uint32_t)(last >> 32), ~(uint32_t)last};
      // (none of the bin's weighs more than its first)
      unsigned long long first = 0;
      for (int i = tid; i < n; i += T) first = s.all[i] > first ? s.all[i] : first;
      most += (double)n * weight(sm_value((uint32_t)(sm_most<T>(first, s.wu) >> 32)));
    }
    set_grain(most);
    if (tid < parts) s.mass[tid] = fine(left);
    if (plan.bin < kSmBins) {
      __syncthreads();
      const unsigned long long last = (unsigned long long)cut.key << 32 | (uint32_t)~cut.col;
      int more = 0;
      for (int i = tid; i < n; i += T) {
        const unsigned long long v = s.all[i];
        if (v < last) continue;
        const double wi = weight(sm_value((uint32_t)(v >> 32)));
        if (passes(wi, (uint32_t)(v >> 32))) {
          atomicAdd(&s.mass[~(uint32_t)v / (uint32_t)S::kPart], fine(wi));
          ++more;
        }
      }
      kept += sm_sum<T>(more, reinterpret_cast<int*>(s.wf));
    }
    __syncthreads();
    all = kept;
    return true;
  }

  // Of s.all's n logits, all of bin `bin`, the one in descending order at which `want` of them (by_mass: that mass)
  // have come; false if they never do.  8 bits of the order and the column at a time, from the first that
  // differ; masses as integers of 2^-50 of the bin's.
  __device__ __forceinline__ bool select(int n, bool by_mass, double want, int bin, unsigned long long* last) {
    const unsigned long long first = s.all[0];
    unsigned long long diff = 0;
    for (int i = tid; i < n; i += T) diff |= s.all[i] ^ first;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) diff |= __shfl_xor(diff, o);
    if ((tid & 63) == 0) s.wu[tid >> 6] = diff;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / 64; ++i) diff |= s.wu[i];
    const int scale = 49 + bin / (int)kSmPerOctave;
    unsigned long long left = 1;                   // (at least one)
    if (by_mass) {
      const double f = ceil(__builtin_ldexp(want, scale));
      if (f > 9e18) return false;
      if (f > 1.0) left = (unsigned long long)f;
    } else if (want > 1.0) {
      left = (unsigned long long)want;
    }
    int shift = diff ? 63 - __builtin_clzll(diff) - 7 : 0;
    shift = shift > 0 ? shift : 0;
    unsigned long long mask = shift < 56 ? ~0ull << (shift + 8) : 0ull, key = first & mask;
    for (bool again = false;; again = true) {
      __syncthreads();
      for (int b = tid; b < 256; b += T) {
        s.mass8[b] = 0;
        s.cnt8[b] = 0;
      }
      __syncthreads();
      for (int i = tid; i < n; i += T) {
        const unsigned long long v = s.all[i];
        if ((v & mask) != key) continue;
        const int d = (int)(v >> shift & 255u);
        atomicAdd(&s.cnt8[d], 1u);
        if (by_mass) atomicAdd(&s.mass8[d], (unsigned long long)(__builtin_ldexp(weight(sm_value((uint32_t)(v >> 32))), scale) + 0.5));
      }
      __syncthreads();
      unsigned long long mine = 0, before;
      if (tid < 256) mine = by_mass ? s.mass8[255 - tid] : s.cnt8[255 - tid];
      const unsigned long long all = sm_scan<T>(mine, s.wu, &before);
      if (!again && all < left) return false;
      if (before < left && left <= before + mine) {
        s.at = 255 - tid;
        s.ahead = before;
      }
      __syncthreads();
      const int d = s.at;
      left -= s.ahead;
      key |= (unsigned long long)d << shift;
      mask |= 255ull << shift;
      if (s.cnt8[d] == 1) break;
      shift = shift > 8 ? shift - 8 : 0;
    }
    for (int i = tid; i < n; i += T)
      if ((s.all[i] & mask) == key) s.last = s.all[i];
    __syncthreads();
    *last = s.last;
    return true;
  }

  // Cuts and draws from the lists' logits down to bin `need`; false if they turn out not to reach the cut.
  __device__ __forceinline__ bool from_lists(Rsrc recs, int need, bool by_min, bool partly, int big, double W) {
    // a run of the lists' slots a thread, so that one sum gives their places
    constexpr int kMost = kSmParts * (P == 256 ? S::kList / 2 : S::kList) / T;
    static_assert(16 * S::kList <= kMost * T);
    const int bits = S::list_bits(parts), slots = parts << bits, run = (slots + T - 1) / T;
    uint64_t v[kMost];
#pragma unroll
    for (int q = 0; q < kMost; ++q) {
      const int i = tid * run + q, p = i >> bits, e = i & ((1 << bits) - 1);
      const bool is = q < run && i < slots && e < s.list[i < slots ? p : 0];
      v[q] = sm_load(recs, is ? p * S::kRec + S::kHead + e : S::kNone);     // (nothing: 0)
    }
    uint32_t in = 0;
    int at0, all = 0;
#pragma unroll
    for (int q = 0; q < kMost; ++q) {
      in |= (v[q] != 0) & ((need >= kSmBins - 1) | (big - r.bin(sm_value((uint32_t)(v[q] >> 32))) <= need)) ? 1u << q : 0u;
      all += v[q] != 0 ? 1 : 0;
    }
    // (both sums in one: at most 2^14 of each)
    const int sums = sm_scan<T>((int)__popc(in) | all << 16, reinterpret_cast<int*>(s.wf), &at0);
    const int n = sums & 0xFFFF;
    at0 &= 0xFFFF;
    all = sums >> 16;
    if (n > kSmSort) return false;
#pragma unroll
    for (int q = 0; q < kMost; ++q)
      if (in >> q & 1u) {
        s.cand[at0] = v[q];
        s.sorting[at0++] = v[q] ^ 0xFFFFFFFFu;
      }
    __syncthreads();
    constexpr int kFew = 256;                      // (1 row with top-k 20: 21 us, by sorting 24)
    if (n <= kFew) {
      // a logit's place is the number of those ahead of it, counted by T / kFew threads
      const int i = tid % kFew;
      const unsigned long long own = s.sorting[i < n ? i : 0];
      int place = 0;
      for (int j = tid / kFew; j < n; j += T / kFew) place += s.sorting[j] > own ? 1 : 0;
      if (tid < kFew) s.place[i] = place;
      __syncthreads();
      if (tid >= kFew && i < n) atomicAdd(&s.place[i], place);
      __syncthreads();
      if (tid < n) s.sorting[s.place[i]] = own;
      __syncthreads();
    } else {
      int size = 64;
      while (size < n) size <<= 1;
      for (int i = n + tid; i < size; i += T) s.sorting[i] = 0;
      __syncthreads();
      sort(size);
    }
    // masses in the tokens' order, a run of them a thread
    constexpr int kMine = kSmSort / T;
    const int own_n = (n + T - 1) / T, r0 = tid * own_n, kk = r.k < n ? (int)r.k : n;
    double own[kMine], mine = 0.0, before;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      own[q] = 0.0;
      if (q < own_n && r0 + q < kk) own[q] = weight(sm_value((uint32_t)(s.sorting[r0 + q] >> 32)));
      mine += own[q];
    }
    const double listed = sm_scan<T>(mine, s.wd, &before);
    const double want = r.p * (r.k < a.n ? listed : W);
    // (what is not here is below all that is, bins never falling as logits rise: so are those of top-k)
    const double least = weight(sm_value((uint32_t)(s.sorting[n - 1] >> 32)));
    const double most = partly ? r.p * (listed + (double)(r.k - n) * least) : want;
    const bool ends = all == n && need >= kSmBins - 1;   // (nothing else is left)
    // min-p's three bins more cover what rounding x * bins may move, while that is below 2^21 (a quarter of a bin)
    const bool min_ends = by_min && (least < r.min_p || fabs(M * (double)r.bins) < 2097152.0);
    // is the end of what is kept among them?
    if (!(partly ? listed >= most : ends || min_ends || (r.k < a.n ? n >= r.k : r.p < 1.0 && listed >= want))) return false;
    int keep = 0, keeps = 0;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int i = r0 + q;
      if (q < own_n && i < kk) {
        if (i == 0 || ((r.p >= 1.0 || before < want) && own[q] >= r.min_p)) ++keep;
        if (i == 0 || ((r.p >= 1.0 || before < most) && own[q] >= r.min_p)) ++keeps;
      }
      before += own[q];
    }
    keep = sm_sum<T>(keep, reinterpret_cast<int*>(s.wf));
    if (partly && sm_sum<T>(keeps, reinterpret_cast<int*>(s.wf)) != keep) return false;
    const unsigned long long last = s.sorting[keep - 1];
    const SmCut cut = {(uint32_t)(last >> 32), ~(uint32_t)last};
    // and in column order
    constexpr int kNone = 0x7FFFFFFF;
    mine = 0.0;
    if (tid == 0) s.found = kNone;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const unsigned long long v1 = s.cand[q < own_n && r0 + q < n ? r0 + q : 0];
      const bool is = q < own_n && r0 + q < n && cut.in((uint32_t)(v1 >> 32), (uint32_t)v1);
      own[q] = 0.0;
      if (is) own[q] = weight(sm_value((uint32_t)(v1 >> 32)));
      mine += own[q];
    }
    const double sum = sm_scan<T>(mine, s.wd, &before);
    const float u = a.u[row];
    const double target = u > 0.0f ? (double)u * sum : 0.0;
    // the first one past target (one thread's last border and the next one's first may differ by a rounding: where
    // target lies between them, the next one's is it), a wave's first for all of it
    int at = kNone;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      before += own[q];
      if (u < 1.0f || !(u > 0.0f)) at = own[q] > 0.0 && before > target && at == kNone ? r0 + q : at;
    }
    const uint64_t some = __ballot(at != kNone);
    if (some && (tid & 63) == __ffsll((unsigned long long)some) - 1) atomicMin(&s.found, at);
    __syncthreads();
    const int found = s.found;
    __syncthreads();                               // (all have read it before some write it again)
    if (found == kNone) {                          // u of 1 or more, or a rounding at the end: the last one
      if (tid == 0) s.found = 0;                   // (the largest logit has a weight, and a place from 0 on)
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kMine; ++q)
        if (own[q] > 0.0) atomicMax(&s.found, r0 + q);
      __syncthreads();
    }
    if (tid == 0) {
      const unsigned long long f = s.cand[s.found];
      const double d = ((double)sm_value((uint32_t)(f >> 32)) - M) * r.c;
      put((uint32_t)f, 0.6931471805599453 * (d - log2(sum)), keep);
    }
    return true;
  }
};

template <bool BF, int T>
__global__ __launch_bounds__(T, 6) void k_sample(SampleArgs a, int parts, uint64_t* recs) {
  __shared__ typename SmPart<BF, T>::Shared s;
  const int64_t row = blockIdx.x / parts;
  SmPart<BF, T> k(a, row, parts, s);
  k.part((int)(blockIdx.x - row * parts), recs + (int64_t)blockIdx.x * SmShape<T>::kRec);
}
template <bool BF, int T>
__global__ __launch_bounds__(kSmJoin) void k_sample_join(SampleArgs a, int parts, SmPlanned* plans, const uint64_t* recs) {
  __shared__ typename SmJoin<BF, T>::Shared s;
  const int64_t row = blockIdx.x;
  SmJoin<BF, T> k(a, row, parts, s);
  k.join(recs + row * parts * SmShape<T>::kRec, plans + row);
}
template <bool BF, int T>
__global__ __launch_bounds__(T, 6) void k_sample_cut(SampleArgs a, int parts, const SmPlanned* plans, uint64_t* recs) {
  __shared__ typename SmPart<BF, T>::Shared s;
  const int64_t row = blockIdx.x / parts;
  const SmPlanned plan = plans[row];
  if (plan.state != 1) return;
  SmPart<BF, T> k(a, row, parts, s);
  k.is_top(plan.M);
  k.cut_part((int)(blockIdx.x - row * parts), plan, recs + (int64_t)blockIdx.x * SmShape<T>::kRec);
}
template <bool BF, int T>
__global__ __launch_bounds__(kSmJoin) void k_sample_cut_join(SampleArgs a, int parts, const SmPlanned* plans, const uint64_t* recs) {
  __shared__ typename SmJoin<BF, T>::Shared s;
  const int64_t row = blockIdx.x;
  const SmPlanned plan = plans[row];
  if (plan.state == 0) return;
  SmJoin<BF, T> k(a, row, parts, s);
  k.is_top(plan.M);
  k.cut_join(plan, recs + row * parts * SmShape<T>::kRec);
}

// Parts of 4096 logits; of 16384 where a row would have more than 64 of them.
struct SmPlan {
  bool wide;              // 1024 threads
  int parts;
  int64_t rec;            // bytes
  int64_t rows;           // of a launch
};
static SmPlan sm_plan(int64_t m, int64_t n) {
  SmPlan p;
  const int64_t few = (n + SmShape<256>::kPart - 1) / SmShape<256>::kPart;
  p.wide = few > kSmParts;
  const int64_t size = p.wide ? SmShape<1024>::kPart : SmShape<256>::kPart;
  p.parts = (int)((n + size - 1) / size);
  p.rec = (p.wide ? SmShape<1024>::kRec : SmShape<256>::kRec) * 8;
  p.rows = (int64_t(64) << 20) / (p.parts * p.rec);
  p.rows = p.rows < 1 ? 1 : p.rows > kSmRows ? kSmRows : p.rows;
  p.rows = p.rows < m ? p.rows : m;
  return p;
}

uint64_t sample_scratch(int64_t m, int64_t n) {
  const SmPlan p = sm_plan(m, n);
  return (uint64_t)(p.rows * (p.parts * p.rec + (int64_t)sizeof(SmPlanned)));
}

template <bool BF, int T>
static void sm_go(hipStream_t s, const SampleArgs& a, int parts, SmPlanned* plans, uint64_t* recs, bool cuts) {
  const dim3 rows((unsigned)a.m), all((unsigned)(a.m * parts));
  hipLaunchKernelGGL((k_sample<BF, T>), all, dim3(T), 0, s, a, parts, recs);
  hipLaunchKernelGGL((k_sample_join<BF, T>), rows, dim3(kSmJoin), 0, s, a, parts, plans, recs);
  if (!cuts) return;
  hipLaunchKernelGGL((k_sample_cut<BF, T>), all, dim3(T), 0, s, a, parts, plans, recs);
  hipLaunchKernelGGL((k_sample_cut_join<BF, T>), rows, dim3(kSmJoin), 0, s, a, parts, plans, recs);
}

hipError_t launch_sample(const SampleArgs& a0, bool bf, void* scratch, hipStream_t s) {
  const SmPlan p = sm_plan(a0.m, a0.n);
  if (p.parts > kSmParts) return hipErrorInvalidValue;
  SampleArgs a = a0;
  uint64_t* const recs = static_cast<uint64_t*>(scratch);
  SmPlanned* const plans = reinterpret_cast<SmPlanned*>(recs + p.rows * p.parts * (p.rec / 8));
  // (without a filter nothing is left for the second pair: a temperature alone keeps one token or all)
  const bool cuts = a.top_k || a.top_p || a.min_p;
  for (int64_t r0 = 0; r0 < a0.m; r0 += p.rows) {
    a.m = a0.m - r0 < p.rows ? a0.m - r0 : p.rows;
    if (p.wide && bf) sm_go<true, 1024>(s, a, p.parts, plans, recs, cuts);
    else if (p.wide) sm_go<false, 1024>(s, a, p.parts, plans, recs, cuts);
    else if (bf) sm_go<true, 256>(s, a, p.parts, plans, recs, cuts);
    else sm_go<false, 256>(s, a, p.parts, plans, recs, cuts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.y = static_cast<const uint8_t*>(a.y) + p.rows * a.ldy * (bf ? 2 : 4);
    if (a.temperature) a.temperature += p.rows;
    if (a.top_k) a.top_k += p.rows;
    if (a.top_p) a.top_p += p.rows;
    if (a.min_p) a.min_p += p.rows;
    a.u += p.rows;
    if (a.token) a.token += p.rows;
    if (a.logp) a.logp += p.rows;
    if (a.kept) a.kept += p.rows;
  }
  return hipSuccess;
}

}  // namespace w12
