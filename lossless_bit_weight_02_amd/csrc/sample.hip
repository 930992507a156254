// A token for each row of logits from temperature, top-k, top-p, min-p and a given random number.
//
// With M the row's largest logit and w = e^((x - M) / T), all three filters keep a prefix of the tokens'
// order (descending logit, equal ones by the lower column), so what is kept is known by its last token.
// The token drawn is the first kept one in column order at which the mass passes u * (mass of all kept).
//
// A row is cut into parts of 16 logits a thread, which a workgroup holds in registers (k_sample).  It leaves
// the part's maximum, its mass, a histogram (count and mass of bins of a 32nd of a power of two of w, from
// the part's maximum down) and, in column order, the part's largest logits as far as whole bins of them
// fit a short list.  The row's last workgroup (counted) joins the parts: the histogram says how far down
// what is kept can reach, and then
//   lists    where everything down to there is in the lists, their logits are ranked, cut and drawn from;
//   no cut   without filters the parts' masses say which part the token is in, and that part is scanned;
//   cut bin  else (thousands kept) a second kernel's parts (k_sample_cut; it has nothing to do for other
//            rows) sum the masses above the bin that the cut falls in and list the bin's logits; the row's
//            last sorts those, cuts exactly, and goes on as without a cut;
//   radix    if even one bin holds too many (thousands of equal logits), or top-p cuts what a top-k of
//            thousands leaves, one workgroup reads the row, 8 bits of the logits' order a time.
//
// A border between two tokens has to fall as it does in the formula: where each border were off by 1e-7, as
// sums of 152064 floats are, one draw in a hundred from a flat row would be a neighbour's.  So weights
// that decide are e^(..) in double (their own 2^f by a polynomial: |f ln 2| < 0.35, 12 terms,
// 1e-14), those below 2^-24 of the maximum in float times an exact power of two (1e-7 of 2^-24), and sums are doubles in a
// fixed order or integers, the same whichever workgroup is last.  The histogram's masses, which only choose
// where to look, are floats rounded to 2^-30.
#include "kv_device.hpp"

namespace w12 {

constexpr int kSmElems = 16;                      // logits of a thread
constexpr int kSmBins = 1024;
constexpr float kSmPerOctave = 32.0f;             // bins of a power of two
constexpr int kSmParts = 64;                      // parts of a row at most
constexpr int kSmCand = 2048;                     // candidates that the lists' way ranks
constexpr int kSmLists = 4096;                    // entries of the lists that it takes
constexpr int kSmSort = 2048;                     // logits of the cut's bin that are sorted
constexpr int kSmAll = 2100000000;                // a cut's bin below every logit's
constexpr int kSmRows = 4096;                     // rows of a launch, each with a count
constexpr int kSmCountStep = 16;                  // counts 64 bytes apart
constexpr uint32_t kSmMasked = 0x007FFFFFu;       // the order of -Inf
constexpr double kSmFine = 4398046511104.0;       // 2^42: masses as integers, 2^20 logits of at most 1

typedef uint32_t sm_u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t sm_u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

template <int T>
struct SmShape {
  static constexpr int kPart = T * kSmElems;
  static constexpr int kList = T / 4;              // entries of a part's list
  static constexpr int kHead = 4;                  // a part's record, in 64-bit words
  static constexpr int kRec = kHead + kList + kSmBins;
};

__device__ __forceinline__ uint32_t sm_order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);    // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float sm_value(uint32_t ord) {
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}

__device__ __forceinline__ void sm_store(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// (of a row's records, `i` in words: as one of the device's dies stored it a moment ago)
constexpr int kAuxAgent = 16;                     // sc1
__device__ __forceinline__ uint64_t sm_load(Rsrc rec, int i) {
  return __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(rec, 8 * i, 0, kAuxAgent));
}

// 16 logits of a thread: V loads of 16 bytes, the workgroup's threads side by side in each.  Columns from n on are -Inf.
template <bool BF, int T>
struct SmLoad {
  static constexpr int kPer = BF ? 8 : 4, kLoads = kSmElems / kPer;
  static __device__ __forceinline__ int column(int e, int tid) { return (e / kPer * T + tid) * kPer + e % kPer; }
  static __device__ __forceinline__ void load(const uint8_t* row, int64_t c0, int64_t n, int tid, float (&x)[kSmElems]) {
    if (c0 + T * kSmElems <= n) {
#pragma unroll
      for (int v = 0; v < kLoads; ++v) {
        const uint8_t* const at = row + (c0 + (int64_t)(v * T + tid) * kPer) * (BF ? 2 : 4);
        if constexpr (BF) {
          const sm_u32x4_a2 w = *reinterpret_cast<const sm_u32x4_a2*>(at);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[8 * v + 2 * i] = __uint_as_float(w[i] << 16);
            x[8 * v + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        } else {
          const sm_u32x4_a4 w = *reinterpret_cast<const sm_u32x4_a4*>(at);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[4 * v + i] = __uint_as_float(w[i]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kSmElems; ++e) {
        const int64_t c = c0 + column(e, tid);
        x[e] = -INFINITY;
        if (c < n) x[e] = BF ? bf16_to_float(reinterpret_cast<const uint16_t*>(row)[c]) : reinterpret_cast<const float*>(row)[c];
      }
    }
  }
};

// 2^t for t <= 0 (below 2^-1000: 0)
__device__ __forceinline__ double sm_exp2(double t) {
  t = t > -1000.0 ? t : -1000.0;
  const double n = __builtin_rint(t);
  const double f = (t - n) * 0.693147180559945309417;
  double p = 1.0 / 479001600.0;
  p = __builtin_fma(p, f, 1.0 / 39916800.0);
  p = __builtin_fma(p, f, 1.0 / 3628800.0);
  p = __builtin_fma(p, f, 1.0 / 362880.0);
  p = __builtin_fma(p, f, 1.0 / 40320.0);
  p = __builtin_fma(p, f, 1.0 / 5040.0);
  p = __builtin_fma(p, f, 1.0 / 720.0);
  p = __builtin_fma(p, f, 1.0 / 120.0);
  p = __builtin_fma(p, f, 1.0 / 24.0);
  p = __builtin_fma(p, f, 1.0 / 6.0);
  p = __builtin_fma(p, f, 0.5);
  p = __builtin_fma(p, f, 1.0);
  p = __builtin_fma(p, f, 1.0);
  return n > -1000.0 ? __builtin_ldexp(p, (int)n) : 0.0;
}

// What a row asks for.
struct SmRow {
  double c;               // log2 e / temperature
  float bins;             // bins of one unit of logit
  bool hard;              // the largest logit
  int64_t k;              // n: off
  double p;               // 1 or more: off
  double min_p;           // 0: off
  __device__ __forceinline__ SmRow(const SampleArgs& a, int64_t row, float temp) {
    hard = temp <= 0.0f;
    c = hard ? 1.4426950408889634 : 1.4426950408889634 / (double)temp;
    bins = (float)(c * kSmPerOctave < 1e30 ? c * kSmPerOctave : 1e30);
    const int32_t kk = a.top_k ? a.top_k[row] : 0;
    const float pp = a.top_p ? a.top_p[row] : 1.0f, mp = a.min_p ? a.min_p[row] : 0.0f;
    const bool one = hard || mp > 1.0f;            // the first token alone
    k = one ? 1 : kk > 0 && kk < a.n ? kk : a.n;
    p = !one && pp < 1.0f ? (pp > 0.0f ? (double)pp : 0.0) : 1.0;
    min_p = !one && mp > 0.0f ? (double)mp : 0.0;
  }
  // bin of a logit above -Inf: never falls as x rises
  __device__ __forceinline__ int bin(float x) const {
    return (int)floorf(fminf(fmaxf(x * bins, -1e9f), 1e9f));
  }
};

// Sums over the workgroup's threads.
template <int T, class V>
__device__ __forceinline__ V sm_scan(V v, V* s_w, V* before) {   // *before: of the threads ahead
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  V in = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const V up = __shfl_up(in, o);
    if (lane >= o) in += up;
  }
  const V ahead = __shfl_up(in, 1);
  __syncthreads();
  if (lane == 63) s_w[w] = in;
  __syncthreads();
  V tot = 0, pre = 0;
#pragma unroll
  for (int i = 0; i < T / 64; ++i) {
    if (i == w) pre = tot;
    tot += s_w[i];
  }
  *before = lane > 0 ? pre + ahead : pre;
  return tot;
}
template <int T, class V>
__device__ __forceinline__ V sm_sum(V v, V* s_w) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
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

template <bool BF, int T>
struct SmKernel {
  using S = SmShape<T>;
  using L = SmLoad<BF, T>;

  // The workgroup's LDS; the row's last one uses the space of the histogram and more for its own.
  struct Shared {
    union {
      unsigned long long hist[kSmBins];
      struct {
        union {
          struct {
            double w[kSmCand];                     // candidates in column order
            double sorted[kSmCand];
          };
          uint64_t raw[kSmLists];                  // the lists, before
        };
        uint32_t key[kSmCand], col[kSmCand];
      } cand;
      unsigned long long sorting[kSmSort];         // the cut's bin: order, then the column's complement
      struct {
        unsigned long long mass[256];
        uint32_t cnt[256];
      } sort;
    };
    double wd[T / 64];
    unsigned long long wu[T / 64];
    float wf[T / 64];
    // the parts
    double scale[kSmParts], total[kSmParts];
    unsigned long long mass[kSmParts];             // of what is kept, in 2^-42
    uint32_t ties[kSmParts];
    float top[kSmParts];
    int shift[kSmParts], bound[kSmParts], list[kSmParts + 1], live[kSmParts];
    int bad, last, n, found;
    int at[4];
    double val[4];
    uint32_t cnt0, key0;
  };

  const SampleArgs& a;
  Shared& s;
  const int tid;
  const int64_t row;
  const uint8_t* const y;
  const int parts;
  const SmRow r;
  double M = 0.0;                                  // the row's largest logit
  uint32_t top = 0;                                // its order

  __device__ __forceinline__ double weight(float x) const { return sm_exp2(((double)x - M) * r.c); }
  __device__ __forceinline__ unsigned long long fine(double w) const { return (unsigned long long)(w * kSmFine + 0.5); }
  __device__ __forceinline__ bool passes(double w, uint32_t key) const { return w >= r.min_p || key == top; }

  __device__ __forceinline__ void put(int64_t token, double logp, int64_t kept) const {
    if (a.token) a.token[row] = (int32_t)token;
    if (a.logp) a.logp[row] = (float)logp;
    if (a.kept) a.kept[row] = (int32_t)kept;
  }

  // A part: its record into rec.
  __device__ __forceinline__ void part(int p, float temp, uint64_t* rec) {
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
      const double t = live ? ((double)x[e] - (double)mx) * r.c : -1e4;
      const float tf = (float)(t > -200.0 ? t : -200.0);
      if (masses) {
        double w;
        if (__ballot(t > -24.0)) {
          w = sm_exp2(t);
        } else {
          const double n = __builtin_rint(t > -1000.0 ? t : -1000.0);
          w = __builtin_ldexp((double)__builtin_amdgcn_exp2f((float)((t > -1000.0 ? t : -1000.0) - n)), (int)n);
        }
        tot += live ? w : 0.0;
      }
      rel[e] = kSmBins;
      if (cuts && live) {
        const int d = big - r.bin(x[e]);
        rel[e] = d < kSmBins ? d : kSmBins - 1;
        atomicAdd(&s.hist[rel[e]], 1ull << 48 | (uint32_t)(__builtin_amdgcn_exp2f(tf) * 1073741824.0f + 0.5f));
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
      constexpr int kBpt = kSmBins / T;
      int mine = 0;
#pragma unroll
      for (int i = 0; i < kBpt; ++i) {
        const unsigned long long h = s.hist[tid * kBpt + i];
        mine += (int)(h >> 48);
        sm_store(rec + S::kHead + S::kList + tid * kBpt + i, h);
      }
      int before;
      sm_scan<T>(mine, reinterpret_cast<int*>(s.wf), &before);
      int fit = 0;
#pragma unroll
      for (int i = 0; i < kBpt; ++i) {
        before += (int)(s.hist[tid * kBpt + i] >> 48);
        fit += before <= S::kList ? 1 : 0;
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
          if (rel[e] <= bound) sm_store(rec + S::kHead + at++, (uint64_t)sm_order(x[e]) << 32 | (uint32_t)(c0 + L::column(e, tid)));
        }
        base += (int)(all >> (16 * v) & 0xFFFFu);
      }
      listed = base;
    }
    if (tid == 0) {
      sm_store(rec, (uint64_t)__float_as_uint(mx) << 32 | (uint32_t)s.bad);
      sm_store(rec + 1, (uint64_t)(uint32_t)big << 32 | (uint32_t)(bound + 1));
      sm_store(rec + 2, (uint64_t)(uint32_t)live << 32 | (uint32_t)listed);
      sm_store(rec + 3, (uint64_t)__double_as_longlong(tot));
    }
  }

  // The token, where `cut` is known and s.mass holds the kept mass of every part (in 2^-42): the part, then in it.
  __device__ __forceinline__ void draw(SmCut cut, int64_t kept) {
    unsigned long long sum = 0;
    for (int p = 0; p < parts; ++p) sum += s.mass[p];
    const float u = a.u[row];
    unsigned long long want = u > 0.0f ? u < 1.0f ? (unsigned long long)((double)u * (double)sum) : sum - 1 : 0;
    if (want >= sum) want = sum - 1;
    unsigned long long left = want;
    int p = 0;
    while (p < parts - 1 && left >= s.mass[p]) left -= s.mass[p++];
    const int64_t c0 = (int64_t)p * S::kPart;
    float x[kSmElems];
    L::load(y, c0, a.n, tid, x);
    unsigned long long m[kSmElems], before = 0, sofar = 0;
    uint32_t in = 0;
    if (tid == 0) s.found = -1;
#pragma unroll
    for (int v = 0; v < L::kLoads; ++v) {
      unsigned long long mine = 0;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int e = v * L::kPer + i;
        const uint32_t key = sm_order(x[e]);
        m[e] = 0;
        if (key > kSmMasked && cut.in(key, (uint32_t)(c0 + L::column(e, tid)))) {
          const double w = weight(x[e]);
          if (passes(w, key)) {
            m[e] = fine(w);
            in |= 1u << e;
          }
        }
        mine += m[e];
      }
      const unsigned long long tot = sm_scan<T>(mine, s.wu, &before);
      before += sofar;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int e = v * L::kPer + i;
        if (before <= left && left < before + m[e]) {
          s.found = (int)(c0 + L::column(e, tid));
          s.val[0] = ((double)x[e] - M) * r.c;
        }
        // (the part's mass and its weights' may differ by a rounding: then the last one)
        before += m[e];
      }
      sofar += tot;
    }
    __syncthreads();
    if (s.found < 0) {
#pragma unroll
      for (int e = 0; e < kSmElems; ++e)
        if (in >> e & 1u) atomicMax(&s.found, (int)(c0 + L::column(e, tid)));
      __syncthreads();
      const int f = s.found;
#pragma unroll
      for (int e = 0; e < kSmElems; ++e)
        if ((int)(c0 + L::column(e, tid)) == f) s.val[0] = ((double)x[e] - M) * r.c;
      __syncthreads();
    }
    if (tid == 0) put(s.found, 0.6931471805599453 * (s.val[0] - log2((double)sum / kSmFine)), kept);
  }

  // Every logit of the row, a part at a time: f(x, key, column, part).
  template <class F, class G>
  __device__ __forceinline__ void each(const F& f, const G& end) {
    for (int p = 0; p < parts; ++p) {
      const int64_t c0 = (int64_t)p * S::kPart;
      float x[kSmElems];
      L::load(y, c0, a.n, tid, x);
#pragma unroll
      for (int e = 0; e < kSmElems; ++e)
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

  // The first token in order at which `want` tokens (by_mass: that mass, in 2^-42) have come, the last one there
  // is where they never do, by 8 bits of the order at a time; *mass: of the tokens up to and with it.
  __device__ SmCut radix(unsigned long long want, bool by_mass, SmCut within, unsigned long long* mass) {
    uint32_t key = 0, mask = 0;
    unsigned long long had_n = 0, had_m = 0, ties = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      __syncthreads();
      for (int b = tid; b < 256; b += T) {
        s.sort.cnt[b] = 0;
        s.sort.mass[b] = 0;
      }
      __syncthreads();
      each([&](float x, uint32_t k, uint32_t col) {
        if ((k & mask) != key || !within.in(k, col)) return;
        atomicAdd(&s.sort.cnt[k >> shift & 255u], 1u);
        atomicAdd(&s.sort.mass[k >> shift & 255u], fine(weight(x)));
      }, [](int) {});
      __syncthreads();
      int bin = 0;
      unsigned long long n = had_n, m = had_m;
      for (int b = 255; b >= 0; --b) {               // (all threads alike)
        const uint32_t c = s.sort.cnt[b];
        if (c == 0) continue;
        bin = b;
        had_n = n;
        had_m = m;
        n += c;
        m += s.sort.mass[b];
        if ((by_mass ? m : n) >= want) break;
      }
      ties = s.sort.cnt[bin];
      key |= (uint32_t)bin << shift;
      mask |= 255u << shift;
    }
    // of the equal ones, as many as it takes: the column of the last of them
    const unsigned long long one = fine(weight(sm_value(key)));
    unsigned long long need = 1;
    const unsigned long long had = by_mass ? had_m : had_n, step = by_mass ? one : 1;
    if (want > had && step > 0) need = (want - had + step - 1) / step;
    if (need > ties) need = ties;
    *mass = had_m + need * one;
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
    float x[kSmElems];
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

  // The cuts by k and p over the row itself, and the end.
  __device__ __forceinline__ void whole_row() {
    const SmCut all = {kSmMasked + 1, 0xFFFFFFFFu};
    SmCut cut = all;
    unsigned long long mass = 0;
    if (r.k < a.n) cut = radix((unsigned long long)r.k, false, all, &mass);
    if (r.p < 1.0) {
      if (!(r.k < a.n)) {
        unsigned long long mine = 0;
        each([&](float x, uint32_t, uint32_t) { mine += fine(weight(x)); }, [](int) {});
        mass = sm_sum<T>(mine, s.wu);
      }
      unsigned long long up_to;
      cut = radix((unsigned long long)ceil(r.p * (double)mass), true, cut, &up_to);
    }
    const int64_t kept = part_masses(cut);
    draw(cut, kept);
  }

  // The row, from its parts' records.
  __device__ __forceinline__ void join(uint64_t* rec0, SmPlanned* plan) {
    const bool cuts = r.k < a.n || r.p < 1.0 || r.min_p > 0.0;
    const Rsrc recs = make_rsrc(rec0, (uint32_t)(parts * S::kRec * 8));
    if (tid == 0) plan->state = 0;
    __syncthreads();
    if (tid < parts) {
      const int at = tid * S::kRec;
      const uint64_t h0 = sm_load(recs, at), h1 = sm_load(recs, at + 1), h2 = sm_load(recs, at + 2), h3 = sm_load(recs, at + 3);
      s.top[tid] = __uint_as_float((uint32_t)(h0 >> 32));
      s.ties[tid] = (uint32_t)h0;                  // bad
      s.shift[tid] = (int)(uint32_t)(h1 >> 32);
      s.bound[tid] = (int)(uint32_t)h1 - 1;
      s.list[tid + 1] = (int)(uint32_t)h2;
      s.live[tid] = (int)(h2 >> 32);
      s.total[tid] = __longlong_as_double((long long)h3);
    }
    __syncthreads();
    bool bad = false;
    float mx = -INFINITY;
    int big = -1000000000;
    for (int p = 0; p < parts; ++p) {
      bad |= s.ties[p] != 0;
      mx = fmaxf(mx, s.top[p]);
      big = s.shift[p] > big ? s.shift[p] : big;
    }
    if (bad || mx == -INFINITY) {
      if (tid == 0) put(-1, bad ? (double)__uint_as_float(0x7FC00000u) : -(double)INFINITY, 0);
      return;
    }
    M = (double)mx;
    top = sm_order(mx);
    __syncthreads();
    if (tid < parts) {
      s.scale[tid] = s.top[tid] > -INFINITY ? sm_exp2(((double)s.top[tid] - M) * r.c) : 0.0;
      s.shift[tid] = big - s.shift[tid];
      s.mass[tid] = fine(s.total[tid] * s.scale[tid]);
    }
    if (tid == 0) {
      s.list[0] = 0;
      for (int p = 0; p < parts; ++p) s.list[p + 1] += s.list[p];
    }
    __syncthreads();
    if (!cuts) {
      int64_t live = 0;
      for (int p = 0; p < parts; ++p) live += s.live[p];
      draw({kSmMasked + 1, 0xFFFFFFFFu}, live);
      return;
    }
    double W = 0.0;                                // (top-k off: the row's mass)
    for (int p = 0; p < parts; ++p) W += s.total[p] * s.scale[p];

    // the row's histogram, a run of bins a thread, and how far down what is kept can reach
    constexpr int kBpt = kSmBins / T;
    int cnt[kBpt];
    double ms[kBpt];
    int cs = 0;
    double md = 0.0;
#pragma unroll
    for (int i = 0; i < kBpt; ++i) {
      cnt[i] = 0;
      ms[i] = 0.0;
    }
    constexpr int kAhead = 8;                      // parts in flight
    for (int p0 = 0; p0 < parts; p0 += kAhead) {
      uint64_t v[kAhead][kBpt];
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        const int p = p0 + z < parts ? p0 + z : parts - 1;
        const int h = p * S::kRec + S::kHead + S::kList, sh = s.shift[p];
#pragma unroll
        for (int i = 0; i < kBpt; ++i) {
          // (the last bin takes what lies below in its part, too)
          const int b = tid * kBpt + i - sh;
          v[z][i] = sm_load(recs, p0 + z < parts && tid * kBpt + i < kSmBins - 1 && b >= 0 ? h + b : (1 << 28) - 1);
        }
      }
#pragma unroll
      for (int z = 0; z < kAhead; ++z) {
        const double sc = s.scale[p0 + z < parts ? p0 + z : parts - 1] * (1.0 / 1073741824.0);
#pragma unroll
        for (int i = 0; i < kBpt; ++i) {
          cnt[i] += (int)(v[z][i] >> 48);
          ms[i] += sc * (double)(v[z][i] & 0xFFFFFFFFFFFFull);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBpt; ++i) {
      cs += cnt[i];
      md += ms[i];
    }
    int c_before;
    double m_before;
    sm_scan<T>(cs, reinterpret_cast<int*>(s.wf), &c_before);
    sm_scan<T>(md, s.wd, &m_before);
    // the first bin with k tokens, or with p of the mass
    int kb = kSmBins - 1;
    if (tid == 0) {
      s.at[0] = kSmBins - 1;
      s.at[1] = kSmBins - 1;
    }
    __syncthreads();
    int c = c_before;
    if (r.k < a.n) {
#pragma unroll
      for (int i = 0; i < kBpt; ++i) {
        if (c < r.k && c + cnt[i] >= r.k && tid * kBpt + i < kSmBins - 1) s.at[0] = tid * kBpt + i;
        c += cnt[i];
      }
      __syncthreads();
      kb = s.at[0];
    }
    int need = kb, pb = kSmBins - 1;
    if (r.p < 1.0 && !(r.k < a.n)) {
      const double want = r.p * W * (1.0 + 1e-5);
      double m = m_before;
#pragma unroll
      for (int i = 0; i < kBpt; ++i) {
        if (m < want && m + ms[i] >= want && tid * kBpt + i < kSmBins - 1) s.at[1] = tid * kBpt + i;
        m += ms[i];
      }
      __syncthreads();
      pb = want > 0.0 ? s.at[1] : 0;
      need = pb < need ? pb : need;
    }
    // (top-k and top-p together: the mass of all k is asked for)
    bool by_min = false;
    if (r.min_p > 0.0 && !(r.k < a.n && r.p < 1.0)) {
      const double f = r.min_p < 1.0 ? -log2(r.min_p) * kSmPerOctave + 3.0 : 3.0;
      if (f < (double)need) {
        need = (int)f;
        by_min = true;
      }
    }
    // whether the lists have all of that
    bool lists = need < kSmBins - 1;
    for (int p = 0; p < parts; ++p) lists = lists && need - s.shift[p] <= s.bound[p];
    if (need >= kSmBins - 1) {
      lists = true;                                // (all of every part)
      for (int p = 0; p < parts; ++p) lists = lists && s.bound[p] == kSmBins - 1;
    }
    if (lists && from_lists(recs, need, by_min, big, W)) return;
    if (tid != 0) return;
    const int bin = r.k < a.n ? kb : r.p < 1.0 ? pb : kSmAll;
    plan->state = r.k < a.n && r.p < 1.0 ? 2 : bin == kSmBins - 1 ? 2 : 1;
    plan->bin = bin;
    plan->big = big;
    plan->M = mx;
    plan->W = W;
  }

  // The second kernel's part of a row with a plan: masses and counts of what lies above the cut's bin (also of
  // those that min-p leaves), and the bin's logits, into the record.
  __device__ __forceinline__ void cut_part(int p, const SmPlanned& plan, uint64_t* rec) {
    const int64_t c0 = (int64_t)p * S::kPart;
    float x[kSmElems];
    L::load(y, c0, a.n, tid, x);
    if (tid == 0) s.n = 0;
    __syncthreads();
    double mass = 0.0;
    unsigned long long left = 0, counts = 0;       // counts: above, and of those the ones min-p leaves << 32
#pragma unroll
    for (int e = 0; e < kSmElems; ++e) {
      const int d = x[e] > -INFINITY ? plan.big - r.bin(x[e]) : 0x7FFFFFFF;
      if (d < plan.bin) {
        const double w = weight(x[e]);
        mass += w;
        const bool in = passes(w, sm_order(x[e]));
        left += in ? fine(w) : 0;
        counts += in ? 1ull << 32 | 1 : 1;
      }
      if (d == plan.bin) {
        const int at = atomicAdd(&s.n, 1);
        if (at < kSmBins) sm_store(rec + S::kHead + S::kList + at, (uint64_t)sm_order(x[e]) << 32 | (uint32_t)~(uint32_t)(c0 + L::column(e, tid)));
      }
    }
    mass = sm_sum<T>(mass, s.wd);
    left = sm_sum<T>(left, s.wu);
    counts = sm_sum<T>(counts, s.wu);
    if (tid == 0) {
      sm_store(rec, (uint64_t)__double_as_longlong(mass));
      sm_store(rec + 1, left);
      sm_store(rec + 2, counts);
      sm_store(rec + 3, (uint64_t)s.n);
    }
  }

  // And the row's last one: the bin sorted and cut, the token drawn.
  __device__ __forceinline__ void cut_join(const SmPlanned& plan, uint64_t* rec0) {
    const Rsrc recs = make_rsrc(rec0, (uint32_t)(parts * S::kRec * 8));
    __syncthreads();
    if (tid < parts) {
      const int at = tid * S::kRec;
      s.total[tid] = __longlong_as_double((long long)sm_load(recs, at));
      s.mass[tid] = sm_load(recs, at + 1);
      const uint64_t c = sm_load(recs, at + 2);
      s.ties[tid] = (uint32_t)c;
      s.live[tid] = (int)(c >> 32);
      s.list[tid + 1] = (int)sm_load(recs, at + 3);
    }
    if (tid == 0) s.list[0] = 0;
    __syncthreads();
    double above = 0.0;
    int64_t count = 0, kept = 0;
    bool fits = true;
    int n = 0;
    for (int p = 0; p < parts; ++p) {
      above += s.total[p];
      count += s.ties[p];
      kept += s.live[p];
      fits = fits && s.list[p + 1] <= kSmBins;
      n += s.list[p + 1];
    }
    if (!fits || n > kSmSort) {
      whole_row();
      return;
    }
    SmCut cut = {kSmMasked + 1, 0xFFFFFFFFu};
    if (plan.bin < kSmBins) {
      __syncthreads();
      if (tid == 0)
        for (int p = 0; p < parts; ++p) s.list[p + 1] += s.list[p];
      __syncthreads();
      int size = 64;                               // the sort's, a power of two
      while (size < n) size <<= 1;
      for (int i = tid; i < size; i += T) {
        unsigned long long v = 0;
        if (i < n) {
          const int p = part_of(i);
          v = sm_load(recs, p * S::kRec + S::kHead + S::kList + (i - s.list[p]));
        }
        s.sorting[i] = v;
      }
      // descending, by runs of twice the length each round
      for (int len = 2; len <= size; len <<= 1)
        for (int step = len >> 1; step > 0; step >>= 1) {
          __syncthreads();
          for (int z = tid; z < size / 2; z += T) {
            const int i = (z / step * 2) * step + z % step, j = i + step;
            const unsigned long long u = s.sorting[i], v = s.sorting[j];
            if ((u < v) == ((i & len) == 0)) {
              s.sorting[i] = v;
              s.sorting[j] = u;
            }
          }
        }
      __syncthreads();
      // the last one kept of them
      constexpr int kMine = kSmSort / T;
      double w[kMine], mine = 0.0, before;
#pragma unroll
      for (int q = 0; q < kMine; ++q) {
        const int i = tid * kMine + q;
        w[q] = i < n ? weight(sm_value((uint32_t)(s.sorting[i] >> 32))) : 0.0;
        mine += w[q];
      }
      const double all = sm_scan<T>(mine, s.wd, &before);
      int upto;                                    // how many are kept
      if (r.k < a.n) {
        upto = (int)(r.k - count);
        if (r.k <= count || r.k > count + n) upto = 0;
      } else {
        const double want = r.p * plan.W - above;
        int short_of = 0;
#pragma unroll
        for (int q = 0; q < kMine; ++q) {
          before += w[q];
          short_of += tid * kMine + q < n && before < want ? 1 : 0;
        }
        upto = sm_sum<T>(short_of, reinterpret_cast<int*>(s.wf)) + 1;
        if ((want <= 0.0 && count > 0) || upto > n || all < want) upto = 0;
      }
      if (upto == 0) {                             // (the histogram's masses were off by a bin)
        whole_row();
        return;
      }
      const unsigned long long last = s.sorting[upto - 1];
      cut = {(uint32_t)(last >> 32), ~(uint32_t)last};
      unsigned long long more = 0;
      for (int i = tid; i < upto; i += T) {
        const unsigned long long v = s.sorting[i];
        const double wi = weight(sm_value((uint32_t)(v >> 32)));
        if (passes(wi, (uint32_t)(v >> 32))) {
          atomicAdd(&s.mass[~(uint32_t)v / (uint32_t)S::kPart], fine(wi));
          ++more;
        }
      }
      kept += (int64_t)sm_sum<T>(more, s.wu);
    }
    __syncthreads();
    draw(cut, kept);
  }

  // the part that entry i of the lists is in
  __device__ __forceinline__ int part_of(int i) const {
    int lo = 0, hi = parts;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.list[mid] <= i) lo = mid;
      else hi = mid;
    }
    return lo;
  }

  // Cuts and draws from the lists' logits down to bin `need`; false if they turn out not to reach the cut.
  __device__ __forceinline__ bool from_lists(Rsrc recs, int need, bool by_min, int big, double W) {
    __syncthreads();
    const int all = s.list[parts];
    if (all > kSmLists) return false;
#pragma unroll 4
    for (int i = tid; i < all; i += T) {
      const int p = part_of(i);
      s.cand.raw[i] = sm_load(recs, p * S::kRec + S::kHead + (i - s.list[p]));
    }
    __syncthreads();
    // a run of the entries a thread, so that one sum gives their places
    const int run = (all + T - 1) / T, i1 = (tid + 1) * run < all ? (tid + 1) * run : all;
    const auto in = [&](int i) {
      return need >= kSmBins - 1 || big - r.bin(sm_value((uint32_t)(s.cand.raw[i] >> 32))) <= need;
    };
    int mine_n = 0, at0;
#pragma unroll 1
    for (int i = tid * run; i < i1; ++i) mine_n += in(i) ? 1 : 0;
    const int n = sm_scan<T>(mine_n, reinterpret_cast<int*>(s.wf), &at0);
    if (n > kSmCand) return false;
#pragma unroll 1
    for (int i = tid * run; i < i1; ++i)
      if (in(i)) {
        s.cand.key[at0] = (uint32_t)(s.cand.raw[i] >> 32);
        s.cand.col[at0++] = (uint32_t)s.cand.raw[i];
      }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < n; i += T) s.cand.w[i] = weight(sm_value(s.cand.key[i]));
    __syncthreads();
    // ranks in the tokens' order
    constexpr int kMine = kSmCand / T;
    int rank[kMine];
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int i = q * T + tid;
      rank[q] = kSmCand;
      if (i >= n) continue;
      const uint32_t key = s.cand.key[i];
      int k = 0;
      for (int j = 0; j < n; ++j) {
        const uint32_t o = s.cand.key[j];
        k += o > key || (o == key && j < i) ? 1 : 0;
      }
      rank[q] = k;
      s.cand.sorted[k] = s.cand.w[i];
    }
    __syncthreads();
    // masses in that order (a run of ranks a thread)
    double own[kMine], mine = 0.0, before;
    const int r0 = tid * kMine, kk = r.k < n ? (int)r.k : n;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      own[q] = r0 + q < kk ? s.cand.sorted[r0 + q] : 0.0;
      mine += own[q];
    }
    const double listed = sm_scan<T>(mine, s.wd, &before);
    const double mass = r.k < a.n ? listed : W, want = r.p * mass;
    const bool ends = s.list[parts] == n && need >= kSmBins - 1;   // (nothing else is left)
    // is the end of what is kept among them?
    if (!ends && !by_min && !(r.k < a.n ? n >= r.k : r.p < 1.0 && listed >= want)) return false;
    int keep = 0;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int i = r0 + q;
      if (i < kk && (i == 0 || ((r.p >= 1.0 || before < want) && own[q] >= r.min_p))) ++keep;
      before += own[q];
    }
    keep = sm_sum<T>(keep, reinterpret_cast<int*>(s.wf));
    // in column order
    mine = 0.0;
    double mw[kMine];
    int at[kMine];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      const int i = q * T + tid;
      if (i < n && rank[q] >= keep) s.cand.w[i] = 0.0;
    }
    if (tid == 0) s.found = -1;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      at[q] = r0 + q;
      mw[q] = at[q] < n ? s.cand.w[at[q]] : 0.0;
      mine += mw[q];
    }
    const double sum = sm_scan<T>(mine, s.wd, &before);
    const float u = a.u[row];
    const double target = u > 0.0f ? u < 1.0f ? (double)u * sum : sum : 0.0;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
      // (the border that the next one starts from is the one this one ends at)
      const double end = before + mw[q];
      if (mw[q] > 0.0 && before <= target && target < end) s.found = at[q];
      before = end;
    }
    __syncthreads();
    if (s.found < 0) {                             // u of 1 or more, or a rounding at the end
#pragma unroll
      for (int q = 0; q < kMine; ++q)
        if (mw[q] > 0.0) atomicMax(&s.found, at[q]);
      __syncthreads();
    }
    if (tid == 0) {
      const int f = s.found;
      const double d = ((double)sm_value(s.cand.key[f]) - M) * r.c;
      put(s.cand.col[f], r.hard ? 0.0 : 0.6931471805599453 * (d - log2(sum)), keep);
    }
    return true;
  }
};

// Whether this is the row's last workgroup to get here, all stores of the others to be seen.
template <class Shared>
__device__ __forceinline__ bool sm_last(uint32_t* count, int parts, Shared& s) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (parts == 1) return true;
  if (threadIdx.x == 0) {
    const uint32_t old = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s.last = old == (uint32_t)parts - 1 ? 1 : 0;
    if (s.last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  const bool last = s.last != 0;
  asm volatile("" ::: "memory");
  return last;
}

template <bool BF, int T>
__global__ __launch_bounds__(T) void k_sample(SampleArgs a, int parts, uint32_t* count, SmPlanned* plans, uint64_t* recs) {
  using K = SmKernel<BF, T>;
  __shared__ typename K::Shared s;
  const int64_t row = blockIdx.x / parts;
  const int p = (int)(blockIdx.x - row * parts);
  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  uint64_t* const rec0 = recs + row * parts * SmShape<T>::kRec;
  K k = {a, s, (int)threadIdx.x, row, static_cast<const uint8_t*>(a.y) + row * a.ldy * (BF ? 2 : 4), parts, SmRow(a, row, temp)};
  k.part(p, temp, rec0 + (int64_t)p * SmShape<T>::kRec);
  if (sm_last(&count[row * kSmCountStep], parts, s)) k.join(rec0, plans + row);
}

template <bool BF, int T>
__global__ __launch_bounds__(T) void k_sample_cut(SampleArgs a, int parts, uint32_t* count, const SmPlanned* plans, uint64_t* recs) {
  using K = SmKernel<BF, T>;
  __shared__ typename K::Shared s;
  const int64_t row = blockIdx.x / parts;
  const SmPlanned plan = plans[row];
  if (plan.state == 0) return;
  const int p = (int)(blockIdx.x - row * parts);
  if (plan.state == 2 && p > 0) return;
  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  uint64_t* const rec0 = recs + row * parts * SmShape<T>::kRec;
  K k = {a, s, (int)threadIdx.x, row, static_cast<const uint8_t*>(a.y) + row * a.ldy * (BF ? 2 : 4), parts, SmRow(a, row, temp)};
  k.M = (double)plan.M;
  k.top = sm_order(plan.M);
  if (plan.state == 2) {
    k.whole_row();
    return;
  }
  k.cut_part(p, plan, rec0 + (int64_t)p * SmShape<T>::kRec);
  if (sm_last(&count[row * kSmCountStep], parts, s)) k.cut_join(plan, rec0);
}

// Parts of 4096 logits while they are few for the chip (a row's latency), else of 16384 (records are then a
// smaller share of what is read).
struct SmPlan {
  bool wide;              // 1024 threads
  int parts;
  int64_t rec;            // bytes
  int64_t rows;           // of a launch
};
static SmPlan sm_plan(const DevInfo& di, int64_t m, int64_t n) {
  SmPlan p;
  const int64_t few = (n + SmShape<256>::kPart - 1) / SmShape<256>::kPart;
  p.wide = few > kSmParts || m * few > (int64_t)di.cus * 4;
  const int64_t size = p.wide ? SmShape<1024>::kPart : SmShape<256>::kPart;
  p.parts = (int)((n + size - 1) / size);
  p.rec = (p.wide ? SmShape<1024>::kRec : SmShape<256>::kRec) * 8;
  p.rows = (int64_t(64) << 20) / (p.parts * p.rec);
  p.rows = p.rows < 1 ? 1 : p.rows > kSmRows ? kSmRows : p.rows;
  p.rows = p.rows < m ? p.rows : m;
  return p;
}

uint64_t sample_scratch(const DevInfo& di, int64_t m, int64_t n, bool, uint64_t* zero) {
  const SmPlan p = sm_plan(di, m, n);
  *zero = (uint64_t)kSmRows * kSmCountStep * sizeof(uint32_t);
  return *zero + (uint64_t)(p.rows * (p.parts * p.rec + (int64_t)sizeof(SmPlanned)));
}

template <bool BF, int T>
static void sm_go(dim3 grid, hipStream_t s, const SampleArgs& a, int parts, uint32_t* count, SmPlanned* plans, uint64_t* recs,
                  bool cuts) {
  hipLaunchKernelGGL((k_sample<BF, T>), grid, dim3(T), 0, s, a, parts, count, plans, recs);
  if (cuts) hipLaunchKernelGGL((k_sample_cut<BF, T>), grid, dim3(T), 0, s, a, parts, count, plans, recs);
}

hipError_t launch_sample(const SampleArgs& a0, bool bf, void* scratch, hipStream_t s) {
  DevInfo di;
  const hipError_t err = dev_info(&di);
  if (err != hipSuccess) return err;
  const SmPlan p = sm_plan(di, a0.m, a0.n);
  if (p.parts > kSmParts) return hipErrorInvalidValue;
  SampleArgs a = a0;
  uint32_t* const count = static_cast<uint32_t*>(scratch);
  SmPlanned* const plans = reinterpret_cast<SmPlanned*>(count + kSmRows * kSmCountStep);
  uint64_t* const recs = reinterpret_cast<uint64_t*>(plans + p.rows);
  const bool cuts = a.top_k || a.top_p || a.min_p;           // (without: nothing for the second kernel)
  for (int64_t r0 = 0; r0 < a0.m; r0 += p.rows) {
    a.m = a0.m - r0 < p.rows ? a0.m - r0 : p.rows;
    const dim3 grid((unsigned)(a.m * p.parts));
    if (p.wide && bf) sm_go<true, 1024>(grid, s, a, p.parts, count, plans, recs, cuts);
    else if (p.wide) sm_go<false, 1024>(grid, s, a, p.parts, count, plans, recs, cuts);
    else if (bf) sm_go<true, 256>(grid, s, a, p.parts, count, plans, recs, cuts);
    else sm_go<false, 256>(grid, s, a, p.parts, count, plans, recs, cuts);
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
