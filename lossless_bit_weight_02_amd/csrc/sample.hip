// A token for each row of logits from temperature, top-k, top-p, min-p and a given random number.
//
// With M the row's largest logit and w = e^((x - M) / T), all three filters keep a prefix of the tokens'
// order (descending logit, equal ones by the lower column), so what is kept is known by its last
// token: the order of that logit (a 32-bit key) and, among the logits equal to it, a column.  The key
// comes from a histogram over 8 of its bits at a time, of counts and of masses; the column from a count
// of the equal logits in column order.  The token itself is the first kept one in column order at
// which the mass passes u * (mass of all kept): a sum over tiles of columns, then over the tile's.
//
// A weight is e^(..) in double times 2^shift, rounded to an integer, 2^shift * n <= 2^62: masses are
// integers, so no sum depends on the order of its terms, and a border between two tokens is off
// by about 2^-shift / 2 a term (152064 columns: 2^-45, some 1e-11 of the row's mass after all of
// them).  In float the borders' errors would add up to 1e-7 each, and the 152064 borders of a
// flat row would send one draw in a hundred to a neighbouring token.
#include "kv_device.hpp"

namespace w12 {

constexpr int kSmThreads = 1024;
constexpr uint32_t kSmMasked = 0x007FFFFFu;       // the order of -Inf

__device__ __forceinline__ uint32_t sm_order(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);    // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float sm_value(uint32_t ord) {
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}

template <bool BF>
__device__ __forceinline__ float sm_logit(const void* row, int64_t c) {
  if constexpr (BF) return bf16_to_float(static_cast<const uint16_t*>(row)[c]);
  else return static_cast<const float*>(row)[c];
}

// A row's weights.
struct SmRow {
  double M, inv;          // largest logit, 1 / temperature
  double unit;            // 2^shift
  double min_p;           // 0: off
  uint32_t top;           // the largest logit's order
  __device__ __forceinline__ double weight(float x) const {
    return x == (float)M ? 1.0 : exp(((double)x - M) * inv);
  }
  __device__ __forceinline__ uint64_t mass(double w) const { return (uint64_t)(w * unit + 0.5); }
};

// The workgroup's sum, and in *before what the threads before this one have; every thread gets both.
__device__ __forceinline__ uint64_t sm_scan(uint64_t v, uint64_t* s_w, uint64_t* before) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint64_t in = v;
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t up = __shfl_up((unsigned long long)in, o);
    if (lane >= o) in += up;
  }
  __syncthreads();
  if (lane == 63) s_w[w] = in;
  __syncthreads();
  uint64_t tot = 0, pre = 0;
  for (int i = 0; i < kSmThreads / 64; ++i) {
    if (i < w) pre += s_w[i];
    tot += s_w[i];
  }
  *before = pre + in - v;
  return tot;
}

// The last token kept, as its order and the number of logits equal to it that are kept.
struct SmCut {
  uint32_t key;
  uint64_t ties;
  uint64_t count;         // tokens of a higher order
  uint64_t mass;          // and their mass
};

// The first token in order at which `want` tokens (by_mass: that mass) have come, the last one there is
// where they never do; eligible are orders at or above `low`.
template <bool BF>
__device__ SmCut sm_cut(const void* y, int64_t n, const SmRow& r, uint32_t low, uint64_t want, bool by_mass,
                        uint32_t* s_cnt, unsigned long long* s_mass, uint64_t* s_out) {
  SmCut c = {0, 0, 0, 0};
  uint32_t mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) {
      s_cnt[threadIdx.x] = 0;
      s_mass[threadIdx.x] = 0;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kSmThreads) {
      const float x = sm_logit<BF>(y, i);
      const uint32_t o = sm_order(x);
      if (o < low || (o & mask) != c.key) continue;
      const uint32_t bin = o >> shift & 255u;
      atomicAdd(&s_cnt[bin], 1u);
      atomicAdd(&s_mass[bin], (unsigned long long)r.mass(r.weight(x)));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      uint64_t cnt = c.count, mass = c.mass;
      for (int bin = 255; bin >= 0; --bin) {
        if (s_cnt[bin] == 0) continue;
        s_out[0] = bin;
        s_out[1] = cnt;
        s_out[2] = mass;
        s_out[3] = s_cnt[bin];
        cnt += s_cnt[bin];
        mass += s_mass[bin];
        if ((by_mass ? mass : cnt) >= want) break;
      }
    }
    __syncthreads();
    c.key |= (uint32_t)s_out[0] << shift;
    c.count = s_out[1];
    c.mass = s_out[2];
    c.ties = s_out[3];
    mask |= 255u << shift;
  }
  // of the equal ones, as many as it takes
  const uint64_t each = by_mass ? r.mass(r.weight(sm_value(c.key))) : 1, had = by_mass ? c.mass : c.count;
  uint64_t need = 1;
  if (want > had && each > 0) need = (want - had + each - 1) / each;
  if (need < c.ties) c.ties = need;
  __syncthreads();
  return c;
}

template <bool BF>
__global__ __launch_bounds__(kSmThreads) void k_sample(SampleArgs a, int shift) {
  __shared__ uint32_t s_cnt[256];
  __shared__ unsigned long long s_mass[256];
  __shared__ uint64_t s_out[4];
  __shared__ uint64_t s_w[kSmThreads / 64];
  __shared__ float s_f[kSmThreads / 64];
  __shared__ int s_bad;
  __shared__ int64_t s_tok;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const uint8_t* const y = static_cast<const uint8_t*>(a.y) + row * a.ldy * (BF ? 2 : 4);
  const float temp = a.temperature ? a.temperature[row] : 1.0f;
  float top = -INFINITY;
  bool bad = temp != temp;
  for (int64_t i = tid; i < a.n; i += kSmThreads) {
    const float x = sm_logit<BF>(y, i);
    bad |= x != x || x == INFINITY;
    top = fmaxf(top, x);
  }
  if (tid == 0) s_bad = 0;
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if ((tid & 63) == 0) s_f[tid >> 6] = top;
  __syncthreads();
  if (bad) s_bad = 1;
  for (int i = 0; i < kSmThreads / 64; ++i) top = fmaxf(top, s_f[i]);
  __syncthreads();
  if (s_bad || top == -INFINITY) {
    if (tid == 0) {
      if (a.token) a.token[row] = -1;
      if (a.logp) a.logp[row] = s_bad ? __uint_as_float(0x7FC00000u) : -INFINITY;
      if (a.kept) a.kept[row] = 0;
    }
    return;
  }
  SmRow r;
  r.M = (double)top;
  r.unit = __longlong_as_double((long long)(1023 + shift) << 52);
  r.top = sm_order(top);
  const bool hard = temp <= 0.0f;
  r.inv = hard ? 0.0 : 1.0 / (double)temp;
  const float mp = a.min_p ? a.min_p[row] : 0.0f;
  r.min_p = mp > 0.0f ? (double)mp : 0.0;
  const int64_t k = hard ? 1 : a.top_k && a.top_k[row] > 0 ? a.top_k[row] : a.n;
  const float p = a.top_p ? a.top_p[row] : 1.0f;

  // the tokens that top-k and then top-p leave: orders above cut.key, and cut.ties equal ones
  SmCut cut = {kSmMasked + 1, ~0ull, 0, 0};
  uint64_t before;
  if (k < a.n) cut = sm_cut<BF>(y, a.n, r, kSmMasked + 1, (uint64_t)k, false, s_cnt, s_mass, s_out);
  if (p < 1.0f && !hard) {
    uint64_t mine = 0;
    uint64_t total;
    if (k < a.n) {
      total = cut.mass + cut.ties * r.mass(r.weight(sm_value(cut.key)));
    } else {
      for (int64_t i = tid; i < a.n; i += kSmThreads) {
        const float x = sm_logit<BF>(y, i);
        if (sm_order(x) > kSmMasked) mine += r.mass(r.weight(x));
      }
      total = sm_scan(mine, s_w, &before);
    }
    const uint64_t part = p > 0.0f ? (uint64_t)ceil((double)p * (double)total) : 0;
    const SmCut pc = sm_cut<BF>(y, a.n, r, cut.key, part, true, s_cnt, s_mass, s_out);
    if (pc.key > cut.key || (pc.key == cut.key && pc.ties < cut.ties)) cut = pc;
  }
  // what is kept, in column order: number and mass, then the token
  const auto pass = [&](bool pick, uint64_t want, uint64_t* count, uint64_t* mass) {
    uint64_t ties = 0, cnt = 0, sum = 0;
    for (int64_t c0 = 0; c0 < a.n; c0 += kSmThreads) {
      const int64_t i = c0 + tid;
      uint32_t o = 0;
      float x = -INFINITY;
      if (i < a.n) {
        x = sm_logit<BF>(y, i);
        o = sm_order(x);
      }
      const bool tie = o == cut.key;
      uint64_t ahead;
      const uint64_t found = sm_scan(tie ? 1 : 0, s_w, &ahead);
      bool in = o > cut.key || (tie && ties + ahead < cut.ties);
      const double w = in ? r.weight(x) : 0.0;
      in = in && (w >= r.min_p || o == r.top);
      ties += found;
      const uint64_t v = in ? r.mass(w) : 0;
      uint64_t pre;
      cnt += sm_scan(in ? 1 : 0, s_w, &pre);
      const uint64_t got = sm_scan(v, s_w, &pre);
      if (pick && sum + pre <= want && want < sum + pre + v) s_tok = i;
      sum += got;
    }
    *count = cnt;
    *mass = sum;
  };
  if (r.min_p > 1.0) cut = {r.top, 1, 0, 0};       // the first token alone
  uint64_t cnt, sum, c2, m2;
  pass(false, 0, &cnt, &sum);
  const float u = a.u[row];
  uint64_t want = u > 0.0f ? u < 1.0f ? (uint64_t)((double)u * (double)sum) : sum - 1 : 0;
  if (want >= sum) want = sum - 1;
  pass(true, want, &c2, &m2);
  __syncthreads();
  if (tid == 0) {
    const int64_t t = s_tok;
    if (a.token) a.token[row] = (int32_t)t;
    if (a.logp) a.logp[row] = hard ? 0.0f : (float)(((double)sm_logit<BF>(y, t) - r.M) * r.inv - log((double)sum / r.unit));
    if (a.kept) a.kept[row] = (int32_t)cnt;
  }
}

uint64_t sample_scratch(const DevInfo&, int64_t, int64_t, bool, uint64_t* zero) {
  *zero = 0;
  return 0;
}

hipError_t launch_sample(const SampleArgs& a0, bool bf, void*, hipStream_t s) {
  SampleArgs a = a0;
  int shift = 62;
  while (shift > 31 && ((int64_t)1 << (62 - shift)) < a.n) --shift;
  constexpr int64_t kRows = int64_t(1) << 21;                // a launch holds fewer than 2^32 work items
  for (int64_t r0 = 0; r0 < a0.m; r0 += kRows) {
    a.m = a0.m - r0 < kRows ? a0.m - r0 : kRows;
    const dim3 grid((unsigned)a.m), block(kSmThreads);
    if (bf) hipLaunchKernelGGL(k_sample<true>, grid, block, 0, s, a, shift);
    else hipLaunchKernelGGL(k_sample<false>, grid, block, 0, s, a, shift);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.y = static_cast<const uint8_t*>(a.y) + kRows * a.ldy * (bf ? 2 : 4);
    if (a.temperature) a.temperature += kRows;
    if (a.top_k) a.top_k += kRows;
    if (a.top_p) a.top_p += kRows;
    if (a.min_p) a.min_p += kRows;
    a.u += kRows;
    if (a.token) a.token += kRows;
    if (a.logp) a.logp += kRows;
    if (a.kept) a.kept += kRows;
  }
  return hipSuccess;
}

}  // namespace w12
