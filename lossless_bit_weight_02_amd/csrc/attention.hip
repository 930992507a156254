// Attention of a step's new tokens over the paged cache.
//
// One wave per row and head walks the places 64 at a time with a running maximum and sum.
#include "kv_device.hpp"

namespace w12 {

template <bool E4M3>
__device__ __forceinline__ float kv_value(const void* p, int64_t at) {
  if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(p)[at], 0);
  else return bf16_to_float(static_cast<const uint16_t*>(p)[at]);
}

template <bool E4M3>
__global__ __launch_bounds__(64) void k_attention(const uint16_t* __restrict__ q, int64_t ldq, int64_t m, int64_t hq,
                                                  KvArgs kv, BatchArgs b, float scale, uint16_t* __restrict__ y,
                                                  int64_t first) {
  __shared__ float s_q[256];
  const int lane = threadIdx.x;
  const int64_t row = first + blockIdx.x / hq, h = blockIdx.x % hq, hk = h / (hq / kv.heads);
  const int64_t s = find_seq(b, row);
  if (s < 0) return;
  const SeqRows sr = seq_rows(b, s, m);
  if (row >= sr.first + sr.count) return;
  const int dim = (int)kv.dim;
  for (int c = lane; c < dim; c += 64) s_q[c] = bf16_to_float(q[row * ldq + h * dim + c]);
  __syncthreads();
  const int64_t base = sr.len - sr.count, j = row - sr.first;
  const float f = scale * (kv.k_scale ? kv.k_scale[hk] : 1.0f);
  float big = -INFINITY, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t t0 = 0; t0 < sr.len; t0 += 64) {
    const int64_t t = t0 + lane, bit = t - base;
    bool sees = t < sr.len && (bit < 0 || (b.tree ? bit < 64 && (b.tree[row] >> (bit & 63) & 1) : bit <= j));
    const int64_t page = sees ? page_of(kv, b, s, t) : -1;
    sees = page >= 0;
    const int64_t at = sees ? page * kv.page_stride + hk * kv.head_stride + (t % kv.page) * kv.token_stride : 0;
    float x = -INFINITY;
    if (sees) {
      x = 0.0f;
      for (int c = 0; c < dim; ++c) x += s_q[c] * kv_value<E4M3>(kv.k, at + c);
      x *= f;
    }
    float top = x;
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float now = fmaxf(big, top), ref = now == -INFINITY ? 0.0f : now;
    const float p = sees ? expf(x - ref) : 0.0f;
    float tot = p;
    for (int o = 32; o > 0; o >>= 1) tot += __shfl_xor(tot, o);
    const float old = expf(big - ref);
    sum = sum * old + tot;
    big = now;
    for (int i = 0; i < 4; ++i) acc[i] *= old;
    for (int l = 0; l < 64; ++l) {
      const float w = __shfl(p, l);
      const int64_t va = __shfl(at, l);
      if (__shfl((int)sees, l))
        for (int i = 0; i * 64 < dim; ++i) acc[i] += w * kv_value<E4M3>(kv.v, va + i * 64 + lane);
    }
  }
  const float vs = kv.v_scale ? kv.v_scale[hk] : 1.0f;
  for (int i = 0; i * 64 < dim; ++i)
    y[(row * hq + h) * dim + i * 64 + lane] = float_to_bf16_rne(sum == 0.0f ? 0.0f : acc[i] / sum * vs);
}

uint64_t attention_scratch(const DevInfo&, int64_t, int64_t, const KvArgs&, const BatchArgs&, uint64_t* zero) {
  *zero = 0;
  return 0;
}

hipError_t launch_attention(const uint16_t* q, int64_t ldq, int64_t m, int64_t hq, const KvArgs& kv,
                            const BatchArgs& b, float scale, uint16_t* y, void*, hipStream_t s) {
  const int64_t rows = (int64_t(1) << 25) / hq;              // a launch holds fewer than 2^32 work items
  for (int64_t r0 = 0; r0 < m; r0 += rows) {
    const dim3 grid((unsigned)((m - r0 < rows ? m - r0 : rows) * hq));
    if (kv.e4m3) hipLaunchKernelGGL(k_attention<true>, grid, dim3(64), 0, s, q, ldq, m, hq, kv, b, scale, y, r0);
    else hipLaunchKernelGGL(k_attention<false>, grid, dim3(64), 0, s, q, ldq, m, hq, kv, b, scale, y, r0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace w12
