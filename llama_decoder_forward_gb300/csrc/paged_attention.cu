// paged_attention.cu - causal grouped-query attention of a chunk of new tokens
// over a paged cache.
//
// out[t, h] = sum_j softmax_j(scale q[t, h] . k[j]) v[j] over the positions
// j <= p, j > p - window, p = L + t.  One warp takes one query row and head and
// walks over its keys with a running maximum and sum; lane i holds the values
// at i * hd / 32 .. of q, k, v and the accumulator.
#include <cuda_fp8.h>
#include <math.h>

#include "paged.cuh"

namespace smol {
namespace {

template <int HD, bool FP8>
__device__ __forceinline__ void load_row(const uint8_t *base, long long slot, int lane, float scale,
                                         float (&f)[HD / 32]) {
  constexpr int E = HD / 32;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const long long i = slot * HD + lane * E + e;
    if constexpr (FP8)
      f[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(base[i], __NV_E4M3))) * scale;
    else
      f[e] = __bfloat162float(reinterpret_cast<const bf16 *>(base)[i]);
  }
}

template <int HD, bool FP8>
__global__ void __launch_bounds__(128) paged_rows_kernel(const PagedAttnParams p) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int b = static_cast<int>(item / (static_cast<long long>(p.c.T) * p.H));
  if (b >= p.c.B) return;
  const int rest = static_cast<int>(item - static_cast<long long>(b) * p.c.T * p.H);
  const int t = rest / p.H, h = rest % p.H, kvh = h / p.G;
  const PagedSeq s = paged_seq(p.c, b, p.kv.max_pages << p.kv.page_shift);
  if (s.bad && lane == 0) set_status(p.status, kDevBadInput);
  if (t >= s.n) return;
  const bf16 *q = reinterpret_cast<const bf16 *>(p.q.data) + paged_row_off(p.q, p.c, s, b, t, h) + lane * E;
  float qf[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[e]);
    acc[e] = 0.f;
  }
  const int at = s.L + t, lo = p.window > 0 ? max(0, at - p.window + 1) : 0;
  for (int j = lo; j <= at; ++j) {
    const int page = paged_page(p.kv, b, j);
    if (page < 0 || page >= p.kv.P) {
      if (lane == 0) set_status(p.status, kDevBadInput);
      continue;
    }
    const long long slot = paged_slot(p.kv, page, j, kvh);
    float kf[E], vf[E];
    load_row<HD, FP8>(p.kv.k, slot, lane, FP8 ? p.kv.ks[slot] : 1.f, kf);
    load_row<HD, FP8>(p.kv.v, slot, lane, FP8 ? p.kv.vs[slot] : 1.f, vf);
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) d += qf[e] * kf[e];
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    d *= p.scale_log2;
    const float mn = fmaxf(m, d), a = exp2f(m - mn), w = exp2f(d - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * vf[e];
  }
  bf16 *o = reinterpret_cast<bf16 *>(p.o.data) + paged_row_off(p.o, p.c, s, b, t, h) + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = __float2bfloat16_rn(acc[e] / l);
}

}  // namespace

size_t paged_attention_ws_bytes(int hd, int H, int KV, int B, int T) { return 1024; }

cudaError_t launch_paged_attention(const PagedAttnParams &p, uint8_t *ws, int sms, cudaStream_t st, int *launches) {
  const unsigned blocks = static_cast<unsigned>(cdiv(static_cast<long long>(p.c.B) * p.c.T * p.H, 4));
  if (p.kv.hd == 64) {
    if (p.kv.e4m3) paged_rows_kernel<64, true><<<blocks, 128, 0, st>>>(p);
    else paged_rows_kernel<64, false><<<blocks, 128, 0, st>>>(p);
  } else {
    if (p.kv.e4m3) paged_rows_kernel<128, true><<<blocks, 128, 0, st>>>(p);
    else paged_rows_kernel<128, false><<<blocks, 128, 0, st>>>(p);
  }
  *launches = 1;
  return cudaGetLastError();
}

}  // namespace smol
