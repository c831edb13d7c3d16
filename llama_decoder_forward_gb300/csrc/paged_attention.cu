// paged_attention.cu - causal grouped-query attention of a chunk of new tokens
// over a paged cache: the kernel for few rows, the combination of partial
// results, and the choice of kernel.
//
// out[t, h] = sum_j softmax_j(scale q[t, h] . k[j]) v[j] over the positions
// j <= p, j > p - window, p = L + t.
#include <math.h>

#include "paged_decode.cuh"
#include "profile.cuh"

namespace smol {
namespace {

constexpr int kCombThreads = 256;

// Units cut by a border between CTAs: CTA c's combines the unit that CTA c began
// and did not finish, from its place 1 and the place 0 of the CTAs behind it up
// to the one in which the unit ends, in that order (the same bits every time).
// One warp for each row; blockIdx.y splits the rows.
template <int HD>
__global__ void __launch_bounds__(kCombThreads) paged_combine_kernel(const PagedAttnParams p, int rows) {
  __shared__ int list[kPagedMaxCtas], n_warp[8], first_end;
  __shared__ float weight[8][kPagedMaxCtas];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  griddep_wait();
  const PagedMeta *metas = paged_meta(p.ws);
  const PagedMeta mine = metas[c];
  if (!mine.out) return;
  if (tid == 0) first_end = p.ctas;
  __syncthreads();
  const int other = c + tid;                      // tid 0: this CTA's own place 1
  PagedMeta mo{};
  if (tid > 0 && other < p.ctas) mo = metas[other];
  if (mo.in && mo.ends) atomicMin(&first_end, other);
  __syncthreads();
  const bool in = tid == 0 || (mo.in && other <= first_end);
  const unsigned vote = __ballot_sync(0xffffffffu, in);
  if (lane == 0) n_warp[warp] = __popc(vote);
  __syncthreads();
  int at = __popc(vote & ((1u << lane) - 1)), n = 0;
  for (int w = 0; w < 8; ++w) {
    if (w < warp) at += n_warp[w];
    n += n_warp[w];
  }
  if (in) list[at] = other;
  __syncthreads();
  const PagedSeq s = paged_seq(p.c, mine.b, paged_cap(p));
  int t0, nt, lo, hi, j0, j1;
  paged_unit_tiles(p, s, mine.qt, t0, nt, lo, hi, j0, j1);
  const int live = nt * p.G;
  for (int r = blockIdx.y * 8 + warp; r < live; r += gridDim.y * 8) {
    float mx = -INFINITY, sum = 0.f;
    for (int i = lane; i < n; i += 32)
      mx = fmaxf(mx, paged_part(p.ws, list[i], i == 0, rows, HD)[rows * HD + 2 * r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    for (int i = lane; i < n; i += 32) {
      const float2 ml = *reinterpret_cast<const float2 *>(paged_part(p.ws, list[i], i == 0, rows, HD) + rows * HD + 2 * r);
      const float a = mx == -INFINITY ? 0.f : ex2_approx(ml.x - mx);
      weight[warp][i] = a;
      sum += a * ml.y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    float acc[HD / 32];
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float *row = paged_part(p.ws, list[i], i == 0, rows, HD) + r * HD + lane * (HD / 32);
      const float a = weight[warp][i];
      if constexpr (HD == 64) {
        const float2 v = *reinterpret_cast<const float2 *>(row);
        acc[0] += a * v.x;
        acc[1] += a * v.y;
      } else {
        const float4 v = *reinterpret_cast<const float4 *>(row);
        acc[0] += a * v.x;
        acc[1] += a * v.y;
        acc[2] += a * v.z;
        acc[3] += a * v.w;
      }
    }
    uint32_t *out = reinterpret_cast<uint32_t *>(
        p.o.data + (paged_unit_row(p.o, p, s, mine.b, t0, mine.kvh, r) + lane * (HD / 32)) * 2);
#pragma unroll
    for (int e = 0; e < HD / 64; ++e)
      out[e] = p.o_f16 ? pack_f16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv) : pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    __syncwarp();                                 // the weights are rewritten
  }
}

template <int HD, bool FP8, int RT>
cudaError_t launch_few(const PagedAttnParams &p, cudaStream_t st) {
  using C = PdCfg<HD, FP8, RT>;
  const cudaError_t e = ensure_smem_attr<paged_few_rows_kernel<HD, FP8, RT>>(C::SMEM);
  if (e != cudaSuccess) return e;
  PagedAttnParams q = p;
  q.bk_shift = C::BK_SHIFT;
  paged_few_rows_kernel<HD, FP8, RT><<<p.ctas, C::THREADS, C::SMEM, st>>>(q);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_combine(const PagedAttnParams &p, int rows, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas, static_cast<unsigned>(cdiv(rows, 32)));
  cfg.blockDim = dim3(kCombThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<HD>, p, rows);
}

}  // namespace

// Rows of a unit: the tile of the kernel that takes the call.
static int unit_rows(int G, int T) {
  const long long r = (long long)T * G;
  return r <= 16 ? 16 : r <= 128 ? 128 : 256;
}

size_t paged_attention_ws_bytes(int hd, int H, int KV, int B, int T) {
  return kPagedPartOff + (size_t)kPagedMaxCtas * 2 * unit_rows(H / KV, T) * (hd + 2) * sizeof(float);
}

cudaError_t launch_paged_attention(const PagedAttnParams &p0, int sms, cudaStream_t st, int *launches) {
  PagedAttnParams p = p0;
  p.ctas = min(sms, kPagedMaxCtas);
  const int rows = unit_rows(p.G, p.c.T);
  p.tt = rows / p.G;
  const bool f8 = p.kv.e4m3, h64 = p.kv.hd == 64, one = rows == 16;
  p.bk_shift = rows >= 128 || !(h64 || f8) ? 7 : 8;
  cudaError_t e;
  prof_before(SMOL_K_DEC_ATTN, st);
  if (rows >= 128) {
    e = launch_paged_tiles(p, st);
  } else if (h64) {
    if (f8) e = one ? launch_few<64, true, 1>(p, st) : launch_few<64, true, 2>(p, st);
    else e = one ? launch_few<64, false, 1>(p, st) : launch_few<64, false, 2>(p, st);
  } else {
    if (f8) e = one ? launch_few<128, true, 1>(p, st) : launch_few<128, true, 2>(p, st);
    else e = one ? launch_few<128, false, 1>(p, st) : launch_few<128, false, 2>(p, st);
  }
  prof_after(SMOL_K_DEC_ATTN, st);
  if (e != cudaSuccess) return e;
  *launches = 1;
  prof_before(SMOL_K_OTHER, st);
  e = h64 ? launch_combine<64>(p, rows, st) : launch_combine<128>(p, rows, st);
  prof_after(SMOL_K_OTHER, st);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

}  // namespace smol
