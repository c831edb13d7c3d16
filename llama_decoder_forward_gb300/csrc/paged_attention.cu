// paged_attention.cu - causal grouped-query attention of a chunk of new tokens
// over a paged cache: the kernel for few rows, the combination of partial
// results, and the choice of kernel.
//
// out[t, h] = sum_j softmax_j(scale q[t, h] . k[j]) v[j] over the positions
// j <= p, j > p - window, p = L + t.
#include <math.h>

#include <algorithm>

#include "paged_decode.cuh"
#include "profile.cuh"

namespace smol {
namespace {

constexpr int kCombThreads = 256;

// The many-rows kernel's units that a border between CTAs cuts: CTA c's of this
// grid combines the unit that CTA c began and did not finish, from that one's place 1
// and the place 0 of the CTAs behind it up to the one in which the unit ends.
// One warp for each row; blockIdx.y splits the rows.
template <int HD>
__global__ void __launch_bounds__(kCombThreads) paged_combine_kernel(const PagedAttnParams p, int rows) {
  __shared__ int first_end;
  __shared__ float weight[8][kPagedMaxCtas];
  const int tid = threadIdx.x, warp = tid >> 5, c = blockIdx.x;
  griddep_wait();
  const PagedMeta *metas = paged_meta(p.ws);
  const PagedMeta mine = metas[c];
  if (!mine.out) return;
  if (tid == 0) first_end = p.ctas - 1;
  __syncthreads();
  const int other = c + 1 + tid;
  if (other < p.ctas && metas[other].in && metas[other].ends) atomicMin(&first_end, other);
  __syncthreads();
  const int n = first_end - c + 1;
  const PagedSeq s = paged_seq(p.c, mine.b, paged_cap(p));
  int t0, nt, lo, hi, j0, j1;
  paged_unit_tiles(p, s, mine.qt, t0, nt, lo, hi, j0, j1);
  for (int r = blockIdx.y * 8 + warp; r < nt * p.G; r += gridDim.y * 8)
    paged_combine_row<HD>(p, rows, c, n, r, weight[warp], paged_unit_row(p.o, p, s, mine.b, t0, mine.kvh, r));
}

template <int HD, bool FP8, int NR>
cudaError_t launch_few(const PagedAttnParams &p, cudaStream_t st) {
  using C = PdCfg<HD, FP8, NR>;
  const cudaError_t e = ensure_smem_attr<paged_few_rows_kernel<HD, FP8, NR>>(C::SMEM);
  if (e != cudaSuccess) return e;
  PagedAttnParams q = p;
  q.bk_shift = C::BK_SHIFT;
  CUtensorMap tq, tk, tv;
  if (!paged_map_q(&tq, p) || !paged_map_pages(&tk, p.kv, p.kv.k, C::KC) || !paged_map_pages(&tv, p.kv, p.kv.v, C::KC))
    return cudaErrorInvalidValue;
  paged_few_rows_kernel<HD, FP8, NR><<<p.ctas, C::THREADS, C::SMEM, st>>>(tq, tk, tv, q);
  return cudaGetLastError();
}

// The most rows that the few-rows kernel takes as one unit (32 sequences of 2000 to 8191
// cached tokens, by it and by the many-rows kernel): bf16 of hd 64 24 rows 42 and 48 us,
// 30 rows 50 and 48; of hd 128 16 rows 70 and 73, 20 rows 84 and 74; e4m3 of hd 128 20
// rows 75 and 160, of hd 64 27 rows 53 and 90.
constexpr int few_rows_most(int hd, bool e4m3) { return e4m3 ? 32 : hd == 64 ? 24 : 16; }

template <int HD, bool FP8>
cudaError_t launch_few(int rows, const PagedAttnParams &p, cudaStream_t st) {
  constexpr int most = few_rows_most(HD, FP8);
  if constexpr (most >= 32)
    if (rows > 24) return launch_few<HD, FP8, 4>(p, st);
  if constexpr (most >= 24)
    if (rows > 16) return launch_few<HD, FP8, 3>(p, st);
  return rows > 8 ? launch_few<HD, FP8, 2>(p, st) : launch_few<HD, FP8, 1>(p, st);
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

// q as [sequences][tokens][heads][hd]: a unit's box is its tokens' heads, 64 columns.
bool paged_map_q(CUtensorMap *map, const PagedAttnParams &p) {
  const bool packed = p.c.row_start != nullptr;
  const uint64_t d[4] = {(uint64_t)p.kv.hd, (uint64_t)p.H, packed ? (uint64_t)p.c.rows : (uint64_t)p.c.T, packed ? 1ull : (uint64_t)p.c.B};
  const uint64_t s[3] = {(uint64_t)p.q.head * 2, (uint64_t)p.q.row * 2, (uint64_t)(packed ? p.kv.hd : p.q.seq) * 2};
  const uint32_t b[4] = {64, (uint32_t)p.G, (uint32_t)p.tt, 1};
  return make_tmap_nd(map, p.q.data, 2, 4, d, s, b, 128);
}

// One layer's pages as [page][kv heads' rows][hd]: boxes of up to box_rows rows of a
// page, 64 columns of bf16 or a row of codes.
bool paged_map_pages(CUtensorMap *map, const PagedKv &kv, const void *base, int box_rows) {
  const uint64_t page = 1ull << kv.page_shift, row = (uint64_t)kv.hd * (kv.e4m3 ? 1 : 2);
  const uint64_t d[3] = {(uint64_t)kv.hd, kv.KV * page, (uint64_t)kv.P}, s[2] = {row, kv.KV * page * row};
  const uint32_t b[3] = {kv.e4m3 ? (uint32_t)kv.hd : 64u, (uint32_t)(page < (uint64_t)box_rows ? page : box_rows), 1};
  return make_tmap_nd(map, base, kv.e4m3 ? 1 : 2, 3, d, s, b, kv.e4m3 && kv.hd == 64 ? 64 : 128);
}

// Rows of a unit: the tile of the kernel that takes the call.  e4m3 chunks of up to 48
// rows go to the few-rows kernel in two halves, which read the same keys (4 heads, 9
// tokens: 129 us, by the many-rows kernel 163; 3 heads, 16 tokens 73 and 92; of 64 rows
// 173 and 167).
static int unit_rows(int G, int T, int hd, bool e4m3) {
  const long long r = (long long)T * G;
  if (r <= few_rows_most(hd, e4m3)) return static_cast<int>((r + 7) / 8 * 8);
  if (e4m3 && r <= 48 && (T + 1) / 2 * G <= 24) return unit_rows(G, (T + 1) / 2, hd, true);
  return r <= 128 ? 128 : 256;
}

size_t paged_attention_ws_bytes(int hd, int H, int KV, int B, int T) {
  return kPagedPartOff + (size_t)kPagedMaxCtas * 2 * std::max(unit_rows(H / KV, T, hd, false), unit_rows(H / KV, T, hd, true)) * (hd + 2) * sizeof(float);
}

cudaError_t launch_paged_attention(const PagedAttnParams &p0, int sms, cudaStream_t st, int *launches) {
  PagedAttnParams p = p0;
  p.ctas = min(sms, kPagedMaxCtas);
  const int rows = unit_rows(p.G, p.c.T, p.kv.hd, p.kv.e4m3);
  p.tt = rows / p.G;
  const bool f8 = p.kv.e4m3, h64 = p.kv.hd == 64;
  p.bk_shift = 7;                                 // the many-rows kernel's tiles; the other one has its own
  cudaError_t e;
  const int kind = rows >= 128 ? SMOL_K_ATTN : SMOL_K_DEC_ATTN;
  prof_before(kind, st);
  if (rows >= 128) {
    e = launch_paged_tiles(p, st);
  } else if (h64) {
    e = f8 ? launch_few<64, true>(rows, p, st) : launch_few<64, false>(rows, p, st);
  } else {
    e = f8 ? launch_few<128, true>(rows, p, st) : launch_few<128, false>(rows, p, st);
  }
  prof_after(kind, st);
  if (e != cudaSuccess) return e;
  *launches = 1;
  if (rows < 128) return cudaSuccess;             // that kernel combines its parts itself
  prof_before(kind, st);
  e = h64 ? launch_combine<64>(p, rows, st) : launch_combine<128>(p, rows, st);
  prof_after(kind, st);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

}  // namespace smol
