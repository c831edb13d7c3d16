// paged_cache.cu - writing a chunk's keys and values into cache pages (bf16, or
// e4m3 codes with one scale for each position and kv head) and reading them back.
//
//   scale = max_d |x_d| / 448,  code_d = e4m3(x_d / scale),  value_d = code_d * scale
//
// 448 is the largest e4m3 number, so the row's largest magnitude takes the
// largest code and nothing saturates.  The quotients are the correctly rounded ones
// (a bare product with 1 / scale would move values next to a border to the other
// code): q = x r with r = 1 / scale correctly rounded, and one correction by the
// residual, q + (x - q scale) r, which Markstein's theorem says is x / scale
// rounded.  The compiler's division, with its checks of range, is for rows whose
// scale is beyond 2^+-100 only: with it for all the kernel was bound by arithmetic,
// at half the bandwidth.
//
// Both are copies bound by memory.  A group of hd / 16 lanes takes one row (a
// token's hd values of one kv head) of the keys and the same row of the values, in
// some of the layers one after the other, so a lane has four independent 16-byte
// loads in flight, the row's maximum needs two or three shuffles, and the search
// for the row's sequence and page is done once.  Consecutive groups take
// consecutive kv heads of a row: contiguous in packed rows, whole 128- or 256-byte
// lines otherwise.  In tensors whose rows of a head lie one behind the other (the dense
// cache's layout) they take consecutive rows of a head: 16 sequences of up to 4096
// tokens, e4m3 to bf16, 77 us, by kv heads 80.
#include <cuda_fp8.h>
#include <math.h>

#include "paged.cuh"

namespace smol {
namespace {

constexpr int kPcThreads = 256;

// The sequence and row index of row r of the chunk's row tensors (packed: the
// sequence that owns row r by a search of row_start; else r = b * T + t); whether
// there is such a row, and it stands at a position.
__device__ __forceinline__ bool chunk_row(const PagedChunk &c, long long r, int cap, int &b, int &t, PagedSeq &s) {
  if (c.row_start) {
    int lo = 0, hi = c.B;                        // row_start[lo] <= r < row_start[hi], if any
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (c.row_start[mid] <= r) lo = mid;
      else hi = mid;
    }
    b = lo;
    s = paged_seq(c, b, cap);
    const long long d = r - s.row0;
    t = d < 0 || d > 0x7fffffff ? -1 : static_cast<int>(d);
  } else {
    b = static_cast<int>(paged_div(r, c.T));
    t = static_cast<int>(r - static_cast<long long>(b) * c.T);
    s = paged_seq(c, b, cap);
  }
  return t >= 0 && t < s.n && !s.moved;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(__half2(h));
}

// A lane's sixteen values of one row (two 16-byte words of bf16) to codes.
template <int LANES>
__device__ __forceinline__ uint4 quantise16(const uint4 (&w)[2], float &scale) {
  float f[16];
  float amax = 0.f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = reinterpret_cast<const uint32_t *>(w)[i];
    const float2 x = unpack_bf16x2(u);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
    amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
    fine &= (u & 0x7f80u) != 0x7f80u && (u & 0x7f800000u) != 0x7f800000u;
  }
  if (!fine) amax = INFINITY;                    // an infinity or NaN: fmaxf drops a NaN, not this
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  scale = amax == INFINITY ? __int_as_float(0x7fffffff) : amax / 448.f;
  const float d = scale > 0.f ? scale : 1.f;     // a row of zeros (or of NaN scale): codes of x itself
  if (d > 7.9e-31f && d < 1.2e30f) {
    const float r = 1.f / d;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float q = f[i] * r;
      f[i] = __fmaf_rn(__fmaf_rn(-q, d, f[i]), r, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = f[i] / d;
  }
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  return make_uint4(c[0], c[1], c[2], c[3]);
}

template <int HD, bool FP8, bool APPEND>
__global__ void __launch_bounds__(kPcThreads) paged_copy_kernel(const PagedKv kv, const PagedChunk c,
                                                                const PagedRows kr, const PagedRows vr,
                                                                long long n_rows, int layers, int per, int by_row) {
  constexpr int LANES = HD / 16;                 // lanes of one row
  const long long g = (static_cast<long long>(blockIdx.x) * kPcThreads + threadIdx.x) / LANES;
  const int part = threadIdx.x % LANES;          // values part * 16 .. + 15
  long long r;
  int h;
  if (by_row) {                                  // g = (b * KV + h) * T + t
    const long long bh = paged_div(g, c.T), b = paged_div(bh, kv.KV);
    h = static_cast<int>(bh - b * kv.KV);
    r = b * c.T + (g - bh * c.T);
  } else {                                       // g = row * KV + h
    r = paged_div(g, kv.KV);
    h = static_cast<int>(g - r * kv.KV);
  }
  const int cap = kv.max_pages << kv.page_shift;
  int b = 0, t = 0, page = -1, x = 0;
  PagedSeq s{};
  bool live = r < n_rows && chunk_row(c, r, cap, b, t, s);
  if (live) {
    x = s.L + t;
    page = paged_page(kv, b, x);
    live = page >= 0 && page < kv.P;
  }
  if (!__any_sync(0xffffffffu, live)) return;    // the shuffles below want whole warps
  const long long slot0 = live ? paged_slot(kv, page, x, h) : 0;
  const long long row0 = live ? paged_row_off(kr, c, s, b, t, h) + part * 16 : 0;
  const long long row1 = live ? paged_row_off(vr, c, s, b, t, h) + part * 16 : 0;
  const int last = min(layers, (static_cast<int>(blockIdx.y) + 1) * per);
#pragma unroll 2
  for (int layer = blockIdx.y * per; layer < last; ++layer) {
    const long long slot = layer * kv.layer_rows + slot0;
    const long long in0 = row0 + layer * kr.layer, in1 = row1 + layer * vr.layer;
    if constexpr (APPEND) {
      uint4 kw[2] = {}, vw[2] = {};
      if (live) {
        const uint4 *ks = reinterpret_cast<const uint4 *>(kr.data + in0 * 2);
        const uint4 *vs = reinterpret_cast<const uint4 *>(vr.data + in1 * 2);
        kw[0] = ks[0];
        kw[1] = ks[1];
        vw[0] = vs[0];
        vw[1] = vs[1];
      }
      if constexpr (FP8) {
        float sk, sv;
        const uint4 ck = quantise16<LANES>(kw, sk), cv = quantise16<LANES>(vw, sv);
        if (live) {
          *reinterpret_cast<uint4 *>(kv.k + slot * HD + part * 16) = ck;
          *reinterpret_cast<uint4 *>(kv.v + slot * HD + part * 16) = cv;
          if (part == 0) {
            kv.ks[slot] = sk;
            kv.vs[slot] = sv;
          }
        }
      } else if (live) {
        uint4 *kd = reinterpret_cast<uint4 *>(kv.k + (slot * HD + part * 16) * 2);
        uint4 *vd = reinterpret_cast<uint4 *>(kv.v + (slot * HD + part * 16) * 2);
        kd[0] = kw[0];
        kd[1] = kw[1];
        vd[0] = vw[0];
        vd[1] = vw[1];
      }
    } else if (live) {
      uint4 kw[2], vw[2];
      if constexpr (FP8) {
        const uint4 ck = *reinterpret_cast<const uint4 *>(kv.k + slot * HD + part * 16);
        const uint4 cv = *reinterpret_cast<const uint4 *>(kv.v + slot * HD + part * 16);
        const float sk = kv.ks[slot], sv = kv.vs[slot];
        const uint32_t *cks = reinterpret_cast<const uint32_t *>(&ck), *cvs = reinterpret_cast<const uint32_t *>(&cv);
  #pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 a = e4m3x2_value((cks[i >> 1] >> ((i & 1) * 16)) & 0xffffu);
          const float2 e = e4m3x2_value((cvs[i >> 1] >> ((i & 1) * 16)) & 0xffffu);
          reinterpret_cast<uint32_t *>(kw)[i] = pack_bf16x2(a.x * sk, a.y * sk);
          reinterpret_cast<uint32_t *>(vw)[i] = pack_bf16x2(e.x * sv, e.y * sv);
        }
      } else {
        const uint4 *ks = reinterpret_cast<const uint4 *>(kv.k + (slot * HD + part * 16) * 2);
        const uint4 *vs = reinterpret_cast<const uint4 *>(kv.v + (slot * HD + part * 16) * 2);
        kw[0] = ks[0];
        kw[1] = ks[1];
        vw[0] = vs[0];
        vw[1] = vs[1];
      }
      uint4 *kd = reinterpret_cast<uint4 *>(kr.data + in0 * 2);
      uint4 *vd = reinterpret_cast<uint4 *>(vr.data + in1 * 2);
      kd[0] = kw[0];
      kd[1] = kw[1];
      vd[0] = vw[0];
      vd[1] = vw[1];
    }
  }
}

template <bool APPEND>
cudaError_t launch_copy(const PagedKv &kv, int layers, const PagedChunk &c, const PagedRows &k, const PagedRows &v,
                        cudaStream_t st) {
  const long long n_rows = c.row_start ? c.rows : static_cast<long long>(c.B) * c.T;
  if (n_rows == 0) return cudaSuccess;
  const long long blocks = cdiv(n_rows * kv.KV * (kv.hd / 16), kPcThreads);
  if (blocks > 0x7fffffffll || layers > 65535) return cudaErrorInvalidConfiguration;
  // layers of a thread: as many as leave some 2000 blocks, eight at most
  const int per = static_cast<int>(max(1ll, min(8ll, blocks * layers / 2000)));
  const int by_row = !c.row_start && c.T > 1 && k.row == kv.hd && v.row == kv.hd;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(cdiv(layers, per)));
  if (kv.hd == 64) {
    if (kv.e4m3) paged_copy_kernel<64, true, APPEND><<<grid, kPcThreads, 0, st>>>(kv, c, k, v, n_rows, layers, per, by_row);
    else paged_copy_kernel<64, false, APPEND><<<grid, kPcThreads, 0, st>>>(kv, c, k, v, n_rows, layers, per, by_row);
  } else {
    if (kv.e4m3) paged_copy_kernel<128, true, APPEND><<<grid, kPcThreads, 0, st>>>(kv, c, k, v, n_rows, layers, per, by_row);
    else paged_copy_kernel<128, false, APPEND><<<grid, kPcThreads, 0, st>>>(kv, c, k, v, n_rows, layers, per, by_row);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedKv &kv, int layers, const PagedChunk &c, const PagedRows &k,
                                const PagedRows &v, cudaStream_t st) {
  return launch_copy<true>(kv, layers, c, k, v, st);
}

cudaError_t launch_paged_read(const PagedKv &kv, int layers, const PagedChunk &c, const PagedRows &k,
                              const PagedRows &v, cudaStream_t st) {
  return launch_copy<false>(kv, layers, c, k, v, st);
}

}  // namespace smol
