// paged_decode.cuh - paged attention of few rows: up to 16 or 32 query rows
// (tokens times heads of a kv head) share a sequence's keys.  Included by
// paged_attention.cu.
//
// Bound by memory: every key and value is read once for at most 32 rows.  What
// counts is bytes in flight, so each of the CTA's eight warps runs by itself: its
// own ring of stages in shared memory, filled by 16-byte asynchronous copies
// (keys outside the rows' sight, and pages that are not there, are filled with
// zeros, so nothing that lies in unused slots is ever computed with), and its own
// running maximum, sum and accumulator over an eighth of each key tile.  No
// barrier is met until a unit ends; then the eight states are merged through
// shared memory, two at a time.
//
// mma.sync m16n8k16 (bf16, fp32 sums): a tcgen05 tile has 128 rows, of which 3 to
// 32 would be used, and its score tile's trip through tensor memory is longer than
// the whole step here.  The fragments of a step stay in registers.
//
// e4m3 codes become bf16 exactly: the code's 7 bits moved to the bf16 exponent and
// mantissa are the value times 2^-120 (subnormal codes included), one exact
// product restores it.  The keys' scales multiply the scores, the values' scales
// the weights, so no dequantised value is rounded.
#pragma once

#include "paged_sched.cuh"

namespace smol {
namespace {

__device__ __forceinline__ void pd_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void pd_ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void pd_ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Two e4m3 codes in the high bytes of the halves of x to a bf16 pair.
__device__ __forceinline__ uint32_t e4m3_bf16x2(uint32_t x) {
  const uint32_t u = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u);
  const uint32_t two120 = 0x7b807b80u;
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&u), *reinterpret_cast<const __nv_bfloat162 *>(&two120));
  return *reinterpret_cast<const uint32_t *>(&v);
}

// A pair of q's values.
__device__ __forceinline__ uint32_t pd_q2(const uint8_t *q, long long off) {
  return *reinterpret_cast<const uint32_t *>(q + off * 2);
}

template <int HD, bool FP8, int RT>
struct PdCfg {
  static constexpr int NW = 8, THREADS = 32 * NW;
  static constexpr int KC = (HD == 128 && !FP8) ? 16 : 32;     // keys of a warp's step: 4 or 8 KB of K and V
  static constexpr int ROWB = HD * (FP8 ? 1 : 2);              // bytes of a key
  static constexpr int CPR = ROWB / 16;                        // 16-byte pieces of a key
  static constexpr int KV_BYTES = KC * ROWB;
  static constexpr int STAGE = 2 * KV_BYTES + (FP8 ? 2 * KC * 4 : 0);
  static constexpr int NS = (FP8 && HD == 64) ? 5 : (FP8 && RT == 2) ? 2 : 3;
  static constexpr int BK_SHIFT = KC == 32 ? 8 : 7;            // keys of a tile: NW * KC
  static constexpr int NT8 = KC / 8;                           // key columns of the score fragments
  static constexpr int ND8 = HD / 8;
  static constexpr int MERGE_WORDS = RT * (ND8 * 4 + 4);       // a thread's state
  static constexpr int OFF_MERGE = NW * NS * STAGE;
  static constexpr int SMEM = OFF_MERGE + 2 * 32 * MERGE_WORDS * 4;   // two warps' states at a time
  static_assert(SMEM <= 227 * 1024 - 1024, "shared memory per CTA");
};

// Byte offset of 16-byte piece c of key row `key`, swizzled so that eight rows'
// same piece (ldmatrix) and, for codes, two rows' four neighbouring pieces (the
// fragment loads of K) meet no bank twice.
template <int CPR>
__device__ __forceinline__ uint32_t pd_off(int key, int c) {
  if constexpr (CPR == 4) return key * 64 + ((c ^ ((key >> 1) & 3)) << 4);          // 64-byte rows
  else if constexpr (CPR == 8) return key * 128 + ((c ^ (((key & 1) << 2) | ((key >> 1) & 3))) << 4);
  else return key * 256 + ((c ^ (key & 7)) << 4);
}

template <int HD, bool FP8, int RT>
__global__ void __launch_bounds__(PdCfg<HD, FP8, RT>::THREADS, 1) paged_few_rows_kernel(const PagedAttnParams p) {
  using C = PdCfg<HD, FP8, RT>;
  constexpr int KC = C::KC, NS = C::NS, CPR = C::CPR, ND8 = C::ND8, NT8 = C::NT8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PagedSchedSmem sched;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x;
  const int g8 = lane >> 2, c4 = lane & 3;        // fragment row and column pair
  uint8_t *ring = smem + warp * NS * C::STAGE;
  float *merge = reinterpret_cast<float *>(smem + C::OFF_MERGE);

  griddep_launch_dependents();
  PagedIter cur = paged_locate<C::THREADS>(p, cta, p.ctas, sched);
  PagedMeta meta{};
  if (cur.left == 0) {
    if (threadIdx.x == 0) paged_meta(p.ws)[cta] = meta;
    return;
  }
  const bool first_in = cur.j > cur.j0;           // begun by an earlier CTA

  // ---- loads: this warp's KC keys of a tile; the page numbers are fetched one
  // step ahead of the copies that need them
  PagedIter ld = cur;
  int page0 = -1, page1 = -1;                     // pages of the first and the second half of the keys
  auto fetch_pages = [&]() {
    page0 = page1 = -1;
    if (ld.left <= 0) return;
    const int x0 = (ld.j << C::BK_SHIFT) + warp * KC, x1 = x0 + 16;
    if (x0 < ld.hi && x0 + 16 > ld.lo) page0 = paged_page(p.kv, ld.b, x0);
    if (KC == 32 && x1 < ld.hi && x1 + 16 > ld.lo) page1 = paged_page(p.kv, ld.b, x1);
  };
  fetch_pages();
  int ld_stage = 0;
  auto produce = [&]() {
    if (ld.left > 0) {
      const int x0 = (ld.j << C::BK_SHIFT) + warp * KC;
      if (x0 < ld.hi && x0 + KC > ld.lo) {
        uint8_t *st = ring + ld_stage * C::STAGE;
        bool ok0 = page0 >= 0 && page0 < p.kv.P, ok1 = page1 >= 0 && page1 < p.kv.P;
        if ((!ok0 && x0 + 16 > ld.lo) || (KC == 32 && !ok1 && x0 + 16 < ld.hi)) set_status(p.status, kDevBadInput);
        const long long s0 = ok0 ? paged_slot(p.kv, page0, x0, ld.kvh) : 0;
        const long long s1 = ok1 ? paged_slot(p.kv, page1, x0 + 16, ld.kvh) : 0;
#pragma unroll
        for (int i = lane; i < KC * CPR; i += 32) {
          const int key = i / CPR, c = i % CPR, x = x0 + key;
          const bool second = KC == 32 && key >= 16;
          const bool ok = (second ? ok1 : ok0) && x >= ld.lo && x < ld.hi;
          const long long slot = (second ? s1 : s0) + (key & 15);
          const long long at = ok ? slot * C::ROWB + c * 16 : 0;
          cp_async16(st + pd_off<CPR>(key, c), p.kv.k + at, ok);
          cp_async16(st + C::KV_BYTES + pd_off<CPR>(key, c), p.kv.v + at, ok);
        }
        if constexpr (FP8) {
          const int x = x0 + lane;
          const bool second = lane >= 16;
          const bool ok = (second ? ok1 : ok0) && x >= ld.lo && x < ld.hi;
          const long long slot = ok ? (second ? s1 : s0) + (lane & 15) : 0;
          cp_async4(st + 2 * C::KV_BYTES + lane * 4, p.kv.ks + slot, ok);
          cp_async4(st + 2 * C::KV_BYTES + (KC + lane) * 4, p.kv.vs + slot, ok);
        }
      }
      paged_next(p, ld);
      fetch_pages();
    }
    cp_async_commit();
    ld_stage = ld_stage + 1 == NS ? 0 : ld_stage + 1;
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) produce();

  // ---- state of the rows: row g8 + 8 i of m-tile rt
  float o[RT][ND8][4], m[RT][2], l[RT][2];
  uint32_t qf[RT][HD / 16][4];
  int at[RT][2];                                  // a row's own position, -1: no such row
  auto begin_unit = [&]() {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = rt * 16 + g8 + 8 * i;
        const bool live = r < cur.nt * p.G;
        at[rt][i] = live ? cur.s.L + cur.t0 + r / p.G : -1;
        m[rt][i] = -INFINITY;
        l[rt][i] = 0.f;
        const long long base = live ? paged_unit_row(p.q, p, cur.s, cur.b, cur.t0, cur.kvh, r) : 0;
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          // codes: a lane's fragments of four k-steps are 16 neighbouring bytes of the key,
          // so step s of group g takes the dims 64 g + 16 c4 + 4 s .. + 3 there
          const int d0 = FP8 ? (ks >> 2) * 64 + 16 * c4 + 4 * (ks & 3) : 16 * ks + 2 * c4;
          const int d1 = FP8 ? d0 + 2 : d0 + 8;
          qf[rt][ks][i] = live ? pd_q2(p.q.data, base + d0) : 0u;
          qf[rt][ks][2 + i] = live ? pd_q2(p.q.data, base + d1) : 0u;
        }
      }
#pragma unroll
      for (int d = 0; d < ND8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[rt][d][e] = 0.f;
    }
  };
  begin_unit();

  int stage = 0;
  bool in_unit = first_in;
  while (true) {
    cp_async_wait<NS - 2>();
    __syncwarp();                                 // every lane's copies, and its reads of the stage to refill
    produce();
    const int x0 = (cur.j << C::BK_SHIFT) + warp * KC;
    if (x0 < cur.hi && x0 + KC > cur.lo) {
      const uint8_t *st = ring + stage * C::STAGE;
      const uint32_t k_s = smem_u32(st), v_s = k_s + C::KV_BYTES;
      const float *scales = reinterpret_cast<const float *>(st + 2 * C::KV_BYTES);
      // ---- S = Q K^T
      float s[RT][NT8][4];
#pragma unroll
      for (int n = 0; n < NT8; ++n) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[rt][n][e] = 0.f;
        if constexpr (FP8) {
          const int key = n * 8 + g8;
#pragma unroll
          for (int gr = 0; gr < HD / 64; ++gr) {
            const uint4 w = *reinterpret_cast<const uint4 *>(st + pd_off<CPR>(key, gr * 4 + c4));
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const uint32_t b0 = e4m3_bf16x2(__byte_perm(ws[q4], 0, 0x1404)), b1 = e4m3_bf16x2(__byte_perm(ws[q4], 0, 0x3424));
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) pd_mma(s[rt][n], qf[rt][gr * 4 + q4], b0, b1);
            }
          }
        } else {
#pragma unroll
          for (int k2 = 0; k2 < HD / 32; ++k2) {
            uint32_t b[4];
            pd_ldsm4(b, k_s + pd_off<CPR>(n * 8 + (lane & 7), k2 * 4 + (lane >> 3)));
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              pd_mma(s[rt][n], qf[rt][2 * k2], b[0], b[1]);
              pd_mma(s[rt][n], qf[rt][2 * k2 + 1], b[2], b[3]);
            }
          }
        }
      }
      // ---- scores in the exp2 domain, masked where a row does not see the key
      const int first_at = cur.s.L + cur.t0;      // the first row's position
      const bool edge = x0 + KC - 1 > first_at || x0 < cur.lo || (p.window > 0 && x0 <= first_at + cur.nt - 1 - p.window) ||
                        RT * 16 > cur.nt * p.G;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NT8; ++n) {
          float2 ks = make_float2(p.scale_log2, p.scale_log2);
          if constexpr (FP8) {
            const float2 t = *reinterpret_cast<const float2 *>(scales + n * 8 + 2 * c4);
            ks.x *= t.x;
            ks.y *= t.y;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = s[rt][n][e] * ((e & 1) ? ks.y : ks.x);
            if (edge) {
              const int x = x0 + n * 8 + 2 * c4 + (e & 1), own = at[rt][e >> 1];
              if (x > own || x < cur.lo || (p.window > 0 && x <= own - p.window)) v = -INFINITY;
            }
            s[rt][n][e] = v;
            mx[e >> 1] = fmaxf(mx[e >> 1], v);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        }
        const bool grows = mx[0] > m[rt][0] || mx[1] > m[rt][1];
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[rt][i], mx[i]);
            const float a = mn == -INFINITY ? 1.f : ex2_approx(m[rt][i] - mn);
            m[rt][i] = mn;
            l[rt][i] *= a;
#pragma unroll
            for (int d = 0; d < ND8; ++d) {
              o[rt][d][2 * i] *= a;
              o[rt][d][2 * i + 1] *= a;
            }
          }
        }
        const float mu[2] = {m[rt][0] == -INFINITY ? 0.f : m[rt][0], m[rt][1] == -INFINITY ? 0.f : m[rt][1]};
#pragma unroll
        for (int n = 0; n < NT8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float w = ex2_approx(s[rt][n][e] - mu[e >> 1]);
            l[rt][e >> 1] += w;
            s[rt][n][e] = w;
          }
      }
      // ---- O += P V; P rounded to bf16, the tensor core's operand type
#pragma unroll
      for (int k16 = 0; k16 < KC / 16; ++k16) {
        uint32_t a[RT][4];
        float2 vs0 = make_float2(1.f, 1.f), vs1 = vs0;
        if constexpr (FP8) {
          vs0 = *reinterpret_cast<const float2 *>(scales + KC + k16 * 16 + 2 * c4);
          vs1 = *reinterpret_cast<const float2 *>(scales + KC + k16 * 16 + 8 + 2 * c4);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float(&f)[4] = s[rt][2 * k16], (&g)[4] = s[rt][2 * k16 + 1];
          a[rt][0] = pack_bf16x2(f[0] * vs0.x, f[1] * vs0.y);
          a[rt][1] = pack_bf16x2(f[2] * vs0.x, f[3] * vs0.y);
          a[rt][2] = pack_bf16x2(g[0] * vs1.x, g[1] * vs1.y);
          a[rt][3] = pack_bf16x2(g[2] * vs1.x, g[3] * vs1.y);
        }
        const int key = k16 * 16 + (lane & 15), half = lane >> 4;
        if constexpr (FP8) {
          // a transposed load gives pairs of neighbouring dims: the even dims of 16 go
          // to one accumulator column block, the odd ones to the next
#pragma unroll
          for (int c2 = 0; c2 < CPR / 2; ++c2) {
            uint32_t b[4];
            pd_ldsm4_t(b, v_s + pd_off<CPR>(key, 2 * c2 + half));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t e0 = e4m3_bf16x2(__byte_perm(b[2 * h], 0, 0x2404)), e1 = e4m3_bf16x2(__byte_perm(b[2 * h + 1], 0, 0x2404));
              const uint32_t d0 = e4m3_bf16x2(b[2 * h] & 0xff00ff00u), d1 = e4m3_bf16x2(b[2 * h + 1] & 0xff00ff00u);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                pd_mma(o[rt][4 * c2 + 2 * h], a[rt], e0, e1);
                pd_mma(o[rt][4 * c2 + 2 * h + 1], a[rt], d0, d1);
              }
            }
          }
        } else {
#pragma unroll
          for (int c2 = 0; c2 < CPR / 2; ++c2) {
            uint32_t b[4];
            pd_ldsm4_t(b, v_s + pd_off<CPR>(key, 2 * c2 + half));
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              pd_mma(o[rt][2 * c2], a[rt], b[0], b[1]);
              pd_mma(o[rt][2 * c2 + 1], a[rt], b[2], b[3]);
            }
          }
        }
      }
    }
    stage = stage + 1 == NS ? 0 : stage + 1;
    const bool unit_ends = cur.j + 1 == cur.j1, last = cur.left == 1;
    if (unit_ends || last) {
      // ---- merge the warps' states: 4, 5 into 0, 1; 6, 7 into 2, 3; 2, 3 into 0, 1; 1 into 0
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[rt][i] += __shfl_xor_sync(0xffffffffu, l[rt][i], 1);
          l[rt][i] += __shfl_xor_sync(0xffffffffu, l[rt][i], 2);
        }
#pragma unroll 1
      for (int step = 0; step < 4; ++step) {
        const int from = step == 0 ? 4 : step == 1 ? 6 : step == 2 ? 2 : 1, to = step == 1 ? 2 : 0, n = step == 3 ? 1 : 2;
        if (warp >= from && warp < from + n) {
          float *dst = merge + (warp - from) * 32 * C::MERGE_WORDS + lane;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int d = 0; d < ND8; ++d)
#pragma unroll
              for (int e = 0; e < 4; ++e) dst[(rt * (ND8 * 4 + 4) + d * 4 + e) * 32] = o[rt][d][e];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              dst[(rt * (ND8 * 4 + 4) + ND8 * 4 + i) * 32] = m[rt][i];
              dst[(rt * (ND8 * 4 + 4) + ND8 * 4 + 2 + i) * 32] = l[rt][i];
            }
          }
        }
        __syncthreads();
        if (warp >= to && warp < to + n) {
          const float *src = merge + (warp - to) * 32 * C::MERGE_WORDS + lane;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const float *sr = src + rt * (ND8 * 4 + 4) * 32;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float m2 = sr[(ND8 * 4 + i) * 32], l2 = sr[(ND8 * 4 + 2 + i) * 32];
              const float mn = fmaxf(m[rt][i], m2);
              const float a = mn == -INFINITY ? 1.f : ex2_approx(m[rt][i] - mn), a2 = mn == -INFINITY ? 1.f : ex2_approx(m2 - mn);
              m[rt][i] = mn;
              l[rt][i] = l[rt][i] * a + l2 * a2;
#pragma unroll
              for (int d = 0; d < ND8; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  o[rt][d][2 * i + e] = o[rt][d][2 * i + e] * a + sr[(d * 4 + 2 * i + e) * 32] * a2;
            }
          }
        }
        __syncthreads();
      }
      const bool whole = unit_ends && !in_unit;
      if (warp == 0) {
        float *part = paged_part(p.ws, cta, in_unit ? 0 : 1, RT * 16, HD);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = rt * 16 + g8 + 8 * i;
            const bool live = at[rt][i] >= 0;
            const float inv = l[rt][i] > 0.f ? 1.f / l[rt][i] : 0.f;
            const long long out = live && whole ? paged_unit_row(p.o, p, cur.s, cur.b, cur.t0, cur.kvh, r) : 0;
            float *row = part + r * HD;
            if (live) {
#pragma unroll
              for (int d = 0; d < ND8; ++d) {
                const float x = o[rt][d][2 * i], y = o[rt][d][2 * i + 1];
                if constexpr (FP8) {
                  if (d & 1) continue;
                  const float x1 = o[rt][d + 1][2 * i], y1 = o[rt][d + 1][2 * i + 1];   // the odd dims
                  const int dim = d * 8 + 4 * c4;
                  if (whole)
                    *reinterpret_cast<uint2 *>(p.o.data + (out + dim) * 2) =
                        p.o_f16 ? make_uint2(pack_f16x2(x * inv, x1 * inv), pack_f16x2(y * inv, y1 * inv))
                                : make_uint2(pack_bf16x2(x * inv, x1 * inv), pack_bf16x2(y * inv, y1 * inv));
                  else
                    *reinterpret_cast<float4 *>(row + dim) = make_float4(x, x1, y, y1);
                } else {
                  const int dim = d * 8 + 2 * c4;
                  if (whole)
                    *reinterpret_cast<uint32_t *>(p.o.data + (out + dim) * 2) =
                        p.o_f16 ? pack_f16x2(x * inv, y * inv) : pack_bf16x2(x * inv, y * inv);
                  else
                    *reinterpret_cast<float2 *>(row + dim) = make_float2(x, y);
                }
              }
              if (!whole && c4 == 0) *reinterpret_cast<float2 *>(part + RT * 16 * HD + 2 * r) = make_float2(m[rt][i], l[rt][i]);
            }
          }
      }
      if (in_unit) {
        meta.in = 1;
        meta.ends = unit_ends;
      } else if (!unit_ends) {
        meta.out = 1;
        meta.b = cur.b;
        meta.qt = cur.qt;
        meta.kvh = cur.kvh;
      }
      if (last) break;
      in_unit = false;
      paged_next(p, cur);
      begin_unit();
    } else {
      paged_next(p, cur);
    }
  }
  cp_async_wait<0>();
  if (threadIdx.x == 0) paged_meta(p.ws)[cta] = meta;
}

}  // namespace
}  // namespace smol
