// paged_attention_tc.cu - paged attention of many rows on tcgen05.
//
// A CTA takes units of up to 256 query rows (tokens times heads of one kv head,
// two tiles of 128) and walks over their key tiles of 128; units and pieces of
// units come from paged_sched.cuh.  Per key tile and query tile:
//   S = Q K^T      tcgen05.mma, M = 128, N = 128, K = hd, fp32 in tensor memory
//   P = exp2(S c - m)   one softmax warpgroup for each query tile, a row per thread;
//                  P is written as bf16 over S in tensor memory
//   O += P V       tcgen05.mma, A from tensor memory, V as stored ([key][dim],
//                  MN-major), N = hd, fp32 in tensor memory
// One thread issues every MMA, S of the next tile behind P V of this one, so that
// the tensor core works on one query tile while the other's exponents are taken.
// A commit behind S of tile i + 1 also says that P V of tile i is done: a softmax
// warpgroup that holds S may rescale O.  It does so only when a row's maximum grows
// by more than 2^8 (P then stays below 256, exact in the fp32 sums).
//
// K and V come from pages of 16 tokens and more, so four loader warps copy 16
// rows at a time (one page number each) with 16-byte asynchronous copies into the
// swizzled operand layout.  Rows outside the sight of the unit, or on a page that
// is not there, are filled with zeros: whatever lies in unused slots, P = 0 meets
// V = 0.  e4m3 codes are loaded to registers a tile ahead and become bf16 exactly;
// the keys' scales multiply the scores, the values' scales P.
//
// Registers: 512 threads start with 128 each; the softmax warpgroups take 184
// (their 128 scores stay in registers), the loaders and the issuer give up theirs.
#include <math.h>

#include "paged_sched.cuh"

namespace smol {
namespace {

constexpr int kTileK = 128;

template <int HD, bool FP8>
struct PtCfg {
  static constexpr int THREADS = 512;
  static constexpr int NSUB = HD / 64;                       // 64-column sub-tiles
  static constexpr int TILE_BYTES = 128 * HD * 2;            // a Q, K or V tile, bf16
  static constexpr int NST = HD == 64 ? 4 : 2;               // K and V stages
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NST * TILE_BYTES;
  static constexpr int OFF_SC = OFF_V + NST * TILE_BYTES;    // [NST][2][128] scales of keys and values
  static constexpr int OFF_BAR = OFF_SC + (FP8 ? NST * 2 * 128 * 4 : 0);
  static constexpr int NBAR = 2 + 4 * NST + 2 + 2 + 2 + 1;
  static constexpr int SMEM = 1024 + OFF_BAR + NBAR * 8 + 16;
  static constexpr int R_SOFTMAX = FP8 ? 168 : 184, R_LOAD = FP8 ? 128 : 96, R_MMA = FP8 ? 48 : 48;
  static_assert(2 * R_SOFTMAX + R_LOAD + R_MMA <= 512, "registers of the block");
  static_assert(SMEM + 400 <= 232448, "shared memory per CTA");
};

enum : int { kPtTimeoutLoad = 0x205, kPtTimeoutMma = 0x206, kPtTimeoutSoftmax = 0x207, kPtTimeoutDrain = 0x208 };

constexpr uint32_t kColS = 0, kColO = 256;                   // tensor memory columns: S (and P), O

__device__ __forceinline__ uint32_t pt_code_pair(uint32_t x) {
  const uint32_t u = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u), two120 = 0x7b807b80u;
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&u), *reinterpret_cast<const __nv_bfloat162 *>(&two120));
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Eight codes (two words) to eight bf16.
__device__ __forceinline__ uint4 pt_codes8(uint32_t a, uint32_t b) {
  return make_uint4(pt_code_pair(__byte_perm(a, 0, 0x1404)), pt_code_pair(__byte_perm(a, 0, 0x3424)),
                    pt_code_pair(__byte_perm(b, 0, 0x1404)), pt_code_pair(__byte_perm(b, 0, 0x3424)));
}

template <int HD, bool FP8>
__global__ void __launch_bounds__(512, 1) paged_tiles_kernel(const PagedAttnParams p) {
  using C = PtCfg<HD, FP8>;
  constexpr int NST = C::NST, NSUB = C::NSUB;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PagedSchedSmem sched;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem + C::OFF_Q, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V;
  float *sSc = reinterpret_cast<float *>(smem + C::OFF_SC);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *q_empty = q_full + 1;
  uint64_t *k_full = q_empty + 1, *k_empty = k_full + NST, *v_full = k_empty + NST, *v_empty = v_full + NST;
  uint64_t *s_full = v_empty + NST, *p_full = s_full + 2, *o_full = p_full + 2, *drain = o_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const uint64_t limit = p.wait_ns;

  griddep_launch_dependents();
  PagedIter it = paged_locate<C::THREADS>(p, cta, p.ctas, sched);
  if (it.left == 0) {                             // the same for the whole CTA
    if (tid == 0) paged_meta(p.ws)[cta] = PagedMeta{};
    return;
  }
  if (tid == 0) {
    mbar_init(q_full, 128);
    mbar_init(q_empty, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 12) {
    setmaxnreg_dec<C::R_MMA>();
    if (warp == 12) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false), kIdO = idesc_bf16_f32(128, HD, true);
      const uint64_t dq = sdesc_kmajor_sw128(smem_u32(sQ)), dk = sdesc_kmajor_sw128(smem_u32(sK));
      const uint64_t dv = sdesc_mnmajor_sw128(smem_u32(sV), 128 * 128);
      const bool me = elect_one();
      bool ok = true, any = false;
      int units = 0;                              // Q loads seen
      uint32_t n1 = 0;                            // key tiles done with the second query tile
      int kst = 0, vst = 0;
      uint32_t kph = 0, vph = 0, n0 = 0;
      PagedIter nx = it;                          // the tile whose S is issued next
      auto issue_s = [&](int h) {
        if (me) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint64_t a = dq + ((h * C::TILE_BYTES + (k >> 2) * (128 * 128) + (k & 3) * 32) >> 4);
            const uint64_t b = dk + ((kst * C::TILE_BYTES + (k >> 2) * (128 * 128) + (k & 3) * 32) >> 4);
            umma_f16(tmem + kColS + h * 128, a, b, kIdS, k > 0);
          }
          umma_commit(&s_full[h]);
        }
        __syncwarp();
      };
      // waits for what S of tile nx needs; new_unit: Q as well
      auto ready_s = [&](bool new_unit) {
        if (new_unit) {
          if (!mbar_wait_bounded(q_full, units & 1, abort_flag, limit)) return false;
          ++units;
        }
        if (!mbar_wait_bounded(&k_full[kst], kph, abort_flag, limit)) return false;
        fence_proxy_async_smem();                 // the copies' writes, before the tensor core reads them
        tc_fence_after_sync();
        return true;
      };
      auto done_s = [&](bool unit_last) {         // S of tile nx issued for each query tile
        if (me) {
          umma_commit(&k_empty[kst]);
          if (unit_last) umma_commit(q_empty);
        }
        if (++kst == NST) {
          kst = 0;
          kph ^= 1;
        }
      };
      ok = ready_s(true);
      if (ok) {
        issue_s(0);
        if (it.nt * p.G > 128) issue_s(1);
        done_s(it.j + 1 == it.j1 || it.left == 1);
        any = true;
      }
      bool first = true;                          // the unit's first key tile: O starts at zero
      while (ok) {
        const bool two = it.nt * p.G > 128, last = it.left == 1, unit_last = last || it.j + 1 == it.j1;
        paged_next(p, nx);
        const bool two_nx = nx.nt * p.G > 128;
        bool s_ready = false;
        if (!mbar_wait_bounded(&v_full[vst], vph, abort_flag, limit)) { ok = false; break; }
        fence_proxy_async_smem();
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (h == 0 || two) {
            if (!mbar_wait_bounded(&p_full[h], (h ? n1 : n0) & 1, abort_flag, limit)) { ok = false; break; }
            tc_fence_after_sync();
            if (me) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_f16_tmem_a(tmem + kColO + h * HD, tmem + kColS + h * 128 + k * 8, dv + ((vst * C::TILE_BYTES + k * 2048) >> 4),
                                kIdO, !(first && k == 0));
              if (unit_last) umma_commit(&o_full[h]);
            }
            __syncwarp();
            if (h) ++n1;
            else ++n0;
          }
          if (!last) {
            if (!s_ready) {
              if (!ready_s(unit_last)) { ok = false; break; }
              s_ready = true;
            }
            if (h == 0 || two_nx) issue_s(h);
          }
        }
        if (!ok) break;
        if (me) umma_commit(&v_empty[vst]);
        if (++vst == NST) {
          vst = 0;
          vph ^= 1;
        }
        if (last) break;
        done_s(nx.j + 1 == nx.j1 || nx.left == 1);
        first = unit_last;
        it = nx;
      }
      if (!ok) {
        set_status(p.status, kPtTimeoutMma);
        *abort_flag = 1;
      }
      if (any) {
        // every MMA issued is done before shared and tensor memory go
        if (me) umma_commit(drain);
        if (!mbar_wait_drain(drain, 0)) set_status(p.status, kPtTimeoutDrain);
      }
    }
  } else if (warp >= 8) {
    if constexpr (C::R_LOAD < 128) setmaxnreg_dec<C::R_LOAD>();
    // ------------------------------------------------------------------ loaders
    const int lt = tid - 256, row16 = lt >> 3, c8 = lt & 7;  // row of 16, 16-byte piece of 128 bytes
    bool ok = true;
    int kst = 0, vst = 0;
    uint32_t ph = 1, vph = 1;                     // the stages start empty
    int units = 0;
    int pages = -1;                               // lane i < 8 of each warp: page of keys 16 i .. of the next tile
    auto fetch_pages = [&](const PagedIter &u) {
      const int x = u.j * kTileK + 16 * (lane & 7);
      pages = -1;
      if (x < u.hi && x + 16 > u.lo) {
        pages = paged_page(p.kv, u.b, x);
        if (pages < 0 || pages >= p.kv.P) {
          set_status(p.status, kDevBadInput);
          pages = -1;
        }
      }
    };
    // slot of this thread's row in pass i of tile u; false: zeros
    auto place = [&](const PagedIter &u, int i, int pg, long long &slot) {
      const int x = u.j * kTileK + 16 * i + row16;
      const int page = __shfl_sync(0xffffffffu, pg, i);
      slot = page >= 0 ? paged_slot(p.kv, page, x, u.kvh) : 0;
      const bool in = page >= 0 && x >= u.lo && x < u.hi;
      if (!in) slot = 0;
      return in;
    };
    fetch_pages(it);
    bool new_unit = true;
    [[maybe_unused]] uint4 raw_k[8], raw_v[8];    // codes of the next tile: pass i, 16 codes of a row at most
    [[maybe_unused]] float raw_ks = 0.f, raw_vs = 0.f, next_ks = 0.f;
    // hd 64: a row's 64 codes are 4 pieces of 16; hd 128: 8.  Passes of 32 or 16 rows.
    constexpr int RPP = HD == 64 ? 32 : 16, NPASS = 128 / RPP;
    const int frow = HD == 64 ? lt >> 2 : lt >> 3, fc = HD == 64 ? lt & 3 : lt & 7;
    auto load_codes = [&](const PagedIter &u, const uint8_t *src, uint4(&raw)[8], const float *sc, float &raw_s) {
#pragma unroll
      for (int i = 0; i < NPASS; ++i) {
        const int key = i * RPP + frow, x = u.j * kTileK + key;
        const int page = __shfl_sync(0xffffffffu, pages, key >> 4);
        const bool in = page >= 0 && x >= u.lo && x < u.hi;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (in) raw[i] = __ldg(reinterpret_cast<const uint4 *>(src + paged_slot(p.kv, page, x, u.kvh) * HD + fc * 16));
      }
      const int x = u.j * kTileK + lt;            // scales: thread lt takes key lt
      const int page = __shfl_sync(0xffffffffu, pages, (lt & 127) >> 4);
      raw_s = page >= 0 && x >= u.lo && x < u.hi ? __ldg(sc + paged_slot(p.kv, page, x, u.kvh)) : 0.f;
    };
    auto store_codes = [&](uint8_t *dst, const uint4(&raw)[8]) {
#pragma unroll
      for (int i = 0; i < NPASS; ++i) {
        const int key = i * RPP + frow, ch = fc * 2;         // two pieces of 8 bf16
        uint8_t *row = dst + (ch >> 3) * (128 * 128) + key * 128;
        *reinterpret_cast<uint4 *>(row + (((ch & 7) ^ (key & 7)) << 4)) = pt_codes8(raw[i].x, raw[i].y);
        *reinterpret_cast<uint4 *>(row + ((((ch + 1) & 7) ^ (key & 7)) << 4)) = pt_codes8(raw[i].z, raw[i].w);
      }
    };
    if constexpr (FP8) {
      load_codes(it, p.kv.k, raw_k, p.kv.ks, raw_ks);
      load_codes(it, p.kv.v, raw_v, p.kv.vs, raw_vs);
    }
    while (true) {
      PagedIter nx = it;
      paged_next(p, nx);
      const bool last = it.left == 1;
      const int cur_pages = pages;
      if (!last) fetch_pages(nx);                 // in use from the next round on
      // ---- K
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&k_empty[kst], ph, abort_flag, limit))) { ok = false; break; }
      uint8_t *dk = sK + kst * C::TILE_BYTES;
      if constexpr (FP8) {
        store_codes(dk, raw_k);
        fence_proxy_async_smem();
        mbar_arrive(&k_full[kst]);
        next_ks = raw_ks;
        if (!last) load_codes(nx, p.kv.k, raw_k, p.kv.ks, raw_ks);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          long long slot;
          const bool in = place(it, i, cur_pages, slot);
          const int key = 16 * i + row16;
#pragma unroll
          for (int sub = 0; sub < NSUB; ++sub)
            cp_async16(dk + sub * (128 * 128) + key * 128 + ((c8 ^ (key & 7)) << 4), p.kv.k + (slot * HD + sub * 64 + c8 * 8) * 2, in);
        }
        cp_async_mbar_arrive(&k_full[kst]);
      }
      // ---- Q of a new unit, behind its first keys
      if (new_unit) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(q_empty, (units & 1) ^ 1, abort_flag, limit))) { ok = false; break; }
        const int rows = it.nt * p.G;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int r = i * 16 + row16;
          if (i * 16 >= ((rows + 127) & ~127)) break;        // the second tile is not used
          const long long base = r < rows ? paged_unit_row(p.q, p, it.s, it.b, it.t0, it.kvh, r) : 0;
          uint8_t *dst = sQ + (r >> 7) * C::TILE_BYTES + (r & 127) * 128 + ((c8 ^ (r & 7)) << 4);
#pragma unroll
          for (int sub = 0; sub < NSUB; ++sub) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < rows) {
              w = *reinterpret_cast<const uint4 *>(p.q.data + (base + sub * 64 + c8 * 8) * 2);
              if (p.q_f16) {
                uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 f = unpack_f16x2(u[e]);
                  u[e] = pack_bf16x2(f.x, f.y);
                }
              }
            }
            *reinterpret_cast<uint4 *>(dst + sub * (128 * 128)) = w;
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
        ++units;
      }
      // ---- V
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&v_empty[vst], vph, abort_flag, limit))) { ok = false; break; }
      uint8_t *dv = sV + vst * C::TILE_BYTES;
      if constexpr (FP8) {
        store_codes(dv, raw_v);
        // both scales go with V: the softmax reads them until it signals P, and V's
        // stage is free only after P V
        sSc[(vst * 2) * 128 + lt] = next_ks * p.scale_log2;
        sSc[(vst * 2 + 1) * 128 + lt] = raw_vs;
        fence_proxy_async_smem();
        mbar_arrive(&v_full[vst]);
        if (!last) load_codes(nx, p.kv.v, raw_v, p.kv.vs, raw_vs);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          long long slot;
          const bool in = place(it, i, cur_pages, slot);
          const int key = 16 * i + row16;
#pragma unroll
          for (int sub = 0; sub < NSUB; ++sub)
            cp_async16(dv + sub * (128 * 128) + key * 128 + ((c8 ^ (key & 7)) << 4), p.kv.v + (slot * HD + sub * 64 + c8 * 8) * 2, in);
        }
        cp_async_mbar_arrive(&v_full[vst]);
      }
      if (++kst == NST) {
        kst = 0;
        ph ^= 1;
      }
      vst = kst;
      vph = ph;
      if (last) break;
      new_unit = it.j + 1 == it.j1;
      it = nx;
    }
    cp_async_wait<0>();
    if (!ok) {
      if (lane == 0) set_status(p.status, kPtTimeoutLoad);
      *abort_flag = 1;
    }
  } else {
    setmaxnreg_inc<C::R_SOFTMAX>();
    // ------------------------------------------------------------------ softmax warpgroup h: rows of query tile h
    const int h = warp >> 2, r = h * 128 + (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + h * 128, tO = tmem + lanes + kColO + h * HD;
    bool ok = true, in_unit = it.j > it.j0, first = true;
    uint32_t n = 0, n_units = 0;                  // key tiles, and units, of this query tile
    int st = 0;
    uint32_t sph = 0;                             // stage and phase of the tile's scales
    PagedMeta meta{};
    float m = -INFINITY, l = 0.f;
    while (true) {
      const bool mine = h == 0 || it.nt * p.G > 128, last = it.left == 1, ends = it.j + 1 == it.j1;
      if (mine) {
        const int t = r / p.G, x0 = it.j * kTileK;
        const bool live = r < it.nt * p.G;
        const int own = live ? it.s.L + it.t0 + t : -1;
        if (first) {
          m = -INFINITY;
          l = 0.f;
        }
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_full[h], n & 1, abort_flag, limit))) { ok = false; break; }
        tc_fence_after_sync();
        uint32_t sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
        tmem_ld_wait();
        if constexpr (FP8) {
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(&v_full[st], sph, abort_flag, limit))) { ok = false; break; }
          // scores times their keys' scales (which hold scale * log2 e already)
          const float4 *sc = reinterpret_cast<const float4 *>(sSc + (st * 2) * 128);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float4 f = sc[e];
            sv[4 * e] = __float_as_uint(__uint_as_float(sv[4 * e]) * f.x);
            sv[4 * e + 1] = __float_as_uint(__uint_as_float(sv[4 * e + 1]) * f.y);
            sv[4 * e + 2] = __float_as_uint(__uint_as_float(sv[4 * e + 2]) * f.z);
            sv[4 * e + 3] = __float_as_uint(__uint_as_float(sv[4 * e + 3]) * f.w);
          }
        }
        const int first_at = it.s.L + it.t0;
        if (x0 + kTileK - 1 > first_at || (p.window > 0 && x0 <= first_at + it.nt - 1 - p.window) || it.nt * p.G < (h + 1) * 128) {
          const int hi = own - x0, lo = p.window > 0 ? own - p.window + 1 - x0 : 0;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (!(e <= hi && e >= lo)) sv[e] = 0xff800000u;
        }
        float mc[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 2)
          mc[(e >> 1) & 3] = fmax3(mc[(e >> 1) & 3], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
        float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
        if (!FP8) mx *= p.scale_log2;             // scale > 0; -inf stays -inf
        float alpha = 1.f;
        const bool grows = mx > m + 8.f && m != -INFINITY;
        if (grows) {
          alpha = ex2_approx(m - mx);
          m = mx;
        } else if (m == -INFINITY) {
          m = mx;
        }
        if (__any_sync(0xffffffffu, grows)) {
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            uint32_t ov[16];
            tmem_ld16(tO + c, ov);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st16(tO + c, ov);
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const float4 *vsc = reinterpret_cast<const float4 *>(sSc + (st * 2 + 1) * 128);
        float2 lsum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const float a = __uint_as_float(sv[half * 64 + 2 * q]), b = __uint_as_float(sv[half * 64 + 2 * q + 1]);
            float2 x;
            if constexpr (FP8) x = fadd2(a, b, -mu, -mu);
            else x = ffma2(a, b, p.scale_log2, -mu);
            x.x = ex2_approx(x.x);
            x.y = ex2_approx(x.y);
            lsum[q & 1] = fadd2(lsum[q & 1].x, lsum[q & 1].y, x.x, x.y);
            if constexpr (FP8) {
              const float4 f = vsc[half * 16 + (q >> 1)];
              x.x *= (q & 1) ? f.z : f.x;
              x.y *= (q & 1) ? f.w : f.y;
            }
            pk[q] = pack_bf16x2(x.x, x.y);        // the tensor core's operand type: half a step is 2^-9
          }
          tmem_st32(tS + half * 32, pk);
        }
        l += (lsum[0].x + lsum[0].y) + (lsum[1].x + lsum[1].y);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&p_full[h]);
        ++n;
        if (ends || last) {
          // ---- the unit (or this CTA's part of it) is done: out, or a partial result
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(&o_full[h], n_units & 1, abort_flag, limit))) { ok = false; break; }
          ++n_units;
          tc_fence_after_sync();
          const bool whole = ends && !in_unit;
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const long long at = live && whole ? paged_unit_row(p.o, p, it.s, it.b, it.t0, it.kvh, r) : 0;
          float *part = paged_part(p.ws, cta, in_unit ? 0 : 1, 256, HD);
          if (live && !whole) *reinterpret_cast<float2 *>(part + 256 * HD + 2 * r) = make_float2(m, l);
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            uint32_t ov[32];
            tmem_ld32(tO + c, ov);
            tmem_ld_wait();
            const float *f = reinterpret_cast<const float *>(ov);
            if (live && whole) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float *g = f + 8 * q;
                const uint4 w = p.q_f16 ? make_uint4(pack_f16x2(g[0] * inv, g[1] * inv), pack_f16x2(g[2] * inv, g[3] * inv),
                                                     pack_f16x2(g[4] * inv, g[5] * inv), pack_f16x2(g[6] * inv, g[7] * inv))
                                        : make_uint4(pack_bf16x2(g[0] * inv, g[1] * inv), pack_bf16x2(g[2] * inv, g[3] * inv),
                                                     pack_bf16x2(g[4] * inv, g[5] * inv), pack_bf16x2(g[6] * inv, g[7] * inv));
                *reinterpret_cast<uint4 *>(p.o.data + (at + c + 8 * q) * 2) = w;
              }
            } else if (live) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<float4 *>(part + r * HD + c + 4 * q) = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
            }
          }
          tc_fence_before_sync();                 // these reads, before the next unit's first P is signalled
        }
      }
      if (++st == NST) {
        st = 0;
        sph ^= 1;
      }
      first = ends;
      if (ends || last) {
        if (in_unit) {
          meta.in = 1;
          meta.ends = ends;
        } else if (!ends) {
          meta.out = 1;
          meta.b = it.b;
          meta.qt = it.qt;
          meta.kvh = it.kvh;
        }
        in_unit = false;
      }
      if (last) break;
      paged_next(p, it);
    }
    if (!ok) {
      if (lane == 0) set_status(p.status, kPtTimeoutSoftmax);
      *abort_flag = 1;
    }
    if (tid == 0) paged_meta(p.ws)[cta] = meta;
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool FP8>
cudaError_t launch_tiles(const PagedAttnParams &p, cudaStream_t st) {
  using C = PtCfg<HD, FP8>;
  cudaError_t e = ensure_smem_attr<paged_tiles_kernel<HD, FP8>>(C::SMEM);
  if (e != cudaSuccess) return e;
  // the register split adds up to 128 a thread: a build that starts with fewer would
  // wait for registers that never come
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, paged_tiles_kernel<HD, FP8>)) != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != 128) return cudaErrorInvalidConfiguration;
  paged_tiles_kernel<HD, FP8><<<p.ctas, C::THREADS, C::SMEM, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedAttnParams &p0, cudaStream_t st) {
  PagedAttnParams p = p0;
  p.tt = 256 / p.G;
  p.bk_shift = 7;
  if (p.kv.hd == 64) return p.kv.e4m3 ? launch_tiles<64, true>(p, st) : launch_tiles<64, false>(p, st);
  return p.kv.e4m3 ? launch_tiles<128, true>(p, st) : launch_tiles<128, false>(p, st);
}

}  // namespace smol
