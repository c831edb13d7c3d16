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
// V = 0.  e4m3 codes are copied ahead and become bf16 exactly on the way to the
// operand tiles; the keys' scales multiply the scores, the values' scales P.
//
// The loaders alone walk the schedule and leave a note of each tile beside its K:
// the walk's registers would have been spilled in the other roles (the issuing
// thread then took 140 cycles for each MMA).  Registers: 512 threads start with 128
// each; the softmax warpgroups take 184 or more (their 128 scores stay in
// registers), the loaders and the issuer give up theirs.
#include <math.h>

#include "paged_sched.cuh"

namespace smol {
namespace {

constexpr int kTileK = 128;

// What the other roles need to know of a key tile, written by the loaders with K.
struct PtInfo {
  int flags;                   // kPt*
  int x0;                      // its first position
  int first_at, rows;          // position of the unit's first row; query rows of the unit
  long long o_base;            // element offset of the unit's first row in out
  int b, qt, kvh, pad;
};
enum : int { kPtNew = 1, kPtTwo = 2, kPtUnitLast = 4, kPtEnds = 8, kPtLast = 16, kPtInUnit = 32 };

template <int HD, bool FP8>
struct PtCfg {
  static constexpr int THREADS = 512;
  static constexpr int NSUB = HD / 64;                       // 64-column sub-tiles
  static constexpr int TILE_BYTES = 128 * HD * 2;            // a Q, K or V tile, bf16
  static constexpr int NST = HD == 64 ? (FP8 ? 3 : 4) : 2;   // K and V stages
  static constexpr int SD = HD == 64 ? 3 : 1;                // tiles of codes under way (e4m3)
  static constexpr int NCH = HD / 16;                        // 16-byte pieces of codes of a tensor's tile for each loader thread
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NST * TILE_BYTES;
  static constexpr int OFF_CODES = OFF_V + NST * TILE_BYTES; // [SD][K, V][NCH][128 threads] 16 bytes
  static constexpr int OFF_CSC = OFF_CODES + (FP8 ? SD * 2 * NCH * 2048 : 0);  // [SD][K, V][128] their scales, if SD > 1
  static constexpr int OFF_SC = OFF_CSC + (FP8 && SD > 1 ? SD * 1024 : 0);     // [NST][2][128] scales of keys and values
  static constexpr int OFF_INFO = OFF_SC + (FP8 ? NST * 2 * 128 * 4 : 0);
  static constexpr int OFF_BAR = OFF_INFO + NST * sizeof(PtInfo);
  static constexpr int NBAR = 2 + 4 * NST + 2 + 2 + 2 + 1;
  static constexpr int USED = OFF_BAR + NBAR * 8 + 16;
  // the tiles want 1024-byte alignment; the block has no other shared memory, so its
  // own usually starts there (checked)
  static constexpr int SMEM = USED + 1008 <= 232448 ? USED + 1008 : 232448;
  static constexpr int R_SOFTMAX = FP8 ? 184 : 192, R_LOAD = FP8 ? 104 : 88, R_MMA = 40;
  static_assert(2 * R_SOFTMAX + R_LOAD + R_MMA <= 512, "registers of the block");
  static_assert(USED <= 232448, "shared memory per CTA");
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
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem + C::OFF_Q, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V;
  float *sSc = reinterpret_cast<float *>(smem + C::OFF_SC);
  PtInfo *sInfo = reinterpret_cast<PtInfo *>(smem + C::OFF_INFO);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *q_empty = q_full + 1;
  uint64_t *k_full = q_empty + 1, *k_empty = k_full + NST, *v_full = k_empty + NST, *v_empty = v_full + NST;
  uint64_t *s_full = v_empty + NST, *p_full = s_full + 2, *o_full = p_full + 2, *drain = o_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, cta = blockIdx.x;
  const uint64_t limit = p.wait_ns;

  griddep_launch_dependents();
  if (smem + C::USED > smem_raw + C::SMEM) {      // no room left by the alignment
    if (tid == 0) {
      set_status(p.status, kPtTimeoutLoad);
      paged_meta(p.ws)[cta] = PagedMeta{};
    }
    return;
  }
  // the schedule's scratch lies where Q will
  PagedIter it = paged_locate<C::THREADS>(p, cta, p.ctas, *reinterpret_cast<PagedSchedSmem *>(sQ));
  if (it.left == 0) {                             // the same for the whole CTA
    if (tid == 0) paged_meta(p.ws)[cta] = PagedMeta{};
    return;
  }
  if (tid == 0) {
    mbar_init(q_full, 128);
    mbar_init(q_empty, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&k_full[i], 128 + 1);             // and the note of the tile
      mbar_init(&k_empty[i], 1 + 8);              // the S MMAs, and each softmax warp has read the tile's info
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
  __syncthreads();                                // also: every thread has its copy of the schedule
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 12) {
    setmaxnreg_dec<C::R_MMA>();
    if (warp == 12) {
      // ---------------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false), kIdO = idesc_bf16_f32(128, HD, true);
      const uint64_t dq = sdesc_kmajor_sw128(smem_u32(sQ)), dk = sdesc_kmajor_sw128(smem_u32(sK));
      const uint64_t dv = sdesc_mnmajor_sw128(smem_u32(sV), 128 * 128);
      bool ok = true, any = false;
      uint32_t units = 0, n0 = 0, n1 = 0;         // Q loads, and key tiles of each query tile, so far
      int kst = 0, vst = 0;
      uint32_t kph = 0, vph = 0;
      int f_next = 0;                             // flags of the tile whose S is issued next
      auto issue_s = [&](int h) {
        if (elect_one()) {
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
      // waits for what S of the next tile needs
      auto ready_s = [&]() {
        if (!mbar_wait_bounded(&k_full[kst], kph, abort_flag, limit)) return false;
        f_next = sInfo[kst].flags;
        if (f_next & kPtNew) {
          if (!mbar_wait_bounded(q_full, units & 1, abort_flag, limit)) return false;
          ++units;
        }
        if (!FP8) fence_proxy_async_smem();       // the asynchronous copies' writes, before the tensor core reads them
        tc_fence_after_sync();
        return true;
      };
      auto done_s = [&]() {                       // S of that tile is issued for each query tile
        if (elect_one()) {
          umma_commit(&k_empty[kst]);
          if (f_next & kPtUnitLast) umma_commit(q_empty);
        }
        __syncwarp();
        if (++kst == NST) {
          kst = 0;
          kph ^= 1;
        }
      };
      ok = ready_s();
      if (ok) {
        issue_s(0);
        if (f_next & kPtTwo) issue_s(1);
        done_s();
        any = true;
      }
      while (ok) {
        const int f = f_next;
        const bool last = f & kPtLast;
        if (!mbar_wait_bounded(&v_full[vst], vph, abort_flag, limit)) { ok = false; break; }
        if (!FP8) fence_proxy_async_smem();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 0 || (f & kPtTwo)) {
            if (!mbar_wait_bounded(&p_full[h], (h ? n1 : n0) & 1, abort_flag, limit)) { ok = false; break; }
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)         // the unit's first tile: O starts at zero
                umma_f16_tmem_a(tmem + kColO + h * HD, tmem + kColS + h * 128 + k * 8, dv + ((vst * C::TILE_BYTES + k * 2048) >> 4),
                                kIdO, k > 0 || !(f & kPtNew));
              if (f & kPtUnitLast) umma_commit(&o_full[h]);
            }
            __syncwarp();
            if (h) ++n1;
            else ++n0;
          }
          if (!last) {
            if (h == 0 && !ready_s()) { ok = false; break; }
            if (h == 0 || (f_next & kPtTwo)) issue_s(h);
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit(&v_empty[vst]);
        __syncwarp();
        if (++vst == NST) {
          vst = 0;
          vph ^= 1;
        }
        if (last) break;
        done_s();
      }
      if (!ok) {
        set_status(p.status, kPtTimeoutMma);
        *abort_flag = 1;
      }
      if (any) {
        // every MMA issued is done before shared and tensor memory go
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        if (!mbar_wait_drain(drain, 0)) set_status(p.status, kPtTimeoutDrain);
      }
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<C::R_LOAD>();
    // ------------------------------------------------------------------ loaders
    const int lt = tid - 256;
    bool ok = true, in_unit = it.j > it.j0, new_unit = true;
    int st = 0;
    uint32_t ph = 1, units = 0;                   // the stages start empty
    // page numbers of a tile: lane i < 8 of each warp has that of keys 16 i ..; fetched ahead
    auto fetch_pages = [&](const PagedIter &u) {
      const int x = u.j * kTileK + 16 * (lane & 7);
      int page = -1;
      if (x < u.hi && x + 16 > u.lo) {
        page = paged_page(p.kv, u.b, x);
        if (page < 0 || page >= p.kv.P) {
          set_status(p.status, kDevBadInput);
          page = -1;
        }
      }
      return page;
    };
    auto write_info = [&](bool last) {
      if (lt == 0) {
        PtInfo f;
        const bool ends = it.j + 1 == it.j1;
        f.rows = it.nt * p.G;
        f.flags = (new_unit ? kPtNew : 0) | (f.rows > 128 ? kPtTwo : 0) | (ends || last ? kPtUnitLast : 0) | (ends ? kPtEnds : 0) |
                  (last ? kPtLast : 0) | (in_unit ? kPtInUnit : 0);
        f.x0 = it.j * kTileK;
        f.first_at = it.s.L + it.t0;
        f.o_base = paged_row_off(p.o, p.c, it.s, it.b, it.t0, it.kvh * p.G);
        f.b = it.b;
        f.qt = it.qt;
        f.kvh = it.kvh;
        sInfo[st] = f;
        mbar_arrive(&k_full[st]);
      }
    };
    // Q of the unit, both query tiles (rows past its last are zeros)
    auto load_q = [&]() {
      const int rows = it.nt * p.G, row16 = lt >> 3, c8 = lt & 7;
      const int used = (rows + 127) & ~127;
#pragma unroll 2
      for (int r = row16; r < used; r += 16) {
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
    };
    if constexpr (!FP8) {
      const int row16 = lt >> 3, c8 = lt & 7;     // row of 16, 16-byte piece of 128 bytes
      // 16 rows at a time: one page, one base address, constant steps in shared memory
      auto copy = [&](uint8_t *dst, const uint8_t *src, int pages) {
        uint8_t *row = dst + row16 * 128 + ((c8 ^ (row16 & 7)) << 4);
        const int x = it.j * kTileK + row16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int page = __shfl_sync(0xffffffffu, pages, i);
          const bool in = page >= 0 && x + 16 * i >= it.lo && x + 16 * i < it.hi;
          const uint8_t *from = src + ((in ? paged_slot(p.kv, page, x + 16 * i, it.kvh) : 0) * HD + c8 * 8) * 2;
#pragma unroll
          for (int sub = 0; sub < NSUB; ++sub) cp_async16(row + sub * (128 * 128) + i * 2048, from + sub * 128, in);
        }
      };
      int pages = fetch_pages(it);
      while (true) {
        PagedIter nx = it;
        paged_next(p, nx);
        const bool last = it.left == 1;
        const int cur = pages;
        if (!last) pages = fetch_pages(nx);       // in use from the next round on
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&k_empty[st], ph, abort_flag, limit))) { ok = false; break; }
        write_info(last);
        copy(sK + st * C::TILE_BYTES, p.kv.k, cur);
        cp_async_mbar_arrive(&k_full[st]);
        if (new_unit) {                           // Q behind the unit's first keys
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(q_empty, (units & 1) ^ 1, abort_flag, limit))) { ok = false; break; }
          load_q();
          ++units;
        }
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&v_empty[st], ph, abort_flag, limit))) { ok = false; break; }
        copy(sV + st * C::TILE_BYTES, p.kv.v, cur);
        cp_async_mbar_arrive(&v_full[st]);
        if (++st == NST) {
          st = 0;
          ph ^= 1;
        }
        if (last) break;
        new_unit = it.j + 1 == it.j1;
        if (new_unit) in_unit = false;
        it = nx;
      }
    } else {
      // codes go to this thread's own places in shared memory SD tiles ahead of their
      // conversion (in registers the prefetch spilled); piece i is keys i * RPP + frow
      constexpr int SD = C::SD, NCH = C::NCH, RPP = 128 / NCH;
      const int frow = lt / NCH, fc = lt % NCH;   // a row's hd bytes are NCH pieces
      uint8_t *codes = smem + C::OFF_CODES + lt * 16;
      // the scales of key lt go the same way; with one tile ahead they wait in registers
      // (shared memory is full) and are fetched behind the last ones' use
      float *codes_sc = reinterpret_cast<float *>(smem + C::OFF_CSC) + lt;
      [[maybe_unused]] float ks = 0.f, vs = 0.f;
      PagedIter ahead = it;
      int slot = 0;
      // (K or V of) tile `ahead` under way
      auto fetch = [&](int which, const uint8_t *src, const float *sc, int pages) {
        uint8_t *dst = codes + (slot * 2 + which) * NCH * 2048;
        const int x0 = ahead.j * kTileK;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int key = i * RPP + frow, x = x0 + key;
          const int page = __shfl_sync(0xffffffffu, pages, key >> 4);
          const bool in = page >= 0 && x >= ahead.lo && x < ahead.hi;
          cp_async16(dst + i * 2048, src + (in ? paged_slot(p.kv, page, x, ahead.kvh) * HD + fc * 16 : 0), in);
        }
        if constexpr (SD > 1) {
          const int page = __shfl_sync(0xffffffffu, pages, lt >> 4);
          const bool in = page >= 0 && x0 + lt >= ahead.lo && x0 + lt < ahead.hi;
          cp_async4(codes_sc + (slot * 2 + which) * 128, sc + (in ? paged_slot(p.kv, page, x0 + lt, ahead.kvh) : 0), in);
        }
        cp_async_commit();
      };
      auto fetch_scales = [&](int pages) {
        const int x = ahead.j * kTileK + lt;
        const int page = __shfl_sync(0xffffffffu, pages, lt >> 4);
        const bool in = page >= 0 && x >= ahead.lo && x < ahead.hi;
        const long long at = in ? paged_slot(p.kv, page, x, ahead.kvh) : 0;
        ks = in ? __ldg(p.kv.ks + at) : 0.f;
        vs = in ? __ldg(p.kv.vs + at) : 0.f;
      };
      auto convert = [&](uint8_t *dst, int which, int at) {
        const uint8_t *src = codes + (at * 2 + which) * NCH * 2048;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int key = i * RPP + frow, ch = fc * 2;       // two pieces of 8 bf16
          const uint4 w = *reinterpret_cast<const uint4 *>(src + i * 2048);
          uint8_t *row = dst + (ch >> 3) * (128 * 128) + key * 128;
          *reinterpret_cast<uint4 *>(row + (((ch & 7) ^ (key & 7)) << 4)) = pt_codes8(w.x, w.y);
          *reinterpret_cast<uint4 *>(row + ((((ch + 1) & 7) ^ (key & 7)) << 4)) = pt_codes8(w.z, w.w);
        }
        fence_proxy_async_smem();
      };
      int pages = fetch_pages(ahead);
#pragma unroll
      for (int d = 0; d < SD; ++d) {
        if (ahead.left > 0) {
          fetch(0, p.kv.k, p.kv.ks, pages);
          fetch(1, p.kv.v, p.kv.vs, pages);
          if (SD == 1) fetch_scales(pages);
          paged_next(p, ahead);
          if (ahead.left > 0) pages = fetch_pages(ahead);
        } else {
          cp_async_commit();
          cp_async_commit();
        }
        slot = slot + 1 == SD ? 0 : slot + 1;
      }
      while (true) {
        const bool last = it.left == 1, more = ahead.left > 0;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&k_empty[st], ph, abort_flag, limit))) { ok = false; break; }
        write_info(last);
        cp_async_wait<2 * SD - 1>();              // this thread's codes of K
        convert(sK + st * C::TILE_BYTES, 0, slot);
        mbar_arrive(&k_full[st]);
        if (more) fetch(0, p.kv.k, p.kv.ks, pages);
        else cp_async_commit();
        if (new_unit) {                           // Q behind the unit's first keys
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(q_empty, (units & 1) ^ 1, abort_flag, limit))) { ok = false; break; }
          load_q();
          ++units;
        }
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&v_empty[st], ph, abort_flag, limit))) { ok = false; break; }
        cp_async_wait<2 * SD - 1>();              // of V
        // both scales go with V: the softmax reads them until it signals P, and V's
        // stage is free only after P V
        if (SD > 1) {
          ks = codes_sc[slot * 256];
          vs = codes_sc[slot * 256 + 128];
        }
        sSc[(st * 2) * 128 + lt] = ks * p.scale_log2;
        sSc[(st * 2 + 1) * 128 + lt] = vs;
        convert(sV + st * C::TILE_BYTES, 1, slot);
        mbar_arrive(&v_full[st]);
        if (more) {
          fetch(1, p.kv.v, p.kv.vs, pages);
          if (SD == 1) fetch_scales(pages);
          paged_next(p, ahead);
          if (ahead.left > 0) pages = fetch_pages(ahead);
        } else {
          cp_async_commit();
        }
        slot = slot + 1 == SD ? 0 : slot + 1;
        if (++st == NST) {
          st = 0;
          ph ^= 1;
        }
        if (last) break;
        new_unit = it.j + 1 == it.j1;
        if (new_unit) in_unit = false;
        paged_next(p, it);
      }
    }
    cp_async_wait<0>();
    if (!ok) {
      if (lane == 0) set_status(p.status, kPtTimeoutLoad);
      *abort_flag = 1;
    }
  } else {
    setmaxnreg_inc<C::R_SOFTMAX>();
    // ------------------------------------------------------------------ softmax warpgroup h: rows of query tile h
    const int h = warp >> 2, r0 = h * 128 + (warp & 3) * 32, r = r0 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + h * 128, tO = tmem + lanes + kColO + h * HD;
    const int tok = r / p.G, head = r - tok * p.G;
    bool ok = true;
    uint32_t n = 0, n_units = 0;                  // key tiles, and units, of this query tile
    int st = 0;
    uint32_t ph = 0;                              // stage and phase of the tile
    PagedMeta meta{};
    float m = -INFINITY, l = 0.f;
    while (true) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&k_full[st], ph, abort_flag, limit))) { ok = false; break; }
      const PtInfo &info = sInfo[st];
      const int f = info.flags, x0 = info.x0, first_at = info.first_at, rows = info.rows;
      const long long o_base = info.o_base;
      if (tid == 0 && (f & kPtUnitLast)) {
        if (f & kPtInUnit) {
          meta.in = 1;
          meta.ends = (f & kPtEnds) != 0;
        } else if (!(f & kPtEnds)) {
          meta.out = 1;
          meta.b = info.b;
          meta.qt = info.qt;
          meta.kvh = info.kvh;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_empty[st]);   // the info may be overwritten
      if (h == 0 || (f & kPtTwo)) {
        const bool work = r0 < rows;              // a warp without rows leaves P as it is: it reaches no other row
        if (f & kPtNew) {
          m = -INFINITY;
          l = 0.f;
        }
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_full[h], n & 1, abort_flag, limit))) { ok = false; break; }
        tc_fence_after_sync();
        if (work) {
          uint32_t sv[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
          tmem_ld_wait();
          if constexpr (FP8) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&v_full[st], ph, abort_flag, limit))) { ok = false; break; }
            // scores times their keys' scales (which hold scale * log2 e already)
            const float4 *sc = reinterpret_cast<const float4 *>(sSc + (st * 2) * 128);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float4 k4 = sc[e];
              const float2 a = fmul2(__uint_as_float(sv[4 * e]), __uint_as_float(sv[4 * e + 1]), k4.x, k4.y);
              const float2 b = fmul2(__uint_as_float(sv[4 * e + 2]), __uint_as_float(sv[4 * e + 3]), k4.z, k4.w);
              sv[4 * e] = __float_as_uint(a.x);
              sv[4 * e + 1] = __float_as_uint(a.y);
              sv[4 * e + 2] = __float_as_uint(b.x);
              sv[4 * e + 3] = __float_as_uint(b.y);
            }
          }
          const int own = first_at + tok;         // past the unit's rows: a row that is not written
          if (x0 + kTileK - 1 > first_at || (p.window > 0 && x0 <= first_at + (rows - 1) / p.G - p.window)) {
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
          if (!FP8) mx *= p.scale_log2;           // scale > 0; -inf stays -inf
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
                const float4 v4 = vsc[half * 16 + (q >> 1)];
                x = (q & 1) ? fmul2(x.x, x.y, v4.z, v4.w) : fmul2(x.x, x.y, v4.x, v4.y);
              }
              pk[q] = pack_bf16x2(x.x, x.y);      // the tensor core's operand type: off by 2^-9 at most
            }
            tmem_st32(tS + half * 32, pk);
          }
          l += (lsum[0].x + lsum[0].y) + (lsum[1].x + lsum[1].y);
          tmem_st_wait();
        }
        tc_fence_before_sync();
        mbar_arrive(&p_full[h]);
        ++n;
        if (f & kPtUnitLast) {
          // ---- the unit (or this CTA's part of it) is done: out, or a partial result
          if (!__all_sync(0xffffffffu, mbar_wait_bounded(&o_full[h], n_units & 1, abort_flag, limit))) { ok = false; break; }
          ++n_units;
          tc_fence_after_sync();
          if (work) {
            const bool whole = (f & (kPtEnds | kPtInUnit)) == kPtEnds, live = r < rows;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const long long at = o_base + tok * p.o.row + head * p.o.head;
            float *part = paged_part(p.ws, cta, f & kPtInUnit ? 0 : 1, 256, HD);
            if (live && !whole) *reinterpret_cast<float2 *>(part + 256 * HD + 2 * r) = make_float2(m, l);
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              uint32_t ov[32];
              tmem_ld32(tO + c, ov);
              tmem_ld_wait();
              const float *o = reinterpret_cast<const float *>(ov);
              if (live && whole) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float *g = o + 8 * q;
                  const uint4 w = p.q_f16 ? make_uint4(pack_f16x2(g[0] * inv, g[1] * inv), pack_f16x2(g[2] * inv, g[3] * inv),
                                                       pack_f16x2(g[4] * inv, g[5] * inv), pack_f16x2(g[6] * inv, g[7] * inv))
                                          : make_uint4(pack_bf16x2(g[0] * inv, g[1] * inv), pack_bf16x2(g[2] * inv, g[3] * inv),
                                                       pack_bf16x2(g[4] * inv, g[5] * inv), pack_bf16x2(g[6] * inv, g[7] * inv));
                  *reinterpret_cast<uint4 *>(p.o.data + (at + c + 8 * q) * 2) = w;
                }
              } else if (live) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  *reinterpret_cast<float4 *>(part + r * HD + c + 4 * q) = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
              }
            }
          }
          tc_fence_before_sync();                 // these reads, before the next unit's first P is signalled
        }
      }
      if (f & kPtLast) break;
      if (++st == NST) {
        st = 0;
        ph ^= 1;
      }
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
