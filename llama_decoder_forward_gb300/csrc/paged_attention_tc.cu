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
// K and V of bf16 pages, and Q, come by TMA straight into the swizzled operand
// layout: a box for each page of a key tile (up to 128 of its rows), the tokens and
// heads of the unit for Q.  A page number outside the pool is a coordinate outside
// the tensor: zeros.  Where a tile reaches past what the unit's rows see, a second
// warp sets V's rows there to zero before the tensor core reads them: whatever lies
// in unused slots, P = 0 meets V = 0.  (Copies by the loader's threads, 16 bytes
// each, took 4,600 cycles for a tile of 64 KB: more than its 32 MMAs.)
// e4m3 codes are copied ahead by bulk copies, as they lie, and four warps turn them
// into bf16 on the way to the operand tiles, exactly; the keys' scales multiply the
// scores, the values' scales P.
//
// One warp alone walks the schedule for the MMA issuer and the softmax, and leaves a
// note of each tile beside its K: the walk's registers would have been spilled in
// those roles.  Registers: 512 threads start with 128 each; the softmax warpgroups
// take 184 or more (their 128 scores stay in registers), the others give up theirs.
// NQ: query tiles of a unit; a call whose units have at most 128 rows leaves the
// second tile's shared memory to more stages.
#include <math.h>

#include "paged_sched.cuh"

namespace smol {
namespace {

constexpr int kTileK = 128;

// What the other roles need to know of a key tile, written by the loader with K.
struct PtInfo {
  int flags;                   // kPt*
  int x0;                      // its first position
  int first_at, rows;          // position of the unit's first row; query rows of the unit
  long long o_base;            // element offset of the unit's first row in out
  int b, qt, kvh;
  int valid;                   // first and behind the last of its keys that some row sees (16 bits each)
};
enum : int { kPtNew = 1, kPtTwo = 2, kPtUnitLast = 4, kPtEnds = 8, kPtLast = 16, kPtInUnit = 32, kPtEdge = 64 };

// The loader's note of a tile of codes, in the slot's place.
struct PtCodes {
  PtInfo info;
  int page[8];                 // pages of the tile's keys
};

template <int HD, bool FP8, int NQ>
struct PtCfg {
  static constexpr int THREADS = 512;
  static constexpr int NSUB = HD / 64;                       // 64-column sub-tiles
  static constexpr int TILE_BYTES = 128 * HD * 2;            // a K or V tile, bf16
  static constexpr int NST = HD == 64 ? 4 : (NQ == 1 && !FP8) ? 3 : 2;   // K and V stages
  static constexpr int SD = HD == 64 ? 3 : NQ == 1 ? 2 : 1;  // tiles of codes under way (e4m3)
  static constexpr int OFF_Q = 0;                            // [NSUB][NQ * 128 rows][64]
  static constexpr int OFF_K = NQ * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NST * TILE_BYTES;
  static constexpr int OFF_CODES = OFF_V + NST * TILE_BYTES; // [SD][K, V][128 keys][HD]
  static constexpr int OFF_SC = OFF_CODES + (FP8 ? SD * 2 * 128 * HD : 0);     // [NST][2][128] scales of keys and values
  static constexpr int OFF_INFO = OFF_SC + (FP8 ? NST * 2 * 128 * 4 : 0);
  static constexpr int OFF_NOTE = OFF_INFO + NST * sizeof(PtInfo);
  static constexpr int OFF_BAR = OFF_NOTE + (FP8 ? SD * sizeof(PtCodes) : 0);
  static constexpr int NBAR = 2 + 5 * NST + 4 * SD + 2 + 2 + 2 + 1;
  static constexpr int USED = OFF_BAR + NBAR * 8 + 16;
  // the tiles want 1024-byte alignment; the block has no other shared memory, so its
  // own usually starts there (checked)
  static constexpr int SMEM = USED + 1008 <= 232448 ? USED + 1008 : 232448;
  static constexpr int R_SOFTMAX = FP8 ? 176 : 192, R_LOAD = FP8 ? 80 : 88, R_MMA = FP8 ? 80 : 40;
  static_assert(2 * R_SOFTMAX + R_LOAD + R_MMA <= 512, "registers of the block");
  static_assert(USED <= 232448, "shared memory per CTA");
};

enum : int { kPtTimeoutLoad = 0x205, kPtTimeoutMma = 0x206, kPtTimeoutSoftmax = 0x207, kPtTimeoutDrain = 0x208 };

constexpr uint32_t kColS = 0, kColO = 256;                   // tensor memory columns: S (and P), O

// Eight codes (two words) to eight bf16, exactly.
__device__ __forceinline__ uint4 pt_codes8(uint32_t a, uint32_t b) {
  const float2 f0 = unpack_e4m3x2(a), f1 = unpack_e4m3x2(a >> 16), f2 = unpack_e4m3x2(b), f3 = unpack_e4m3x2(b >> 16);
  return make_uint4(pack_bf16x2(f0.x, f0.y), pack_bf16x2(f1.x, f1.y), pack_bf16x2(f2.x, f2.y), pack_bf16x2(f3.x, f3.y));
}

template <int HD, bool FP8, int NQ>
__global__ void __launch_bounds__(512, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PagedAttnParams p) {
  using C = PtCfg<HD, FP8, NQ>;
  constexpr int NST = C::NST, NSUB = C::NSUB, SD = C::SD;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem + C::OFF_Q, *sK = smem + C::OFF_K, *sV = smem + C::OFF_V;
  float *sSc = reinterpret_cast<float *>(smem + C::OFF_SC);
  PtInfo *sInfo = reinterpret_cast<PtInfo *>(smem + C::OFF_INFO);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *q_empty = q_full + 1;
  uint64_t *k_full = q_empty + 1, *k_empty = k_full + NST, *v_full = k_empty + NST, *v_empty = v_full + NST;
  uint64_t *v_raw = v_empty + NST, *c_full = v_raw + NST;   // V landed but not yet cleared; codes of K and V landed [SD][2]
  uint64_t *c_empty = c_full + 2 * SD;            // and read by the four converting warps
  uint64_t *s_full = c_empty + 2 * SD, *p_full = s_full + 2, *o_full = p_full + 2, *drain = o_full + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, cta = blockIdx.x;
  const uint64_t limit = p.wait_ns;
  // the other roles' warps give up as one: their lanes go on to instructions of the whole warp
  auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, limit)); };

  griddep_launch_dependents();
  if (smem + C::USED > smem_raw + C::SMEM) {      // no room left by the alignment
    if (tid == 0) {
      set_status(p.status, kPtTimeoutLoad);
      paged_meta(p.ws)[cta] = PagedMeta{};
    }
    return;
  }
  if (tid == 0) {
    tma_prefetch_desc(&tmQ);
    if (!FP8) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  // the schedule's scratch lies where Q will
  PagedIter it = paged_locate<C::THREADS>(p, cta, p.ctas, *reinterpret_cast<PagedSchedSmem *>(sQ));
  if (it.left == 0) {                             // the same for the whole CTA
    if (tid == 0) paged_meta(p.ws)[cta] = PagedMeta{};
    return;
  }
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(&k_full[i], FP8 ? 128 : 1);
      mbar_init(&k_empty[i], FP8 ? 1 + 8 : 1 + 9);   // the S MMAs, and each reader of the tile's note
      mbar_init(&v_full[i], FP8 ? 128 : 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&v_raw[i], 1);
    }
    for (int i = 0; i < 2 * SD; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], 4);
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

  // ---- what the loading warps share
  const int box = min(1 << p.kv.page_shift, kTileK), n_box = kTileK / box;   // rows of a page in a tile, pages of a tile
  // page numbers of a tile: lane i < n_box of the warp has that of keys i * box ..; -1: not in
  // sight, P: no such page
  auto fetch_pages = [&](const PagedIter &u) {
    const int x = u.j * kTileK + box * lane;
    int page = -1;
    if (lane < n_box && x < u.hi && x + box > u.lo) {
      page = paged_page(p.kv, u.b, x);
      if (page < 0 || page >= p.kv.P) {
        set_status(p.status, kDevBadInput);
        page = p.kv.P;
      }
    }
    return page;
  };
  auto note_of = [&](const PagedIter &it, bool new_unit, bool in_unit) {
    PtInfo f;
    const bool last = it.left == 1;
    const bool ends = it.j + 1 == it.j1;
    f.x0 = it.j * kTileK;
    f.rows = it.nt * p.G;
    f.valid = max(0, it.lo - f.x0) | (min(kTileK, it.hi - f.x0) << 16);
    f.flags = (new_unit ? kPtNew : 0) | (f.rows > 128 ? kPtTwo : 0) | (ends || last ? kPtUnitLast : 0) | (ends ? kPtEnds : 0) |
              (last ? kPtLast : 0) | (in_unit ? kPtInUnit : 0) | (f.valid != kTileK << 16 ? kPtEdge : 0);
    f.first_at = it.s.L + it.t0;
    f.o_base = paged_row_off(p.o, p.c, it.s, it.b, it.t0, it.kvh * p.G);
    f.b = it.b;
    f.qt = it.qt;
    f.kvh = it.kvh;
    return f;
  };
  // Q of the unit: its tokens' heads are the rows, in both tiles (rows past the sequence's last
  // are whatever follows them, or zeros: they reach no other row)
  auto load_q = [&](const PagedIter &it) {        // one lane
    mbar_arrive_expect_tx(q_full, NSUB * 128 * p.tt * p.G);
#pragma unroll
    for (int sub = 0; sub < NSUB; ++sub)
      tma_load_4d(sQ + sub * (NQ * 128 * 128), &tmQ, q_full, sub * 64, it.kvh * p.G, static_cast<int>(it.s.row0) + it.t0,
                  p.c.row_start ? 0 : it.b);
  };

  if (warp >= 12) {
    setmaxnreg_dec<C::R_MMA>();
    if (warp == 12 && elect_one()) {
      // ---------------------------------------------------------------- MMA issuer: one thread, which
      // gives up by itself (as a warp with votes: 2048 tokens on 32,000 449 us, so 426)
      auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, abort_flag, limit); };
      constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, false), kIdO = idesc_bf16_f32(128, HD, true);
      const uint64_t dq = sdesc_kmajor_sw128(smem_u32(sQ)), dk = sdesc_kmajor_sw128(smem_u32(sK));
      const uint64_t dv = sdesc_mnmajor_sw128(smem_u32(sV), 128 * 128);
      bool ok = true, any = false;
      uint32_t units = 0, n0 = 0, n1 = 0;         // Q loads, and key tiles of each query tile, so far
      int kst = 0, vst = 0;
      uint32_t kph = 0, vph = 0;
      int f_next = 0;                             // flags of the tile whose S is issued next
      auto issue_s = [&](int h) {
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint64_t a = dq + (((k >> 2) * (NQ * 128 * 128) + h * (128 * 128) + (k & 3) * 32) >> 4);
          const uint64_t b = dk + ((kst * C::TILE_BYTES + (k >> 2) * (128 * 128) + (k & 3) * 32) >> 4);
          umma_f16(tmem + kColS + h * 128, a, b, kIdS, k > 0);
        }
        umma_commit(&s_full[h]);
      };
      // waits for what S of the next tile needs
      auto ready_s = [&]() {
        if (!wait(&k_full[kst], kph)) return false;
        f_next = sInfo[kst].flags;
        if (f_next & kPtNew) {
          if (!wait(q_full, units & 1)) return false;
          ++units;
        }
        tc_fence_after_sync();
        return true;
      };
      auto done_s = [&]() {                       // S of that tile is issued for each query tile
        umma_commit(&k_empty[kst]);
        if (f_next & kPtUnitLast) umma_commit(q_empty);
        if (++kst == NST) {
          kst = 0;
          kph ^= 1;
        }
      };
      // the one wait that keeps a short limit, outside the loop; the other roles then see the abort
      // flag.  (Its code at all twenty waits: 24 packed chunks 332 to 347 us for 288 to 300, 2048
      // tokens on 32,000 484 for 451, for the instructions to fetch; in the issuer's loop 462.)
      ok = mbar_wait_limit(&k_full[0], 0, abort_flag, limit) && ready_s();
      if (ok) {
        issue_s(0);
        if (f_next & kPtTwo) issue_s(1);
        done_s();
        any = true;
      }
      while (ok) {
        const int f = f_next;
        const bool last = f & kPtLast;
        if (!wait(&v_full[vst], vph)) { ok = false; break; }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 0 || (f & kPtTwo)) {
            if (!wait(&p_full[h], (h ? n1 : n0) & 1)) { ok = false; break; }
            tc_fence_after_sync();
#pragma unroll
            for (int k = 0; k < 8; ++k)           // the unit's first tile: O starts at zero
              umma_f16_tmem_a(tmem + kColO + h * HD, tmem + kColS + h * 128 + k * 8, dv + ((vst * C::TILE_BYTES + k * 2048) >> 4),
                              kIdO, k > 0 || !(f & kPtNew));
            if (f & kPtUnitLast) umma_commit(&o_full[h]);
            if (h) ++n1;
            else ++n0;
          }
          if (!last) {
            if (h == 0 && !ready_s()) { ok = false; break; }
            if (h == 0 || (f_next & kPtTwo)) issue_s(h);
          }
        }
        if (!ok) break;
        umma_commit(&v_empty[vst]);
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
        umma_commit(drain);
        if (!mbar_wait_drain(drain, 0)) set_status(p.status, kPtTimeoutDrain);
      }
    }
    if (FP8 && warp == 13) {
      // ---------------------------------------------------------------- codes on their way, SD tiles ahead
      bool ok = true, in_unit = it.j > it.j0, new_unit = true;
      int slot = 0;
      uint32_t cph = 1, n = 0, units = 0;         // the slots start empty
      uint8_t *codes = smem + C::OFF_CODES;
      PtCodes *notes = reinterpret_cast<PtCodes *>(smem + C::OFF_NOTE);
      auto fetch = [&](int which, const uint8_t *src, int page) {
        const bool mine = page >= 0 && page < p.kv.P;
        const unsigned in = __ballot_sync(0xffffffffu, mine);
        uint64_t *bar = &c_full[slot * 2 + which];
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(in) * box * HD);
        __syncwarp();
        if (mine)
          bulk_load(codes + (slot * 2 + which) * 128 * HD + lane * box * HD,
                    src + paged_slot(p.kv, page, it.j * kTileK + lane * box, it.kvh) * HD, box * HD, bar);
        __syncwarp();
      };
      int pages = fetch_pages(it);
      while (true) {
        PagedIter nx = it;
        paged_next(p, nx);
        const bool last = it.left == 1;
        const int cur = pages;
        if (!last) pages = fetch_pages(nx);       // in use from the next round on
        if (!wait(&c_empty[slot * 2], cph)) { ok = false; break; }
        if (!wait(&c_empty[slot * 2 + 1], cph)) { ok = false; break; }
        if (lane < 8) notes[slot].page[lane] = cur;
        if (lane == 0) notes[slot].info = note_of(it, new_unit, in_unit);
        __syncwarp();                             // before lane 0's arrivals
        fetch(0, p.kv.k, cur);
        fetch(1, p.kv.v, cur);
        ++n;
        if (new_unit) {                           // Q behind the unit's first keys
          if (!wait(q_empty, (units & 1) ^ 1)) { ok = false; break; }
          if (lane == 0) load_q(it);
          __syncwarp();
          ++units;
        }
        if (++slot == SD) {
          slot = 0;
          cph ^= 1;
        }
        if (last) break;
        new_unit = it.j + 1 == it.j1;
        if (new_unit) in_unit = false;
        it = nx;
      }
      if (!ok) {
        if (lane == 0) set_status(p.status, kPtTimeoutLoad);
        *abort_flag = 1;
      }
      // what this warp has asked for lands before the block's shared memory goes, also where it
      // came to its end and the warps that would have waited gave up
      bool done = units == 0 || mbar_wait_drain(q_full, (units - 1) & 1);
      for (uint32_t k = n > SD ? n - SD : 0; k < n; ++k)
        for (int w = 0; w < 2; ++w) done &= mbar_wait_drain(&c_full[(k % SD) * 2 + w], (k / SD) & 1);
      if (!done && lane == 0) set_status(p.status, kPtTimeoutDrain);
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<C::R_LOAD>();
    // ------------------------------------------------------------------ loaders
    bool ok = true;
    int st = 0;
    uint32_t ph = 1;                              // the stages start empty
    if constexpr (!FP8) {
      if (warp == 8) {
        bool in_unit = it.j > it.j0, new_unit = true;
        uint32_t units = 0;
        // a box for each page and 64 columns; every lane issues its own page's
        auto copy = [&](uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int page) {
          const unsigned in = __ballot_sync(0xffffffffu, page >= 0);
          if (lane == 0) mbar_arrive_expect_tx(bar, __popc(in) * box * HD * 2);
          __syncwarp();
          if (page >= 0) {
            const int y = (it.kvh << p.kv.page_shift) + ((it.j * kTileK) & ((1 << p.kv.page_shift) - 1));
#pragma unroll
            for (int sub = 0; sub < NSUB; ++sub) tma_load_3d(dst + sub * (128 * 128) + lane * box * 128, map, bar, sub * 64, y, page);
          }
          __syncwarp();
        };
        int pages = fetch_pages(it);
        uint32_t nk = 0, nv = 0, edges = 0, raw = 0;   // tiles asked for; stages whose V went to v_raw, and its phase
        while (true) {
          PagedIter nx = it;
          paged_next(p, nx);
          const bool last = it.left == 1;
          const int cur = pages;
          if (!last) pages = fetch_pages(nx);     // in use from the next round on
          if (!wait(&k_empty[st], ph)) { ok = false; break; }
          if (lane == 0) sInfo[st] = note_of(it, new_unit, in_unit);   // before this lane's arrival in copy()
          copy(sK + st * C::TILE_BYTES, &tmK, &k_full[st], cur);
          ++nk;
          if (new_unit) {                         // Q behind the unit's first keys
            if (!wait(q_empty, (units & 1) ^ 1)) { ok = false; break; }
            if (lane == 0) load_q(it);
            __syncwarp();
            ++units;
          }
          if (!wait(&v_empty[st], ph)) { ok = false; break; }
          const bool edge = it.lo > it.j * kTileK || it.hi < (it.j + 1) * kTileK;
          copy(sV + st * C::TILE_BYTES, &tmV, edge ? &v_raw[st] : &v_full[st], cur);
          ++nv;
          edges = (edges & ~(1u << st)) | (edge ? 1u << st : 0u);
          if (edge) raw ^= 1u << st;
          if (++st == NST) {
            st = 0;
            ph ^= 1;
          }
          if (last) break;
          new_unit = it.j + 1 == it.j1;
          if (new_unit) in_unit = false;
          it = nx;
        }
        if (!ok) {
          if (lane == 0) set_status(p.status, kPtTimeoutLoad);
          *abort_flag = 1;
        }
        // what this warp has asked for lands before the block's shared memory goes, also where it
        // came to its end and the warps that would have waited gave up
        bool done = units == 0 || mbar_wait_drain(q_full, (units - 1) & 1);
        for (uint32_t n = nk > NST ? nk - NST : 0; n < nk; ++n) done &= mbar_wait_drain(&k_full[n % NST], (n / NST) & 1);
        for (uint32_t n = nv > NST ? nv - NST : 0; n < nv; ++n) {
          const uint32_t s = n % NST;
          done &= (edges >> s) & 1 ? mbar_wait_drain(&v_raw[s], ((raw >> s) & 1) ^ 1) : mbar_wait_drain(&v_full[s], (n / NST) & 1);
        }
        if (!done && lane == 0) set_status(p.status, kPtTimeoutDrain);
      } else if (warp == 9) {
        // V of tiles that reach past what the unit's rows see: zeros there
        uint32_t raw = 0;                         // phase of each stage's v_raw
        ph = 0;
        while (true) {
          if (!wait(&k_full[st], ph)) { ok = false; break; }
          const int f = sInfo[st].flags, valid = sInfo[st].valid;
          __syncwarp();
          if (lane == 0) mbar_arrive(&k_empty[st]);
          if (f & kPtEdge) {
            if (!wait(&v_raw[st], (raw >> st) & 1)) { ok = false; break; }
            raw ^= 1u << st;
            const int from = valid & 0xffff, to = valid >> 16, gone = 128 - (to - from);
            for (int i = lane; i < gone * 8 * NSUB; i += 32) {
              int key = (i >> 3) % gone;
              const int sub = (i >> 3) / gone;
              if (key >= from) key += to - from;
              *reinterpret_cast<uint4 *>(sV + st * C::TILE_BYTES + sub * (128 * 128) + key * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[st]);
          }
          if (++st == NST) {
            st = 0;
            ph ^= 1;
          }
          if (f & kPtLast) break;
        }
        if (!ok) {
          if (lane == 0) set_status(p.status, kPtTimeoutLoad);
          *abort_flag = 1;
        }
      }
    } else {
      // ---- codes of a slot to the operand tiles
      constexpr int NCH = HD / 16, RPP = 128 / NCH;   // 16-byte pieces of a key's codes; keys of a pass
      const int lt = tid - 256, frow = lt / NCH, fc = lt % NCH;   // this thread's key of a pass, and piece
      const uint8_t *codes = smem + C::OFF_CODES + lt * 16;
      // where its two pieces of 8 bf16 go; hd 128: the upper half writes them in the other
      // order, so that the halves' stores meet different banks
      const int swap = HD == 128 ? fc >> 2 : 0;
      const uint32_t to0 = ((fc * 2) >> 3) * (128 * 128) + frow * 128 + (((fc * 2 + swap) & 7) ^ (frow & 7)) * 16;
      const uint32_t to1 = ((fc * 2) >> 3) * (128 * 128) + frow * 128 + (((fc * 2 + 1 - swap) & 7) ^ (frow & 7)) * 16;
      int slot = 0;
      uint32_t cph = 0;
      auto convert = [&](uint8_t *dst, int which, int valid, bool edge) {
        const uint8_t *src = codes + (slot * 2 + which) * 128 * HD;
        const int from = valid & 0xffff, to = valid >> 16;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          uint4 w = *reinterpret_cast<const uint4 *>(src + i * 2048);
          // keys out of sight: zeros, whatever is there
          if (edge && (i * RPP + frow < from || i * RPP + frow >= to)) w = make_uint4(0, 0, 0, 0);
          const uint4 a = pt_codes8(w.x, w.y), b = pt_codes8(w.z, w.w);
          *reinterpret_cast<uint4 *>(dst + to0 + i * RPP * 128) = swap ? b : a;
          *reinterpret_cast<uint4 *>(dst + to1 + i * RPP * 128) = swap ? a : b;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c_empty[slot * 2 + which]);
      };
      while (true) {
        if (!wait(&c_full[slot * 2], cph)) { ok = false; break; }
        const PtCodes &note = reinterpret_cast<const PtCodes *>(smem + C::OFF_NOTE)[slot];
        const int valid = note.info.valid, f = note.info.flags, page = note.page[lt / box];
        const bool edge = f & kPtEdge, in = page >= 0 && page < p.kv.P && lt >= (valid & 0xffff) && lt < valid >> 16;
        const long long at = in ? paged_slot(p.kv, page, note.info.x0 + lt, note.info.kvh) : 0;
        const float ks = in ? __ldg(p.kv.ks + at) : 0.f, vs = in ? __ldg(p.kv.vs + at) : 0.f;   // of key lt, for later
        if (!wait(&k_empty[st], ph)) { ok = false; break; }
        if (lt == 0) sInfo[st] = note.info;
        convert(sK + st * C::TILE_BYTES, 0, valid, edge);
        mbar_arrive(&k_full[st]);
        if (!wait(&c_full[slot * 2 + 1], cph)) { ok = false; break; }
        if (!wait(&v_empty[st], ph)) { ok = false; break; }
        // both scales go with V: the softmax reads them until it signals P, and V's
        // stage is free only after P V
        sSc[(st * 2) * 128 + lt] = ks * p.scale_log2;
        sSc[(st * 2 + 1) * 128 + lt] = vs;
        convert(sV + st * C::TILE_BYTES, 1, valid, edge);
        mbar_arrive(&v_full[st]);
        if (++slot == SD) {
          slot = 0;
          cph ^= 1;
        }
        if (++st == NST) {
          st = 0;
          ph ^= 1;
        }
        if (f & kPtLast) break;
      }
      if (!ok) {
        if (lane == 0) set_status(p.status, kPtTimeoutLoad);
        *abort_flag = 1;
      }
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
      if (!wait(&k_full[st], ph)) { ok = false; break; }
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
        if (!wait(&s_full[h], n & 1)) { ok = false; break; }
        tc_fence_after_sync();
        if (work) {
          uint32_t sv[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
          tmem_ld_wait();
          if constexpr (FP8) {
            if (!wait(&v_full[st], ph)) { ok = false; break; }
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
              pk[q] = pack_bf16x2(x.x, x.y);      // the tensor core's operand type: off by 2^-8 of the value at most
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
          if (!wait(&o_full[h], n_units & 1)) { ok = false; break; }
          ++n_units;
          tc_fence_after_sync();
          if (work) {
            const bool whole = (f & (kPtEnds | kPtInUnit)) == kPtEnds, live = r < rows;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const long long at = o_base + tok * p.o.row + head * p.o.head;
            float *part = paged_part(p.ws, cta, f & kPtInUnit ? 0 : 1, NQ * 128, HD);
            if (live && !whole) *reinterpret_cast<float2 *>(part + NQ * 128 * HD + 2 * r) = make_float2(m, l);
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
                  const uint4 w = p.o_f16 ? make_uint4(pack_f16x2(g[0] * inv, g[1] * inv), pack_f16x2(g[2] * inv, g[3] * inv),
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
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool FP8, int NQ>
cudaError_t launch_tiles(const PagedAttnParams &p, cudaStream_t st) {
  using C = PtCfg<HD, FP8, NQ>;
  cudaError_t e = ensure_smem_attr<paged_tiles_kernel<HD, FP8, NQ>>(C::SMEM);
  if (e != cudaSuccess) return e;
  // the register split adds up to 128 a thread: a build that starts with fewer would
  // wait for registers that never come
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes a;
    if ((e = cudaFuncGetAttributes(&a, paged_tiles_kernel<HD, FP8, NQ>)) != cudaSuccess) return e;
    regs.store(a.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != 128) return cudaErrorInvalidConfiguration;
  CUtensorMap tq, tk{}, tv{};
  if (!paged_map_q(&tq, p)) return cudaErrorInvalidValue;
  if (!FP8 && (!paged_map_pages(&tk, p.kv, p.kv.k, kTileK) || !paged_map_pages(&tv, p.kv, p.kv.v, kTileK))) return cudaErrorInvalidValue;
  paged_tiles_kernel<HD, FP8, NQ><<<p.ctas, C::THREADS, C::SMEM, st>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template <int HD, bool FP8>
cudaError_t launch_tiles_q(const PagedAttnParams &p, cudaStream_t st) {
  return (long long)p.c.T * p.G <= 128 ? launch_tiles<HD, FP8, 1>(p, st) : launch_tiles<HD, FP8, 2>(p, st);
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedAttnParams &p, cudaStream_t st) {
  if (p.kv.hd == 64) return p.kv.e4m3 ? launch_tiles_q<64, true>(p, st) : launch_tiles_q<64, false>(p, st);
  return p.kv.e4m3 ? launch_tiles_q<128, true>(p, st) : launch_tiles_q<128, false>(p, st);
}

}  // namespace smol
