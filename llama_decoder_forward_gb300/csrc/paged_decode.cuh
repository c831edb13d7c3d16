// paged_decode.cuh - paged attention of few rows: up to 16 or 32 query rows
// (tokens times heads of a kv head) share a sequence's keys.  Included by
// paged_attention.cu.
//
// Bound by memory: every key and value is read once for at most 32 rows.  What
// counts is bytes in flight, so each of the CTA's eight warps runs by itself: its
// own ring of stages in shared memory, filled by TMA boxes that one lane asks for
// (a box for each page), and its own running maximum, sum and accumulator over an
// eighth of each key tile.  No barrier of the CTA is met until a unit ends; then the
// eight states are merged through shared memory, two at a time.  A unit that
// several CTAs share is finished by the one that comes last: it combines all their
// parts, in the CTAs' order (the same bits every time).
//
// mma.sync m16n8k16 (bf16, fp32 sums): a tcgen05 tile has 128 rows, of which 3 to
// 32 would be used, and its score tile's trip through tensor memory is longer than
// the whole step here.  The fragments of a step stay in registers; with 32 rows the
// queries' are read from shared memory each time (they would spill).
//
// e4m3 codes become bf16 exactly, by way of f16 and fp32: four cycles of the integer
// pipe for a pair (shifting the bits into place took eight).
// The keys' scales multiply the scores, the values' scales the weights, so no
// dequantised value is rounded.
//
// Slots outside the rows' sight may hold anything: their scores are replaced before
// they are looked at, their values (and values' scales) set to zero.
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
__device__ __forceinline__ uint4 pd_lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 pd_lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int HD, bool FP8, int RT>
struct PdCfg {
  static constexpr int NW = 8, THREADS = 32 * NW;
  static constexpr int KC = (HD == 128 && !FP8) ? 16 : 32;     // keys of a warp's step: 4 or 8 KB of K and V
  static constexpr int NSUB = FP8 ? 1 : HD / 64;               // boxes across a key (128 bytes each, or 64)
  static constexpr int ROWB = FP8 ? HD : 128;                  // bytes of a key in a box
  static constexpr int SUB_BYTES = KC * ROWB;
  static constexpr int KV_BYTES = NSUB * SUB_BYTES;
  static constexpr int STAGE = 2 * KV_BYTES;
  static constexpr int NS = STAGE == 4096 ? 5 : RT == 2 && HD == 128 ? 2 : 3;
  static constexpr int BK_SHIFT = KC == 32 ? 8 : 7;            // keys of a tile: NW * KC
  static constexpr int NT8 = KC / 8;                           // key columns of the score fragments
  static constexpr int ND8 = HD / 8;
  static constexpr bool Q_REGS = RT == 1;                      // the queries' fragments stay in registers
  static constexpr int Q_BYTES = RT * 16 * HD * 2;             // [HD / 64][RT * 16 rows][64]
  static constexpr int MERGE_WORDS = RT * (ND8 * 4 + 4);       // a thread's state
  static constexpr int OFF_SC = NW * NS * STAGE;               // of each stage: scales of the keys, and of the values
  static constexpr int OFF_NOTE = OFF_SC + (FP8 ? NW * NS * 2 * KC * 4 : 0);
  static constexpr int OFF_Q = (OFF_NOTE + NW * NS * 64 + 1023) / 1024 * 1024;   // [2] this unit's and the next one's
  static constexpr int OFF_MERGE = OFF_Q + 2 * Q_BYTES;        // two warps' states at a time
  static constexpr int MERGE_BYTES = 2 * 32 * MERGE_WORDS * 4;
  static constexpr int OFF_BAR = OFF_MERGE + MERGE_BYTES;      // [NW][NS] stages, [2] Q
  static constexpr int USED = OFF_BAR + (NW * NS + 2) * 8 + 16;
  static constexpr int SMEM = USED + 1008 <= 232448 ? USED + 1008 : 232448;
  static_assert(USED <= 232448, "shared memory per CTA");
  static_assert(MERGE_BYTES >= 8 * kPagedMaxCtas * 4 + (int)sizeof(PagedSchedSmem), "room for the parts' weights, and the schedule");
};

// A warp's note of a step, beside its keys.
struct PdNote {
  int x0, lo, hi;              // the warp's first position; the positions that some row of the unit sees
  int first_at, rows;          // the unit's first row's position; its rows
  int flags;                   // kPd*
  int b, kvh, t0, row0;        // the unit
  int j01;                     // its key tiles, and the first one's place in the line
  long long u0;
  int pad[2];
};
static_assert(sizeof(PdNote) == 64, "note");

enum : int { kPdFirst = 1, kPdEnds = 2, kPdLast = 4 };       // the unit's first tile here, its last tile, this CTA's last
enum : int { kPdTimeout = 0x209 };

template <int HD, bool FP8, int RT>
__global__ void __launch_bounds__(PdCfg<HD, FP8, RT>::THREADS, 1)
    paged_few_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const PagedAttnParams p) {
  using C = PdCfg<HD, FP8, RT>;
  constexpr int KC = C::KC, NS = C::NS, ND8 = C::ND8, NT8 = C::NT8, NSUB = C::NSUB;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), cta = blockIdx.x;
  const int g8 = lane >> 2, c4 = lane & 3;        // fragment row and column pair
  if (smem + C::USED > smem_raw + C::SMEM) {      // no room left by the alignment
    if (tid == 0) set_status(p.status, kPdTimeout);
    return;
  }
  uint8_t *ring = smem + warp * NS * C::STAGE;
  float *ring_sc = reinterpret_cast<float *>(smem + C::OFF_SC) + warp * NS * 2 * KC;
  PdNote *notes = reinterpret_cast<PdNote *>(smem + C::OFF_NOTE + warp * NS * 64);   // 64 bytes each
  float *merge = reinterpret_cast<float *>(smem + C::OFF_MERGE);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + warp * NS;
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + C::NW * NS;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(q_full + 2);
  volatile int *s_parts = abort_flag + 1;         // [2] a unit to combine: its first CTA, and how many

  if (tid == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  PagedSchedSmem &sched = *reinterpret_cast<PagedSchedSmem *>(merge);
  PagedIter ld = paged_locate<C::THREADS>(p, cta, p.ctas, sched);
  if (ld.left == 0) return;                       // the same for the whole CTA
  const long long total = sched.total;
  const int workers = sched.workers;
  if (lane == 0)
    for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
  if (tid == 0) {
    mbar_init(&q_full[0], 1);
    mbar_init(&q_full[1], 1);
    *abort_flag = 0;
  }
  if (lane == 0) fence_barrier_init();
  __syncthreads();

  bool alive = true;                              // false: a wait gave up, nothing more is asked for
  // ---- Q of a unit by TMA: its tokens' heads are the rows (rows past its last are
  // whatever follows, or zeros: they reach no other row)
  PagedIter qn = ld;                              // the unit whose Q is asked for next (warp 0)
  uint32_t nq = 0;
  auto ask_q = [&]() {
    if (qn.left > 0 && alive) {
      if (lane == 0) {
        uint64_t *bar = &q_full[nq & 1];
        mbar_arrive_expect_tx(bar, (HD / 64) * 128 * p.tt * p.G);
#pragma unroll
        for (int sub = 0; sub < HD / 64; ++sub)
          tma_load_4d(smem + C::OFF_Q + (nq & 1) * C::Q_BYTES + sub * (RT * 16 * 128), &tmQ, bar, sub * 64, qn.kvh * p.G,
                      qn.s.row0 + qn.t0, p.c.row_start ? 0 : qn.b);
      }
      ++nq;
      qn.left -= qn.j1 - qn.j - 1;                // to the unit's last tile, and over it
      qn.j = qn.j1 - 1;
      paged_next(p, qn);
    }
    __syncwarp();
  };

  // ---- loads: this warp's KC keys of a tile; the page numbers are fetched one
  // step ahead of the boxes that need them
  const int box = min(1 << p.kv.page_shift, KC), n_box = KC / box;
  int page = -1;                                  // lane i < n_box: of keys i * box ..
  bool first_tile = true;
  const bool started_inside = ld.j > ld.j0;       // the first unit was begun by an earlier CTA
  uint32_t asked = 0;                             // steps asked for
  auto fetch_page = [&]() {
    page = -1;
    if (ld.left > 0 && lane < n_box) {
      const int x = (ld.j << C::BK_SHIFT) + warp * KC + lane * box;
      if (x < ld.hi && x + box > ld.lo) page = paged_page(p.kv, ld.b, x);
    }
  };
  fetch_page();
  int ld_stage = 0;
  auto produce = [&]() {
    if (ld.left > 0) {
      uint8_t *st = ring + ld_stage * C::STAGE;
      uint64_t *bar = &full[ld_stage];
      const int x0 = (ld.j << C::BK_SHIFT) + warp * KC;
      const bool mine = lane < n_box && x0 + lane * box < ld.hi && x0 + (lane + 1) * box > ld.lo;
      const bool there = page >= 0 && page < p.kv.P;
      if (mine && !there) set_status(p.status, kDevBadInput);
      const unsigned in = __ballot_sync(0xffffffffu, mine), good = __ballot_sync(0xffffffffu, mine && there);
      if (lane == 0) {
        PdNote *note = &notes[ld_stage];
        note->x0 = x0;
        note->lo = ld.lo;
        note->hi = ld.hi;
        note->first_at = ld.s.L + ld.t0;
        note->rows = ld.nt * p.G;
        note->flags = (first_tile ? kPdFirst : 0) | (ld.j + 1 == ld.j1 ? kPdEnds : 0) | (ld.left == 1 ? kPdLast : 0);
        note->b = ld.b;
        note->kvh = ld.kvh;
        note->t0 = ld.t0;
        note->row0 = ld.s.row0;
        note->j01 = ld.j1 - ld.j0;
        note->u0 = ld.u0;
        // a box on no page comes as zeros (its scales stay what they were)
        if (alive) mbar_arrive_expect_tx(bar, __popc(in) * box * C::ROWB * NSUB * 2 + (FP8 ? __popc(good) * box * 8 : 0));
      }
      __syncwarp();
      if (mine && alive) {
        const int y = (ld.kvh << p.kv.page_shift) + (x0 & ((1 << p.kv.page_shift) - 1)), z = there ? page : p.kv.P;
#pragma unroll
        for (int sub = 0; sub < NSUB; ++sub) {
          tma_load_3d(st + sub * C::SUB_BYTES + lane * box * C::ROWB, &tmK, bar, sub * 64, y, z);
          tma_load_3d(st + C::KV_BYTES + sub * C::SUB_BYTES + lane * box * C::ROWB, &tmV, bar, sub * 64, y, z);
        }
        if (FP8 && there) {
          const long long at = paged_slot(p.kv, page, x0 + lane * box, ld.kvh);
          bulk_load(ring_sc + ld_stage * 2 * KC + lane * box, p.kv.ks + at, box * 4, bar);
          bulk_load(ring_sc + ld_stage * 2 * KC + KC + lane * box, p.kv.vs + at, box * 4, bar);
        }
      }
      __syncwarp();
      if (alive) ++asked;
      first_tile = ld.j + 1 == ld.j1;
      paged_next(p, ld);
      fetch_page();
    }
    ld_stage = ld_stage + 1 == NS ? 0 : ld_stage + 1;
  };
  if (warp == 0) {
    ask_q();
    ask_q();
  }
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) produce();

  // ---- state of the rows: row g8 + 8 i of m-tile rt
  float o[RT][ND8][4], m[RT][2], l[RT][2];
  [[maybe_unused]] uint32_t qf[RT][HD / 16][4];
  uint32_t units = 0, phase = 0;
  int stage = 0;
  // A fragments of k-step ks.  Codes: a lane's B fragments of four k-steps are 16
  // neighbouring bytes of the key, so step s of group g takes the dims
  // 64 g + 16 c4 + 4 s .. + 3 there, and the queries' fragments the same.
  auto load_a = [&](uint32_t q_s, int rt, int ks, uint32_t (&a)[4]) {
    const uint32_t sub = q_s + (ks >> 2) * (RT * 16 * 128) + rt * (16 * 128);
    if constexpr (FP8) {
      const int ch = 2 * c4 + ((ks & 3) >> 1);
      const uint2 u = pd_lds64(sub + g8 * 128 + ((ch ^ g8) << 4) + (ks & 1) * 8);
      const uint2 v = pd_lds64(sub + (g8 + 8) * 128 + ((ch ^ g8) << 4) + (ks & 1) * 8);
      a[0] = u.x;
      a[1] = v.x;
      a[2] = u.y;
      a[3] = v.y;
    } else {
      pd_ldsm4(a, sub + (lane & 15) * 128 + ((((ks & 3) * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
    }
  };
  // where this lane's pieces of the keys and values lie in a box (the boxes' swizzle:
  // 128-byte rows by the row's last three bits, 64-byte rows by its bits 1 and 2)
  // codes of hd 128: fragment column n reads key (n >> 1) + 4 (n & 1) of eight, so that
  // two rows' pieces meet different banks; the weights' columns follow
  constexpr bool PERM = FP8 && HD == 128;
  auto key_of = [](int n) { return PERM ? (n & ~7) | ((n & 7) >> 1) | ((n & 1) << 2) : n; };
  while (true) {
    if (alive && !__all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], phase, abort_flag, p.wait_ns))) {
      // give up: what was asked for has a second to land, and the rest is done without
      set_status(p.status, kPdTimeout);
      *abort_flag = 1;
      alive = false;
    }
    __syncwarp();
    produce();                                    // into the stage read last, which every lane has left
    const uint8_t *st = ring + stage * C::STAGE;
    const PdNote *note = &notes[stage];
    const int x0 = note->x0, lo = note->lo, hi = note->hi, first_at = note->first_at, rows = note->rows, flags = note->flags;
    const uint32_t q_s = smem_u32(smem + C::OFF_Q + (units & 1) * C::Q_BYTES);
    if (flags & kPdFirst) {
      // ---- a new unit
      if (alive && !__all_sync(0xffffffffu, mbar_wait_bounded(&q_full[units & 1], (units >> 1) & 1, abort_flag, p.wait_ns))) {
        set_status(p.status, kPdTimeout);
        *abort_flag = 1;
        alive = false;
      }
      if constexpr (C::Q_REGS) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) load_a(q_s, rt, ks, qf[rt][ks]);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[rt][i] = -INFINITY;
          l[rt][i] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < ND8; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[rt][d][e] = 0.f;
      }
    }
    if (x0 < hi && x0 + KC > lo) {
      const uint32_t k_s = smem_u32(st), v_s = k_s + C::KV_BYTES;
      float *scales = ring_sc + stage * 2 * KC;
      if (x0 < lo || x0 + KC > hi) {
        // keys out of sight: their values (and the values' scales) become zeros
        if (FP8 && lane < KC && (x0 + lane < lo || x0 + lane >= hi)) scales[KC + lane] = 0.f;
        for (int i = lane; i < C::KV_BYTES / 16; i += 32) {
          const int key = i / (C::ROWB / 16) % KC;
          if (x0 + key < lo || x0 + key >= hi)
            *reinterpret_cast<uint4 *>(ring + stage * C::STAGE + C::KV_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();                 // before the stage's next boxes
        __syncwarp();
      }
      // ---- S = Q K^T
      float s[RT][NT8][4];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int n = 0; n < NT8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[rt][n][e] = 0.f;
      if constexpr (FP8) {
#pragma unroll
        for (int gr = 0; gr < HD / 64; ++gr) {
          uint4 w[NT8];
#pragma unroll
          for (int n = 0; n < NT8; ++n) {
            const int key = n * 8 + key_of(g8);
            const uint32_t ch = gr * 4 + c4;
            w[n] = pd_lds128(k_s + key * C::ROWB + ((HD == 64 ? ch ^ ((key >> 1) & 3) : ch ^ (key & 7)) << 4));
          }
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t a[RT][4];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              if constexpr (C::Q_REGS) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[rt][e] = qf[rt][gr * 4 + q4][e];
              } else {
                load_a(q_s, rt, gr * 4 + q4, a[rt]);
              }
            }
#pragma unroll
            for (int n = 0; n < NT8; ++n) {
              const uint32_t u = q4 == 0 ? w[n].x : q4 == 1 ? w[n].y : q4 == 2 ? w[n].z : w[n].w;
              const float2 f0 = unpack_e4m3x2(u), f1 = unpack_e4m3x2(u >> 16);
              const uint32_t b0 = pack_bf16x2(f0.x, f0.y), b1 = pack_bf16x2(f1.x, f1.y);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) pd_mma(s[rt][n], a[rt], b0, b1);
            }
          }
        }
      } else {
        const uint32_t k_lane = k_s + (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
#pragma unroll
        for (int k2 = 0; k2 < HD / 32; ++k2) {
          uint32_t a[RT][2][4];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (C::Q_REGS) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[rt][h][e] = qf[rt][2 * k2 + h][e];
              } else {
                load_a(q_s, rt, 2 * k2 + h, a[rt][h]);
              }
            }
#pragma unroll
          for (int n = 0; n < NT8; ++n) {
            uint32_t b[4];
            pd_ldsm4(b, (k_lane ^ ((k2 & 1) * 64)) + (k2 >> 1) * C::SUB_BYTES + n * 1024);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              pd_mma(s[rt][n], a[rt][0], b[0], b[1]);
              pd_mma(s[rt][n], a[rt][1], b[2], b[3]);
            }
          }
        }
      }
      // ---- scores in the exp2 domain, replaced where a row does not see the key
      const bool edge = x0 + KC - 1 > first_at || x0 < lo || (p.window > 0 && x0 <= first_at + (rows - 1) / p.G - p.window);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if constexpr (FP8) {
#pragma unroll
          for (int n = 0; n < NT8; ++n) {
            const float k0 = scales[n * 8 + key_of(2 * c4)] * p.scale_log2, k1 = scales[n * 8 + key_of(2 * c4 + 1)] * p.scale_log2;
            s[rt][n][0] *= k0;
            s[rt][n][1] *= k1;
            s[rt][n][2] *= k0;
            s[rt][n][3] *= k1;
          }
        }
        if (edge) {
          int own[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) own[i] = first_at + (rt * 16 + g8 + 8 * i) / p.G;   // past the unit's rows: not written
#pragma unroll
          for (int n = 0; n < NT8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = x0 + n * 8 + key_of(2 * c4 + (e & 1));
              if (x > own[e >> 1] || (p.window > 0 && x <= own[e >> 1] - p.window)) s[rt][n][e] = -INFINITY;
            }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < NT8; ++n) {
          mx[0] = fmax3(mx[0], s[rt][n][0], s[rt][n][1]);
          mx[1] = fmax3(mx[1], s[rt][n][2], s[rt][n][3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
          if (!FP8) mx[i] *= p.scale_log2;        // scale > 0; -inf stays -inf
        }
        if (__any_sync(0xffffffffu, mx[0] > m[rt][0] || mx[1] > m[rt][1])) {
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
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mu = m[rt][i] == -INFINITY ? 0.f : m[rt][i];
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int n = 0; n < NT8; ++n) {
            float2 x;
            if constexpr (FP8) x = fadd2(s[rt][n][2 * i], s[rt][n][2 * i + 1], -mu, -mu);
            else x = ffma2(s[rt][n][2 * i], s[rt][n][2 * i + 1], p.scale_log2, -mu);
            x.x = ex2_approx(x.x);
            x.y = ex2_approx(x.y);
            sum = fadd2(sum.x, sum.y, x.x, x.y);
            s[rt][n][2 * i] = x.x;
            s[rt][n][2 * i + 1] = x.y;
          }
          l[rt][i] += sum.x + sum.y;
        }
      }
      // ---- O += P V; P rounded to bf16, the tensor core's operand type
#pragma unroll
      for (int k16 = 0; k16 < KC / 16; ++k16) {
        uint32_t a[RT][4];
        float2 vs0 = make_float2(1.f, 1.f), vs1 = vs0;
        if constexpr (FP8) {
          vs0 = make_float2(scales[KC + k16 * 16 + key_of(2 * c4)], scales[KC + k16 * 16 + key_of(2 * c4 + 1)]);
          vs1 = make_float2(scales[KC + k16 * 16 + 8 + key_of(2 * c4)], scales[KC + k16 * 16 + 8 + key_of(2 * c4 + 1)]);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float(&f)[4] = s[rt][2 * k16], (&g)[4] = s[rt][2 * k16 + 1];
          a[rt][0] = pack_bf16x2(f[0] * vs0.x, f[1] * vs0.y);
          a[rt][1] = pack_bf16x2(f[2] * vs0.x, f[3] * vs0.y);
          a[rt][2] = pack_bf16x2(g[0] * vs1.x, g[1] * vs1.y);
          a[rt][3] = pack_bf16x2(g[2] * vs1.x, g[3] * vs1.y);
        }
        if constexpr (FP8) {
          // a transposed load gives pairs of neighbouring dims: the even dims of 16 go
          // to one accumulator column block, the odd ones to the next
          const int key = k16 * 16 + key_of(lane & 15);
          const uint32_t row = v_s + key * C::ROWB;
#pragma unroll
          for (int c2 = 0; c2 < HD / 32; ++c2) {
            uint32_t b[4];
            const uint32_t ch = 2 * c2 + (lane >> 4);
            pd_ldsm4_t(b, row + ((HD == 64 ? ch ^ ((key >> 1) & 3) : ch ^ (key & 7)) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float2 p0 = unpack_e4m3x2(b[2 * h]), p1 = unpack_e4m3x2(b[2 * h] >> 16);
              const float2 p2 = unpack_e4m3x2(b[2 * h + 1]), p3 = unpack_e4m3x2(b[2 * h + 1] >> 16);
              const uint32_t e0 = pack_bf16x2(p0.x, p1.x), e1 = pack_bf16x2(p2.x, p3.x);
              const uint32_t d0 = pack_bf16x2(p0.y, p1.y), d1 = pack_bf16x2(p2.y, p3.y);
#pragma unroll
              for (int rt = 0; rt < RT; ++rt) {
                pd_mma(o[rt][4 * c2 + 2 * h], a[rt], e0, e1);
                pd_mma(o[rt][4 * c2 + 2 * h + 1], a[rt], d0, d1);
              }
            }
          }
        } else {
          const uint32_t v_lane = v_s + k16 * 2048 + (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
#pragma unroll
          for (int c2 = 0; c2 < HD / 16; ++c2) {
            uint32_t b[4];
            pd_ldsm4_t(b, (v_lane ^ ((c2 & 3) * 32)) + (c2 >> 2) * C::SUB_BYTES);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              pd_mma(o[rt][2 * c2], a[rt], b[0], b[1]);
              pd_mma(o[rt][2 * c2 + 1], a[rt], b[2], b[3]);
            }
          }
        }
      }
    }
    if (flags & (kPdEnds | kPdLast)) {
      // ---- the unit, or this CTA's part of it, is done: merge the warps' states: 4, 5
      // into 0, 1; 6, 7 into 2, 3; 2, 3 into 0, 1; 1 into 0
      const PdNote u = *note;
      const bool in_unit = units == 0 && started_inside, whole = (flags & kPdEnds) && !in_unit;
      PagedSeq us{};
      us.row0 = u.row0;
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
          float4 *dst = reinterpret_cast<float4 *>(merge + (warp - from) * 32 * C::MERGE_WORDS) + lane;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int d = 0; d < ND8; ++d)
              dst[(rt * (ND8 + 1) + d) * 32] = make_float4(o[rt][d][0], o[rt][d][1], o[rt][d][2], o[rt][d][3]);
            dst[(rt * (ND8 + 1) + ND8) * 32] = make_float4(m[rt][0], m[rt][1], l[rt][0], l[rt][1]);
          }
        }
        __syncthreads();
        if (warp >= to && warp < to + n) {
          const float4 *src = reinterpret_cast<const float4 *>(merge + (warp - to) * 32 * C::MERGE_WORDS) + lane;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const float4 other = src[(rt * (ND8 + 1) + ND8) * 32];
            const float m2[2] = {other.x, other.y}, l2[2] = {other.z, other.w};
            float a[2], a2[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float mn = fmaxf(m[rt][i], m2[i]);
              a[i] = mn == -INFINITY ? 1.f : ex2_approx(m[rt][i] - mn);
              a2[i] = mn == -INFINITY ? 1.f : ex2_approx(m2[i] - mn);
              m[rt][i] = mn;
              l[rt][i] = l[rt][i] * a[i] + l2[i] * a2[i];
            }
#pragma unroll
            for (int d = 0; d < ND8; ++d) {
              const float4 v = src[(rt * (ND8 + 1) + d) * 32];
              o[rt][d][0] = o[rt][d][0] * a[0] + v.x * a2[0];
              o[rt][d][1] = o[rt][d][1] * a[0] + v.y * a2[0];
              o[rt][d][2] = o[rt][d][2] * a[1] + v.z * a2[1];
              o[rt][d][3] = o[rt][d][3] * a[1] + v.w * a2[1];
            }
          }
        }
        __syncthreads();
      }
      if (warp == 0) {
        float *part = paged_part(p.ws, cta, in_unit ? 0 : 1, RT * 16, HD);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = rt * 16 + g8 + 8 * i;
            if (r >= rows) continue;
            const float inv = l[rt][i] > 0.f ? 1.f / l[rt][i] : 0.f;
            const long long out = whole ? paged_unit_row(p.o, p, us, u.b, u.t0, u.kvh, r) : 0;
            float *row = part + r * HD;
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
                  __stcg(reinterpret_cast<float4 *>(row + dim), make_float4(x, x1, y, y1));
              } else {
                const int dim = d * 8 + 2 * c4;
                if (whole)
                  *reinterpret_cast<uint32_t *>(p.o.data + (out + dim) * 2) =
                      p.o_f16 ? pack_f16x2(x * inv, y * inv) : pack_bf16x2(x * inv, y * inv);
                else
                  __stcg(reinterpret_cast<float2 *>(row + dim), make_float2(x, y));
              }
            }
            if (!whole && c4 == 0) __stcg(reinterpret_cast<float2 *>(part + RT * 16 * HD + 2 * r), make_float2(m[rt][i], l[rt][i]));
          }
      }
      if (!whole) {
        // ---- the CTA that brings a unit's last part combines them all
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const int c0 = paged_worker_of(u.u0, total, workers), n = paged_worker_of(u.u0 + u.j01 - 1, total, workers) - c0 + 1;
          int *count = reinterpret_cast<int *>(p.ws + kPagedCountOff) + c0;
          const bool mine = atomicAdd(count, 1) == n - 1;
          if (mine) atomicExch(count, 0);         // for the next call
          s_parts[0] = c0;
          s_parts[1] = mine ? n : 0;
        }
        __syncthreads();
        const int c0 = s_parts[0], n = s_parts[1];
        if (n > 0) {
          __threadfence();
          float *weight = merge + warp * kPagedMaxCtas;
          for (int r = warp; r < rows; r += C::NW)
            paged_combine_row<HD>(p, RT * 16, c0, n, r, weight, paged_unit_row(p.o, p, us, u.b, u.t0, u.kvh, r));
          __syncthreads();
        }
      }
      ++units;
      if (flags & kPdLast) break;
      if (warp == 0) ask_q();                     // of the unit after the next
    }
    if (++stage == NS) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!alive) {
    // what this warp asked for lands before the block's shared memory goes
    bool done = true;
    for (uint32_t k = asked > NS ? asked - NS : 0; k < asked; ++k) done &= mbar_wait_drain(&full[k % NS], (k / NS) & 1);
    for (uint32_t k = nq > 2 ? nq - 2 : 0; k < nq; ++k) done &= mbar_wait_drain(&q_full[k & 1], (k >> 1) & 1);
    if (!done) set_status(p.status, kPdTimeout);
  }
}

}  // namespace
}  // namespace smol
