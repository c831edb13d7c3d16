// paged_decode.cuh - paged attention of few rows: up to 8, 16, 24 or 32 query rows
// (tokens times heads of a kv head) share a sequence's keys.  Included by
// paged_attention.cu.
//
// Every key and value is read once for at most 32 rows, so bytes in flight count:
// each of the CTA's eight warps runs by itself, with its own ring of stages in shared
// memory, filled by TMA boxes that one lane asks for (a box for each page), and its own
// running maximum, sum and accumulator over an eighth of each key tile.  No barrier of
// the CTA is met until a unit ends; then the eight states are merged through shared
// memory, two or four at a time.  A unit that several CTAs share is finished by the one
// that comes last: it combines all their parts, in the CTAs' order (the same bits every
// time).
//
// 64 sequences of one token on 1024 to 4096 cached ones, hd 64, 3 heads each (126 MB):
// 29.4 us, 4.3 TB/s.  Of a CTA's 48,000 cycles 6,500 pass before its first key, 28,000
// in 13 steps, 14,000 at the ends of two units.  e4m3, hd 128, 20 rows, 32 sequences
// (171 MB): 74 us, bound by the steps (4,700 cycles for 32 keys of each warp).
//
// mma.sync m16n8k16 (bf16, fp32 sums): a tcgen05 tile has 128 rows, of which 3 to
// 32 would be used, and its score tile's trip through tensor memory is longer than
// the whole step here.  The products are taken as S^T = K Q^T and O^T = V^T P^T: keys
// and dims are the 16 rows of an instruction, the queries its 8 columns, and 3 of them
// cost half of what they would as rows.  With two warps in a quarter of the SM a step
// is a chain of waits for results (the tensor pipe is busy 5 to 20 % of the time), so
// fewer instructions count, and large steps: half the keys in each of 16 warps took
// longer (e4m3, 32 sequences of 2000 to 8191 tokens, hd 64: 36 us, 64 keys in each of
// eight 30, 32 keys 33).  A lane has two query columns of eight, its own rows' maxima
// and sums, and P^T is turned by movmatrix between the products.  The fragments of a
// step stay in registers; with more than 16 rows the queries' are read from shared
// memory each time (they would spill).
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
// The transpose of an 8x8 tile of 16-bit values.
__device__ __forceinline__ uint32_t pd_turn(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int HD, bool FP8, int NR>
struct PdCfg {
  static constexpr int NW = 8, THREADS = 32 * NW;
  static constexpr int KC = HD == 128 ? (FP8 ? 32 : 16) : FP8 && NR <= 2 ? 64 : 32;   // keys of a warp's step: 4 or 8 KB of K and V
  static constexpr int NSUB = FP8 ? 1 : HD / 64;               // boxes across a key (128 bytes each, or 64)
  static constexpr int ROWB = FP8 ? HD : 128;                  // bytes of a key in a box
  static constexpr int SUB_BYTES = KC * ROWB;
  static constexpr int KV_BYTES = NSUB * SUB_BYTES;
  static constexpr int STAGE = 2 * KV_BYTES;
  static constexpr int NS = STAGE == 4096 ? 5 : NR > 2 && HD == 128 ? 2 : 3;   // by shared memory
  static constexpr int BK_SHIFT = KC == 64 ? 9 : KC == 32 ? 8 : 7;   // keys of a tile: NW * KC
  static constexpr int KT = KC / 16, DT = HD / 16;             // 16-row tiles of S^T and of O^T
  static constexpr int ROWS = 8 * NR;
  static constexpr bool Q_REGS = NR <= 2;                      // the queries' fragments stay in registers
  static constexpr int Q_BYTES = ROWS * HD * 2;                // [HD / 64][ROWS][64]
  static constexpr int STATE_BYTES = 32 * NR * (DT + 1) * 16;  // a warp's sums, maxima and row sums
  static constexpr int OFF_SC = NW * NS * STAGE;               // of each stage: scales of the keys, and of the values
  static constexpr int OFF_NOTE = OFF_SC + (FP8 ? NW * NS * 2 * KC * 4 : 0);
  static constexpr int OFF_Q = (OFF_NOTE + NW * NS * 64 + 1023) / 1024 * 1024;   // [2] this unit's and the next one's
  static constexpr int OFF_MERGE = OFF_Q + 2 * Q_BYTES;        // some warps' states; then the unit's rows
  static constexpr int BAR_BYTES = (NW * NS + 2) * 8 + 16;     // [NW][NS] stages, [2] Q
  static constexpr int MERGE_WARPS = OFF_MERGE + 4 * STATE_BYTES + BAR_BYTES + 128 <= 232448 ? 4 : 2;
  static constexpr int TILE_LD = HD + 4;                       // words of a row of the merged unit
  static constexpr int TILE_BYTES = ROWS * (TILE_LD + 2) * 4;
  static constexpr int SCHED_BYTES = 8 * kPagedMaxCtas * 4 + (int)sizeof(PagedSchedSmem);   // the parts' weights, and the schedule
  static constexpr int MERGE_BYTES =
      (MERGE_WARPS * STATE_BYTES > SCHED_BYTES ? MERGE_WARPS * STATE_BYTES : SCHED_BYTES) / 16 * 16 + 16;
  static constexpr int OFF_BAR = OFF_MERGE + MERGE_BYTES;
  static constexpr int OFF_WALK = OFF_BAR + (BAR_BYTES + 15) / 16 * 16;
  static constexpr int USED = OFF_WALK + (NR > 3 ? (int)sizeof(PagedIter) : 0);   // warp 0's walk over the queries
  static constexpr int SMEM = USED + 1008 <= 232448 ? USED + 1008 : 232448;
  static_assert(USED <= 232448, "shared memory per CTA");
  static_assert(MERGE_BYTES >= TILE_BYTES, "room for the merged unit");
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

template <int HD, bool FP8, int NR>
__global__ void __launch_bounds__(PdCfg<HD, FP8, NR>::THREADS, 1)
    paged_few_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const PagedAttnParams p) {
  using C = PdCfg<HD, FP8, NR>;
  constexpr int KC = C::KC, KT = C::KT, DT = C::DT, NS = C::NS, NSUB = C::NSUB;
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
  // (with 32 rows the walk lies in shared memory: in registers, where every warp would
  // hold it, it makes the accumulators spill; e4m3, hd 128: 95 us, in registers 107)
  PagedIter q_own;
  PagedIter &next_q = NR > 3 ? *reinterpret_cast<PagedIter *>(smem + C::OFF_WALK) : q_own;
  if (NR <= 3 || tid == 0) next_q = ld;
  uint32_t nq = 0;
  auto ask_q = [&]() {
    PagedIter qn = next_q;                        // the unit whose Q is asked for next
    __syncwarp();
    if (qn.left > 0 && alive) {
      if (lane == 0) {
        uint64_t *bar = &q_full[nq & 1];
        mbar_arrive_expect_tx(bar, (HD / 64) * 128 * p.tt * p.G);
#pragma unroll
        for (int sub = 0; sub < HD / 64; ++sub)
          tma_load_4d(smem + C::OFF_Q + (nq & 1) * C::Q_BYTES + sub * (C::ROWS * 128), &tmQ, bar, sub * 64, qn.kvh * p.G,
                      qn.s.row0 + qn.t0, p.c.row_start ? 0 : qn.b);
      }
      ++nq;
      qn.left -= qn.j1 - qn.j - 1;                // to the unit's last tile, and over it
      qn.j = qn.j1 - 1;
      paged_next(p, qn);
      if (NR <= 3 || lane == 0) next_q = qn;
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
    __syncwarp();
    ask_q();
    ask_q();
  }
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) produce();

  // ---- state of the rows: this lane's are 8 nt + 2 c4 + i
  float o[DT][NR][4], m[NR][2], l[NR][2];
  [[maybe_unused]] uint32_t qf[NR][DT][2];
  uint32_t units = 0, phase = 0;
  int stage = 0;
  // the queries' fragments of k-steps 2 k2 and 2 k2 + 1.  Codes: a lane's pieces of four
  // k-steps are 16 neighbouring bytes of the key, so step s of group g takes the dims
  // 64 g + 16 c4 + 4 s .. + 3 there, and the queries' fragments the same.
  auto load_q = [&](uint32_t q_s, int nt, int k2, uint32_t (&b)[4]) {
    const uint32_t sub = q_s + (k2 >> 1) * (C::ROWS * 128) + nt * 1024;
    if constexpr (FP8) {
      const uint4 v = pd_lds128(sub + g8 * 128 + (((2 * c4 + (k2 & 1)) ^ g8) << 4));
      b[0] = v.x;
      b[1] = v.y;
      b[2] = v.z;
      b[3] = v.w;
    } else {
      pd_ldsm4(b, sub + (lane & 7) * 128 + ((((k2 & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4));
    }
  };
  auto take_q = [&](uint32_t q_s, int k2, uint32_t (&b)[NR][4]) {
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
      if constexpr (C::Q_REGS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[nt][e] = qf[nt][2 * k2 + (e >> 1)][e & 1];
      } else {
        load_q(q_s, nt, k2, b[nt]);
      }
    }
  };
  // where this lane's pieces of the keys and values lie in a box (the boxes' swizzle:
  // 128-byte rows by the row's last three bits, 64-byte rows by its bits 1 and 2)
  // codes of hd 128: fragment row n reads key (n >> 1) + 4 (n & 1) of eight, so that
  // two rows' pieces meet different banks; the values' columns follow
  constexpr bool PERM = FP8 && HD == 128;
  auto key_of = [](int n) { return PERM ? (n & ~7) | ((n & 7) >> 1) | ((n & 1) << 2) : n; };
  while (true) {
    if (alive && !__all_sync(0xffffffffu, mbar_wait_limit(&full[stage], phase, abort_flag, p.wait_ns))) {
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
      if (alive && !__all_sync(0xffffffffu, mbar_wait_limit(&q_full[units & 1], (units >> 1) & 1, abort_flag, p.wait_ns))) {
        set_status(p.status, kPdTimeout);
        *abort_flag = 1;
        alive = false;
      }
      if constexpr (C::Q_REGS) {
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int k2 = 0; k2 < DT / 2; ++k2) {
            uint32_t b[4];
            load_q(q_s, nt, k2, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) qf[nt][2 * k2 + (e >> 1)][e & 1] = b[e];
          }
      }
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[nt][i] = -INFINITY;
          l[nt][i] = 0.f;
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][nt][e] = 0.f;
      }
    }
    if (x0 < hi && x0 + KC > lo) {
      const uint32_t k_s = smem_u32(st), v_s = k_s + C::KV_BYTES;
      float *scales = ring_sc + stage * 2 * KC;
      if (x0 < lo || x0 + KC > hi) {
        // keys out of sight: their values (and the values' scales) become zeros
        if (FP8)
          for (int i = lane; i < KC; i += 32)
            if (x0 + i < lo || x0 + i >= hi) scales[KC + i] = 0.f;
        for (int i = lane; i < C::KV_BYTES / 16; i += 32) {
          const int key = i / (C::ROWB / 16) % KC;
          if (x0 + key < lo || x0 + key >= hi)
            *reinterpret_cast<uint4 *>(ring + stage * C::STAGE + C::KV_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();                 // before the stage's next boxes
        __syncwarp();
      }
      // ---- S^T = K Q^T: key 16 t + g8 (+ 8 from element 2 on), row 8 nt + 2 c4 + (e & 1)
      float s[KT][NR][4];
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][nt][e] = 0.f;
      if constexpr (FP8) {
#pragma unroll
        for (int gr = 0; gr < HD / 64; ++gr) {
          uint4 w[2 * KT];
#pragma unroll
          for (int n = 0; n < 2 * KT; ++n) {
            const int key = n * 8 + key_of(g8);
            const uint32_t ch = gr * 4 + c4;
            w[n] = pd_lds128(k_s + key * C::ROWB + ((HD == 64 ? ch ^ ((key >> 1) & 3) : ch ^ (key & 7)) << 4));
          }
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            uint32_t b[NR][4];
            take_q(q_s, gr * 2 + k2, b);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int t = 0; t < KT; ++t) {
                const int q4 = 2 * k2 + h;
                uint32_t a[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  const uint4 &v = w[2 * t + n];
                  const uint32_t u = q4 == 0 ? v.x : q4 == 1 ? v.y : q4 == 2 ? v.z : v.w;
                  const float2 f0 = unpack_e4m3x2(u), f1 = unpack_e4m3x2(u >> 16);
                  a[n] = pack_bf16x2(f0.x, f0.y);
                  a[2 + n] = pack_bf16x2(f1.x, f1.y);
                }
#pragma unroll
                for (int nt = 0; nt < NR; ++nt) pd_mma(s[t][nt], a, b[nt][2 * h], b[nt][2 * h + 1]);
              }
          }
        }
      } else {
        const uint32_t k_lane = k_s + (lane & 15) * 128;
#pragma unroll
        for (int k2 = 0; k2 < DT / 2; ++k2) {
          uint32_t b[NR][4];
          take_q(q_s, k2, b);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < KT; ++t) {
              uint32_t a[4];
              pd_ldsm4(a, k_lane + (k2 >> 1) * C::SUB_BYTES + t * 2048 + (((((k2 & 1) * 2 + h) * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
              for (int nt = 0; nt < NR; ++nt) pd_mma(s[t][nt], a, b[nt][2 * h], b[nt][2 * h + 1]);
            }
        }
      }
      // ---- scores in the exp2 domain, replaced where a row does not see the key
      const bool edge = x0 + KC - 1 > first_at || x0 < lo || (p.window > 0 && x0 <= first_at + (rows - 1) / p.G - p.window);
      if constexpr (FP8) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const float k0 = scales[t * 16 + key_of(g8)] * p.scale_log2, k1 = scales[t * 16 + 8 + key_of(g8)] * p.scale_log2;
#pragma unroll
          for (int nt = 0; nt < NR; ++nt) {
            s[t][nt][0] *= k0;
            s[t][nt][1] *= k0;
            s[t][nt][2] *= k1;
            s[t][nt][3] *= k1;
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NR; ++nt) {
        if (edge) {
          int own[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) own[i] = first_at + (nt * 8 + 2 * c4 + i) / p.G;   // past the unit's rows: not written
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = x0 + t * 16 + (e >> 1) * 8 + key_of(g8);
              if (x > own[e & 1] || (p.window > 0 && x <= own[e & 1] - p.window)) s[t][nt][e] = -INFINITY;
            }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          mx[0] = fmax3(mx[0], s[t][nt][0], s[t][nt][2]);
          mx[1] = fmax3(mx[1], s[t][nt][1], s[t][nt][3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], x));
          if (!FP8) mx[i] *= p.scale_log2;        // scale > 0; -inf stays -inf
        }
        if (__any_sync(0xffffffffu, mx[0] > m[nt][0] || mx[1] > m[nt][1])) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[nt][i], mx[i]);
            const float a = mn == -INFINITY ? 1.f : ex2_approx(m[nt][i] - mn);
            m[nt][i] = mn;
            l[nt][i] *= a;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              o[d][nt][i] *= a;
              o[d][nt][2 + i] *= a;
            }
          }
        }
        const float mu0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], mu1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
        float2 sum = make_float2(l[nt][0], l[nt][1]);
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float &f0 = s[t][nt][2 * h], &f1 = s[t][nt][2 * h + 1];
            float2 x;
            if constexpr (FP8) x = fadd2(f0, f1, -mu0, -mu1);
            else x = make_float2(fmaf(f0, p.scale_log2, -mu0), fmaf(f1, p.scale_log2, -mu1));
            f0 = ex2_approx(x.x);
            f1 = ex2_approx(x.y);
            sum = fadd2(sum.x, sum.y, f0, f1);
          }
        l[nt][0] = sum.x;
        l[nt][1] = sum.y;
      }
      // ---- O^T += V^T P^T; P rounded to bf16, the tensor core's operand type
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        uint32_t b[NR][2];
        float v0 = 1.f, v1 = 1.f;
        if constexpr (FP8) {
          v0 = scales[KC + t * 16 + key_of(g8)];
          v1 = scales[KC + t * 16 + 8 + key_of(g8)];
        }
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
          b[nt][0] = pd_turn(pack_bf16x2(s[t][nt][0] * v0, s[t][nt][1] * v0));
          b[nt][1] = pd_turn(pack_bf16x2(s[t][nt][2] * v1, s[t][nt][3] * v1));
        }
        if constexpr (FP8) {
          // a transposed load gives pairs of neighbouring dims: the even dims of 16 are a
          // tile's rows 0 .. 7, the odd ones its rows 8 .. 15
          const int key = t * 16 + key_of(lane & 15);
          const uint32_t row = v_s + key * C::ROWB;
#pragma unroll
          for (int c2 = 0; c2 < DT / 2; ++c2) {
            uint32_t u[4];
            const uint32_t ch = 2 * c2 + (lane >> 4);
            pd_ldsm4_t(u, row + ((HD == 64 ? ch ^ ((key >> 1) & 3) : ch ^ (key & 7)) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float2 p0 = unpack_e4m3x2(u[2 * h]), p1 = unpack_e4m3x2(u[2 * h] >> 16);
              const float2 p2 = unpack_e4m3x2(u[2 * h + 1]), p3 = unpack_e4m3x2(u[2 * h + 1] >> 16);
              const uint32_t a[4] = {pack_bf16x2(p0.x, p1.x), pack_bf16x2(p0.y, p1.y), pack_bf16x2(p2.x, p3.x),
                                     pack_bf16x2(p2.y, p3.y)};
#pragma unroll
              for (int nt = 0; nt < NR; ++nt) pd_mma(o[2 * c2 + h][nt], a, b[nt][0], b[nt][1]);
            }
          }
        } else {
          const uint32_t v_lane = v_s + t * 2048 + (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            uint32_t u[4];
            pd_ldsm4_t(u, (v_lane ^ ((d & 3) * 32)) + (d >> 2) * C::SUB_BYTES);
            const uint32_t a[4] = {u[0], u[2], u[1], u[3]};
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) pd_mma(o[d][nt], a, b[nt][0], b[nt][1]);
          }
        }
      }
    }
    if (flags & (kPdEnds | kPdLast)) {
      // ---- the unit, or this CTA's part of it, is done: merge the warps' states, those of
      // MERGE_WARPS warps at a time: 4 .. 7 into 0 .. 3, 2 and 3 into 0 and 1, 1 into 0
      const PdNote u = *note;
      const bool in_unit = units == 0 && started_inside, whole = (flags & kPdEnds) && !in_unit;
      PagedSeq us{};
      us.row0 = u.row0;
#pragma unroll
      for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x);
#pragma unroll 1
      for (int half = 4; half; half >>= 1) {
#pragma unroll 1
        for (int to = 0; to < half; to += C::MERGE_WARPS) {
          const int from = half + to, n = min(half, C::MERGE_WARPS);
          if (warp >= from && warp < from + n) {
            float4 *dst = reinterpret_cast<float4 *>(smem + C::OFF_MERGE + (warp - from) * C::STATE_BYTES) + lane;
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
              for (int d = 0; d < DT; ++d)
                dst[(nt * (DT + 1) + d) * 32] = make_float4(o[d][nt][0], o[d][nt][1], o[d][nt][2], o[d][nt][3]);
              dst[(nt * (DT + 1) + DT) * 32] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
            }
          }
          __syncthreads();
          if (warp >= to && warp < to + n) {
            const float4 *src = reinterpret_cast<const float4 *>(smem + C::OFF_MERGE + (warp - to) * C::STATE_BYTES) + lane;
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
              const float4 other = src[(nt * (DT + 1) + DT) * 32];
              const float m2[2] = {other.x, other.y}, l2[2] = {other.z, other.w};
              float a[2], a2[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float mn = fmaxf(m[nt][i], m2[i]);
                a[i] = mn == -INFINITY ? 1.f : ex2_approx(m[nt][i] - mn);
                a2[i] = mn == -INFINITY ? 1.f : ex2_approx(m2[i] - mn);
                m[nt][i] = mn;
                l[nt][i] = l[nt][i] * a[i] + l2[i] * a2[i];
              }
#pragma unroll
              for (int d = 0; d < DT; ++d) {
                const float4 v = src[(nt * (DT + 1) + d) * 32];
                o[d][nt][0] = o[d][nt][0] * a[0] + v.x * a2[0];
                o[d][nt][1] = o[d][nt][1] * a[1] + v.y * a2[1];
                o[d][nt][2] = o[d][nt][2] * a[0] + v.z * a2[0];
                o[d][nt][3] = o[d][nt][3] * a[1] + v.w * a2[1];
              }
            }
          }
          __syncthreads();
        }
      }
      // ---- the rows through shared memory, then a warp for each
      float2 *ml = reinterpret_cast<float2 *>(merge + C::ROWS * C::TILE_LD);
      if (warp == 0) {
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = nt * 8 + 2 * c4 + i;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              float *to = merge + r * C::TILE_LD + d * 16 + (FP8 ? 2 * g8 : g8);
              to[0] = o[d][nt][i];
              to[FP8 ? 1 : 8] = o[d][nt][2 + i];
            }
            if (g8 == 0) ml[r] = make_float2(m[nt][i], l[nt][i]);
          }
      }
      __syncthreads();
      float *part = paged_part(p.ws, cta, in_unit ? 0 : 1, C::ROWS, HD);
      for (int r = warp; r < rows; r += C::NW) {
        const float *row = merge + r * C::TILE_LD + lane * (HD / 32);
        const float2 st = ml[r];
        const float inv = st.y > 0.f ? 1.f / st.y : 0.f;
        uint8_t *to = p.o.data + 2 * (whole ? paged_unit_row(p.o, p, us, u.b, u.t0, u.kvh, r) + lane * (HD / 32) : 0);
        if constexpr (HD == 64) {
          const float2 v = *reinterpret_cast<const float2 *>(row);
          if (whole)
            *reinterpret_cast<uint32_t *>(to) = p.o_f16 ? pack_f16x2(v.x * inv, v.y * inv) : pack_bf16x2(v.x * inv, v.y * inv);
          else
            __stcg(reinterpret_cast<float2 *>(part + r * HD) + lane, v);
        } else {
          const float4 v = *reinterpret_cast<const float4 *>(row);
          if (whole)
            *reinterpret_cast<uint2 *>(to) =
                p.o_f16 ? make_uint2(pack_f16x2(v.x * inv, v.y * inv), pack_f16x2(v.z * inv, v.w * inv))
                        : make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
          else
            __stcg(reinterpret_cast<float4 *>(part + r * HD) + lane, v);
        }
        if (!whole && lane == 0) __stcg(reinterpret_cast<float2 *>(part + C::ROWS * HD + 2 * r), st);
      }
      if (whole) __syncthreads();                 // before the next unit's states
      if (!whole) {
        // ---- the CTA that brings a unit's last part combines them all.  The barriers
        // around make thread 0's fences stand for the whole CTA's parts.
        __syncthreads();
        if (tid == 0) {
          const int c0 = paged_worker_of(u.u0, total, workers), n = paged_worker_of(u.u0 + u.j01 - 1, total, workers) - c0 + 1;
          int *count = paged_counts(p.status) + c0;
          __threadfence();
          const bool mine = atomicAdd(count, 1) == n - 1;
          if (mine) {
            __threadfence();
            atomicExch(count, 0);                 // for the next call
          }
          s_parts[0] = c0;
          s_parts[1] = mine ? n : 0;
        }
        __syncthreads();
        const int c0 = s_parts[0], n = s_parts[1];
        if (n > 0) {
          float *weight = merge + warp * kPagedMaxCtas;
          for (int r = warp; r < rows; r += C::NW)
            paged_combine_row<HD>(p, C::ROWS, c0, n, r, weight, paged_unit_row(p.o, p, us, u.b, u.t0, u.kvh, r));
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
