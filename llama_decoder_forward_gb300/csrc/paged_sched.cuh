// paged_sched.cuh - how the paged attention kernels share a call's work among
// their CTAs, and where a CTA leaves what it has of a unit it does not finish.
//
// A unit is one sequence, one kv head and a tile of `tt` query tokens (with all
// g heads of each: tt * g rows that read the same keys).  Its work is a number of
// tiles of `1 << bk_shift` keys, from the first that its first row's window shows
// to the one of its last row.  The units of a call in the order (sequence, query
// tile, kv head) form one line of tiles, cut into equal pieces, one for each CTA:
// long caches, short ones, single tokens and chunks balance without a plan made
// on the host.  A unit cut by a border is finished by the combining kernel from
// the CTAs' partial results (unnormalised sums, row maxima and row sums).
#pragma once

#include "paged.cuh"

namespace smol {

// One unit of the line and the tile a worker stands at.
struct PagedIter {
  int b, qt, kvh, j;           // sequence, query tile, kv head, key tile
  int j0, j1;                  // the unit's key tiles
  int t0, nt;                  // its first token, and how many
  int lo, hi;                  // the positions that some row of it sees: [lo, hi)
  PagedSeq s;
  int left;                    // tiles of this worker still to do, this one included
  long long u0;                // the unit's first tile in the line
};

__device__ __forceinline__ int paged_cap(const PagedAttnParams &p) { return p.kv.max_pages << p.kv.page_shift; }

__device__ __forceinline__ void paged_unit_tiles(const PagedAttnParams &p, const PagedSeq &s, int qt, int &t0, int &nt,
                                                 int &lo, int &hi, int &j0, int &j1) {
  t0 = qt * p.tt;
  nt = min(p.tt, s.n - t0);
  hi = s.L + t0 + nt;
  lo = p.window > 0 ? max(0, s.L + t0 - p.window + 1) : 0;
  j0 = lo >> p.bk_shift;
  j1 = (hi + (1 << p.bk_shift) - 1) >> p.bk_shift;
}

__device__ __forceinline__ void paged_set_unit(const PagedAttnParams &p, PagedIter &it) {
  paged_unit_tiles(p, it.s, it.qt, it.t0, it.nt, it.lo, it.hi, it.j0, it.j1);
}

// To the next tile; past the unit's last one, to the next unit's first.
__device__ __forceinline__ void paged_next(const PagedAttnParams &p, PagedIter &it) {
  if (--it.left <= 0) return;
  if (++it.j < it.j1) return;
  it.u0 += it.j1 - it.j0;
  if (++it.kvh == p.kv.KV) {
    it.kvh = 0;
    if (++it.qt * p.tt >= it.s.n) {
      it.qt = 0;
      do {
        ++it.b;                                   // there is a further unit: left > 0
        it.s = paged_seq(p.c, it.b, paged_cap(p));
      } while (it.s.n == 0 && it.b + 1 < p.c.B);
    }
  }
  paged_set_unit(p, it);
  it.j = it.j0;
}

// Tiles of one sequence.
__device__ __forceinline__ long long paged_seq_tiles(const PagedAttnParams &p, const PagedSeq &s) {
  long long sum = 0;
  for (int qt = 0; qt * p.tt < s.n; ++qt) {
    int t0, nt, lo, hi, j0, j1;
    paged_unit_tiles(p, s, qt, t0, nt, lo, hi, j0, j1);
    sum += j1 - j0;
  }
  return sum * p.kv.KV;
}

struct PagedSchedSmem {
  long long warp_sum[32], total;
  int workers;
  PagedIter start;
};

// The worker that has tile x of the line.
__device__ __forceinline__ int paged_worker_of(long long x, long long total, int workers) {
  return static_cast<int>(paged_div((x + 1) * workers - 1, total));
}

// Worker `w` of `workers`: its first tile and how many it has (left == 0: none; the
// line is cut for as many workers as it has tiles, at most).  Called by all THREADS
// threads of the CTA.
template <int THREADS>
__device__ __forceinline__ PagedIter paged_locate(const PagedAttnParams &p, int w, int workers, PagedSchedSmem &sm) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = paged_cap(p);
  // the whole line
  long long mine = 0, first = 0;
  for (int b = tid; b < p.c.B; b += THREADS) {
    const PagedSeq s = paged_seq(p.c, b, cap);
    if (s.bad && w == 0) set_status(p.status, kDevBadInput);
    const long long n = paged_seq_tiles(p, s);
    if (b == tid) first = n;
    mine += n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sm.warp_sum[warp] = mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) total += sm.warp_sum[i];
  __syncthreads();
  PagedIter it{};
  if (total < workers) workers = static_cast<int>(total);
  if (tid == 0) {
    sm.total = total;
    sm.workers = workers;
  }
  if (w >= workers) return it;                    // the same for the whole CTA
  const long long from = paged_div(total * w, workers), to = paged_div(total * (w + 1), workers);
  // the sequence that holds tile `from`, THREADS sequences at a time
  long long before = 0;
  for (int base = 0; base < p.c.B; base += THREADS) {
    const int b = base + tid;
    long long n = first;
    PagedSeq s{};
    if (b < p.c.B) {
      s = paged_seq(p.c, b, cap);
      if (base) n = paged_seq_tiles(p, s);
    } else {
      n = 0;
    }
    long long inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) sm.warp_sum[warp] = inc;
    __syncthreads();
    long long pre = before + inc - n, round = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i < warp) pre += sm.warp_sum[i];
      round += sm.warp_sum[i];
    }
    if (pre <= from && from < pre + n) {
      it.b = b;
      it.s = s;
      it.left = static_cast<int>(to - from);
      long long off = from - pre;
      for (it.qt = 0;; ++it.qt) {
        paged_set_unit(p, it);
        const long long unit = it.j1 - it.j0, all = unit * p.kv.KV;
        if (off < all) {
          it.kvh = static_cast<int>(paged_div(off, unit));
          it.j = it.j0 + static_cast<int>(off - it.kvh * unit);
          it.u0 = from - (it.j - it.j0);
          break;
        }
        off -= all;
      }
      sm.start = it;
    }
    before += round;
    __syncthreads();
    if (from < before) break;                     // the same for the whole CTA
  }
  return sm.start;
}

// ---------------------------------------------------------------- partial results
// Each CTA has two places: 0 for a unit begun by an earlier CTA, 1 for one that
// it begins and does not finish.
struct PagedMeta {
  int in, ends;                // place 0 is used; that unit ends in this CTA
  int out;                     // place 1 is used
  int b, qt, kvh;              // place 1's unit
};
// (The few-rows kernel needs no note: it finds a unit's CTAs by arithmetic.)
constexpr int kPagedMaxCtas = 160;
// Behind the status word, in its block of 1024 bytes: a counter for each CTA, of the
// parts of the unit that it began.  They are zero between calls, the one thing that a
// call finds as an earlier one left it, so they lie where no size of a call moves
// them (the model's forward has its activations between that block and `ws`).
constexpr size_t kPagedCountOff = 256;
static_assert(kPagedCountOff + kPagedMaxCtas * sizeof(int) <= 1024, "the counters lie in the status block");
__device__ __forceinline__ int *paged_counts(int *status) { return status + kPagedCountOff / sizeof(int); }
// In `ws`, written before they are read in each call: the notes; the parts.
constexpr size_t kPagedMetaOff = 1024, kPagedPartOff = kPagedMetaOff + kPagedMaxCtas * sizeof(PagedMeta) + 256;

// Place of CTA c: rows of HD sums, then (maximum, sum) of each row.
__device__ __forceinline__ float *paged_part(uint8_t *ws, int c, int place, int rows, int hd) {
  return reinterpret_cast<float *>(ws + kPagedPartOff) + (static_cast<long long>(c) * 2 + place) * rows * (hd + 2);
}
__device__ __forceinline__ PagedMeta *paged_meta(uint8_t *ws) { return reinterpret_cast<PagedMeta *>(ws + kPagedMetaOff); }

// Row r of a unit from its n parts: CTA c0's place 1 and the place 0 of the ones
// behind it, in that order; o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.  One
// warp; `weight`: n floats of shared memory of its own; `out`: the row's offset.
template <int HD>
__device__ __forceinline__ void paged_combine_row(const PagedAttnParams &p, int rows, int c0, int n, int r, float *weight,
                                                  long long out) {
  const int lane = threadIdx.x & 31;
  constexpr int kHeld = (kPagedMaxCtas + 31) / 32;
  float2 ml[kHeld];                               // this lane's parts' maxima and sums
  float mx = -INFINITY, sum = 0.f;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = lane + 32 * k;
    ml[k] = make_float2(-INFINITY, 0.f);
    if (i < n) ml[k] = __ldcg(reinterpret_cast<const float2 *>(paged_part(p.ws, c0 + i, i == 0, rows, HD) + rows * HD + 2 * r));
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) mx = fmaxf(mx, ml[k].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = lane + 32 * k;
    const float a = mx == -INFINITY ? 0.f : ex2_approx(ml[k].x - mx);
    if (i < n) weight[i] = a;
    sum += a * ml[k].y;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  float acc[HD / 32];
#pragma unroll
  for (int e = 0; e < HD / 32; ++e) acc[e] = 0.f;
#pragma unroll 8
  for (int i = 0; i < n; ++i) {
    const float *row = paged_part(p.ws, c0 + i, i == 0, rows, HD) + r * HD + lane * (HD / 32);
    const float a = weight[i];
    if constexpr (HD == 64) {
      const float2 v = __ldcg(reinterpret_cast<const float2 *>(row));
      acc[0] += a * v.x;
      acc[1] += a * v.y;
    } else {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(row));
      acc[0] += a * v.x;
      acc[1] += a * v.y;
      acc[2] += a * v.z;
      acc[3] += a * v.w;
    }
  }
  uint32_t *to = reinterpret_cast<uint32_t *>(p.o.data + (out + lane * (HD / 32)) * 2);
#pragma unroll
  for (int e = 0; e < HD / 64; ++e)
    to[e] = p.o_f16 ? pack_f16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv) : pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  __syncwarp();                                   // the weights are rewritten
}

// Element offset of row r (token r / g, head r % g) of a unit in q or out.
__device__ __forceinline__ long long paged_unit_row(const PagedRows &x, const PagedAttnParams &p, const PagedSeq &s, int b,
                                                    int t0, int kvh, int r) {
  const int t = r / p.G;
  return paged_row_off(x, p.c, s, b, t0 + t, kvh * p.G + (r - t * p.G));
}

}  // namespace smol
