// verify.cu - verification of drafted tokens against the target's probabilities.
//
// p_i is the target's distribution after the tokens before draft i: the softmax
// of logits / temperature over what top-k and top-p leave (the rules of
// sample.cu), q_i the drafter's.  Draft x_i stays iff u_i q_i(x_i) < p_i(x_i); at
// the first that does not, the next token is drawn from max(p_i - q_i, 0), and
// from the row behind the drafts where all stay: then the tokens are distributed
// as the target's own.  The draw is the first index in vocabulary order at which
// the running sum exceeds u times the whole.
//
// Exactness.  A row of 50,000 or more running sums has a border within 1e-7 of u
// once in a hundred draws, so fp32 sums would pick another token than the
// definition.  Here a token's mass is e = 2^((l - l_max) log2(e) / temperature) as
// an integer in units of 2^-44, from an exponential good to some 2^-44 (mass_of),
// and every sum is a 64-bit integer: exact, and the same in any order.  The
// borders are then off by the masses' own errors only: some 1e-11 of the whole where
// those have both signs, up to V 2^-45 (4e-9 at V = 131072) where a long tail of equal
// values shares one, or falls below half a unit altogether.
//
// Two launches.
//   rows    one CTA for each target row, which it reads one to three times (from L2
//           after the first; in registers it would take half of them, and the spills
//           cost more).  bf16 logits take few distinct values, so the row becomes a
//           histogram over the values, and the exponential is taken once for each value
//           that occurs: a tenth of the row and less.  The counters of the values of
//           magnitude below 512 have 16 bits, two in a word, so that two CTAs of 512
//           threads share an SM (few rows: one of 1024 threads).  Where one ran over,
//           which the sum shows, or larger values count, the row is read again for 16,384
//           values at a time, with counters of 32 bits.  The sum, the k-th largest value
//           and the top-p cut are prefix sums over the histogram.
//           With top-k up to 256 another kernel does this without a histogram, two
//           CTAs on an SM: the k-th largest of the threads' own maxima is a bound
//           below which none of the k largest lies, and what reaches it, a little
//           more than k tokens, goes to a list in shared memory on which the filters
//           work token by token, in descending order (64 sequences of up to 5 drafts, V =
//           49152, top-k 50: the whole call takes 19 us, with the histogram 50).
//   choice  one cluster of eight CTAs for each sequence: the acceptances, then
//           the draw over one row, an eighth of the vocabulary for each CTA (or from
//           the row's list, one token for each thread of one CTA).
#include <math.h>

#include "common.cuh"
#include "prims.cuh"
#include "profile.cuh"
#include "verify.cuh"

namespace smol {
namespace {

typedef unsigned long long u64;

constexpr int kTopThreads = 512;     // of the kernel for a small top-k, and the tokens of its list
constexpr int kTopMaxK = 256;        // the largest top-k it takes
constexpr int kBatch = 6;            // 16-byte loads in flight in each thread
constexpr int kLoKey = 0x3c00, kHiKey = 0xc400;   // order keys of the values of magnitude below 512
constexpr int kPairs = (kHiKey - kLoKey) / 2;
constexpr int kWindow = 16384;       // keys that are counted together in 32 bits
constexpr int kRows = 0x10000 / 32;  // rows of 32 neighbouring values
constexpr int kChoiceThreads = 512;  // the most drafts of a sequence, too
constexpr int kChoiceCtas = 8;
constexpr float kMinLog2 = -45.f;    // 2^x below half a unit of 2^-44 counts as 0

// ---------------------------------------------------------------- masses
// 2^(j / 256), j = -128 .. 128, each as a sum of two floats: from 2^-0.5 by
// products with 2^(1/256), each rounded at 2^-63 (off by 2^-55 at most).
struct Pow2Table {
  float2 v[257];
  constexpr Pow2Table() : v() {
    unsigned __int128 x = 0x5a827999fcef3242ull;               // 2^-0.5 in units of 2^-63
    for (int j = 0; j < 257; ++j) {
      const u64 t = static_cast<u64>((x + 1) >> 1);            // units of 2^-62
      const float hi = static_cast<float>(static_cast<double>(t));
      const long long rest = static_cast<long long>(t - static_cast<u64>(static_cast<double>(hi)));
      v[j].x = static_cast<float>(static_cast<double>(hi) / 4611686018427387904.0);
      v[j].y = static_cast<float>(static_cast<double>(rest) / 4611686018427387904.0);
      // 2^(1/256) - 1 in units of 2^-63
      x += (x * 0x0058d7d2d5e5f6b1ull + (static_cast<unsigned __int128>(1) << 62)) >> 63;
    }
  }
};
__device__ constexpr Pow2Table kPow2{};

// Exponentials of one row: y = (l - l_max) * c with c = log2(e) / temperature.
struct MassCtx {
  float lmax, c_hi, c_lo;
  const float2 *table;               // kPow2 in shared memory
};

// round(2^44 * 2^y): the difference and the product are carried as sums of two
// floats (Dekker's and Knuth's exact sums and products), y is split into a whole
// number, 256ths from the table and a remainder r, |r| <= 2^-9, whose 2^r - 1 is
// a short series (Tang's table-driven exponential): the leading term in two
// floats, the others below 2^-18 in one.  Off by half a unit and, rarely, up to
// three (against extended precision, 1.2 million values).  Whole numbers come from
// adding 1.5 * 2^23: the conversion instructions share a slow pipe.
__device__ __forceinline__ u64 mass_of(const MassCtx &m, float l) {
  constexpr float kMagic = 12582912.f;
  constexpr int kMagicBits = 0x4b400000;
  const float dh = __fsub_rn(l, m.lmax);
  float yh = __fmul_rn(dh, m.c_hi);
  // not -inf, not NaN; and no value above l_max, which bins without tokens name: the
  // table's index is 0 .. 256 for y <= 0 only
  const bool counts = yh >= kMinLog2 && yh <= 0.f;
  yh = counts ? yh : 0.f;
  const float bb = __fsub_rn(dh, l);
  const float dl = __fsub_rn(__fsub_rn(l, __fsub_rn(dh, bb)), __fadd_rn(m.lmax, bb));
  const float yl = __fadd_rn(__fmaf_rn(dh, m.c_hi, -yh), __fmaf_rn(dh, m.c_lo, __fmul_rn(dl, m.c_hi)));
  const float ns = __fadd_rn(yh, kMagic), n = __fsub_rn(ns, kMagic);
  const float f = __fsub_rn(yh, n);
  const float js = __fmaf_rn(f, 256.f, kMagic), j = __fsub_rn(js, kMagic);
  const float f2 = __fmaf_rn(j, -0.00390625f, f);
  const float rh = __fadd_rn(f2, yl);
  const float rl = __fsub_rn(yl, __fsub_rn(rh, f2));
  // ln 2 as a sum of two floats; ln2^2 / 2, ln2^3 / 6, ln2^4 / 24
  constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654299957768e-9f;
  const float ph = __fmul_rn(rh, kLn2Hi);
  const float pl = __fadd_rn(__fmaf_rn(rh, kLn2Hi, -ph), __fmaf_rn(rh, kLn2Lo, __fmul_rn(rl, kLn2Hi)));
  const float s = __fmaf_rn(__fmaf_rn(rh, 0.009618129107628f, 0.055504108664822f), rh, 0.240226506959101f);
  const float rest = __fmaf_rn(__fmul_rn(rh, rh), s, pl);
  const float h = __fadd_rn(ph, rest), lo = __fsub_rn(rest, __fsub_rn(h, ph));   // 2^r - 1
  const float2 t = m.table[__float_as_int(js) - kMagicBits + 128];
  // t (1 + h + lo)
  const float p = __fmul_rn(t.x, h), pe = __fmaf_rn(t.x, h, -p);
  const float eh = __fadd_rn(t.x, p);
  const float el = __fadd_rn(__fsub_rn(p, __fsub_rn(eh, t.x)), __fadd_rn(__fmaf_rn(t.x, lo, pe), __fmaf_rn(t.y, h, t.y)));
  // in units of 2^-44: whole multiples of 2^23 (at most 2^21.5 of them), and the rest
  const float scale = __int_as_float((127 + 44 + __float_as_int(ns) - kMagicBits) << 23);
  const float v = __fmul_rn(eh, scale);
  const float his = __fmaf_rn(v, 1.1920928955078125e-7f, kMagic);
  const float rem = __fmaf_rn(__fsub_rn(his, kMagic), -8388608.f, v);
  const float los = __fadd_rn(__fmaf_rn(el, scale, rem), kMagic);
  const long long mass = static_cast<long long>(__float_as_int(his) - kMagicBits) * 8388608ll + (__float_as_int(los) - kMagicBits);
  return counts ? static_cast<u64>(mass) : dh == 0.f ? 1ull << 44 : 0ull;   // l_max itself where c is infinite
}

// floor(q * z) for z < 2^63 (a q that is negative or NaN counts as 0, one of 2 or
// more as just under 2).
__device__ __forceinline__ u64 scaled_floor(float q, u64 z) {
  if (!(q > 0.f)) return 0;
  const uint32_t bits = min(__float_as_uint(q), 0x3fffffffu);
  const int ex = static_cast<int>(bits >> 23);
  const u64 man = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int s = 150 - max(ex, 1);                                     // q = man * 2^-s, s >= 23
  const u64 lo = man * z, hi = __umul64hi(man, z);
  if (s >= 64) return s >= 128 ? 0 : hi >> (s - 64);
  return (hi << (64 - s)) | (lo >> s);
}

// z as a sum of two floats, to 2^-48.
__device__ __forceinline__ float rest_of(u64 z, float zh) {
  return __ll2float_rn(static_cast<long long>(z - __float2ull_rn(zh)));
}

// max(m - q z, 0), the product as a sum of two floats: off by less than a unit where
// it matters, next to a mass of at most 2^44.
__device__ __forceinline__ u64 mass_less(u64 m, float q, float zh, float zl) {
  constexpr float kMagic = 12582912.f;
  const float ph = __fmul_rn(q, zh), pl = __fmaf_rn(q, zl, __fmaf_rn(q, zh, -ph));
  if (!(ph > 0.f)) return m;                      // also a NaN
  if (ph >= 17592186044416.f) return 0;           // 2^44: no mass is larger
  const float his = __fmaf_rn(ph, 1.1920928955078125e-7f, kMagic);
  const float los = __fadd_rn(__fadd_rn(__fmaf_rn(__fsub_rn(his, kMagic), -8388608.f, ph), pl), kMagic);
  const long long have = static_cast<long long>(__float_as_int(his) - 0x4b400000) * 8388608ll + (__float_as_int(los) - 0x4b400000);
  const long long left = static_cast<long long>(m) - have;
  return left > 0 ? static_cast<u64>(left) : 0;
}
__device__ __forceinline__ u64 mass_less(u64 m, float q, u64 z) {
  const float zh = __ull2float_rn(z);
  return mass_less(m, q, zh, rest_of(z, zh));
}

// ---------------------------------------------------------------- rows in chunks
// A row of V bf16 as chunks of eight tokens whose 16 bytes are aligned: chunk c
// holds the tokens base + 8 c .. + 7, base in (-8, 0].  Tokens outside the row
// read as -infinity (mass 0, below every other value).
struct Row {
  const uint16_t *p;
  int V, base, chunks;
};

__device__ __forceinline__ Row make_row(const uint16_t *p, int V) {
  Row r;
  r.p = p;
  r.V = V;
  const int past = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) >> 1);   // tokens past a 16-byte border
  r.base = -past;
  r.chunks = (V + past + 7) >> 3;
  return r;
}

__device__ __forceinline__ uint4 load_chunk(const Row &r, int c) {
  const int i = r.base + 8 * c;
  if (i >= 0 && i + 8 <= r.V) return *reinterpret_cast<const uint4 *>(r.p + i);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int a = i + 2 * e;
    const uint32_t lo = a >= 0 && a < r.V ? r.p[a] : 0xff80u, hi = a + 1 >= 0 && a + 1 < r.V ? r.p[a + 1] : 0xff80u;
    w[e] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Element e of a chunk of eight 16-bit values.
__device__ __forceinline__ uint32_t chunk_half(const uint4 &c, int e) {
  const uint32_t w = (e >> 1) == 0 ? c.x : (e >> 1) == 1 ? c.y : (e >> 1) == 2 ? c.z : c.w;
  return (e & 1) ? w >> 16 : w & 0xffffu;
}

// bf16_order_key of two values: all bits of a negative one flipped, the sign of
// another; adding +0 has turned -0 into +0.
__device__ __forceinline__ uint32_t order_key2(uint32_t w) {
  const __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&w), __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)));
  w = *reinterpret_cast<const uint32_t *>(&v);
  uint32_t sign;                                  // 0xffff where negative (the bytes' sign replicated)
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(sign) : "r"(w));
  return w ^ (sign | 0x80008000u);
}

__device__ __forceinline__ uint4 chunk_keys(const uint4 &c) {
  return make_uint4(order_key2(c.x), order_key2(c.y), order_key2(c.z), order_key2(c.w));
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {   // of two pairs of 16 bits
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The larger of the upper keys and of the lower ones, side by side.
__device__ __forceinline__ uint32_t chunk_max2(const uint4 &k) { return max2(max2(k.x, k.y), max2(k.z, k.w)); }

__device__ __forceinline__ float key_value(uint32_t key) {
  const uint32_t bits = (key & 0x8000u) ? key & 0x7fffu : ~key & 0xffffu;
  return __uint_as_float(bits << 16);
}

// Adds `by` to the counter at `to`, and 1 to n, where d < span, without a branch.
__device__ __forceinline__ void count_in(uint32_t to, uint32_t by, uint32_t d, uint32_t span, uint32_t &n) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %3, %4;\n\t@p red.shared.add.u32 [%1], %2;\n\t@p add.u32 %0, %0, 1;\n\t}"
               : "+r"(n)
               : "r"(to), "r"(by), "r"(d), "r"(span)
               : "memory");
}

// ---------------------------------------------------------------- block sums
template <int THREADS>
__device__ __forceinline__ u64 block_scan(u64 v, u64 *sh, u64 *total) {   // exclusive
  constexpr int W = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const u64 w = lane < W ? sh[lane] : 0;
    u64 wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 t = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += t;
    }
    if (lane < W) sh[lane] = wi - w;
    if (lane == 31) sh[32] = wi;
  }
  __syncthreads();
  const u64 before = sh[warp];
  *total = sh[32];
  __syncthreads();
  return before + inc - v;
}

// Sum over the block (exact), for every thread.
template <int THREADS>
__device__ __forceinline__ u64 block_sum(u64 v, u64 *sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 t = (threadIdx.x & 31) < THREADS / 32 ? sh[threadIdx.x & 31] : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  __syncthreads();                                // sh may be reused
  return t;
}

__device__ __forceinline__ u64 warp_max(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---------------------------------------------------------------- rows
struct RowSmem {
  unsigned hist[kPairs];             // two counters of 16 bits in a word, or one of 32 bits for each of kWindow keys
  unsigned row_count[kRows];  // tokens, and masses, of 32 neighbouring values, the largest first
  u64 row_mass[kRows];
  float2 table[257];
  u64 red[33];
  unsigned bins[32];
  u64 before_mass, z, t_cut;
  unsigned before_count;
  int found, bin, x_cut;
};

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) verify_rows_kernel(const VerifyParams p) {
  constexpr int WARPS = THREADS / 32, PER = kRows / THREADS;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  RowSmem &S = *reinterpret_cast<RowSmem *>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / (p.T + 1), i = blockIdx.x - b * (p.T + 1);
  griddep_launch_dependents();
  int n = p.T;
  if (p.n_draft) {
    const int v = p.n_draft[b];
    n = min(max(v, 0), p.T);
    if (n != v && i == 0 && tid == 0) set_status(p.status, kDevBadInput);
  }
  const long long at = static_cast<long long>(b) * p.T + i;
  if (i >= n && i < p.T && p.p_draft && tid == 0) p.p_draft[at] = 0.f;   // no draft in this row
  if (i > n) return;
  const Row row = make_row(p.logits + static_cast<long long>(blockIdx.x) * p.ld, p.V);

  // fn(chunk, its eight order keys in pairs), over this thread's chunks, a batch of
  // loads at a time; `between` runs with the first batch under way and is given the
  // largest of its keys by a call
  auto for_chunks = [&](auto &&fn, auto &&between) {
    bool start = true;
    for (int c0 = tid; start || c0 < row.chunks; c0 += kBatch * THREADS) {
      uint4 w[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (c0 + k * THREADS < row.chunks) w[k] = load_chunk(row, c0 + k * THREADS);
      if (start)
        between([&] {
          uint32_t top2 = 0;
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            if (c0 + k * THREADS < row.chunks) top2 = max2(top2, chunk_max2(chunk_keys(w[k])));
          return max(top2 & 0xffffu, top2 >> 16);
        });
      start = false;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (c0 + k * THREADS < row.chunks) fn(c0 + k * THREADS, chunk_keys(w[k]));
    }
  };
  auto nothing = [](auto &&) {};
  auto block_max = [&](uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (lane == 0) S.red[warp] = v;
    __syncthreads();
    v = __reduce_max_sync(0xffffffffu, lane < WARPS ? static_cast<uint32_t>(S.red[lane]) : 0u);
    __syncthreads();
    return v;
  };
  auto clear = [&] {
    for (int k = tid; k < kPairs / 4; k += THREADS) reinterpret_cast<uint4 *>(S.hist)[k] = make_uint4(0, 0, 0, 0);
  };
  // a value below l_max - 32 temperature has mass 0 (45 ln 2 = 31.2): the smallest key
  // that counts (one to spare for the truncation)
  auto least_key = [&](uint32_t kmax) {
    const float least = key_value(kmax) - 32.f * p.temperature;
    if (!(least > -INFINITY)) return 0u;
    const uint32_t k = bf16_order_key(static_cast<uint16_t>(__float_as_uint(least) >> 16));
    return k > 0 ? k - 1 : 0u;
  };
  // one pass for the values of magnitude below 512: the keys' maximum, and how many of
  // this thread's were counted.  The largest of the first batch bounds what is counted.
  uint32_t counted = 0;
  auto count_packed = [&] {
    uint32_t top2 = 0, from = 0, span = 0;
    const uint32_t base = smem_u32(S.hist) - 2 * kLoKey;
    for_chunks([&](int, const uint4 &k) {
      top2 = max2(top2, chunk_max2(k));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t key = chunk_half(k, e);
        count_in(base + 2 * (key & 0xfffeu), 1u + (key & 1u) * 0xffffu, key - from, span, counted);
      }
    }, [&](auto &&first_max) {
      clear();
      from = max(least_key(block_max(first_max())), static_cast<uint32_t>(kLoKey));
      span = from < kHiKey ? kHiKey - from : 0u;
    });
    return max(top2 & 0xffffu, top2 >> 16);
  };
  // the keys of one window of kWindow, those >= from
  auto count_window = [&](int window, uint32_t from) {
    const uint32_t low = 0x10000u - (window + 1) * kWindow, lo = max(low, from), span = low + kWindow - lo;
    const uint32_t base = smem_u32(S.hist) - 4 * low;
    uint32_t all = 0;
    for_chunks([&](int, const uint4 &k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) count_in(base + 4 * chunk_half(k, e), 1u, chunk_half(k, e) - lo, span, all);
    }, [&](auto &&) {
      clear();
      __syncthreads();
    });
    __syncthreads();
  };

  // ---- the largest value, with the histogram on the way
  const bool use_k = p.top_k > 0 && p.top_k < p.V, use_p = p.top_p < 1.f;
  u64 best = 0;
  if (p.greedy) {
    for_chunks([&](int c, const uint4 &k) {       // chunks ascend: the first of equal values stays
      const uint32_t t2 = chunk_max2(k), t = max(t2 & 0xffffu, t2 >> 16);
      if (t > static_cast<uint32_t>(best >> 32)) {
        int x = 0;
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (chunk_half(k, e) == t) x = row.base + 8 * c + e;
        best = argmax_pack(t, x);
      }
    }, nothing);
  } else {
    best = argmax_pack(count_packed(), 0);
  }
  best = warp_max(best);
  if (lane == 0) S.red[warp] = best;
  for (int k = tid; k < 257; k += THREADS) S.table[k] = kPow2.v[k];
  if (tid == 0) S.x_cut = p.V;
  __syncthreads();
  best = warp_max(lane < WARPS ? S.red[lane] : 0);
  __syncthreads();
  const uint32_t kmax = static_cast<uint32_t>(best >> 32);
  const float lmax = key_value(kmax);
  const bool fine = lmax > -INFINITY && lmax < INFINITY;              // NaN and infinities: no distribution
  VerifyRow out{};
  out.listed = -1;
  out.argmax = fine && p.greedy ? argmax_index(best) : -1;
  out.lmax = lmax;
  const int x = i < n ? p.drafts[at] : -1;
  const bool x_ok = x >= 0 && x < p.V;
  if (tid == 0 && (!fine || (i < n && !x_ok))) set_status(p.status, kDevBadInput);
  if (p.greedy || !fine) {
    out.z = fine ? 1 : 0;
    out.mx = fine && x_ok && x == out.argmax ? 1 : 0;
    if (tid == 0) {
      p.rows[blockIdx.x] = out;
      if (i < n && p.p_draft) p.p_draft[at] = out.mx ? 1.f : 0.f;
    }
    return;
  }
  const MassCtx mc = MassCtx{lmax, p.c_hi, p.c_lo, S.table};
  // ---- counts and masses of rows of 32 neighbouring values, the largest first: row r has
  // the keys 0xffff - 32 r - (0 .. 31)
  for (int k = tid; k < kRows; k += THREADS) {
    S.row_count[k] = 0;
    S.row_mass[k] = 0;
  }
  __syncthreads();
  constexpr int kPacked = -1;
  int resident = kPacked;                         // what the histogram holds, or the window
  u64 total_m = 0;
  unsigned held = 0;
  // a warp looks through its blocks of 64 keys first: two in each lane
  {
    constexpr int BLOCKS = kPairs / 32 / WARPS;
    static_assert(BLOCKS * 32 * WARPS == kPairs && BLOCKS <= 64, "the same number of blocks for every warp");
    const unsigned *mine = S.hist + warp * 32 + lane;
    u64 some = 0;
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) some |= static_cast<u64>(__any_sync(0xffffffffu, mine[k * THREADS] != 0) ? 1 : 0) << k;
#pragma unroll 1
    for (; some; some &= some - 1) {
      const int k = __ffsll(static_cast<long long>(some)) - 1, block = warp + k * WARPS;
      const unsigned w = mine[k * THREADS], c0 = w & 0xffffu, c1 = w >> 16;
      const uint32_t key = kLoKey + 64 * block + 2 * lane;
      u64 ms = 0;
      if (c0) ms = mass_of(mc, key_value(key)) * c0;
      if (c1) ms += mass_of(mc, key_value(key + 1)) * c1;
      held += c0 + c1;
      if (!use_k && !use_p) {                     // only the whole sum is wanted
        total_m += ms;
      } else {
        unsigned cs = c0 + c1;
#pragma unroll
        for (int o = 8; o; o >>= 1) {
          cs += __shfl_xor_sync(0xffffffffu, cs, o);
          ms += __shfl_xor_sync(0xffffffffu, ms, o);
        }
        if ((lane & 15) == 0) {
          const int r = (0xffff - static_cast<int>(key)) >> 5;        // the lower 32 keys are the later row
          S.row_count[r] = cs;
          S.row_mass[r] = ms;
        }
      }
    }
  }
  const uint32_t least = least_key(kmax);
  // a counter of 16 bits that ran over takes 65,535 or 65,536 from the sum
  const bool spoilt = block_sum<THREADS>(static_cast<int>(held - counted), S.red) != 0;
  if (!use_k && !use_p) total_m = block_sum<THREADS>(total_m, S.red);
  if (spoilt || kmax >= kHiKey || least < kLoKey) {
    // so did one, or values of 512 and more count: a window of the keys at a time, with
    // counters of 32 bits, down to the smallest key that counts or the k-th largest
    u64 have = 0;
    for (int k = tid; k < kRows; k += THREADS) {
      S.row_count[k] = 0;
      S.row_mass[k] = 0;
    }
    for (int window = 0; window < 0x10000 / kWindow; ++window) {
      if (0xffffu - window * kWindow < least || (use_k && have >= static_cast<u64>(p.top_k))) break;
      resident = window;
      count_window(window, least);
      unsigned mine = 0;
      for (int j = warp; j < kWindow / 32; j += WARPS) {
        const unsigned c = S.hist[kWindow - 1 - 32 * j - lane];
        if (!__any_sync(0xffffffffu, c != 0)) continue;
        const int r = window * (kWindow / 32) + j;
        u64 ms = c ? mass_of(mc, key_value(0xffffu - 32 * r - lane)) * c : 0;
        const unsigned cs = __reduce_add_sync(0xffffffffu, c);
#pragma unroll
        for (int o = 16; o; o >>= 1) ms += __shfl_xor_sync(0xffffffffu, ms, o);
        mine += c;
        if (lane == 0) {
          S.row_count[r] = cs;
          S.row_mass[r] = ms;
        }
      }
      have += block_sum<THREADS>(mine, S.red);
    }
  }
  // prefix sums over the rows, PER for each thread
  u64 total_c = 0, pc = 0, pm = 0, m_of[PER] = {}, mm = 0;
  unsigned c_of[PER] = {}, cc = 0;
  if (use_k || use_p || resident != kPacked) {
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      cc += c_of[q] = S.row_count[PER * tid + q];
      mm += m_of[q] = S.row_mass[PER * tid + q];
    }
    pc = block_scan<THREADS>(cc, S.red, &total_c);
    pm = block_scan<THREADS>(mm, S.red, &total_m);
  }

  // the counters of one row of 32 values, into S.bins
  auto fetch_bins = [&](int r) {
    const int top = 0xffff - 32 * r;
    const bool here = resident == kPacked || r / (kWindow / 32) == resident;
    if (tid < 32)
      S.bins[tid] = !here                 ? 0u
                    : resident == kPacked ? reinterpret_cast<const uint16_t *>(S.hist)[top - tid - kLoKey]
                                          : S.hist[kWindow - 1 - 32 * (r % (kWindow / 32)) - tid];
    __syncthreads();
    if (here) return;
    for_chunks([&](int, const uint4 &k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t d = static_cast<uint32_t>(top) - chunk_half(k, e);
        if (d < 32u) atomicAdd(&S.bins[d], 1u);
      }
    }, nothing);
    __syncthreads();
  };
  auto key_of = [&](int r, int bin) { return static_cast<uint32_t>(0xffff - 32 * r - bin); };

  // ---- top-k: the k-th largest value; where fewer than k have a mass, all stay
  uint32_t vcut = 0;                              // values above stay, and of this one the tokens up to xcut
  int xcut = p.V;
  u64 z = total_m;
  const u64 k_th = static_cast<u64>(max(p.top_k, 0));
  if (use_k && total_c >= k_th) {
    u64 c_before = pc, m_before = pm;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (c_before < k_th && k_th <= c_before + c_of[q]) {
        S.found = PER * tid + q;
        S.before_count = static_cast<unsigned>(c_before);
        S.before_mass = m_before;
      }
      c_before += c_of[q];
      m_before += m_of[q];
    }
    __syncthreads();
    const int r = S.found;
    fetch_bins(r);
    if (warp == 0) {
      const unsigned c = S.bins[lane];
      unsigned ci = c;
      const u64 m = c ? mass_of(mc, key_value(key_of(r, lane))) * c : 0;
      u64 mi = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned tc = __shfl_up_sync(0xffffffffu, ci, o);
        const u64 tm = __shfl_up_sync(0xffffffffu, mi, o);
        if (lane >= o) {
          ci += tc;
          mi += tm;
        }
      }
      const int bin = __ffs(__ballot_sync(0xffffffffu, S.before_count + ci >= k_th)) - 1;
      if (lane == bin) {
        S.bin = bin;
        S.z = S.before_mass + mi;
      }
    }
    __syncthreads();
    vcut = key_of(r, S.bin);
    z = S.z;
    __syncthreads();
  }
  // ---- top-p: the value at which the running mass first exceeds top_p of the whole
  if (use_p) {
    if (tid == 0) {
      S.found = -1;
      S.t_cut = static_cast<u64>(static_cast<double>(p.top_p) * static_cast<double>(z));
    }
    __syncthreads();
    const u64 goal = S.t_cut;                     // a whole sum exceeds top_p z iff it exceeds its floor
    auto over = [&](u64 v) { return v > goal; };
    u64 m_before = pm;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      if (!over(m_before) && over(m_before + m_of[q])) {
        S.found = PER * tid + q;
        S.before_mass = m_before;
      }
      m_before += m_of[q];
    }
    __syncthreads();
    const int r = S.found;                        // found: z > goal
    if (r >= 0) {
      fetch_bins(r);
      if (warp == 0) {
        const unsigned c = S.bins[lane];
        const u64 one = c ? mass_of(mc, key_value(key_of(r, lane))) : 0, m = one * c;
        u64 mi = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 tm = __shfl_up_sync(0xffffffffu, mi, o);
          if (lane >= o) mi += tm;
        }
        const int bin = __ffs(__ballot_sync(0xffffffffu, over(S.before_mass + mi))) - 1;
        if (lane == bin) {
          // equal values have equal masses: the first t + 1 of them in index order stay
          const u64 above = S.before_mass + mi - m;
          const u64 tc = min((goal - above) / one, static_cast<u64>(c - 1));
          S.bin = bin;
          S.t_cut = tc + 1 < c ? tc : ~0ull;      // ~0: all of them
          S.z = above + (tc + 1) * one;
        }
      }
      __syncthreads();
      const uint32_t v = key_of(r, S.bin);
      const u64 tc = S.t_cut;
      z = S.z;
      vcut = v;
      if (tc != ~0ull) {
        // the index of the (t + 1)-th token of this value: counts in vocabulary
        // order, a round of a chunk for each thread at a time
        u64 seen = 0;
        for (int c_first = 0; c_first < row.chunks; c_first += THREADS) {
          const int c = c_first + tid;
          uint4 k = make_uint4(0, 0, 0, 0);       // key 0 is a NaN, never the cut
          if (c < row.chunks) k = chunk_keys(load_chunk(row, c));
          unsigned mine = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) mine += chunk_half(k, e) == v;
          u64 all;
          u64 rank = seen + block_scan<THREADS>(mine, S.red, &all);
          if (rank <= tc && tc < rank + mine) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (chunk_half(k, e) == v && rank++ == tc) S.x_cut = row.base + 8 * c + e;
          }
          seen += all;
          if (seen > tc) break;                   // the same for every thread
        }
        __syncthreads();
        xcut = S.x_cut;
      }
    }
  }
  if (tid == 0) {
    out.z = z;
    out.vcut = vcut;
    out.xcut = xcut;
    if (x_ok) {
      const uint32_t key = bf16_order_key(row.p[x]);
      if (key > vcut || (key == vcut && x <= xcut)) out.mx = mass_of(mc, key_value(key));
    }
    p.rows[blockIdx.x] = out;
    if (i < n && p.p_draft) p.p_draft[at] = static_cast<float>(static_cast<double>(out.mx) / static_cast<double>(z));
  }
}

// ---------------------------------------------------------------- rows, small top-k
struct TopSmem {
  float2 table[257];
  u64 red[33];
  alignas(16) u64 token[kTopThreads];    // order key, and the index's complement: larger goes before
  u64 z;
  unsigned n, best, vcut;
  int x_cut;
};

__global__ void __launch_bounds__(kTopThreads, 2) verify_top_kernel(const VerifyParams p) {
  __shared__ TopSmem S;
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = blockIdx.x / (p.T + 1), i = blockIdx.x - b * (p.T + 1);
  griddep_launch_dependents();
  int n_draft = p.T;
  if (p.n_draft) {
    const int v = p.n_draft[b];
    n_draft = min(max(v, 0), p.T);
    if (n_draft != v && i == 0 && tid == 0) set_status(p.status, kDevBadInput);
  }
  const long long at = static_cast<long long>(b) * p.T + i;
  if (i >= n_draft && i < p.T && p.p_draft && tid == 0) p.p_draft[at] = 0.f;   // no draft in this row
  if (i > n_draft) return;
  const Row row = make_row(p.logits + static_cast<long long>(blockIdx.x) * p.ld, p.V);
  const int x_in = i < n_draft ? p.drafts[at] : -1;
  const bool x_ok = x_in >= 0 && x_in < p.V;
  auto for_chunks = [&](auto &&fn) {              // fn(chunk, its eight order keys in pairs), some loads at a time
    for (int c0 = tid; c0 < row.chunks; c0 += kBatch * kTopThreads) {
      uint4 w[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (c0 + k * kTopThreads < row.chunks) w[k] = load_chunk(row, c0 + k * kTopThreads);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (c0 + k * kTopThreads < row.chunks) fn(c0 + k * kTopThreads, chunk_keys(w[k]));
    }
  };
  for (int k = tid; k < 257; k += kTopThreads) S.table[k] = kPow2.v[k];
  if (tid == 0) {
    S.n = S.best = 0;
    S.x_cut = -1;
  }
  uint32_t top2 = 0;                              // two maxima side by side
  for_chunks([&](int, const uint4 &k) { top2 = max2(top2, chunk_max2(k)); });
  const uint32_t my_max = max(top2 & 0xffffu, top2 >> 16);
  __syncthreads();
  const uint32_t warp_best = __reduce_max_sync(0xffffffffu, my_max);
  if (lane == 0) atomicMax(&S.best, warp_best);
  // the largest bound that k of the maxima reach, bit by bit (0: fewer than k threads have a chunk)
  auto bound_of = [&](auto &&reach) {
    uint32_t t = 0;
#pragma unroll 1
    for (uint32_t bit = 0x8000u; bit; bit >>= 1)
      if (reach(t | bit)) t |= bit;
    return t;
  };
  const uint32_t least = bound_of([&](uint32_t t) { return __syncthreads_count(my_max >= t) >= p.top_k; });
  const float lmax = key_value(S.best);
  const bool fine = lmax > -INFINITY && lmax < INFINITY;              // NaN and infinities: no distribution
  if (tid == 0 && (!fine || (i < n_draft && !x_ok))) set_status(p.status, kDevBadInput);
  VerifyRow out{};
  out.argmax = out.listed = -1;
  out.lmax = lmax;
  if (!fine) {
    if (tid == 0) {
      p.rows[blockIdx.x] = out;
      if (i < n_draft && p.p_draft) p.p_draft[at] = 0.f;
    }
    return;
  }
  const MassCtx mc{lmax, p.c_hi, p.c_lo, S.table};
  const bool use_p = p.top_p < 1.f;
  uint32_t vcut = 0;                              // values above stay, and of this one the tokens up to xcut
  int xcut = p.V;
  u64 z = 0;
  // ---- what reaches the bound
  for_chunks([&](int c, const uint4 &k) {
    const uint32_t t2 = chunk_max2(k);
    if (max(t2 & 0xffffu, t2 >> 16) < least) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int x = row.base + 8 * c + e;
      if (chunk_half(k, e) < least || x < 0 || x >= p.V) continue;
      const unsigned to = atomicAdd(&S.n, 1u);
      if (to < kTopThreads) S.token[to] = argmax_pack(chunk_half(k, e), x);
    }
  });
  __syncthreads();
  const int n = static_cast<int>(S.n);
  if (n >= p.top_k && n <= kTopThreads) {
    // in descending order, equal values in index order: a token's place is the number before it
    const u64 token = tid < n ? S.token[tid] : 0;
    int place = tid;
    if (tid < n) {
      place = 0;
      int i = 0;
#pragma unroll 8
      for (; i + 1 < n; i += 2) {
        const ulonglong2 two = *reinterpret_cast<const ulonglong2 *>(&S.token[i]);
        place += (two.x > token) + (two.y > token);
      }
      if (i < n) place += S.token[i] > token;
    }
    __syncthreads();
    S.token[place] = token;
    __syncthreads();
    const u64 own = S.token[tid];
    const uint32_t key = static_cast<uint32_t>(own >> 32);
    const int x = argmax_index(own);
    vcut = static_cast<uint32_t>(S.token[p.top_k - 1] >> 32);         // the k-th largest value
    const u64 mass = tid < n && key >= vcut ? mass_of(mc, key_value(key)) : 0;
    const u64 before = block_scan<kTopThreads>(mass, S.red, &z);
    bool stays = mass != 0;
    if (use_p) {
      // a token stays while what comes before it does not exceed top_p of the whole
      const u64 goal = static_cast<u64>(static_cast<double>(p.top_p) * static_cast<double>(z));
      stays = stays && before <= goal;
    }
    const int many = __syncthreads_count(stays);  // the first ones: masses descend, sums grow
    if (use_p) {
      if (tid == many - 1) {
        S.z = before + mass;
        S.vcut = key;
        S.x_cut = x;
      }
      __syncthreads();
      z = S.z;
      vcut = S.vcut;
      xcut = S.x_cut;
    }
    if (stays && tid < kVerifyList) p.lists[static_cast<long long>(blockIdx.x) * kVerifyList + tid] = VerifyToken{mass, x, 0};
    if (many <= kVerifyList) out.listed = many;
  } else {
    // ---- fewer chunks than k, or many equal values: by passes over the row
    auto mass_from = [&](uint32_t t) {
      u64 m = 0;
      for_chunks([&](int, const uint4 &k) {
#pragma unroll 1
        for (int e = 0; e < 8; ++e)
          if (chunk_half(k, e) >= t) m += mass_of(mc, key_value(chunk_half(k, e)));
      });
      return block_sum<kTopThreads>(m, S.red);
    };
    auto count_from_key = [&](uint32_t t) {
      u64 m = 0;
      for_chunks([&](int c, const uint4 &k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int x = row.base + 8 * c + e;
          m += chunk_half(k, e) >= t && x >= 0 && x < p.V;
        }
      });
      return block_sum<kTopThreads>(m, S.red);
    };
    vcut = bound_of([&](uint32_t t) { return count_from_key(t) >= static_cast<u64>(p.top_k); });
    z = mass_from(vcut);
    if (use_p) {
      const u64 goal = static_cast<u64>(static_cast<double>(p.top_p) * static_cast<double>(z));
      const uint32_t v = bound_of([&](uint32_t t) { return mass_from(t) > goal; });   // at least the k-th largest: z > goal
      const u64 above = mass_from(v + 1), one = mass_of(mc, key_value(v));
      const u64 c = count_from_key(v) - count_from_key(v + 1), tc = min((goal - above) / one, c - 1);
      z = above + (tc + 1) * one;
      vcut = v;
      // the index of the (tc + 1)-th token of this value, a round of chunks at a time
      u64 seen = 0;
      for (int c_first = 0; c_first < row.chunks && seen <= tc; c_first += kTopThreads) {
        const int cc = c_first + tid;
        uint4 k = make_uint4(0, 0, 0, 0);         // key 0 is a NaN, never the cut
        if (cc < row.chunks) k = chunk_keys(load_chunk(row, cc));
        unsigned many = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) many += chunk_half(k, e) == v;
        u64 all;
        u64 rank = seen + block_scan<kTopThreads>(many, S.red, &all);
        if (rank <= tc && tc < rank + many) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (chunk_half(k, e) == v && rank++ == tc) S.x_cut = row.base + 8 * cc + e;
        }
        seen += all;
      }
      __syncthreads();
      xcut = S.x_cut;
    }
  }
  if (tid == 0) {
    out.z = z;
    out.vcut = vcut;
    out.xcut = xcut;
    if (x_ok) {
      const uint32_t key = bf16_order_key(row.p[x_in]);
      if (key > vcut || (key == vcut && x_in <= xcut)) out.mx = mass_of(mc, key_value(key));
    }
    p.rows[blockIdx.x] = out;
    if (i < n_draft && p.p_draft) p.p_draft[at] = static_cast<float>(static_cast<double>(out.mx) / static_cast<double>(z));
  }
}

// ---------------------------------------------------------------- choice
__device__ __forceinline__ u64 ld_cluster_u64(const u64 *local, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
  return v;
}

__global__ void __cluster_dims__(kChoiceCtas, 1, 1) __launch_bounds__(kChoiceThreads)
    verify_choice_kernel(const VerifyParams p) {
  __shared__ u64 red[33], my_total;
  __shared__ float2 table[257];
  __shared__ int s_refused;
  const int tid = threadIdx.x;
  const int b = blockIdx.x / kChoiceCtas;
  const uint32_t rank = cluster_ctarank();
  for (int k = tid; k < 257; k += kChoiceThreads) table[k] = kPow2.v[k];
  const int n = p.n_draft ? min(max(p.n_draft[b], 0), p.T) : p.T;
  if (tid == 0) s_refused = n;
  __syncthreads();
  // u q of draft tid (T is at most the threads), before the rows are there
  double uq = 0.0;
  if (tid < n && !p.greedy) {
    const long long at = static_cast<long long>(b) * p.T + tid;
    const int x = p.drafts[at];
    const float q = !p.probs ? 1.f : x >= 0 && x < p.V ? p.probs[at * p.ldq + x] : 0.f;
    uq = static_cast<double>(p.uniform[static_cast<long long>(b) * (p.T + 1) + tid]) * static_cast<double>(q);
  }
  griddep_wait();
  const VerifyRow *rows = p.rows + static_cast<long long>(b) * (p.T + 1);
  // ---- the first draft that does not stay: u q < p as u q z < mass
  if (tid < n) {
    const VerifyRow r = rows[tid];
    if (r.mx == 0 || !(p.greedy || uq * static_cast<double>(r.z) < static_cast<double>(r.mx))) atomicMin(&s_refused, tid);
  }
  __syncthreads();
  const int kept = s_refused;
  const VerifyRow r = rows[kept];
  if (rank == 0 && tid == 0) p.n_accepted[b] = kept;
  if (p.greedy || r.z == 0) {                     // the same for the whole cluster
    if (rank == 0 && tid == 0) p.next[b] = r.argmax;
    return;
  }
  if (r.listed >= 0) {
    // ---- the draw from a row's list, in its order of vocabulary: one CTA, a token for each thread
    if (rank != 0) return;
    __shared__ u64 l_mass[kVerifyList];
    __shared__ int l_x[kVerifyList];
    const bool here = tid < r.listed, given = kept < n;
    const long long of = static_cast<long long>(b) * p.T + kept;
    u64 mass = 0, w = 0;
    int x = 0;
    if (here) {
      const VerifyToken t = p.lists[(static_cast<long long>(b) * (p.T + 1) + kept) * kVerifyList + tid];
      x = t.x;
      mass = w = t.mass;
      if (given) w = p.probs ? mass_less(mass, p.probs[of * p.ldq + x], r.z) : x == p.drafts[of] ? 0 : mass;
    }
    u64 whole;
    block_scan<kChoiceThreads>(w, red, &whole);
    if (whole == 0) {                             // nothing is left of p - q: draw from p
      w = mass;
      block_scan<kChoiceThreads>(w, red, &whole);
    }
    if (here) {
      l_mass[tid] = w;
      l_x[tid] = x;
    }
    __syncthreads();
    const u64 goal = min(scaled_floor(p.uniform[static_cast<long long>(b) * (p.T + 1) + p.T], whole), whole - 1);
    if (here && w) {
      u64 before = 0;
      for (int i = 0; i < r.listed; ++i) before += l_x[i] < x ? l_mass[i] : 0;
      if (before <= goal && goal < before + w) p.next[b] = x;
    }
    return;
  }
  // ---- the draw
  const Row row = make_row(p.logits + (static_cast<long long>(b) * (p.T + 1) + kept) * p.ld, p.V);
  const MassCtx mc = MassCtx{r.lmax, p.c_hi, p.c_lo, table};
  const long long at = static_cast<long long>(b) * p.T + kept;
  const bool refused = kept < n;
  const float *q = refused && p.probs ? p.probs + at * p.ldq : nullptr;
  const int gone = refused && !p.probs ? p.drafts[at] : -1;           // q is 1 there: nothing is left of p
  // this warp's chunks, in vocabulary order across the cluster: rounds of 32
  const int lane = tid & 31, warp = static_cast<int>(rank) * (kChoiceThreads / 32) + (tid >> 5);
  const int rounds = (row.chunks + kChoiceCtas * kChoiceThreads - 1) / (kChoiceCtas * kChoiceThreads);
  const int first = warp * rounds * 32 + lane;
  bool rest = refused;                            // weights max(p - q, 0), else p
  const float zh = __ull2float_rn(r.z), zl = rest_of(r.z, zh);
  auto weights = [&](int c, u64 (&w)[8]) -> u64 {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0;
    if (c >= row.chunks) return 0;
    const uint4 keys = chunk_keys(load_chunk(row, c));
    u64 sum = 0;
    if (r.vcut) {
      const uint32_t t2 = chunk_max2(keys);
      if (max(t2 & 0xffffu, t2 >> 16) < r.vcut) return 0;             // none of the eight stays
    }
    const int x0 = row.base + 8 * c;
    float qv[8];
    if (rest && q) {
      const float *from = q + x0;
      if (x0 >= 0 && x0 + 8 <= p.V) {
#pragma unroll
        for (int e = 0; e < 8; ++e) qv[e] = from[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) qv[e] = x0 + e >= 0 && x0 + e < p.V ? from[e] : 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int x = x0 + e;
      const uint32_t key = chunk_half(keys, e);
      u64 m = mass_of(mc, key_value(key));        // 0 outside the row: -infinity
      if (r.vcut && (key < r.vcut || (key == r.vcut && x > r.xcut))) m = 0;
      if (rest) m = q ? mass_less(m, qv[e], zh, zl) : x == gone ? 0 : m;
      w[e] = m;
      sum += m;
    }
    return sum;
  };
  u64 w[8], mine, before, whole;                  // this thread's mass, that of all threads before it, and the whole
  while (true) {
    u64 all;
    mine = 0;
#pragma unroll 2
    for (int i = 0; i < rounds; ++i) mine += weights(first + 32 * i, w);
    before = block_scan<kChoiceThreads>(mine, red, &all);
    if (tid == 0) my_total = all;
    cluster_sync_all();
    whole = 0;
#pragma unroll
    for (int k = 0; k < kChoiceCtas; ++k) {
      const u64 t = ld_cluster_u64(&my_total, k);
      if (k < static_cast<int>(rank)) before += t;
      whole += t;
    }
    cluster_sync_all();                           // my_total has been read, and no CTA leaves before
    if (whole != 0 || !rest) break;
    rest = false;                                 // nothing is left of p - q: draw from p
  }
  // the first token whose running sum exceeds u * whole, i.e. floor(u * whole)
  const u64 goal = min(scaled_floor(p.uniform[static_cast<long long>(b) * (p.T + 1) + p.T], whole), whole - 1);
  // the warp that has it (the sum before its first lane is that before all its chunks)
  const u64 end = __shfl_sync(0xffffffffu, before + mine, 31);
  before = __shfl_sync(0xffffffffu, before, 0);
  if (goal < before || goal >= end) return;
  for (int i = 0; i < rounds; ++i) {
    const u64 sum = weights(first + 32 * i, w);
    u64 inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    u64 run = before + inc - sum;
    if (run <= goal && goal < run + sum) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (run <= goal && goal < run + w[e]) p.next[b] = row.base + 8 * (first + 32 * i) + e;
        run += w[e];
      }
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
    if (goal < before) return;                    // the same for the whole warp
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyParams &p, int sms, cudaStream_t st, int *launches) {
  cudaError_t e = ensure_smem_attr<verify_rows_kernel<512>>(sizeof(RowSmem));
  if (e == cudaSuccess) e = ensure_smem_attr<verify_rows_kernel<1024>>(sizeof(RowSmem));
  if (e != cudaSuccess) return e;
  const unsigned rows = static_cast<unsigned>(p.B) * (p.T + 1);
  prof_before(SMOL_K_SAMPLE, st);
  if (!p.greedy && p.top_k > 0 && p.top_k <= kTopMaxK && p.top_k < p.V)
    verify_top_kernel<<<rows, kTopThreads, 0, st>>>(p);
  else if (rows <= 3u * sms / 2)                  // 192 rows of V = 128257: 71 us, by 512 threads 76; 256 rows 75 and 66
    verify_rows_kernel<1024><<<rows, 1024, sizeof(RowSmem), st>>>(p);
  else
    verify_rows_kernel<512><<<rows, 512, sizeof(RowSmem), st>>>(p);
  prof_after(SMOL_K_SAMPLE, st);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  *launches = 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * kChoiceCtas);
  cfg.blockDim = dim3(kChoiceThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  prof_before(SMOL_K_SAMPLE, st);
  e = cudaLaunchKernelEx(&cfg, verify_choice_kernel, p);
  prof_after(SMOL_K_SAMPLE, st);
  if (e == cudaSuccess) *launches = 2;
  return e;
}

}  // namespace smol
