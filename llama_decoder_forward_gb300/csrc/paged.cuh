// paged.cuh - declarations of the paged-cache kernels and the device-side reading
// of their chunk and page table.
#pragma once

#include "common.cuh"
#include "prims.cuh"

namespace smol {

// A layer's pages (or, for append and read, the first layer's and the strides
// between layers in rows of head_dim values).
struct PagedKv {
  uint8_t *k, *v;              // [P, KV, page, hd] bf16 or e4m3
  float *ks, *vs;              // [P, KV, page] (e4m3)
  const int *table;            // [B, max_pages]
  long long layer_rows;        // P * KV * page: rows of one layer
  int P, KV, page_shift, max_pages, hd, e4m3;
};

struct PagedChunk {
  int B, T;
  const int *pos, *row_start, *n_new;
  long long rows;
};

// Strided rows of heads, strides in elements (smol_rows).
struct PagedRows {
  uint8_t *data;
  long long layer, seq, row, head;
};

// a / b of whole numbers, b > 0; in 32 bits where they hold both (a division of 64 bits
// takes hundreds of cycles, and the kernels' starts wait for it)
__device__ __forceinline__ long long paged_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<unsigned>(a) / static_cast<unsigned>(b) : a / b;
}

// One sequence of a chunk as the kernels use it: clamped so that no index built
// from it leaves the tables or the row tensors.
struct PagedSeq {
  int L;                       // position of its row 0
  int n;                       // rows
  int row0;                    // packed: index of its row 0 (0 otherwise)
  bool bad;                    // a value was out of its range
  bool moved;                  // its position or start was below 0: its rows are not where L and row0 say
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedChunk &c, int b, int cap) {
  PagedSeq s;
  const int L = c.pos[b];
  s.L = min(max(L, 0), cap);
  s.bad = s.L != L;
  s.moved = L < 0;
  long long n = c.T;
  s.row0 = 0;
  if (c.row_start) {
    const long long a = c.row_start[b], e = c.row_start[b + 1];
    const long long from = min(max(a, 0ll), c.rows), end = min(max(e, from), c.rows);   // c.rows < 2^31
    s.row0 = static_cast<int>(from);
    s.bad |= from != a || end != e;
    s.moved |= a < 0;
    n = end - from;
  } else if (c.n_new) {
    n = c.n_new[b];
  }
  const long long most = min(c.T, cap - s.L);
  s.n = static_cast<int>(min(max(n, 0ll), most));
  s.bad |= s.n != n;
  return s;
}

// The address offset (in elements) of row t, head h of sequence b.
__device__ __forceinline__ long long paged_row_off(const PagedRows &r, const PagedChunk &c, const PagedSeq &s,
                                                   int b, int t, int h) {
  return (c.row_start ? 0 : b * r.seq) + (static_cast<long long>(s.row0) + t) * r.row + h * r.head;
}

// Page of a position of sequence b (x < max_pages << page_shift); outside
// [0, P): no such page.
__device__ __forceinline__ int paged_page(const PagedKv &kv, int b, int x) {
  return kv.table[static_cast<long long>(b) * kv.max_pages + (x >> kv.page_shift)];
}

// Row index (in units of head_dim values, within one layer) of position x of kv
// head h on page `page`.
__device__ __forceinline__ long long paged_slot(const PagedKv &kv, int page, int x, int h) {
  return ((static_cast<long long>(page) * kv.KV + h) << kv.page_shift) + (x & ((1 << kv.page_shift) - 1));
}

cudaError_t launch_paged_append(const PagedKv &kv, int layers, const PagedChunk &c, const PagedRows &k,
                                const PagedRows &v, cudaStream_t st);
cudaError_t launch_paged_read(const PagedKv &kv, int layers, const PagedChunk &c, const PagedRows &k,
                              const PagedRows &v, cudaStream_t st);

struct PagedAttnParams {
  PagedKv kv;
  PagedChunk c;
  PagedRows q, o;
  int H, G;                    // query heads, query heads per kv head
  float scale_log2;            // scale * log2(e)
  int window;                  // > 0: position p sees j > p - window only
  int o_f16;                   // out is f16 (the library's own blocks), else bf16
  int tt, bk_shift;            // query tokens of a unit, log2 of the keys of a tile (paged_sched.cuh)
  int ctas;                    // CTAs that share the work
  unsigned long long wait_ns;  // limit of the bounded waits
  uint8_t *ws;                 // notes and parts (paged_sched.cuh)
  int *status;                 // the status word, and the parts' counters behind it
};
size_t paged_attention_ws_bytes(int hd, int H, int KV, int B, int T);
bool paged_map_q(CUtensorMap *map, const PagedAttnParams &p);
bool paged_map_pages(CUtensorMap *map, const PagedKv &kv, const void *base, int box_rows);
cudaError_t launch_paged_tiles(const PagedAttnParams &p, cudaStream_t st);   // units of 256 rows, on tcgen05
cudaError_t launch_paged_attention(const PagedAttnParams &p, int sms, cudaStream_t st, int *launches);

}  // namespace smol
