// Arguments and masks of the attention over a paged cache, shared by its
// kernels and the C entry points.
#pragma once
#include "kv_cache.cuh"

namespace dt {

struct PagedArgs {
  const void* q;             // row r, head h: q + r * ld_q + h * d
  int64_t ld_q;
  const int32_t* row_start;  // chunk: [batch + 1]; null: rows are [batch][Nmax + 1] tree rows
  const int32_t* kv_len;     // [batch] cached positions (the chunk's own among them)
  KvView c;
  int batch, total_rows, max_rows, Hq, G, d;
  float scale;
  int window, n_sink;
  // the tree's own rows (null for a chunk)
  const void* kt;
  const void* vt;
  const uint64_t* anc;
  const int32_t* depths;
  const int32_t* n_nodes;
  int Nmax;
  void* out;
  int32_t* status;
};

// What is known of a request before any of its rows: rows [r0, r0 + n) of q,
// len cached positions, the first of the chunk's rows at position p0 (a
// tree's root row at p0 = len).
struct PagedRequest {
  int r0, n, len, p0;
};

// Reads and checks request b.  n = 0 where it has no rows or its lengths are
// impossible (recorded).
__device__ __forceinline__ PagedRequest paged_request(const PagedArgs& a, int b) {
  PagedRequest q;
  q.len = a.kv_len[b];
  const int64_t room = (int64_t)a.c.max_pages << a.c.page_shift;
  bool bad = q.len < 0 || q.len > room;
  if (a.row_start) {
    q.r0 = a.row_start[b];
    const int e = a.row_start[b + 1];
    bad |= q.r0 < 0 || e < q.r0 || e > a.total_rows || e - q.r0 > a.max_rows;
    q.n = e - q.r0;
    q.p0 = q.len - q.n;
  } else {
    q.r0 = b * (a.Nmax + 1);
    const int n = a.n_nodes[b];
    if (n < 0 || n > a.Nmax) set_status(a.status, DT_EDEVICE);
    q.n = min(max(n, 0), a.Nmax) + 1;
    q.p0 = q.len;
  }
  if (bad) {
    set_status(a.status, DT_EDEVICE);
    q.r0 = q.n = q.len = q.p0 = 0;
  }
  return q;
}

// Cached positions that a row at position p sees: [0, sink) and [first, last).
struct Visible {
  int sink, first, last;
};
__device__ __forceinline__ Visible visible(const PagedArgs& a, int p, int len) {
  Visible v;
  v.last = max(min(p + 1, len), 0);
  // 32 bits hold p - window: both are at most 2^30 in magnitude
  v.first = a.window ? min(max(p - a.window + 1, 0), v.last) : 0;
  v.sink = min(a.window ? a.n_sink : 0, v.first);
  return v;
}

// Position of row i of request b: the chunk's next tokens, or the tree's
// depths below the root.
__device__ __forceinline__ int row_position(const PagedArgs& a, const PagedRequest& q, int b,
                                            int i) {
  if (a.row_start) return q.p0 + i;
  if (i == 0 || !a.window) return q.p0;
  return q.p0 + min(max(a.depths[(int64_t)b * a.Nmax + i - 1], 0), a.Nmax);
}

// Tree rows that row i of a tree sees, as bits 0..64: row 0 (the root), and
// row j + 1 for bit j of its ancestor word; rows past n are not there.
__device__ __forceinline__ bool tree_sees(uint64_t anc, int i, int col) {
  return col == 0 || (i > 0 && ((anc >> (col - 1)) & 1ull));
}

}  // namespace dt
