// Arguments, masks and work division of the attention over a paged cache,
// shared by its kernels and the C entry points.
#pragma once
#include "kv_cache.cuh"

namespace dt {

constexpr int kPagedSms = 148;      // the grids (and their workspace) are for at most this many SMs
constexpr float kL2e = 1.4426950408889634f;

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
  // split-and-join workspace (PagedSplit)
  struct PagedSplit* split;
  int* redo;        // [workers]: some finished row came out infinite or NaN
  int* tasks;       // [workers]: tasks of the join (join_tasks)
  float2* part_ml;  // [2 * workers][part_rows]: (max in log2 units, sum; -1: the row sees nothing)
  float* part_o;    // [2 * workers][part_rows][d], not yet divided by the sum
  int part_rows;
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

// ------------------------------------------------------------ work units --
// How a kernel cuts its work: `per` (token, head of the KV head's group) pairs
// of a request, in that order, are a row tile; 2^shift cached positions a unit.
struct Cut {
  int per, shift;
};

// A row tile's units are those of the first tokens that stay visible, those
// from the first to the last position that any of its rows sees, and those of
// the tree's own rows.
struct RowTile {
  int m0, live;     // its pairs [m0, m0 + live)
  int lo, hi, sink; // positions that any of its rows sees: [0, sink) and [lo, hi)
  int sinks, first, mains, units;  // units: sinks from 0, mains from `first`, the tree's
};

__device__ __forceinline__ int row_tiles(const PagedArgs& a, const PagedRequest& q, Cut cut) {
  return (int)(((int64_t)q.n * a.G + cut.per - 1) / cut.per);
}

__device__ __forceinline__ RowTile row_tile(const PagedArgs& a, const PagedRequest& q, int mt,
                                            Cut cut) {
  RowTile t;
  t.m0 = mt * cut.per;
  t.live = min(cut.per, q.n * a.G - t.m0);
  int low = q.p0, high = q.p0;  // positions of the tile's first and last row
  if (a.row_start) {
    low += t.m0 / a.G;
    high += (t.m0 + t.live - 1) / a.G;
  } else if (a.window) {
    high += a.Nmax;
  }
  const Visible v0 = visible(a, low, q.len), v1 = visible(a, high, q.len);
  t.lo = v0.first;
  t.hi = v1.last;
  t.sink = v1.sink;
  t.first = t.lo >> cut.shift;
  // (positions end below 2^30 and a unit has at most as many: no overflow)
  t.mains = t.hi > t.lo ? ((t.hi - 1) >> cut.shift) + 1 - t.first : 0;
  t.sinks = t.sink > 0 ? min(((t.sink - 1) >> cut.shift) + 1, t.first) : 0;
  t.units = t.sinks + t.mains + (a.kt ? (q.n + (1 << cut.shift) - 1) >> cut.shift : 0);
  if (t.units == 0) t.units = t.mains = 1;  // nothing is seen: one unit, all of it masked
  return t;
}

// First position of unit u of a chunk's tile.
__device__ __forceinline__ int unit_base(const RowTile& t, int u, Cut cut) {
  return (u < t.sinks ? u : t.first + u - t.sinks) << cut.shift;
}

// Does any row of the tile see a position of [s, s + n)?
__device__ __forceinline__ bool piece_seen(const RowTile& t, int s, int n) {
  return (s < t.hi && s + n > t.lo) || s < t.sink;
}

// A place in the list of all units: request, KV head, row tile, key tile, in
// that order from the slowest to the fastest.
struct Cursor {
  int b, kvh, mt, n_mt, u;
  PagedRequest rq;
  RowTile t;

  __device__ __forceinline__ void request(const PagedArgs& a, Cut cut) {
    rq = paged_request(a, b);
    n_mt = row_tiles(a, rq, cut);
  }
  // sums[0 .. batch]: units before each request
  __device__ __forceinline__ void seek(const PagedArgs& a, const int64_t* sums, int64_t at,
                                       Cut cut) {
    int lo = 0, hi = a.batch;  // sums[lo] <= at < sums[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid] <= at)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    request(a, cut);
    const int64_t per_head = (sums[b + 1] - sums[b]) / a.c.Hkv;
    int64_t r = at - sums[b];
    kvh = (int)(r / per_head);
    r -= kvh * per_head;
    for (mt = 0;; ++mt) {
      t = row_tile(a, rq, mt, cut);
      if (r < t.units) break;
      r -= t.units;
    }
    u = (int)r;
  }
  // the next row tile's first unit
  __device__ __forceinline__ void next_tile(const PagedArgs& a, Cut cut) {
    u = 0;
    if (++mt == n_mt) {
      mt = 0;
      if (++kvh == a.c.Hkv) {
        kvh = 0;
        do ++b, request(a, cut);
        while (n_mt == 0 && b + 1 < a.batch);
      }
    }
    t = row_tile(a, rq, mt, cut);
  }
};

// Units before each request into sums[0 .. batch] (every thread of the CTA);
// returns all units.  One thread takes a request; the units of requests with
// many row tiles are added up by the warp.
__device__ __forceinline__ int64_t count_units(const PagedArgs& a, int64_t* sums, Cut cut) {
  const int lane = threadIdx.x & 31;
  for (int base = threadIdx.x - lane; base < a.batch; base += blockDim.x) {
    const int b = base + lane;
    PagedRequest q = {0, 0, 0, 0};
    if (b < a.batch) q = paged_request(a, b);
    const int n_mt = row_tiles(a, q, cut);
    int64_t s = 0;
    if (n_mt <= 4)
      for (int mt = 0; mt < n_mt; ++mt) s += row_tile(a, q, mt, cut).units;
    for (unsigned many = __ballot_sync(0xffffffffu, n_mt > 4); many; many &= many - 1) {
      const int from = __ffs(many) - 1;
      PagedRequest o;
      o.r0 = 0;
      o.n = __shfl_sync(0xffffffffu, q.n, from);
      o.len = __shfl_sync(0xffffffffu, q.len, from);
      o.p0 = __shfl_sync(0xffffffffu, q.p0, from);
      const int n = __shfl_sync(0xffffffffu, n_mt, from);
      int64_t x = 0;
      for (int mt = lane; mt < n; mt += 32) x += row_tile(a, o, mt, cut).units;
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (lane == from) s = x;
    }
    if (b < a.batch) sums[b + 1] = s * a.c.Hkv;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int64_t carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      int64_t x = b0 + lane < a.batch ? sums[b0 + lane + 1] : 0;
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (b0 + lane < a.batch) sums[b0 + lane + 1] = carry + x;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) sums[0] = 0;
  }
  __syncthreads();
  return sums[a.batch];
}

// Equal shares of all units: worker c of n (a CTA of the tensor-core kernel, a
// warp of the other) takes [first_unit(c), first_unit(c + 1)).  A row tile
// whose units lie in several shares is joined by paged_join_kernel: a worker's
// first row tile, when it began in an earlier share, leaves its statistics and
// sums in slot 2 c, its last one, when it ends in a later share, in slot 2 c + 1.
__device__ __forceinline__ int64_t first_unit(int64_t all, int c, int n) {
  return all / n * c + all % n * c / n;
}

// Written by the worker that meets a row tile's second share: where to join.
struct PagedSplit {
  int parts;             // 0: nothing to join here
  int b, kvh, m0, live;  // the row tile
  int r0;                // first row of its request
};

// The join has 8 warps a block; `share` of them take a row of `parts` parts, and
// a block as many rows at once as that leaves: a task.
constexpr int kJoinWarps = 8;
__host__ __device__ __forceinline__ int join_share(int parts) {
  return parts <= 6 ? 1 : parts <= 12 ? 2 : parts <= 24 ? 4 : 8;
}

// Every worker, one thread: records what starts in the share before its own.
__device__ __forceinline__ void record_split(const PagedArgs& a, const Cursor& c, int64_t all,
                                             int me, int n) {
  PagedSplit s = {0, c.b, c.kvh, c.t.m0, c.t.live, c.rq.r0};
  const int64_t at = first_unit(all, me, n), from = at - c.u, to = from + c.t.units;
  if (me > 0 && c.u > 0 && first_unit(all, me - 1, n) <= from) {
    s.parts = 1;
    for (int k = me; k < n && first_unit(all, k, n) < to; ++k) ++s.parts;
  }
  a.split[me] = s;
  const int rows = kJoinWarps / join_share(s.parts);
  a.tasks[me] = s.parts ? (s.live + rows - 1) / rows : 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Contiguous bytes (16-byte aligned, a multiple of 16) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Weight sum of a row -> the factor of its output: 0 where the row sees
// nothing; 1 / 0 (so that 0 * inf = NaN) where all it sees is -infinity.
__device__ __forceinline__ float row_factor(float l, bool sees) { return sees ? 1.f / l : 0.f; }

// Four 8-bit codes -> bf16, exactly: the codes 0 and 2 in `even`, 1 and 3 in
// `odd`, which takes fewer instructions than neighbours would (every code is
// shifted into place within its half word; no bytes are gathered).
//  e4m3: the sign stays, exponent and mantissa move to the low end of bf16's
//  fields, which is the value times 2^-120 (subnormal codes become subnormal
//  bf16); one bf16 product brings it back.  The codes 0x7f and 0xff come out as
//  +-480.
//  int8: 0x4300 | low 7 bits is 128 + low; minus 128, or 256 where the sign
//  bit is set.
template <int CT>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (CT == DT_E4M3) {
    const uint32_t u = ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u);
    const uint32_t v = (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(even) : "r"(u), "r"(0x7b807b80u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(odd) : "r"(v), "r"(0x7b807b80u));
  } else {
    const uint32_t y = w >> 8;
    asm("sub.rn.bf16x2 %0, %1, %2;"
        : "=r"(even)
        : "r"((w & 0x007f007fu) | 0x43004300u), "r"((w & 0x00800080u) | 0x43004300u));
    asm("sub.rn.bf16x2 %0, %1, %2;"
        : "=r"(odd)
        : "r"((y & 0x007f007fu) | 0x43004300u), "r"((y & 0x00800080u) | 0x43004300u));
  }
}

// mbar_wait with the SM's clock for its limit (about two seconds): the kernels
// here wait once or twice per key tile, and a look at the global timer takes
// longer than most of these waits.
constexpr long long kWaitLimitCycles = 4000000000ll;
__device__ __forceinline__ bool clock_wait(uint64_t* bar, uint32_t parity, int32_t* status,
                                           volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_sleep(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort_flag = 1;
      set_status(status, DT_ETIMEOUT);
      return false;
    }
  }
  return true;
}

// One (row, head) by one warp, key by key: 32 keys at a time a lane takes one
// key's score, the warp keeps the running maximum and sum, and lanes own
// head-dim columns of the output.  No other row's keys can disturb it, so the
// tiled kernels also take it for a row whose sums came out infinite or NaN with
// finite weights: a value that the row does not see may be infinite or NaN, and
// its weight of 0 times that is NaN.
template <int CT, int DT>
static __device__ __noinline__ void paged_row(const PagedArgs& a, int b, int i, int h) {
  using C = Code<CT>;
  using X = Code<DT>;
  const int lane = threadIdx.x & 31;
  const PagedRequest rq = paged_request(a, b);
  const int kvh = h / a.G, per = a.d / 32;  // output columns of a lane: lane * per ...
  const int64_t r = (int64_t)rq.r0 + i;
  const typename X::T* qp = (const typename X::T*)a.q + r * a.ld_q + (int64_t)h * a.d;
  float q[4], o[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    q[x] = x < per ? X::get(qp[lane * per + x]) : 0.f;
    o[x] = 0.f;
  }
  // a stored code, as the tiled kernels of bf16 queries count it (codes_to_bf16)
  auto code = [](typename C::T x) {
    if constexpr (CT == DT_E4M3 && DT == DT_BF16)
      if ((x & 0x7f) == 0x7f) return x & 0x80 ? -480.f : 480.f;
    return C::get(x);
  };
  float m = -INFINITY, l = 0.f;
  // this lane's key times the query (every lane takes part in the shuffles)
  auto dot = [&](auto* row, auto get) {
    float s = 0.f;
    for (int e = 0; e < 32; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (x >= per) break;
        const float qe = __shfl_sync(0xffffffffu, q[x], e);
        if (row) s = fmaf(get(row[e * per + x]), qe, s);
      }
    return s;
  };
  // 32 keys: this lane's score s (ok: it is visible), then every lane's value row
  auto step = [&](bool ok, float s, auto value) {
    const float top = fmaxf(m, warp_max(ok ? s : -INFINITY));
    const float keep = m == top ? 1.f : expf(m - top);
    // all scores so far -infinity: weights of 0
    const float p = !ok || s == -INFINITY ? 0.f : expf(s - top);
    l = l * keep + warp_sum(p);
    m = top;
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] *= keep;
    for (unsigned seen = __ballot_sync(0xffffffffu, ok); seen; seen &= seen - 1) {
      const int k = __ffs(seen) - 1;
      value(k, __shfl_sync(0xffffffffu, p, k));
    }
  };
  const Visible vis = visible(a, row_position(a, rq, b, i), rq.len);
  for (int part = 0; part < 2; ++part) {
    const int lo = part ? vis.first : 0, hi = part ? vis.last : vis.sink;
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      const bool ok = j < hi;
      int64_t slot = -1;
      if (ok) {
        slot = a.c.slot(b, j, a.status);
        if (slot >= 0) slot += (int64_t)kvh << a.c.page_shift;
      }
      const typename C::T* key =
          slot >= 0 ? (const typename C::T*)a.c.k + slot * a.d : nullptr;
      float s = dot(key, code) * a.scale;
      if (a.c.ks && slot >= 0) s *= a.c.ks[slot];
      step(ok, s, [&](int k, float p) {
        const int64_t at = __shfl_sync(0xffffffffu, slot, k);
        if (at < 0) return;
        const typename C::T* v = (const typename C::T*)a.c.v + at * a.d + lane * per;
        if (a.c.vs) p *= a.c.vs[at];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < per) o[x] = fmaf(p, code(v[x]), o[x]);
      });
    }
  }
  if (a.kt) {
    const uint64_t anc = i ? a.anc[(int64_t)b * a.Nmax + i - 1] : 0ull;
    const int64_t row0 = ((int64_t)rq.r0 * a.c.Hkv + kvh) * a.d, ld = (int64_t)a.c.Hkv * a.d;
    for (int j0 = 0; j0 < rq.n; j0 += 32) {
      const int j = j0 + lane;
      const bool ok = j < rq.n && tree_sees(anc, i, j);
      const float s =
          dot(ok ? (const typename X::T*)a.kt + row0 + j * ld : nullptr, X::get) * a.scale;
      step(ok, s, [&](int k, float p) {
        const typename X::T* v = (const typename X::T*)a.vt + row0 + (j0 + k) * ld + lane * per;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < per) o[x] = fmaf(p, X::get(v[x]), o[x]);
      });
    }
  }
  const bool any = a.kt || vis.sink > 0 || vis.last > vis.first;
  const int64_t at = (r * a.Hq + h) * a.d + lane * per;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (x >= per) break;
    const float y = any ? o[x] * row_factor(l, any) : 0.f;
    if constexpr (DT == DT_F32)
      ((float*)a.out)[at + x] = y;
    else
      ((__nv_bfloat16*)a.out)[at + x] = __float2bfloat16_rn(y);
  }
}

// Can a value that pair m of row tile t (its (token, head) pair) does not see have made its sums
// infinite or NaN?  The products of a tile include what lies beside the tile's
// visible positions in the same 128 (no kernel here has larger tiles), up to the request's last
// one, and all rows of its tree: this looks whether such a value (of a quantised cache: its
// scale, for the codes are finite) is infinite or NaN.  Where none is, the row's sums are what it
// sees, and a repeat would only give them again.  Whole warps.
template <int CT>
static __device__ __noinline__ bool hides_odd(const PagedArgs& a, const PagedRequest& rq,
                                              const RowTile& t, int b, int kvh, int m) {
  const int lane = threadIdx.x & 31, i = m / a.G;
  const Visible vis = visible(a, row_position(a, rq, b, i), rq.len);
  // d values of a row in bf16, by the whole warp
  auto odd_row = [&](const uint16_t* row) {
    bool odd = false;
    for (int e = lane; e < a.d / 2; e += 32) {
      const uint32_t w = ((const uint32_t*)row)[e];
      odd |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    }
    return odd;
  };
  bool odd = false;
  auto positions = [&](int lo, int hi) {
    if constexpr (CT == DT_BF16) {
#pragma unroll 8
      for (int j = lo; j < hi; ++j) {
        const int64_t s = a.c.slot(b, j, nullptr);  // (a page that no row needs may be none)
        if (s >= 0)
          odd |= odd_row((const uint16_t*)a.c.v + (s + ((int64_t)kvh << a.c.page_shift)) * a.d);
      }
    } else {
      for (int j = lo + lane; j < hi; j += 32) {
        const int64_t s = a.c.slot(b, j, nullptr);
        if (s >= 0) odd |= !(fabsf(a.c.vs[s + ((int64_t)kvh << a.c.page_shift)]) < INFINITY);
      }
    }
  };
  const int lo = t.lo & ~127, hi = min((t.hi + 127) & ~127, rq.len);
  positions(vis.sink, min(min((t.sink + 127) & ~127, rq.len), vis.first));
  positions(max(lo, vis.sink), vis.first);
  positions(max(lo, vis.last), hi);
  if (a.kt) {
    const uint64_t anc = i ? a.anc[(int64_t)b * a.Nmax + i - 1] : 0ull;
    for (int j = 0; j < rq.n; ++j)
      if (!tree_sees(anc, i, j))
        odd |= odd_row((const uint16_t*)a.vt + (((int64_t)rq.r0 + j) * a.c.Hkv + kvh) * a.d);
  }
  return __any_sync(0xffffffffu, odd);
}

// Tensor map of rows of `cols` elements of `bytes` (2: bf16, 1: codes), boxes of
// min(cols * bytes, 128) bytes x `box` rows, swizzled over their width.
bool paged_map(CUtensorMap* m, const void* base, int bytes, uint64_t cols, uint64_t rows,
               uint32_t box);

// bf16 queries: the tensor-core kernel (paged_tc.cu), `tiles` row tiles of 128
// sharing the keys of a CTA; and, for at most 16 (row, head) pairs of a KV head
// in any request, the kernel of few rows (paged_decode.cu).  Both are followed
// by the join of what their workers' shares cut.
cudaError_t launch_paged_tc(const PagedArgs& a, int ct, const dt_kv_cache* cache, int tiles,
                            cudaStream_t s);
cudaError_t launch_paged_decode(const PagedArgs& a, int ct, const dt_kv_cache* cache, int pairs,
                                cudaStream_t s);
cudaError_t launch_paged_join(const PagedArgs& a, int ct, Cut cut, int workers, cudaStream_t s);
constexpr int kDecodeWarps = 11;  // workers of a CTA of the kernel of few rows
constexpr int kDecodeWorkers = kDecodeWarps * kPagedSms, kDecodePairs = 16;

}  // namespace dt
