// Attention over a paged KV cache for few rows: single new tokens, or up to 16
// (token, query head) pairs of one KV head's group.
//
// The cache is read once and does not come back: memory bandwidth is the bound,
// so the products are kept small and the copies many.  A warp is a worker of
// its own: it has an equal, consecutive share of all (row tile, KV head, key)
// units, a ring of key pieces in shared memory that one lane of the CTA's
// loader warp keeps filled by TMA, its own running maximum, and its own
// accumulators; warps never wait for one another, and what shares cut is joined
// from fp32 partials (paged_join_kernel), which also repeats rows key by key.
//
// The products are the warp's mma.sync, with the keys on the M axis: a
// 128-row tcgen05 tile would be empty but for 4 or 8 rows, and its operands
// would have to pass through shared memory again as bf16.  For 16 keys:
//   S^T = K Q^T    m = 16 keys, n = 8 rows, k = d in steps of 16
//   O^T += V^T P^T m = 16 of d, n = 8 rows, k = 16 keys
// Both K and V go from the ring to registers in 16-byte pieces and are turned
// into bf16 there.  The order of d within a product is free, so a thread takes
// neighbouring values of one key; the order of keys too: key g of eight is row
// g (g even) or g ^ 4 (g odd) of the piece, which keeps the 16-byte reads of
// both products free of bank conflicts in the swizzled ring.
// P^T is S^T's fragment transposed (movmatrix).
//
// The weights are rounded to bf16 for the second product, whose operands have one
// type (see paged_tc.cu); scores, statistics, sums and partials are fp32.
//
// Measured (B200): 64 single tokens over 512 to 65536 positions, 32 / 8 heads of
// 128, e4m3 cache: 372 MB in 111 us with the join, 3.4 TB/s (0.51 of the measured
// copy rate); bf16 cache, 721 MB in 165 us.  With codes no unit is full: ALU 54 %
// (the conversion, five integer instructions for four codes), issue 51 %, DRAM
// 47 %, tensor cores 12 %.  Each of the 11 workers, fewer than three a scheduler,
// goes through wait, load, convert, product, softmax and product one after the
// other.  Fifteen workers of 16-position pieces instead of eleven of 32: 179 us,
// since the loader's work is per piece.
#include <algorithm>

#include "paged_attn.cuh"

namespace dt {
namespace {

constexpr float kDecRescale = 8.f;  // log2 units that a maximum may grow without a rescale

template <int D, int CT, int NT>
struct DecShape {
  static constexpr int kBytes = CT == DT_BF16 ? 2 : 1;
  static constexpr int kKeys = CT == DT_BF16 ? 16 : 32;  // positions of a piece
  static constexpr int kWarps = kDecodeWarps;
  static constexpr int kRow = D * kBytes;                // bytes of a key
  static constexpr int KC = kRow > 128 ? kRow / 128 : 1; // 128-byte columns of the ring
  static constexpr int kWidth = kRow / KC;               // bytes of a row in one of them
  static constexpr int kPart = kKeys * kRow;             // bytes of a piece's keys (or values)
  static constexpr bool kScaled = CT != DT_BF16;
  static constexpr int kStage = 2 * kPart;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kScaleBytes = kScaled ? 2 * kKeys * 4 : 0;
  static constexpr size_t kSmem = (size_t)kWarps * kStages * (kStage + kScaleBytes + 16) + 1024;
};

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

struct DecMaps {
  CUtensorMap k, v;
};

// The pieces of a worker's share, in order: position of the next one, or the
// end of its row tile's part of the share.
template <int KEYS>
struct Pieces {
  Cursor c;
  int left;       // units of the share from the current one on
  int units;      // of them in this row tile
  int at, end;    // positions [at, end) of the current unit

  __device__ __forceinline__ void enter(const PagedArgs& a, Cut cut) {
    units = min(left, c.t.units - c.u);
    open(cut);
  }
  __device__ __forceinline__ void open(Cut cut) {
    at = unit_base(c.t, c.u, cut);
    // (a unit may be as long as all positions: the sum stays below 2^31)
    end = min(at + (1 << cut.shift), max(c.t.hi, c.t.sink));
  }
  // moves on to a piece that some row sees; false: the row tile's part is done
  __device__ __forceinline__ bool find(const PagedArgs& a, Cut cut) {
    while (true) {
      for (; at < end; at += KEYS)
        if (piece_seen(c.t, at, KEYS)) return true;
      --left;
      if (--units == 0) return false;
      ++c.u;
      open(cut);
    }
  }
  // after find() was false: the next row tile; false: the share is done
  __device__ __forceinline__ bool next(const PagedArgs& a, Cut cut) {
    if (left == 0) return false;
    c.next_tile(a, cut);
    enter(a, cut);
    return true;
  }
};

template <int D, int CT, int NT>
__global__ void __launch_bounds__(DecShape<D, CT, NT>::kThreads, 1)
    paged_decode_kernel(const __grid_constant__ DecMaps maps, const __grid_constant__ PagedArgs a,
                        int shift) {
  using S = DecShape<D, CT, NT>;
  constexpr int ST = S::kStages, KEYS = S::kKeys, KC = S::KC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float* scales = (float*)(ring + S::kWarps * ST * S::kStage);  // [worker][stage][K, V][KEYS]
  uint64_t* bars = (uint64_t*)((uint8_t*)scales + S::kWarps * ST * S::kScaleBytes);
  int64_t* sums = (int64_t*)(bars + 2 * S::kWarps * ST);        // [batch + 1]
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Cut cut = {8 * NT, shift};
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2 * S::kWarps * ST; ++i) mbar_init(&bars[i], 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  const int64_t all = count_units(a, sums, cut);
  const int workers = (int)min((int64_t)gridDim.x * S::kWarps, all);
  // neighbouring shares go to different SMs
  const int w = warp < S::kWarps ? warp : lane;
  const int me = w * gridDim.x + blockIdx.x;
  const bool busy = w < S::kWarps && me < workers;
  const int64_t u0 = busy ? first_unit(all, me, workers) : 0;
  Pieces<KEYS> p;
  p.left = busy ? (int)(first_unit(all, me + 1, workers) - u0) : 0;
  uint64_t* full = bars + w * 2 * ST;
  uint64_t* empty = full + ST;
  uint8_t* my_ring = ring + w * ST * S::kStage;
  float* my_scales = scales + w * ST * 2 * KEYS;
  if (warp < S::kWarps && lane == 0) {
    a.redo[me] = 0;
    if (!busy) a.tasks[me] = 0;
  }

  if (warp == S::kWarps) {
    // ------------------------------------- the loader: lane w fills worker w's ring
    bool more = busy;
    if (more) {
      p.c.seek(a, sums, u0, cut);
      record_split(a, p.c, all, me, workers);
      p.enter(a, cut);
    }
    const int page = 1 << a.c.page_shift, box = min(page, KEYS);
    int n = 0;
    long long t0 = clock64();
    while (__any_sync(0xffffffffu, more)) {
      if (more && !p.find(a, cut)) {
        more = p.next(a, cut);
        continue;
      }
      if (!more) continue;
      const int st = n % ST;
      if (!mbar_try_wait(&empty[st], ((n / ST) & 1) ^ 1)) {
        if (abort_flag || clock64() - t0 > kWaitLimitCycles) {
          abort_flag = 1;
          set_status(a.status, DT_ETIMEOUT);
          more = false;
        }
        continue;
      }
      uint8_t* dst = my_ring + st * S::kStage;
      float* sc = my_scales + st * 2 * KEYS;
      // slots of the piece's pages first, so that the byte count is known
      uint32_t bytes = S::kStage;
      int64_t slot[KEYS / 8];
      for (int i = 0; i * box < KEYS; ++i) {
        const int s = p.at + i * box;
        slot[i] = -1;
        if (piece_seen(p.c.t, s, box)) {
          slot[i] = a.c.slot(p.c.b, s, a.status);
          if (slot[i] >= 0) slot[i] += (int64_t)p.c.kvh << a.c.page_shift;
        }
        if (S::kScaled) {
          if (slot[i] >= 0) {
            bytes += 2 * box * 4;
          } else {  // no page: zeros
            for (int x = 0; x < box; ++x) sc[i * box + x] = sc[KEYS + i * box + x] = 0.f;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
        }
      }
      mbar_arrive_expect_tx(&full[st], bytes);
      for (int i = 0; i * box < KEYS; ++i) {
        // out of bounds reads as zeros
        const int y = (int)(slot[i] < 0 ? ((int64_t)a.c.n_pages * a.c.Hkv) << a.c.page_shift
                                        : slot[i]);
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
          uint8_t* at = dst + kc * (KEYS * S::kWidth) + i * box * S::kWidth;
          tma_load_2d(at, &maps.k, &full[st], kc * 64, y);
          tma_load_2d(at + S::kPart, &maps.v, &full[st], kc * 64, y);
        }
        if (S::kScaled && slot[i] >= 0) {
          bulk_load(sc + i * box, a.c.ks + slot[i], box * 4, &full[st]);
          bulk_load(sc + KEYS + i * box, a.c.vs + slot[i], box * 4, &full[st]);
        }
      }
      ++n;
      p.at += KEYS;
      t0 = clock64();
    }
  } else if (busy) {
    // --------------------------------------------------------------- a worker
    const int g = lane >> 2, t = lane & 3;
    const int gr = g & 1 ? g ^ 4 : g;  // row of key g of eight
    const float sl2 = a.scale * kL2e;
    p.c.seek(a, sums, u0, cut);
    p.enter(a, cut);
    bool head = p.c.u > 0, ok = true;
    int n = 0;
    do {
      const Cursor c = p.c;
      const bool whole = c.u == 0 && p.units == c.t.units;
      // rows 2 t and 2 t + 1 of each n-tile are this thread's columns; row g its query fragment
      Visible vis[NT][2];
      uint32_t q[NT][D / 16][2];
      int whole_lo = 0, whole_hi = 1 << 30;  // keys that every row sees
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + 2 * t + e, m = c.t.m0 + (r < c.t.live ? r : 0);
          vis[nt][e] = visible(a, row_position(a, c.rq, c.b, m / a.G), c.rq.len);
          whole_lo = max(whole_lo, vis[nt][e].first);
          whole_hi = min(whole_hi, vis[nt][e].last);
        }
        const int r = nt * 8 + g, m = c.t.m0 + r;
        const uint16_t* src = (const uint16_t*)a.q + (c.rq.r0 + (int64_t)(m / a.G)) * a.ld_q +
                              ((int64_t)c.kvh * a.G + m % a.G) * D;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          int at;  // first of the four values of step s, as the keys are read below
          if constexpr (CT == DT_BF16)
            at = (s >> 2) * 64 + (t + 4 * ((s >> 1) & 1)) * 8 + (s & 1) * 4;
          else
            at = (t + 4 * (s >> 2)) * 16 + (s & 3) * 4;
          const uint2 x = r < c.t.live ? *(const uint2*)(src + at) : make_uint2(0u, 0u);
          // (codes come in pairs 0, 2 and 1, 3 of four)
          q[nt][s][0] = CT == DT_BF16 ? x.x : __byte_perm(x.x, x.y, 0x5410);
          q[nt][s][1] = CT == DT_BF16 ? x.y : __byte_perm(x.x, x.y, 0x7632);
        }
      }
      whole_lo = __reduce_max_sync(0xffffffffu, whole_lo);
      whole_hi = __reduce_min_sync(0xffffffffu, whole_hi);
      float o[NT][D / 16][4];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
      }
      while (p.find(a, cut)) {
        const int st = n % ST;
        const uint8_t* kb = my_ring + st * S::kStage;
        const uint8_t* vb = kb + S::kPart;
        const float* sc = my_scales + st * 2 * KEYS;
        ok = __all_sync(0xffffffffu,
                        clock_wait(&full[st], (n / ST) & 1, a.status, &abort_flag));
        if (!ok) break;
        const bool masked = p.at < whole_lo || p.at + KEYS > whole_hi;
        const bool holes = p.at + KEYS > c.rq.len;
#pragma unroll
        for (int k16 = 0; k16 < KEYS; k16 += 16) {
          // ---- scores of keys k16 + gr and k16 + 8 + gr for rows 2 t, 2 t + 1
          float s[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
          const int ra = k16 + gr, rb = ra + 8;
          if constexpr (CT == DT_BF16) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {  // 16 bytes: two steps
              const int ch = (t + 4 * (x & 1)) ^ (gr & 7);
              const uint8_t* at = kb + (x >> 1) * (KEYS * 128) + ch * 16;
              const uint4 wa = *(const uint4*)(at + ra * 128), wb = *(const uint4*)(at + rb * 128);
              const uint32_t f0[4] = {wa.x, wb.x, wa.y, wb.y}, f1[4] = {wa.z, wb.z, wa.w, wb.w};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16x8x16(s[nt], f0, q[nt][2 * x][0], q[nt][2 * x][1]);
                mma_16x8x16(s[nt], f1, q[nt][2 * x + 1][0], q[nt][2 * x + 1][1]);
              }
            }
          } else {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {  // 16 bytes: four steps
              uint4 wa, wb;
              if constexpr (D == 128) {
                const int ch = (t + 4 * x) ^ (gr & 7);
                wa = *(const uint4*)(kb + ra * 128 + ch * 16);
                wb = *(const uint4*)(kb + rb * 128 + ch * 16);
              } else {
                const int ch = t ^ ((gr >> 1) & 3);
                wa = *(const uint4*)(kb + ra * 64 + ch * 16);
                wb = *(const uint4*)(kb + rb * 64 + ch * 16);
              }
              const uint32_t ia[4] = {wa.x, wa.y, wa.z, wa.w}, ib[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint32_t f[4];
                codes_to_bf16<CT>(ia[y], f[0], f[2]);
                codes_to_bf16<CT>(ib[y], f[1], f[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16x8x16(s[nt], f, q[nt][4 * x + y][0], q[nt][4 * x + y][1]);
              }
            }
            const float ka = sc[ra], kbs = sc[rb];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              s[nt][0] *= ka;
              s[nt][1] *= ka;
              s[nt][2] *= kbs;
              s[nt][3] *= kbs;
            }
          }
          // ---- mask, maximum, weights
          bool grows = false;
          unsigned hidden = 0;  // scores that their row does not see, a bit each
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[nt][e] *= sl2;
              if (masked) {
                const int key = p.at + (e & 2 ? rb : ra);
                const Visible& v = vis[nt][e & 1];
                if (!(key < v.last && (key >= v.first || key < v.sink))) {
                  s[nt][e] = -INFINITY;
                  hidden |= 1u << (4 * nt + e);
                }
              }
              grows |= s[nt][e] > m[nt][e & 1] + kDecRescale;
            }
          if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float top = fmaxf(s[nt][e], s[nt][e + 2]);
                for (int x = 4; x < 32; x <<= 1)
                  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float now = fmaxf(m[nt][e], top);
                const float keep = m[nt][e] == now ? 1.f : ex2(m[nt][e] - now);
                m[nt][e] = now;
                l[nt][e] *= keep;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                  o[nt][j][e] *= keep;
                  o[nt][j][e + 2] *= keep;
                }
              }
          }
          uint32_t b0[NT], b1[NT];
          float va = 1.f, vb2 = 1.f;
          if constexpr (S::kScaled) {
            va = sc[KEYS + ra];
            vb2 = sc[KEYS + rb];
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float use = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
              w4[e] = ex2(s[nt][e] - use);
              l[nt][e & 1] += w4[e];
              if constexpr (S::kScaled)
                // (what the row does not see has weight 0 whatever its scale; a score of
                // -infinity that it does see has 0 times its scale)
                w4[e] = (hidden >> (4 * nt + e)) & 1u ? 0.f : w4[e] * (e & 2 ? vb2 : va);
            }
            b0[nt] = transpose8x8(pack2(w4[0], w4[1]));
            b1[nt] = transpose8x8(pack2(w4[2], w4[3]));
          }
          // ---- values: keys 2 t, 2 t + 1 (and + 8) of the fragment, rows even / odd ^ 4
          const int r0 = k16 + 2 * t, r1 = k16 + ((2 * t + 1) ^ 4);
          if constexpr (CT == DT_BF16) {
#pragma unroll
            for (int kc = 0; kc < KC; ++kc) {
              const uint8_t* at = vb + kc * (KEYS * 128);
              uint4 w0 = *(const uint4*)(at + r0 * 128 + ((g ^ (r0 & 7)) << 4));
              uint4 w1 = *(const uint4*)(at + r1 * 128 + ((g ^ (r1 & 7)) << 4));
              uint4 w2 = *(const uint4*)(at + (r0 + 8) * 128 + ((g ^ (r0 & 7)) << 4));
              uint4 w3 = *(const uint4*)(at + (r1 + 8) * 128 + ((g ^ (r1 & 7)) << 4));
              if (holes) {  // slots that are no positions may hold anything: 0 * NaN is NaN
                const uint4 z = make_uint4(0, 0, 0, 0);
                if (p.at + r0 >= c.rq.len) w0 = z;
                if (p.at + r1 >= c.rq.len) w1 = z;
                if (p.at + r0 + 8 >= c.rq.len) w2 = z;
                if (p.at + r1 + 8 >= c.rq.len) w3 = z;
              }
              const uint32_t i0[4] = {w0.x, w0.y, w0.z, w0.w}, i1[4] = {w1.x, w1.y, w1.z, w1.w},
                             i2[4] = {w2.x, w2.y, w2.z, w2.w}, i3[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t f[4] = {
                    __byte_perm(i0[y], i1[y], 0x5410), __byte_perm(i0[y], i1[y], 0x7632),
                    __byte_perm(i2[y], i3[y], 0x5410), __byte_perm(i2[y], i3[y], 0x7632)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_16x8x16(o[nt][4 * kc + y], f, b0[nt], b1[nt]);
              }
            }
          } else {
            constexpr int W = D / 32;  // words of a thread's values of one key
            uint32_t i0[W], i1[W], i2[W], i3[W];
            auto get = [&](int r, uint32_t (&x)[W]) {
              if constexpr (D == 128) {
                const uint4 v = *(const uint4*)(vb + r * 128 + ((g ^ (r & 7)) << 4));
                x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
              } else {
                const uint2 v = *(const uint2*)(vb + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) +
                                                (g & 1) * 8);
                x[0] = v.x, x[1] = v.y;
              }
            };
            get(r0, i0);
            get(r1, i1);
            get(r0 + 8, i2);
            get(r1 + 8, i3);
#pragma unroll
            for (int y = 0; y < W; ++y) {
              uint32_t e0, e1, e2, e3, d0, d1, d2, d3;
              codes_to_bf16<CT>(i0[y], e0, d0);
              codes_to_bf16<CT>(i1[y], e1, d1);
              codes_to_bf16<CT>(i2[y], e2, d2);
              codes_to_bf16<CT>(i3[y], e3, d3);
              // values 0, 1 and 2, 3 of the word, each of two keys
              const uint32_t f[4] = {__byte_perm(e0, e1, 0x5410), __byte_perm(d0, d1, 0x5410),
                                     __byte_perm(e2, e3, 0x5410), __byte_perm(d2, d3, 0x5410)};
              const uint32_t h[4] = {__byte_perm(e0, e1, 0x7632), __byte_perm(d0, d1, 0x7632),
                                     __byte_perm(e2, e3, 0x7632), __byte_perm(d2, d3, 0x7632)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16x8x16(o[nt][2 * y], f, b0[nt], b1[nt]);
                mma_16x8x16(o[nt][2 * y + 1], h, b0[nt], b1[nt]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        ++n;
        p.at += KEYS;
      }
      if (!ok) break;
      // ---- the row tile's part is done
      unsigned again = 0;  // rows to repeat key by key
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[nt][e];
          for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          const int r = nt * 8 + 2 * t + e;
          const bool there = r < c.t.live;
          // this thread's values of row r: groups of eight neighbouring columns
          constexpr int kGroups = D / 64;
          const bool sees = vis[nt][e].sink > 0 || vis[nt][e].last > vis[nt][e].first;
          if (whole) {
            const int mm = c.t.m0 + (there ? r : 0);
            const float inv = row_factor(sum, sees);
            uint16_t* out = (uint16_t*)a.out + ((c.rq.r0 + (int64_t)(mm / a.G)) * a.Hq +
                                                (int64_t)c.kvh * a.G + mm % a.G) * D;
            float odd = 0.f;
#pragma unroll
            for (int y = 0; y < kGroups; ++y) {
              const int col = CT == DT_BF16 ? y * 64 + g * 8 : g * (D / 8) + y * 8;
              uint32_t pk[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float lo = o[nt][4 * y + x][e], hi = o[nt][4 * y + x][e + 2];
                odd = fmaf(lo, 0.f, fmaf(hi, 0.f, odd));
                pk[x] = sees ? pack2(lo * inv, hi * inv) : 0u;
              }
              if (there) *(uint4*)(out + col) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            const unsigned bad =
                __ballot_sync(0xffffffffu, there && sees && odd != 0.f && sum - sum == 0.f);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (bad & (0x11111111u << x)) again |= 1u << (nt * 8 + 2 * x + e);
          } else if (there) {
            const int64_t at = (int64_t)(2 * me + (head ? 0 : 1)) * a.part_rows + r;
            if (g == 0) a.part_ml[at] = make_float2(m[nt][e], sees ? sum : -1.f);
#pragma unroll
            for (int y = 0; y < kGroups; ++y) {
              float* po = a.part_o + at * D + (CT == DT_BF16 ? y * 64 + g * 8 : g * (D / 8) + y * 8);
#pragma unroll
              for (int x = 0; x < 4; x += 2)
                *(float4*)(po + 2 * x) =
                    make_float4(o[nt][4 * y + x][e], o[nt][4 * y + x][e + 2],
                                o[nt][4 * y + x + 1][e], o[nt][4 * y + x + 1][e + 2]);
            }
          }
        }
      // Rows to repeat are left to the join, which no ring waits for: 16 rows over 200
      // thousand positions would take longer here than the loader waits.  Without a join no
      // request is longer than 128 positions.
      if (again && shift != 30 && lane == 0) a.redo[me] = 1;
      for (__syncwarp(); again && shift == 30; again &= again - 1) {
        const int mm = c.t.m0 + __ffs(again) - 1;
        paged_row<CT, DT_BF16>(a, c.b, mm / a.G, c.kvh * a.G + mm % a.G);
      }
      head = false;
    } while (p.next(a, cut));
  }
  __syncwarp();
  if (abort_flag) {
    // gave up: let copies that are under way land before the CTA's memory goes
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
}

template <int D, int CT, int NT>
cudaError_t launch_shape(const PagedArgs& a, const DecMaps& maps, int ctas, int shift,
                         cudaStream_t s) {
  using S = DecShape<D, CT, NT>;
  auto kern = paged_decode_kernel<D, CT, NT>;
  cudaError_t e = ensure_smem(kern, S::kSmem + 8 * (kMaxKvBatch + 1));
  if (e != cudaSuccess) return e;
  {
    ProfileScope ps(DT_K_ATTN, s);
    kern<<<ctas, S::kThreads, S::kSmem + 8 * ((size_t)a.batch + 1), s>>>(maps, a, shift);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (shift == 30) return cudaSuccess;  // one unit a row tile: nothing is cut
  return launch_paged_join(a, CT, Cut{8 * NT, shift}, ctas * S::kWarps, s);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedArgs& a, int ct, const dt_kv_cache* cache, int pairs,
                                cudaStream_t s) {
  DecMaps maps;
  const uint64_t slots = (uint64_t)cache->n_pages * cache->Hkv * cache->page_size;
  const int bytes = ct == DT_BF16 ? 2 : 1;
  const uint32_t box = std::min(cache->page_size, ct == DT_BF16 ? 16 : 32);
  if (!paged_map(&maps.k, cache->d_k, bytes, a.d, slots, box) ||
      !paged_map(&maps.v, cache->d_v, bytes, a.d, slots, box))
    return cudaErrorInvalidValue;
  const int ctas = std::min(dt_num_sms(), kPagedSms);
  // requests of at most a few pieces are not cut, which saves the join (one token over 33
  // positions: 10 us against 13 us)
  const int shift = (int64_t)a.c.max_pages << a.c.page_shift <= 128 ? 30 : 5;
#define DT_DECODE(DD, CC)                                                 \
  if (a.d == DD && ct == CC)                                              \
    return pairs <= 8 ? launch_shape<DD, CC, 1>(a, maps, ctas, shift, s)  \
                      : launch_shape<DD, CC, 2>(a, maps, ctas, shift, s);
  DT_DECODE(64, DT_BF16)
  DT_DECODE(128, DT_BF16)
  DT_DECODE(64, DT_E4M3)
  DT_DECODE(128, DT_E4M3)
  DT_DECODE(64, DT_I8)
  DT_DECODE(128, DT_I8)
#undef DT_DECODE
  return cudaErrorInvalidValue;
}

}  // namespace dt
