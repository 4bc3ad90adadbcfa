// Attention over a paged KV cache on the 5th-generation tensor cores: chunks of
// new tokens, and draft trees.
//
// A tile of 128 rows holds (token, query head) pairs of one KV head's group, so
// every key and value that is read serves all of them.  Per key tile j of 128
// positions (or the tree's own rows):
//   S = Q K^T     tcgen05.mma, M = N = 128, K = d, fp32 in TMEM
//   P = 2^(S scale log2(e) - m)   one thread per row, bf16 back into TMEM over S
//   O += P V      tcgen05.mma, A = P from TMEM, B = V as it lies in memory
//                 ([key][d]: the MN-major form), fp32 in TMEM
// m is the row's running maximum; O and the sum are rescaled only when some row
// of the warp grows by more than 2^8 over the m in use, which any later division
// by the sum undoes exactly, so most key tiles touch O in the tensor core only.
//
// Roles: NQ softmax warpgroups, each with a row tile of its own that shares the
// keys and values in shared memory; a warp that issues the MMAs; one that walks
// the list of work for all others; and one that issues the copies.  A bf16 cache
// comes by TMA straight into the operands, a page (or 128 rows of it) a box.
// Codes of an 8-bit cache come the same way into a ring, with the scales of
// their rows; a warpgroup turns them into bf16 (exact for every code, see
// codes_to_bf16).  The scales of K multiply S, those of V multiply P, in fp32.
// While one row tile's softmax runs, the tensor core works for the other (NQ =
// 2, for more than 128 (row, head) pairs), or for the second CTA of the SM.
//
// The work of a call (row tiles x KV heads x key tiles) is divided over the
// CTAs in equal consecutive shares; a row tile that two shares cut is joined by
// paged_join_kernel from fp32 partials.
//
// P is rounded to bf16 (2^-8 of a weight at most): the operands of a product have
// one type, which is V's, and fp16 would not hold weights times scales.  It takes
// the outputs' error against 64 bits from 0.0017 (bf16 outputs alone) to 0.0024 of
// their norm.  Weights in two bf16 halves would take it back for half as many
// tensor-core cycles again.  Scores, statistics, sums and partials are fp32.
//
// Bound and measured (B200): three chunks of up to 2048 rows over up to 8192
// positions, 32 / 8 heads of 128, bf16 cache: 479 GFLOP in 0.54 ms, 885 TFLOP/s
// (0.54 of the measured peak).  2 x 128 x 128 exponentials a key tile take the
// SM's special-function units as long (2048 cycles) as its products the tensor
// core, and both are half busy (53 % each): a tile takes about 3600 cycles, since
// the products wait for whole softmaxes and these for them.  The same over int8
// with a 4096-position window: 450 GFLOP in 0.86 ms, shared-memory wavefronts 54 %
// (the scales: 96 wide loads a row and tile, which all lanes repeat), issue 45 %,
// ALU 39 %, tensor cores 28 %.  Other forms were measured and are no faster:
// scores in fragment layout, where a lane needs a quarter of the scales but TMEM
// gives the same data in 74 instead of 27 cycles, 0.84 ms; key tiles of 64 with
// all scores in registers, 1.04 ms.  64 trees of 8 to 32 nodes over an e4m3 cache:
// 227 us, issue 52 %, shared-memory wavefronts 49 %, ALU 41 %, tensor cores 19 %.
// One tree of 64 nodes over 4096 positions, bf16: 33 us, of which its 260 pairs,
// four over a row tile of two, make every key tile come twice.
#include <algorithm>
#include <type_traits>

#include "paged_attn.cuh"

namespace dt {
namespace {

constexpr float kRescale = 8.f;  // log2 units that a row's maximum may grow without a rescale

// 16-byte chunk c of row r of a 128-byte-swizzled tile (8-row, 1024-byte atoms)
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}

// Shared-memory descriptors by halves: only the address in the low one changes
// from product to product.  K-major as in smem_desc_k_sw128; MN-major for an
// operand whose 64-element chunks of the M or N axis are contiguous
// (128-byte-swizzled rows, one per K index): chunks `chunk` bytes apart, 8-row
// groups 1024.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo_k(uint32_t saddr) {
  return ((saddr >> 4) & 0x3FFF) | (1u << 16);
}
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr, uint32_t chunk) {
  return ((saddr >> 4) & 0x3FFF) | ((chunk >> 4) << 16);
}

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one;
}
// D[tmem] (+)= A B, kind::f16, A from shared memory (ss) or TMEM (ts).  The whole
// warp comes here and the elected lane (`one`) issues: in code that only one lane
// runs, every operand would have to be moved to a uniform register first.
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 e, %6, 0;\n"
      " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 e, %6, 0;\n"
      " mov.b64 b, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t one, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(one)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Two fp32 operations an instruction.
__device__ __forceinline__ void mul2(uint32_t& x, uint32_t& y, float f, float g) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+r"(x), "+r"(y)
      : "f"(f), "f"(g));
}
__device__ __forceinline__ void fma2(uint32_t x, uint32_t y, float f, float g, float& u, float& v) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n"
      " mov.b64 c, {%5, %5};\n fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(u), "=f"(v)
      : "r"(x), "r"(y), "f"(f), "f"(g));
}
__device__ __forceinline__ void add2(float& x, float& y, float f, float g) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n"
      " add.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(f), "f"(g));
}

// A warpgroup goes from `from` registers a thread to `to`.
template <int from, int to>
__device__ __forceinline__ void deal_regs() {
  if constexpr (to > from)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(to));
  else if constexpr (to < from)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(to));
}

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// What a row sees, as bits over 32 neighbouring columns of a key tile.
struct RowMask {
  Visible vis;
  uint32_t tree[3];  // tree rows 0..64
  // columns [32 w, 32 w + 32) of the tile of KT keys at `base` (Item::base)
  template <int KT>
  __device__ __forceinline__ uint32_t word(int base, int w) const {
    if (base < 0) {
      w += (-1 - base) * (KT / 32);
      return w == 0 ? tree[0] : w == 1 ? tree[1] : w == 2 ? tree[2] : 0u;
    }
    const int at = base + 32 * w;
    return low_bits(vis.last - at) & (~low_bits(vis.first - at) | low_bits(vis.sink - at));
  }
};

// A row tile's part of a CTA's share, as the schedule hands it to the other roles.
struct Item {
  int b, kvh, m0, live;       // request, KV head, (row, head) pairs [m0, m0 + live)
  int r0, n, len, p0;         // PagedRequest
  int u, seg, units, sinks;   // units [u, u + seg) of RowTile's
  int first, lo, hi, sink;
  // first position of a unit; -1 - t: the tree's rows KT t, KT t + 1, ...
  template <int KT>
  __device__ __forceinline__ int base(const PagedArgs& a, int unit) const {
    const int tree = a.kt ? unit - units + (n + KT - 1) / KT : -1;
    return tree >= 0 ? -1 - tree : (unit < sinks ? unit : first + unit - sinks) * KT;
  }
  __device__ __forceinline__ bool seen(int s, int count) const {
    return (s < hi && s + count > lo) || s < sink;
  }
};
static_assert(sizeof(Item) % 16 == 0);

template <int D, int CT, int NQ>
struct TcShape {
  static constexpr bool kTma = CT == DT_BF16;
  static constexpr int KC = D / 64;
  // positions of a key tile: 64 where two CTAs with their codes share an SM
  static constexpr int KT = kTma || NQ == 2 ? 128 : 64, kShift = KT == 128 ? 7 : 6;
  static constexpr int kQChunk = 128 * 128, kQTile = KC * kQChunk;  // 128 rows x 64 bf16, x D
  static constexpr int kChunk = KT * 128, kTile = KC * kChunk;      // of keys or values
  // key tiles in flight; codes have a ring of their own in front (half a tile: keys or values)
  static constexpr int kStages = kTma && (NQ == 2 || D == 64) ? 2 : 1;
  static constexpr int kCodes = 4, kCodeBytes = KT * D;
  static constexpr int kScales = 4;             // tiles of row scales (see the loader)
  // 32-column parts of S that a row keeps in registers between its two passes: all of them, or
  // one at a time, read twice (TMEM gives 32 columns in 27 cycles; a spill costs more)
  static constexpr int kKeep = kTma && NQ == 2 ? 4 : 1;
  // Where registers are scarce the warps come in whole warpgroups and deal them
  // out anew: more for the softmax (S in registers), less for the others.  (A
  // function call in the kernel would undo this: the compiler then allots the
  // least of them to all.  And nothing hot may spill: next to this much shared
  // memory the L1 is too small for it.)
  static constexpr bool kDeal = NQ == 2 || !kTma;
  static constexpr int kSoftRegs = kTma ? 200 : NQ == 2 ? 168 : 128;
  static constexpr int kLoadRegs = kTma ? 104 : NQ == 2 ? 88 : 56;
  static constexpr int kMmaRegs = kTma ? kLoadRegs : NQ == 2 ? 88 : 56;
  // registers a thread at launch (the most that the launch bounds leave), and
  // that the shares add up to no more
  static constexpr int kLaunchRegs = NQ == 1 ? 80 : kTma ? 168 : 128;
  static_assert(NQ == 2 ? (kTma ? 2 * kSoftRegs + kLoadRegs <= 3 * kLaunchRegs
                                : 2 * kSoftRegs + kLoadRegs + kMmaRegs <= 4 * kLaunchRegs)
                        : kTma || kSoftRegs + kLoadRegs + kMmaRegs <= 3 * kLaunchRegs);
  static constexpr int kSoft = 128 * NQ;
  // warps of the MMAs, of the schedule, of TMA, and idle ones that fill a warpgroup; what turns
  // codes into bf16 is a warpgroup of its own
  static constexpr int kMma = kDeal ? 128 : 96;
  static constexpr int kLoad = kTma ? 0 : 128;
  static constexpr int kItemUsers = 2 + 4 * NQ + kLoad / 32;  // MMAs, TMA, softmax, codes
  static constexpr int kThreads = kSoft + kMma + kLoad;
  static constexpr int kItems = 4;  // row tiles that the schedule is ahead
  static constexpr int kPerSm = NQ == 2 ? 1 : 2;
  // TMEM columns: S at 128 q, O at 128 NQ + D q, P where neither is.  Only for D = 128 with
  // tiles of 128 keys is there no room left: P then lies over the upper half of S.  The next S
  // follows the product that reads P in the pipe, and products of one shape (here 128 x 128
  // both) are carried out in the order of their issue.  Of other shapes that is not promised.
  static constexpr uint32_t kTmemCols = NQ == 2 ? 512 : 256;
  static constexpr uint32_t p_at(uint32_t q) {
    return D == 128 && KT == 128 ? 128 * q + 64 : NQ == 2 ? 384 + 64 * q : KT == 64 ? 64 : 192;
  }
  static constexpr int kRows = 128 * NQ;
  static constexpr int kBars = 4 * kStages + 4 * NQ + kScales + 2 * kCodes + 2 * kItems;
  static constexpr size_t kCoded =
      kTma ? 0 : (size_t)kCodes * kCodeBytes + kScales * (2 * KT * 4);
  static constexpr size_t kSmem = (size_t)NQ * kQTile + 2 * kStages * kTile + kCoded +
                                  kItems * sizeof(Item) + kBars * 8 + 16 + 1024;
};

struct TcMaps {
  CUtensorMap k, v;    // the cache, [slots][D], boxes of min(D, 128 bytes) x min(page, key tile)
  CUtensorMap kt, vt;  // the tree's rows, [rows][Hkv * D], boxes of 64 x (Nmax + 1)
};

template <int D, int CT, int NQ>
__global__ void __launch_bounds__(TcShape<D, CT, NQ>::kThreads, TcShape<D, CT, NQ>::kPerSm)
    paged_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ PagedArgs a) {
  using S = TcShape<D, CT, NQ>;
  constexpr int KC = S::KC, ST = S::kStages, KT = S::KT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;                              // Q [NQ][KC][128 rows][128 B]
  uint8_t* sk = sq + NQ * S::kQTile;               // K [ST][KC][KT keys][128 B]
  uint8_t* sv = sk + ST * S::kTile;                // V [ST][KC][KT keys][128 B]
  // 8-bit caches: halves of tiles (keys, values) as codes, scales of tiles
  uint8_t* scode = (uint8_t*)(sv + ST * S::kTile);                       // [kCodes][KT][D]
  float* sscale = (float*)(scode + (S::kTma ? 0 : S::kCodes * S::kCodeBytes));  // [kScales][K, V][KT]
  Item* items = (Item*)(sscale + (S::kTma ? 0 : S::kScales * 2 * KT));   // [kItems]
  uint64_t* bars = (uint64_t*)(items + S::kItems);
  uint64_t* k_full = bars;
  uint64_t* k_empty = k_full + ST;
  uint64_t* v_full = k_empty + ST;
  uint64_t* v_empty = v_full + ST;
  uint64_t* q_full = v_empty + ST;
  uint64_t* s_full = q_full + NQ;
  uint64_t* p_full = s_full + NQ;
  uint64_t* o_full = p_full + NQ;
  uint64_t* c_full = o_full + NQ;                  // the scales of a tile are there
  uint64_t* w_full = c_full + S::kScales;          // a half's codes are there
  uint64_t* w_empty = w_full + S::kCodes;
  uint64_t* i_full = w_empty + S::kCodes;          // an item is there
  uint64_t* i_empty = i_full + S::kItems;
  uint32_t* tslot = (uint32_t*)(i_empty + S::kItems);
  volatile int* abort_flag = (volatile int*)(tslot + 1);
  int64_t* sums = (int64_t*)(tslot + 4);           // [batch + 1]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr Cut cut = {S::kRows, S::kShift};
  constexpr int kWarpMma = 4 * NQ, kWarpPlan = kWarpMma + 1;
  constexpr int kWarpTma = kWarpMma + 2, kWarpLoad = kWarpMma + S::kMma / 32;
  pdl_launch_dependents();  // the join may be scheduled (it waits for this grid)
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&k_full[i], S::kTma ? 1 : 128);
      mbar_init(&v_full[i], S::kTma ? 1 : 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int q = 0; q < NQ; ++q) {
      mbar_init(&q_full[q], 128);
      mbar_init(&s_full[q], 1);
      mbar_init(&p_full[q], 128);
      mbar_init(&o_full[q], 1);
    }
    for (int i = 0; i < S::kScales; ++i) mbar_init(&c_full[i], 128);
    for (int i = 0; i < S::kItems; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], S::kItemUsers);
    }
    for (int i = 0; i < S::kCodes; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 4);
    }
    *abort_flag = 0;
    a.redo[blockIdx.x] = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(tslot, S::kTmemCols);
    tc_fence_before();
  }
  const int64_t all = count_units(a, sums, cut);  // synchronises the CTA
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const int shares = (int)min((int64_t)gridDim.x, all), cta = blockIdx.x;
  const int64_t u0 = cta < shares ? first_unit(all, cta, shares) : 0;
  int left = cta < shares ? (int)(first_unit(all, cta + 1, shares) - u0) : 0;
  if (cta >= shares && tid == 0) a.tasks[cta] = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return clock_wait(bar, parity, a.status, abort_flag);
  };
  auto wait_item = [&](int n) { return wait(&i_full[n % S::kItems], (n / S::kItems) & 1); };
  auto free_item = [&](int n) { mbar_arrive(&i_empty[n % S::kItems]); };

  // The deal stands in each role's own branch, where the compiler allots by it,
  // and every warp takes part in it, with work or without: a share is raised
  // once the others have been lowered.
  if (warp >= kWarpMma) {
    if constexpr (S::kDeal && S::kTma) deal_regs<S::kLaunchRegs, S::kLoadRegs>();
    if (warp < kWarpLoad) {
      if constexpr (S::kDeal && !S::kTma) deal_regs<S::kLaunchRegs, S::kMmaRegs>();
      if (warp == kWarpPlan && lane == 0 && left > 0) {
        // ------------------------------------------------------ the schedule
        Cursor c;
        c.seek(a, sums, u0, cut);
        record_split(a, c, all, cta, shares);
        for (int n = 0;; ++n) {
          if (!wait(&i_empty[n % S::kItems], ((n / S::kItems) & 1) ^ 1)) break;
          const int seg = min(left, c.t.units - c.u);
          Item& it = items[n % S::kItems];
          it = {c.b,   c.kvh, c.t.m0,    c.t.live,  c.rq.r0,   c.rq.n, c.rq.len, c.rq.p0,
                c.u,   seg,   c.t.units, c.t.sinks, c.t.first, c.t.lo, c.t.hi,   c.t.sink};
          mbar_arrive(&i_full[n % S::kItems]);
          left -= seg;
          if (left == 0) break;
          c.next_tile(a, cut);
        }
      } else if (warp == kWarpMma && left > 0) {
        // ---------------------------------------------------------- the MMAs
        constexpr uint32_t is = idesc_bf16_f32(128, KT);
        constexpr uint32_t io = idesc_bf16_f32(128, D) | (1u << 16);  // B is MN-major
        const uint32_t one = elect_lane();
        int ns = 0, np = 0;                  // key tiles whose S / O was issued
        uint32_t q_in = 0, p_in = 0;         // phases of q_full and p_full, a bit each
        int ni = 0, in_item = 0, pairs = 0;  // items taken; units left of one, its row tiles
        bool ok = true;
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
          ok = __all_sync(0xffffffffu, ok && wait(bar, parity));
          tc_fence_after();
        };
        auto take = [&] {
          wait_all(&i_full[ni % S::kItems], (ni / S::kItems) & 1);
          pairs = items[ni % S::kItems].live > 128 ? 2 : 1;
          in_item = items[ni % S::kItems].seg;
          __syncwarp();  // (the schedule writes items by plain stores, which an arrive does order)
          if (one) free_item(ni);
          ++ni;
        };
        take();
        int live_q = 0, live_next = pairs;
        bool first = true, first_next = true;
        // turn t: O of unit t - 1, S of unit t
        for (int more = left; ok; --more) {
          const bool pv = live_q > 0, sc = more > 0;
          if (pv) wait_all(&v_full[np % ST], (np / ST) & 1);
          const uint32_t va = desc_lo_mn(smem_u32(sv) + np % ST * S::kTile, S::kChunk);
          const uint32_t ka = desc_lo_k(smem_u32(sk) + ns % ST * S::kTile);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (q < live_q) {
              wait_all(&p_full[q], (p_in >> q) & 1);
              p_in ^= 1u << q;
              if (!ok) break;
#pragma unroll
              for (int s = 0; s < KT / 16; ++s)
                mma_ts(one, tmem + NQ * 128 + q * D, tmem + S::p_at(q) + 8 * s, va + 128 * s, io,
                       !first || s != 0);
              // (between tiles s_full of the next one says it: it tracks all products so far)
              if (!sc || first_next) commit_if(one, &o_full[q]);
            }
            if (sc && q < live_next) {
              if (q == 0) wait_all(&k_full[ns % ST], (ns / ST) & 1);
              if (first_next) {
                wait_all(&q_full[q], (q_in >> q) & 1);
                q_in ^= 1u << q;
              }
              if (!ok) break;
              const uint32_t qa = desc_lo_k(smem_u32(sq) + q * S::kQTile);
#pragma unroll
              for (int s = 0; s < 4 * KC; ++s)
                mma_ss(one, tmem + q * 128, qa + (s >> 2) * (S::kQChunk >> 4) + (s & 3) * 2,
                       ka + (s >> 2) * (S::kChunk >> 4) + (s & 3) * 2, is, s != 0);
              commit_if(one, &s_full[q]);
            }
          }
          if (!ok) break;
          if (pv) {
            commit_if(one, &v_empty[np % ST]);
            ++np;
          }
          if (!sc) break;
          commit_if(one, &k_empty[ns % ST]);
          ++ns;
          live_q = live_next;
          first = first_next;
          first_next = --in_item == 0;
          if (first_next && more > 1) {
            take();
            live_next = pairs;
          }
        }
      } else if (warp == kWarpTma) {
        // ------------------------------------------------------------- copies
        // bf16: into the operands' places; codes: half a tile at a time into
        // their ring, with the tile's scales beside the keys
        const int page = 1 << a.c.page_shift, box = min(page, KT);
        bool ok = true;
        int g = 0;
        for (int n = 0; left > 0 && ok; ++n) {
          ok = __all_sync(0xffffffffu, wait_item(n));
          if (!ok) break;
          const Item& it = items[n % S::kItems];
          left -= it.seg;
          for (int k = 0; k < it.seg && ok; ++k, ++g) {
            const int base = it.template base<KT>(a, it.u + k);
            const bool mine = base < 0 ? lane == 0 : lane * box < KT;
            // a piece that no row sees, or on a page that is none: out of bounds, read as zeros
            int slot = -1;
            if (base >= 0 && mine && it.seen(base + lane * box, box)) {
              const int64_t at = a.c.slot(it.b, base + lane * box, a.status);
              if (at >= 0) slot = (int)(at + ((int64_t)it.kvh << a.c.page_shift));
            }
            const int y = slot >= 0 ? slot : (int)(((int64_t)a.c.n_pages * a.c.Hkv) << a.c.page_shift);
#pragma unroll 1
            for (int part = 0; part < 2 && ok; ++part) {
              const CUtensorMap* map = part ? &maps.v : &maps.k;
              if constexpr (S::kTma) {
                const int st = g % ST;
                uint64_t* full = (part ? v_full : k_full) + st;
                uint8_t* dst = (part ? sv : sk) + st * S::kTile;
                ok = __all_sync(0xffffffffu, wait((part ? v_empty : k_empty) + st, ((g / ST) & 1) ^ 1));
                if (!ok) break;
                if (lane == 0)
                  mbar_arrive_expect_tx(full, base < 0 ? (uint32_t)(a.Nmax + 1) * D * 2
                                                       : (uint32_t)S::kTile);
                __syncwarp();
                if (mine) {
#pragma unroll
                  for (int kc = 0; kc < KC; ++kc) {
                    if (base < 0)
                      tma_load_2d(dst + kc * S::kChunk, part ? &maps.vt : &maps.kt, full,
                                  it.kvh * D + kc * 64, it.r0);
                    else
                      tma_load_2d(dst + kc * S::kChunk + lane * box * 128, map, full, kc * 64, y);
                  }
                }
              } else {
                const int x = 2 * g + part, st = x % S::kCodes;
                float* scales = sscale + (g % S::kScales) * 2 * KT;
                // The scales' place was last used by tile g - 4.  w_empty says that the keys
                // of tile g - 2 were turned; before them the values of tile g - 3, which had
                // waited for the product with those of tile g - 4: its softmax is done.
                ok = __all_sync(0xffffffffu, wait(&w_empty[st], ((x / S::kCodes) & 1) ^ 1));
                if (!ok) break;
                if (base < 0) {  // the tree's rows come as bf16, without scales
                  if (part == 0)
                    for (int i = lane; i < 2 * KT; i += 32) scales[i] = 1.f;
                  fence_async_smem();
                  __syncwarp();
                  if (lane == 0) mbar_arrive(&w_full[st]);
                } else {
                  const unsigned there = __ballot_sync(0xffffffffu, mine && slot >= 0);
                  if (part == 0 && mine && slot < 0) {
                    for (int i = 0; i < box; ++i)
                      scales[lane * box + i] = scales[KT + lane * box + i] = 0.f;
                    fence_async_smem();
                  }
                  __syncwarp();
                  if (lane == 0)
                    mbar_arrive_expect_tx(&w_full[st], S::kCodeBytes +
                                                           (part ? 0 : __popc(there) * box * 8));
                  __syncwarp();
                  if (mine) {
                    tma_load_2d(scode + st * S::kCodeBytes + lane * box * D, map, &w_full[st], 0, y);
                    if (part == 0 && slot >= 0) {
                      bulk_load(scales + lane * box, a.c.ks + slot, box * 4, &w_full[st]);
                      bulk_load(scales + KT + lane * box, a.c.vs + slot, box * 4, &w_full[st]);
                    }
                  }
                }
              }
              __syncwarp();
            }
          }
          __syncwarp();
          if (lane == 0) free_item(n);
        }
      }
    } else if constexpr (!S::kTma) {
      // ---------------------------------------------------- codes into operands
      // A thread turns every 128th 16-byte piece of a half tile into bf16.  Eight
      // lanes take the same columns of eight neighbouring rows, in which the
      // swizzles of both rings put them into different banks.
      deal_regs<S::kLaunchRegs, S::kLoadRegs>();
      constexpr int kRowPieces = D / 16, kPieces = KT * kRowPieces / 128;
      constexpr int kStep = 128 / kRowPieces;  // rows from one of a thread's pieces to the next
      const int lw = warp - kWarpLoad;
      const int piece = (lane >> 3) + (D == 128 ? 4 * (lw & 1) : 0);
      const int row0 = (lane & 7) + 8 * (D == 128 ? lw >> 1 : lw);
      const uint32_t from = row0 * D + (D == 128 ? (piece ^ (row0 & 7)) << 4
                                                 : (piece ^ ((row0 >> 1) & 3)) << 4);
      const uint32_t to0 = (piece >> 2) * S::kChunk + sw128(row0, (piece & 3) * 2),
                     to1 = (piece >> 2) * S::kChunk + sw128(row0, (piece & 3) * 2 + 1);
      static_assert(ST == 1 && S::kScales == 4 && S::kCodes == 4);
      bool ok = true;
      int g = 0;
      for (int n = 0; left > 0 && ok; ++n) {
        ok = __all_sync(0xffffffffu, wait_item(n));
        if (!ok) break;
        const Item& it = items[n % S::kItems];
        left -= it.seg;
        const int lo = it.lo, hi = it.hi;
        for (int k = 0; k < it.seg && ok; ++k, ++g) {
          const int base = it.template base<KT>(a, it.u + k);
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            const int x = 2 * g + part, st = x % S::kCodes;
            uint8_t* dst = part ? sv : sk;
            ok = __all_sync(0xffffffffu, wait(&w_full[st], (x / S::kCodes) & 1));
            if (!ok) break;
            uint4 w[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
              w[i] = *(const uint4*)(scode + st * S::kCodeBytes + from + i * kStep * D);
            ok = __all_sync(0xffffffffu, wait(part ? v_empty : k_empty, (g & 1) ^ 1));
            if (!ok) break;
            if (base >= 0) {
#pragma unroll
              for (int i = 0; i < kPieces; ++i) {
                uint32_t o[8];
                const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t even, odd;
                  codes_to_bf16<CT>(in[e], even, odd);
                  o[2 * e] = __byte_perm(even, odd, 0x5410);
                  o[2 * e + 1] = __byte_perm(even, odd, 0x7632);
                }
                *(uint4*)(dst + to0 + i * kStep * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                *(uint4*)(dst + to1 + i * kStep * 128) = make_uint4(o[4], o[5], o[6], o[7]);
              }
            } else {
              const uint16_t* rows = (const uint16_t*)(part ? a.vt : a.kt);
#pragma unroll 2
              for (int y = tid & 127; y < KT * KC * 8; y += 128) {
                const int cc = y % (KC * 8), r = y / (KC * 8), at = (-1 - base) * KT + r;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (at < it.n)
                  v = *(const uint4*)(rows + (((int64_t)it.r0 + at) * a.c.Hkv + it.kvh) * D + cc * 8);
                *(uint4*)(dst + (cc >> 3) * S::kChunk + sw128(r, cc & 7)) = v;
              }
            }
            // A place that no row sees may have any scale, and a weight of 0 times it need not be
            // 0: a NaN there (a pool never cleared, a page whose last owner was not finite) would
            // send all rows of the tile to paged_row, 6.2 ms instead of 0.06 ms for three chunks of
            // 200 rows over up to 3000 positions.  (Cleared here, before the softmax reads it; a
            // select there, where the masks are, made the whole call 3 to 7 % longer.)
            if (part == 0 && base >= 0 && (base < lo || base + KT > hi) && (tid & 127) < KT &&
                !it.seen(base + (tid & 127), 1))
              sscale[g % S::kScales * 2 * KT + KT + (tid & 127)] = 0.f;
            fence_async_smem();
            mbar_arrive(part ? v_full : k_full);
            if (part == 0) mbar_arrive(&c_full[g % S::kScales]);
            // The codes' place is freed once the codes have been used and behind the fence: an
            // arrive alone orders this thread's loads before other threads' loads and stores,
            // not before a copy's writes (the async proxy).  An earlier form arrived between the
            // loads and the wait for the operand's place and, with P over scores of another
            // shape (p_at), gave wrong outputs under load.  Both were changed in one step; which
            // of the two was seen there has not been established, and neither is promised to work.
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_empty[st]);
          }
        }
        __syncwarp();
        if (lane == 0) free_item(n);
      }
    }
  } else {
    // ------------------------------------------------------------ the softmax
    if constexpr (S::kDeal) deal_regs<S::kLaunchRegs, S::kSoftRegs>();
    const int q = warp >> 2, row = tid & 127;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + quad + q * 128, to = tmem + quad + NQ * 128 + q * D;
    const uint32_t tp = tmem + quad + S::p_at(q);
    uint8_t* my_q = sq + q * S::kQTile;
    const float sl2 = a.scale * kL2e;
    // item n's queries into shared memory, zeros where there is no row
    auto start_q = [&](int n) {
      const Item& it = items[n % S::kItems];
      const int m0 = it.m0 + q * 128, live = it.live - q * 128, r0 = it.r0, h0 = it.kvh * a.G;
#pragma unroll 4
      for (int x = row; x < 128 * KC * 8; x += 128) {
        const int cc = x % (KC * 8), r = x / (KC * 8), m = m0 + (r < live ? r : 0);
        cp16(smem_u32(my_q + (cc >> 3) * S::kQChunk + sw128(r, cc & 7)),
             (const uint16_t*)a.q + (r0 + (int64_t)(m / a.G)) * a.ld_q +
                 ((int64_t)h0 + m % a.G) * D + cc * 8,
             r < live);
      }
    };
    auto finish_q = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async_smem();
      mbar_arrive(&q_full[q]);
    };
    bool ok = true, q_started = false;
    int n_done = 0, n_item = 0;  // key tiles and row tiles of this warpgroup's barriers
    int g = 0;                   // key tiles of the CTA
    for (int n = 0; left > 0; ++n) {
      ok = __all_sync(0xffffffffu, wait_item(n));
      if (!ok) break;
      const Item& it = items[n % S::kItems];
      const int seg = it.seg, live = it.live - q * 128;
      left -= seg;
      if (live <= 0) {  // no row of this item is in the second row tile
        g += seg;
        __syncwarp();
        if (lane == 0) free_item(n);
        continue;
      }
      if (!q_started) {
        start_q(n);
        finish_q();
      }
      q_started = false;
      const bool head = it.u > 0, whole = it.u == 0 && seg == it.units;
      const bool there = row < live;
      const int m_at = it.m0 + q * 128 + (there ? row : 0);
      const int i = m_at / a.G, h = it.kvh * a.G + m_at % a.G;
      const PagedRequest rq = {it.r0, it.n, it.len, it.p0};
      RowMask mask;
      mask.vis = visible(a, row_position(a, rq, it.b, i), rq.len);
      mask.tree[0] = mask.tree[1] = mask.tree[2] = 0;
      if (a.kt) {
        const uint64_t anc = i ? a.anc[(int64_t)it.b * a.Nmax + i - 1] : 0ull;
        mask.tree[0] = (1u | ((uint32_t)anc << 1)) & low_bits(rq.n);
        mask.tree[1] = (uint32_t)(anc >> 31) & low_bits(rq.n - 32);
        mask.tree[2] = (uint32_t)(anc >> 63) & low_bits(rq.n - 64);
      }
      const bool sees = a.kt || mask.vis.sink > 0 || mask.vis.last > mask.vis.first;
      // key tiles in [whole_lo, whole_hi) need no mask for any row of the warp
      const int whole_lo = __reduce_max_sync(0xffffffffu, mask.vis.first);
      const int whole_hi = __reduce_min_sync(0xffffffffu, mask.vis.last);
      float m = -INFINITY, l = 0.f;
      // O times a factor per row: the products so far are complete (s_full)
      auto rescale = [&](float keep) {
#pragma unroll 1
        for (int w = 0; w < D / 16; ++w) {
          uint32_t x[16];
          tmem_ld16_nowait(to + 16 * w, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * keep);
          tmem_st16(to + 16 * w, x);
        }
      };
      for (int k = 0; k < seg; ++k, ++g, ++n_done) {
        const int base = it.template base<KT>(a, it.u + k);
        const bool masked = base < whole_lo || base + KT > whole_hi;
        ok = wait(&s_full[q], n_done & 1);
        if constexpr (!S::kTma)
          ok = ok && wait(&c_full[g % S::kScales], (g / S::kScales) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (k == seg - 1 && left > 0) {
          // S is complete, so Q's place is free: the next row tile's is on its way
          ok = __all_sync(0xffffffffu, wait_item(n + 1));
          if (!ok) break;
          q_started = items[(n + 1) % S::kItems].live > q * 128;
          if (q_started) start_q(n + 1);
        }
        {
          constexpr int kKeep = S::kKeep, kParts = KT / 32;
          // (a scale of NaN at a place that a row does not see, but another row of the tile
          // does, makes its sum NaN, with a finite weight sum: such rows are done again, see
          // paged_row)
          const float* scales = sscale + g % S::kScales * 2 * KT;
          // ---- the row's largest score of this tile
          uint32_t r[kKeep][32];
          auto load = [&](int w0) {
#pragma unroll
            for (int w = w0; w < w0 + kKeep; ++w) tmem_ld32(ts + 32 * w, r[w - w0]);
            tmem_wait_ld();
            if constexpr (!S::kTma) {  // times the keys' scales
#pragma unroll
              for (int w = w0; w < w0 + kKeep; ++w)
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const float4 f = *(const float4*)(scales + 32 * w + e);
                  uint32_t* x = r[w - w0] + e;
                  mul2(x[0], x[1], f.x, f.y);
                  mul2(x[2], x[3], f.z, f.w);
                }
            }
            if (masked) {
#pragma unroll
              for (int w = w0; w < w0 + kKeep; ++w) {
                const uint32_t see = mask.template word<KT>(base, w);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  r[w - w0][e] = (see >> e) & 1u ? r[w - w0][e] : 0xff800000u;
              }
            }
          };
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int w0 = kParts - kKeep; w0 >= 0; w0 -= kKeep) {
            load(w0);
#pragma unroll
            for (int w = 0; w < kKeep; ++w)
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                t4[(e / 2) % 4] = fmaxf(fmaxf(t4[(e / 2) % 4], __uint_as_float(r[w][e])),
                                        __uint_as_float(r[w][e + 1]));
          }
          const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * sl2;
          // ---- the maximum in use
          if (k == 0) {
            m = top;
          } else if (__any_sync(0xffffffffu, top > m + kRescale)) {
            const float now = fmaxf(m, top);
            const float keep = m == now ? 1.f : ex2(m - now);
            l *= keep;
            m = now;
            rescale(keep);
          }
          const float less = m == -INFINITY ? 0.f : -m;
          // ---- weights, in bf16 for the second product
          float la[4] = {0.f, 0.f, 0.f, 0.f};
          // (from the last part on: P's parts lie over parts of S that were read already)
#pragma unroll (kKeep == 1 ? 1 : kParts)
          for (int w = kParts - 1; w >= 0; --w) {
            if (kKeep == 1) load(w);
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              uint32_t* x = r[kKeep == 1 ? 0 : w] + e;
              float p[4];
              fma2(x[0], x[1], sl2, less, p[0], p[1]);
              fma2(x[2], x[3], sl2, less, p[2], p[3]);
#pragma unroll
              for (int y = 0; y < 4; ++y) p[y] = ex2(p[y]);
              add2(la[0], la[1], p[0], p[1]);
              add2(la[2], la[3], p[2], p[3]);
              if constexpr (!S::kTma) {  // times the values' scales
                const float4 f = *(const float4*)(scales + KT + 32 * w + e);
                uint32_t z[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) z[y] = __float_as_uint(p[y]);
                mul2(z[0], z[1], f.x, f.y);
                mul2(z[2], z[3], f.z, f.w);
#pragma unroll
                for (int y = 0; y < 4; ++y) p[y] = __uint_as_float(z[y]);
              }
              pk[e / 2] = pack2(p[0], p[1]);
              pk[e / 2 + 1] = pack2(p[2], p[3]);
            }
            tmem_st16(tp + 16 * w, pk);
          }
          l += (la[0] + la[1]) + (la[2] + la[3]);
        }
        if constexpr (S::kTma) {
          // V rows that are no positions of the request may hold anything: zeros, before 0 * NaN
          const int valid = base < 0 ? rq.n : rq.len - base;
          if (valid < KT) {
            ok = __all_sync(0xffffffffu, wait(&v_full[g % ST], (g / ST) & 1));
            if (!ok) break;
            uint8_t* v = sv + (g % ST) * S::kTile;
#pragma unroll 1
            for (int x = row; x < 128 * KC * 8; x += 128) {
              const int r8 = x / (KC * 8), cc = x % (KC * 8);
              if (r8 >= valid)
                *(uint4*)(v + (cc >> 3) * S::kChunk + sw128(r8, cc & 7)) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[q]);
      }
      if (!ok) break;
      if (q_started) finish_q();
      ok = __all_sync(0xffffffffu, wait(&o_full[q], n_item & 1));
      if (!ok) break;
      ++n_item;
      tc_fence_after();
      if (whole) {
        const float inv = row_factor(l, sees);
        uint16_t* out = (uint16_t*)a.out + (((int64_t)rq.r0 + i) * a.Hq + h) * D;
        float odd = 0.f;  // NaN once an output is infinite or NaN
#pragma unroll 1
        for (int w = 0; w < D / 32; ++w) {
          uint32_t r[32];
          tmem_ld32(to + 32 * w, r);
          tmem_wait_ld();
          uint4 pk[4];
          uint32_t* pw = (uint32_t*)pk;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float x = __uint_as_float(r[e]), y = __uint_as_float(r[e + 1]);
            odd = fmaf(x, 0.f, fmaf(y, 0.f, odd));
            pw[e / 2] = sees ? pack2(x * inv, y * inv) : 0u;
          }
          if (there) {
#pragma unroll
            for (int e = 0; e < 4; ++e) *(uint4*)(out + 32 * w + 8 * e) = pk[e];
          }
        }
        // finite weights, but not their sums with the values: the join looks at them again
        if (there && sees && odd != 0.f && l - l == 0.f) a.redo[cta] = 1;
      } else {
        const int64_t at = (int64_t)(2 * cta + (head ? 0 : 1)) * a.part_rows + q * 128 + row;
        float* po = a.part_o + at * D;
        if (there) a.part_ml[at] = make_float2(m, sees ? l : -1.f);
#pragma unroll 1
        for (int w = 0; w < D / 32; ++w) {
          uint32_t r[32];
          tmem_ld32(to + 32 * w, r);
          tmem_wait_ld();
          if (there) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *(uint4*)(po + 32 * w + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) free_item(n);
    }
  }
  __syncwarp();
  if (*abort_flag) {
    // gave up: let copies and products that are under way land before the CTA's memory goes
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

template <int D, int CT, int NQ>
cudaError_t launch_shape(const PagedArgs& a, const TcMaps& maps, int ctas, cudaStream_t s) {
  using S = TcShape<D, CT, NQ>;
  const size_t smem = S::kSmem + 8 * ((size_t)a.batch + 1);
  auto kern = paged_tc_kernel<D, CT, NQ>;
  if constexpr (S::kDeal) {
    // the deal counts on the registers that a thread has at launch
    static const bool as_compiled = [kern] {
      cudaFuncAttributes f;
      return cudaFuncGetAttributes(&f, kern) == cudaSuccess && f.numRegs == S::kLaunchRegs;
    }();
    if (!as_compiled) return cudaErrorInvalidKernelImage;
  }
  // the limit is raised once, to the most that any batch needs
  cudaError_t e = ensure_smem(kern, S::kSmem + 8 * (kMaxKvBatch + 1));
  if (e != cudaSuccess) return e;
  {
    ProfileScope ps(DT_K_ATTN, s);
    kern<<<ctas, S::kThreads, smem, s>>>(maps, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_paged_join(a, CT, Cut{S::kRows, S::kShift}, ctas, s);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedArgs& a, int ct, const dt_kv_cache* cache, int tiles,
                            cudaStream_t s) {
  TcMaps maps = {};
  const int bytes = ct == DT_BF16 ? 2 : 1;
  const uint64_t slots = (uint64_t)cache->n_pages * cache->Hkv * cache->page_size;
  const uint32_t box = std::min(cache->page_size, bytes == 2 || tiles == 2 ? 128 : 64);
  if (!paged_map(&maps.k, cache->d_k, bytes, a.d, slots, box) ||
      !paged_map(&maps.v, cache->d_v, bytes, a.d, slots, box))
    return cudaErrorInvalidValue;
  if (a.kt && bytes == 2) {
    const uint64_t cols = (uint64_t)cache->Hkv * a.d;
    if (!paged_map(&maps.kt, a.kt, 2, cols, a.total_rows, a.Nmax + 1) ||
        !paged_map(&maps.vt, a.vt, 2, cols, a.total_rows, a.Nmax + 1))
      return cudaErrorInvalidValue;
  }
  const int sms = std::min(dt_num_sms(), kPagedSms), ctas = tiles == 2 ? sms : 2 * sms;
#define DT_PAGED(DD, CC)                                               \
  if (a.d == DD && ct == CC)                                           \
    return tiles == 2 ? launch_shape<DD, CC, 2>(a, maps, ctas, s)      \
                      : launch_shape<DD, CC, 1>(a, maps, ctas, s);
  DT_PAGED(64, DT_BF16)
  DT_PAGED(128, DT_BF16)
  DT_PAGED(64, DT_E4M3)
  DT_PAGED(128, DT_E4M3)
  DT_PAGED(64, DT_I8)
  DT_PAGED(128, DT_I8)
#undef DT_PAGED
  return cudaErrorInvalidValue;
}

}  // namespace dt
