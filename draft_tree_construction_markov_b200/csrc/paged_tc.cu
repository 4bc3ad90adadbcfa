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
// keys and values in shared memory; one thread that issues the MMAs; and the
// loaders.  A bf16 cache comes by TMA, a page (or 128 rows of it) a box; an
// 8-bit cache is read with 16-byte loads a tile ahead, turned into bf16 (exact
// for every code, see codes_to_bf16) and stored swizzled by a warpgroup, with
// the row scales beside it: those of K multiply S, those of V multiply P.
// While one row tile's softmax runs, the tensor core works for the other (NQ =
// 2), or for the second CTA of the SM (NQ = 1).
//
// The work of a call (row tiles x KV heads x key tiles) is divided over the
// CTAs in equal consecutive shares; a row tile that two shares cut is joined by
// paged_join_kernel from fp32 partials.
#include <algorithm>

#include "paged_attn.cuh"

namespace dt {
namespace {

constexpr float kRescale = 8.f;  // log2 units that a row's maximum may grow without a rescale

// 16-byte chunk c of row r of a 128-byte-swizzled tile (8-row, 1024-byte atoms)
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}

// Descriptor of an operand whose 64-element chunks of the M or N axis are
// contiguous (128-byte-swizzled rows, one per K index): chunks `chunk` bytes
// apart, 8-row groups 1024.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t chunk) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((chunk >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
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
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int D, int CT, int NQ>
struct TcShape {
  static constexpr bool kTma = CT == DT_BF16;
  static constexpr int KC = D / 64;
  static constexpr int kChunk = 128 * 128;      // bytes of 128 rows x 64 bf16
  static constexpr int kOperand = KC * kChunk;  // bytes of 128 rows x D
  // key tiles in flight: a second one where shared memory has room for it
  static constexpr int kStages = NQ == 2 || D == 64 ? 2 : 1;
  static constexpr int kScales = 4;             // tiles of row scales (see the loader)
  static constexpr int kSoft = 128 * NQ;
  static constexpr int kLoad = kTma ? 32 : 128;
  static constexpr int kThreads = kSoft + 32 + kLoad;
  static constexpr int kPerSm = NQ == 2 ? 1 : 2;
  static constexpr uint32_t kTmemCols = NQ == 2 ? 512 : 256;  // S: 128 columns a row tile, O: D
  static constexpr int kRows = 128 * NQ;
  static constexpr int kBars = 4 * kStages + 4 * NQ + kScales;
  static constexpr size_t kSmem = (size_t)(NQ + 2 * kStages) * kOperand +
                                  (kTma ? 0 : kScales * 2 * 128 * 4) + kBars * 8 + 32 + 1024;
};

struct TcMaps {
  CUtensorMap k, v;    // the cache, [slots][D], boxes of 64 x min(page, 128)
  CUtensorMap kt, vt;  // the tree's rows, [rows][Hkv * D], boxes of 64 x (Nmax + 1)
};

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// What a row sees, as bits over 32 neighbouring columns of a key tile.
struct RowMask {
  Visible vis;
  uint64_t tree;  // tree rows 0..63; row 64 in `top`
  uint32_t top;
  // columns [32 w, 32 w + 32) of the tile at position `base` (-1: the tree's)
  __device__ __forceinline__ uint32_t word(int base, int w) const {
    if (base < 0) return w == 0 ? (uint32_t)tree : w == 1 ? (uint32_t)(tree >> 32) : w == 2 ? top : 0u;
    const int at = base + 32 * w;
    return low_bits(vis.last - at) & (~low_bits(vis.first - at) | low_bits(vis.sink - at));
  }
};

template <int D, int CT, int NQ>
__global__ void __launch_bounds__(TcShape<D, CT, NQ>::kThreads, TcShape<D, CT, NQ>::kPerSm)
    paged_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ PagedArgs a) {
  using S = TcShape<D, CT, NQ>;
  constexpr int KC = S::KC, ST = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;                              // Q [NQ][KC][128 rows][128 B]
  uint8_t* sk = sq + NQ * S::kOperand;             // K [ST][KC][128 keys][128 B]
  uint8_t* sv = sk + ST * S::kOperand;             // V [ST][KC][128 keys][128 B]
  float* sscale = (float*)(sv + ST * S::kOperand); // [kScales][K, V][128]
  uint64_t* bars = (uint64_t*)((uint8_t*)sscale + (S::kTma ? 0 : S::kScales * 2 * 128 * 4));
  uint64_t* k_full = bars;
  uint64_t* k_empty = k_full + ST;
  uint64_t* v_full = k_empty + ST;
  uint64_t* v_empty = v_full + ST;
  uint64_t* q_full = v_empty + ST;
  uint64_t* s_full = q_full + NQ;
  uint64_t* p_full = s_full + NQ;
  uint64_t* o_full = p_full + NQ;
  uint64_t* c_full = o_full + NQ;                  // the scales of a tile are there
  uint32_t* tslot = (uint32_t*)(c_full + S::kScales);
  volatile int* abort_flag = (volatile int*)(tslot + 1);
  int64_t* sums = (int64_t*)(tslot + 4);           // [batch + 1]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr Cut cut = {S::kRows, 7};
  static_assert(kTcKeys == 1 << 7);
  constexpr int kWarpMma = 4 * NQ, kWarpLoad = kWarpMma + 1;
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
    *abort_flag = 0;
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
  if (cta >= shares && tid == 0) a.split[cta].parts = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity, a.status, abort_flag);
  };

  if (left == 0) {
    // nothing to do: fall through to the end
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ the MMAs
    if (lane == 0) {
      constexpr uint32_t is = idesc_bf16_f32(128, 128);
      constexpr uint32_t io = idesc_bf16_f32(128, D) | (1u << 16);  // B is MN-major
      Cursor c;
      c.seek(a, sums, u0, cut);
      record_split(a, c, all, cta, shares);
      int ns = 0, np = 0;                // key tiles whose S / O was issued
      int nq_in[NQ] = {}, np_in[NQ] = {};  // phases of q_full and p_full
      bool ok = true;
      auto scores = [&](int q, bool first) {
        if (first) {
          ok = ok && wait(&q_full[q], nq_in[q] & 1);
          ++nq_in[q];
          tc_fence_after();
        }
        if (!ok) return;
        const uint32_t qa = smem_u32(sq + q * S::kOperand),
                       ka = smem_u32(sk + (ns % ST) * S::kOperand);
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
          const uint64_t da = smem_desc_k_sw128(qa + kc * S::kChunk);
          const uint64_t db = smem_desc_k_sw128(ka + kc * S::kChunk);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tc_mma_bf16(tmem + q * 128, da + 2 * s, db + 2 * s, is, (kc | s) != 0);
        }
        tc_commit(&s_full[q]);
      };
      int live_q = c.t.live > 128 ? 2 : 1;
      bool first = true;
      ok = wait(&k_full[0], 0);
      tc_fence_after();
      for (int q = 0; q < NQ && q < live_q; ++q) scores(q, true);
      if (ok) tc_commit(&k_empty[0]);
      ++ns;
      while (ok) {
        // the unit after this one
        int live_next = live_q;
        bool first_next = false;
        if (left > 1 && ++c.u == c.t.units) {
          c.next_tile(a, cut);
          live_next = c.t.live > 128 ? 2 : 1;
          first_next = true;
        }
        ok = ok && wait(&v_full[np % ST], (np / ST) & 1);
        const uint64_t dv =
            smem_desc_mn_sw128(smem_u32(sv + (np % ST) * S::kOperand), S::kChunk);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (q < live_q) {
            ok = ok && wait(&p_full[q], np_in[q] & 1);
            ++np_in[q];
            tc_fence_after();
            if (!ok) break;
#pragma unroll
            for (int s = 0; s < 8; ++s)
              tc_mma_ts(tmem + NQ * 128 + q * D, tmem + q * 128 + 8 * s, dv + 128 * s, io,
                        !first || s != 0);
            tc_commit(&o_full[q]);
          }
          if (left > 1 && q < live_next) {
            if (q == 0) {
              ok = ok && wait(&k_full[ns % ST], (ns / ST) & 1);
              tc_fence_after();
            }
            scores(q, first_next);
          }
        }
        if (!ok) break;
        tc_commit(&v_empty[np % ST]);
        ++np;
        if (--left == 0) break;
        tc_commit(&k_empty[ns % ST]);
        ++ns;
        live_q = live_next;
        first = first_next;
      }
    }
  } else if (warp >= kWarpLoad) {
    // ------------------------------------------------------------ the loads
    Cursor c;
    c.seek(a, sums, u0, cut);
    bool ok = true;
    if constexpr (S::kTma) {
      const int page = 1 << a.c.page_shift, box = min(page, 128);
      for (int g = 0; left > 0 && ok; ++g, --left) {
        const int base = unit_base(a, c.t, c.u, cut), st = g % ST;
        const uint32_t parity = ((g / ST) & 1) ^ 1;
        int y = 0;
        const bool mine = base < 0 ? lane == 0 : lane * box < kTcKeys;
        if (base >= 0 && mine) {
          const int s = base + lane * box;
          // a piece that no row sees, or on a page that is none: out of bounds, read as zeros
          int64_t slot = -1;
          if (piece_seen(c.t, s, box)) slot = a.c.slot(c.b, s, a.status);
          y = (int)(slot < 0 ? ((int64_t)a.c.n_pages * a.c.Hkv) << a.c.page_shift
                             : slot + ((int64_t)c.kvh << a.c.page_shift));
        }
        const uint32_t bytes = base < 0 ? (uint32_t)(a.Nmax + 1) * D * 2 : (uint32_t)S::kOperand;
        auto load = [&](const CUtensorMap* cached, const CUtensorMap* tree, uint8_t* dst,
                        uint64_t* full, uint64_t* empty) {
          ok = ok && __all_sync(0xffffffffu, wait(empty, parity));
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(full, bytes);
          __syncwarp();
          if (!mine) return;
#pragma unroll
          for (int kc = 0; kc < KC; ++kc) {
            if (base < 0)
              tma_load_2d(dst + kc * S::kChunk, tree, full, c.kvh * D + kc * 64, c.rq.r0);
            else
              tma_load_2d(dst + kc * S::kChunk + lane * box * 128, cached, full, kc * 64, y);
          }
        };
        load(&maps.k, &maps.kt, sk + st * S::kOperand, &k_full[st], &k_empty[st]);
        __syncwarp();
        load(&maps.v, &maps.vt, sv + st * S::kOperand, &v_full[st], &v_empty[st]);
        __syncwarp();
        if (left > 1 && ++c.u == c.t.units) c.next_tile(a, cut);
      }
    } else {
      // 8-bit codes: a thread takes every 128th 16-byte piece of the tile
      constexpr int kRowPieces = D / 16, kPieces = 128 * kRowPieces / 128;
      const int lt = tid - kWarpLoad * 32;
      const int piece = lt % kRowPieces;
      uint4 kw[kPieces], vw[kPieces];
      float kscale = 0.f, vscale = 0.f;
      // slot of the tile's position j for this KV head, or -1
      auto slot_of = [&](int base, int j) -> int64_t {
        const int s = base + j;
        if (!piece_seen(c.t, s, 1)) return -1;
        const int64_t slot = a.c.slot(c.b, s, a.status);
        return slot < 0 ? -1 : slot + ((int64_t)c.kvh << a.c.page_shift);
      };
      auto fetch = [&](const void* cache, const float* scales, uint4 (&w)[kPieces], float& scale) {
        const int base = unit_base(a, c.t, c.u, cut);
        if (base < 0) return;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int64_t slot = slot_of(base, (lt + i * 128) / kRowPieces);
          w[i] = slot < 0 ? make_uint4(0, 0, 0, 0)
                          : __ldg((const uint4*)((const uint8_t*)cache + slot * D + piece * 16));
        }
        const int64_t slot = slot_of(base, lt);
        scale = slot < 0 ? 0.f : __ldg(scales + slot);
      };
      // the tile into shared memory as bf16: codes that are in registers, or the tree's rows
      auto place = [&](uint8_t* dst, const void* tree, const uint4 (&w)[kPieces]) {
        if (unit_base(a, c.t, c.u, cut) < 0) {
          const uint16_t* rows = (const uint16_t*)tree;
          for (int x = lt; x < 128 * KC * 8; x += 128) {
            const int cc = x % (KC * 8), r = x / (KC * 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < c.rq.n)
              v = *(const uint4*)(rows + (((int64_t)c.rq.r0 + r) * a.c.Hkv + c.kvh) * D + cc * 8);
            *(uint4*)(dst + (cc >> 3) * S::kChunk + sw128(r, cc & 7)) = v;
          }
          return;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int r = (lt + i * 128) / kRowPieces;
          uint32_t o[8];
          const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) codes_to_bf16<CT>(in[e], o[2 * e], o[2 * e + 1]);
          uint8_t* at = dst + (piece >> 2) * S::kChunk;
          const int c0 = (piece & 3) * 2;
          // the lanes of the second 64 columns store their halves in the other order: all 32 banks
          const int odd = piece >> 2;
          *(uint4*)(at + sw128(r, c0 + odd)) =
              odd ? make_uint4(o[4], o[5], o[6], o[7]) : make_uint4(o[0], o[1], o[2], o[3]);
          *(uint4*)(at + sw128(r, c0 + 1 - odd)) =
              odd ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(o[4], o[5], o[6], o[7]);
        }
      };
      fetch(a.c.k, a.c.ks, kw, kscale);
      fetch(a.c.v, a.c.vs, vw, vscale);
      for (int g = 0; left > 0; ++g, --left) {
        const int st = g % ST;
        const uint32_t parity = ((g / ST) & 1) ^ 1;
        const bool tree = unit_base(a, c.t, c.u, cut) < 0;
        // The scales' slot was last used by tile g - 4.  k_empty means that S of
        // tile g - ST is complete, which was issued only after the softmax of
        // the tile before it had handed over P; so tile g - ST - 1 >= g - 4 is done.
        float* scales = sscale + (g % S::kScales) * 256;
        Cursor now = c;
        ok = ok && wait(&k_empty[st], parity);
        if (!__all_sync(0xffffffffu, ok)) break;
        place(sk + st * S::kOperand, a.kt, kw);
        scales[lt] = tree ? 1.f : kscale;
        scales[128 + lt] = tree ? 1.f : vscale;
        fence_async_smem();
        mbar_arrive(&k_full[st]);
        mbar_arrive(&c_full[g % S::kScales]);
        // the next tile's loads are on their way while this one is worked on
        bool more = left > 1;
        if (more && ++c.u == c.t.units) c.next_tile(a, cut);
        if (more) fetch(a.c.k, a.c.ks, kw, kscale);
        Cursor next = c;
        c = now;
        ok = wait(&v_empty[st], parity);
        if (!__all_sync(0xffffffffu, ok)) break;
        place(sv + st * S::kOperand, a.vt, vw);
        fence_async_smem();
        mbar_arrive(&v_full[st]);
        c = next;
        if (more) fetch(a.c.v, a.c.vs, vw, vscale);
      }
    }
  } else {
    // ---------------------------------------------------------- the softmax
    const int q = warp >> 2, row = tid & 127;
    const uint32_t quad = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + quad + q * 128, to = tmem + quad + NQ * 128 + q * D;
    uint8_t* my_q = sq + q * S::kOperand;
    const float sl2 = a.scale * kL2e;
    Cursor c;
    c.seek(a, sums, u0, cut);
    // the row tile's queries into shared memory, zeros where there is no row
    auto load_q = [&](const Cursor& c) {
      for (int x = row; x < 128 * KC * 8; x += 128) {
        const int cc = x % (KC * 8), r = x / (KC * 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q * 128 + r < c.t.live) {
          const int m = c.t.m0 + q * 128 + r;
          v = *(const uint4*)((const uint16_t*)a.q + (c.rq.r0 + (int64_t)(m / a.G)) * a.ld_q +
                              ((int64_t)c.kvh * a.G + m % a.G) * D + cc * 8);
        }
        *(uint4*)(my_q + (cc >> 3) * S::kChunk + sw128(r, cc & 7)) = v;
      }
      fence_async_smem();
      mbar_arrive(&q_full[q]);
    };
    if (q * 128 < c.t.live) load_q(c);
    bool ok = true;
    int n_done = 0;  // key tiles of this row tile's barriers
    int g = 0;       // key tiles of the CTA
    bool head = c.u > 0;
    while (left > 0) {
      const int seg = min(left, c.t.units - c.u);
      if (q * 128 >= c.t.live) {  // no row of this item is in the second row tile
        g += seg;
        left -= seg;
        head = false;
        if (left > 0) {
          c.next_tile(a, cut);
          if (q * 128 < c.t.live) load_q(c);
        }
        continue;
      }
      const bool there = q * 128 + row < c.t.live;
      const int m_at = c.t.m0 + q * 128 + (there ? row : 0);
      const int i = m_at / a.G, h = c.kvh * a.G + m_at % a.G;
      RowMask mask;
      mask.vis = visible(a, row_position(a, c.rq, c.b, i), c.rq.len);
      mask.tree = 0;
      mask.top = 0;
      if (a.kt) {
        const uint64_t anc = i ? a.anc[(int64_t)c.b * a.Nmax + i - 1] : 0ull;
        mask.tree = 1ull | (anc << 1);
        mask.top = (uint32_t)(anc >> 63);
        if (c.rq.n < 64) mask.tree &= (1ull << c.rq.n) - 1;
        if (c.rq.n < 65) mask.top = 0;
      }
      // key tiles in [whole_lo, whole_hi) need no mask for any row of the tile
      int whole_lo = mask.vis.first, whole_hi = mask.vis.last;
      whole_lo = __reduce_max_sync(0xffffffffu, whole_lo);
      whole_hi = __reduce_min_sync(0xffffffffu, whole_hi);
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < seg; ++k, ++g, ++n_done) {
        const int base = unit_base(a, c.t, c.u + k, cut);
        const bool masked = base < whole_lo || base + kTcKeys > whole_hi;
        const float* scales = sscale + (g % S::kScales) * 256;
        ok = ok && wait(&s_full[q], n_done & 1);
        if constexpr (!S::kTma)
          ok = ok && wait(&c_full[g % S::kScales], (g / S::kScales) & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // ---- the row's largest score of this tile
        float top = -INFINITY;
        uint32_t r[32];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          tmem_ld32(ts + 32 * w, r);
          tmem_wait_ld();
          const uint32_t see = masked ? mask.word(base, w) : 0xffffffffu;
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 sc = make_float4(1.f, 1.f, 1.f, 1.f);
            if constexpr (!S::kTma) sc = *(const float4*)(scales + 32 * w + e);
            const float f[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float s = __uint_as_float(r[e + x]);
              if constexpr (!S::kTma) s *= f[x];
              if (masked) s = (see >> (e + x)) & 1u ? s : -INFINITY;
              t4[x] = fmaxf(t4[x], s);
            }
          }
          top = fmaxf(top, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
        }
        top *= sl2;
        // ---- the maximum in use
        if (k == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + kRescale)) {
          const float now = fmaxf(m, top);
          const float keep = m == now ? 1.f : ex2(m - now);
          l *= keep;
          m = now;
          ok = wait(&o_full[q], (n_done - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            tmem_ld32(to + 32 * w, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * keep);
            tmem_st32(to + 32 * w, r);
          }
        }
        const float use = m == -INFINITY ? 0.f : m;
        // ---- weights, in bf16 for the second product, over the scores
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          tmem_ld32(ts + 32 * w, r);
          tmem_wait_ld();
          const uint32_t see = masked ? mask.word(base, w) : 0xffffffffu;
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 sc = make_float4(1.f, 1.f, 1.f, 1.f), vc = sc;
            if constexpr (!S::kTma) {
              sc = *(const float4*)(scales + 32 * w + e);
              vc = *(const float4*)(scales + 128 + 32 * w + e);
            }
            const float f[4] = {sc.x, sc.y, sc.z, sc.w}, fv[4] = {vc.x, vc.y, vc.z, vc.w};
            float p[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float s = __uint_as_float(r[e + x]);
              if constexpr (!S::kTma) s *= f[x];
              p[x] = ex2(fmaf(s, sl2, -use));
              if (masked) p[x] = (see >> (e + x)) & 1u ? p[x] : 0.f;
              l4[x] += p[x];
              if constexpr (!S::kTma) {
                p[x] *= fv[x];
                if (masked) p[x] = (see >> (e + x)) & 1u ? p[x] : 0.f;
              }
            }
            pk[e / 2] = pack2(p[0], p[1]);
            pk[e / 2 + 1] = pack2(p[2], p[3]);
          }
          tmem_st16(ts + 16 * w, pk);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        if constexpr (S::kTma) {
          // V rows that are no positions of the request may hold anything: zeros, before 0 * NaN
          const int valid = base < 0 ? c.rq.n : c.rq.len - base;
          if (valid < kTcKeys) {
            ok = wait(&v_full[g % ST], (g / ST) & 1);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            uint8_t* v = sv + (g % ST) * S::kOperand;
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
      left -= seg;
      const bool whole = c.u == 0 && seg == c.t.units;
      const Cursor now = c;
      if (left > 0) {
        c.next_tile(a, cut);
        if (q * 128 < c.t.live) load_q(c);
      }
      ok = __all_sync(0xffffffffu, wait(&o_full[q], (n_done - 1) & 1));
      if (!ok) break;
      tc_fence_after();
      if (whole) {
        const bool sees = a.kt || mask.vis.sink > 0 || mask.vis.last > mask.vis.first;
        const float inv = row_factor(l, sees);
        uint16_t* out = (uint16_t*)a.out + (((int64_t)now.rq.r0 + i) * a.Hq + h) * D;
        float odd = 0.f;  // NaN once an output is infinite or NaN
        uint32_t r[32];
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
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
        // finite weights, but not their sums with the values
        unsigned again = __ballot_sync(0xffffffffu, there && sees && odd != 0.f && l - l == 0.f);
        for (; again; again &= again - 1) {
          const int from = __ffs(again) - 1;
          paged_row<CT, DT_BF16>(a, now.b, __shfl_sync(0xffffffffu, i, from),
                                 __shfl_sync(0xffffffffu, h, from));
        }
      } else {
        const int64_t at = (int64_t)(2 * cta + (head ? 0 : 1)) * a.part_rows + q * 128 + row;
        float* po = a.part_o + at * D;
        uint32_t r[32];
        if (there) a.part_ml[at] = make_float2(m, l);
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
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
      head = false;
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
  // the limit is raised once, to the most that any batch needs
  cudaError_t e = ensure_smem(kern, S::kSmem + 8 * (kMaxKvBatch + 1));
  if (e != cudaSuccess) return e;
  {
    ProfileScope ps(DT_K_ATTN, s);
    kern<<<ctas, S::kThreads, smem, s>>>(maps, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch_paged_join(a, CT, Cut{S::kRows, 7}, ctas, s);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedArgs& a, int ct, const dt_kv_cache* cache, int tiles,
                            cudaStream_t s) {
  TcMaps maps = {};
  if (ct == DT_BF16) {
    const uint64_t slots = (uint64_t)cache->n_pages * cache->Hkv * cache->page_size;
    const uint32_t box = std::min(cache->page_size, 128);
    if (!paged_map(&maps.k, cache->d_k, 2, a.d, slots, box) ||
        !paged_map(&maps.v, cache->d_v, 2, a.d, slots, box))
      return cudaErrorInvalidValue;
    if (a.kt) {
      const uint64_t cols = (uint64_t)cache->Hkv * a.d;
      if (!paged_map(&maps.kt, a.kt, 2, cols, a.total_rows, a.Nmax + 1) ||
          !paged_map(&maps.vt, a.vt, 2, cols, a.total_rows, a.Nmax + 1))
        return cudaErrorInvalidValue;
    }
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
