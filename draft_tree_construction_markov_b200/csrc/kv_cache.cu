// Rows quantised as they enter a paged KV cache, and read back.
//
// Write: a row of one head is d values x; with a = max(max |x|, 2^-100) and X
// the largest code (448 or 127), scale = a / X and code = round(x * (X / a)).
// The product with the one quotient X / a (instead of a quotient per value) is
// part of the definition: it costs one multiplication per value and its fp32
// rounding moves a code only where x * X / a is within 2^-24 of a border.
// 2^-100 keeps X / a finite.  Read: code * scale, rounded once.
//
// Both only move data, and what bounds them is memory bandwidth: a warp takes
// a token, looks its request and slot up once, and asks for up to kUnroll pieces
// of 8 values a lane of K and of V before it works on the first.  d / 8
// neighbouring lanes own a head row and find its largest magnitude with shuffles.
// Measured (B200): 25 thousand rows of 8 heads of 128 from a fused bf16 projection
// into e4m3, 154 MB in 41 us (3.7 TB/s; a thread a piece, each looking its row up,
// took 55 us), issue slots 74 % and ALU 56 % busy, DRAM 37 %; into bf16, 203 MB in
// 40 us; fp32 rows into e4m3, 255 MB in 69 us.  112 thousand int8 rows read back as
// bf16, 696 MB in 113 us (6.2 TB/s, 0.94 of the measured copy rate; 160 us before).
#include "kv_cache.cuh"

namespace dt {
namespace {

constexpr int kKvThreads = 256;
constexpr int kPer = 8;     // values of a piece
constexpr int kUnroll = 4;  // pieces of K, and of V, that a lane has on their way

// A piece as it lies in memory, 8 values of type DT; VEC: 16-byte aligned.
// (Pieces wait in this form: turned into fp32 at once they would take twice the
// registers, and half the warps would fit.)
template <int DT>
struct Piece {
  static constexpr int W = DT == DT_F32 ? 8 : DT == DT_BF16 ? 4 : 2;
  uint32_t w[W];
};
template <int DT, bool VEC>
__device__ __forceinline__ Piece<DT> load8(const void* base, int64_t off) {
  Piece<DT> r;
  if constexpr (DT == DT_F32) {
    const uint32_t* p = (const uint32_t*)base + off;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      if constexpr (VEC) {
        const uint4 x = *(const uint4*)(p + i);
        r.w[i] = x.x, r.w[i + 1] = x.y, r.w[i + 2] = x.z, r.w[i + 3] = x.w;
      } else {
#pragma unroll
        for (int e = i; e < i + 4; ++e) r.w[e] = p[e];
      }
    }
  } else if constexpr (DT == DT_BF16) {
    const uint16_t* p = (const uint16_t*)base + off;
    if constexpr (VEC) {
      const uint4 x = *(const uint4*)p;
      r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    }
  } else {
    const uint2 x = *(const uint2*)((const uint8_t*)base + off);
    r.w[0] = x.x, r.w[1] = x.y;
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void values8(const Piece<DT>& r, float scale, float (&x)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (DT == DT_F32)
      x[i] = __uint_as_float(r.w[i]);
    else if constexpr (DT == DT_BF16)
      x[i] = __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
    else
      x[i] = Code<DT>::get((typename Code<DT>::T)((r.w[i / 4] >> (8 * (i & 3))) & 0xff)) * scale;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t off, const float (&x)[kPer]) {
  if constexpr (DT == DT_F32) {
    float4* p = (float4*)((float*)base + off);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *(uint4*)((uint16_t*)base + off) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                  pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

// One head row's piece into the cache; `lanes` = d / 8 lanes share the row.
// Every lane of the warp takes part in the shuffles; slot < 0 stores nothing.
template <int CT>
__device__ __forceinline__ void put8(void* cache, float* scales, int64_t slot, int d, int at,
                                     const float (&x)[kPer]) {
  if constexpr (CT == DT_F32 || CT == DT_BF16) {
    if (slot >= 0) store8<CT>(cache, slot * d + at, x);
  } else {
    constexpr float top = CT == DT_E4M3 ? 448.f : 127.f;
    // magnitudes compare as integers, with infinity and NaN above all numbers
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    for (int o = d / kPer / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool finite = m < 0x7f800000u;
    const float a = fmaxf(__uint_as_float(m), 7.888609052210118e-31f);  // 2^-100
    const float inv = __fdiv_rn(top, a);
    uint32_t w[2] = {0, 0};
    if (finite) {
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        uint32_t two;
        if constexpr (CT == DT_E4M3) {
          uint16_t r;
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
              : "=h"(r)
              : "f"(x[i + 1] * inv), "f"(x[i] * inv));
          two = r;
        } else {
          const int lo = min(max(__float2int_rn(x[i] * inv), -127), 127);
          const int hi = min(max(__float2int_rn(x[i + 1] * inv), -127), 127);
          two = (uint32_t)(lo & 0xff) | ((uint32_t)(hi & 0xff) << 8);
        }
        w[i >> 2] |= two << (8 * (i & 2));
      }
    }
    if (slot >= 0) {
      *(uint2*)((uint8_t*)cache + slot * d + at) = make_uint2(w[0], w[1]);
      if (at == 0) scales[slot] = finite ? __fdiv_rn(a, top) : __uint_as_float(0x7fc00000u);
    }
  }
}

struct WriteArgs {
  const void* k;
  const void* v;
  int64_t ld_k, ld_v;
  const int32_t* row_start;  // write: [batch + 1]
  const int32_t* acc;        // commit: [batch][Bk]
  const int32_t* n_acc;      // commit: [batch]
  const int32_t* pos;        // [batch]
  int batch, total_rows, Bk, Nmax, d;
  KvView c;
  int32_t* status;
};

// a warp per row (commit: batch * (Bk + 1) rows)
template <int ST, int CT, bool VEC, bool COMMIT>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(WriteArgs a) {
  const int lane = threadIdx.x & 31, d = a.d, shift = d == 128 ? 7 : 6;
  const int r = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  int b = -1;
  int64_t src = 0, p = 0;
  if (COMMIT) {
    b = r / (a.Bk + 1);
    const int i = r % (a.Bk + 1);
    if (b >= a.batch) return;
    const int n = a.n_acc[b];
    if (n < 0 || n > a.Bk) set_status(a.status, DT_EDEVICE);
    if (n < 0 || i > min(n, a.Bk)) return;
    const int node = i ? a.acc[(int64_t)b * a.Bk + i - 1] : -1;
    if (node < -1 || node >= a.Nmax || (i && node < 0)) {
      set_status(a.status, DT_EDEVICE);
      return;
    }
    src = (int64_t)b * (a.Nmax + 1) + node + 1;
    p = (int64_t)a.pos[b] + i;
  } else {
    if (r >= a.total_rows) return;
    b = row_request_warp(a.row_start, a.pos, a.batch, r, p);
    if (b < 0) return;
    src = r;
  }
  if (p < 0 || p >= 1ll << 31) {
    set_status(a.status, DT_EDEVICE);
    return;
  }
  const int64_t slot = a.c.slot(b, (int)p, a.status);
  if (slot < 0) return;
  const int all = a.c.Hkv * d / kPer;
  for (int x0 = lane; x0 - lane < all; x0 += 32 * kUnroll) {  // (whole warps: put8 shuffles)
    Piece<ST> k[kUnroll] = {}, v[kUnroll] = {};
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = x0 + 32 * u;
      if (x < all) {
        k[u] = load8<ST, VEC>(a.k, src * a.ld_k + x * kPer);
        v[u] = load8<ST, VEC>(a.v, src * a.ld_v + x * kPer);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = x0 + 32 * u, h = x * kPer >> shift, at = (x * kPer) & (d - 1);
      if (x - lane >= all) break;
      const int64_t to = x < all ? slot + ((int64_t)h << a.c.page_shift) : -1;
      float y[kPer];
      values8<ST>(k[u], 1.f, y);
      put8<CT>(a.c.k, a.c.ks, to, d, at, y);
      values8<ST>(v[u], 1.f, y);
      put8<CT>(a.c.v, a.c.vs, to, d, at, y);
    }
  }
}

struct ReadArgs {
  KvView c;
  const int32_t* row_start;
  const int32_t* pos;
  int batch, total_rows, d;
  void* k_out;
  void* v_out;
  int32_t* status;
};

template <int CT, int OT>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(ReadArgs a) {
  const int lane = threadIdx.x & 31, d = a.d, shift = d == 128 ? 7 : 6;
  const int r = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  if (r >= a.total_rows) return;
  int64_t p = 0, slot = -1;
  const int b = row_request_warp(a.row_start, a.pos, a.batch, r, p);
  if (b < 0) return;
  if (p < 0 || p >= 1ll << 31)
    set_status(a.status, DT_EDEVICE);
  else
    slot = a.c.slot(b, (int)p, a.status);
  const int all = a.c.Hkv * d / kPer;
  const int64_t out = (int64_t)r * a.c.Hkv * d;
  constexpr bool kScaled = CT == DT_E4M3 || CT == DT_I8;
  for (int x0 = lane; x0 < all; x0 += 32 * kUnroll) {
    Piece<CT> k[kUnroll] = {}, v[kUnroll] = {};
    float ks[kUnroll], vs[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = x0 + 32 * u, h = x * kPer >> shift, at = (x * kPer) & (d - 1);
      ks[u] = vs[u] = 0.f;
      if (x < all && slot >= 0) {
        const int64_t from = slot + ((int64_t)h << a.c.page_shift);
        k[u] = load8<CT, true>(a.c.k, from * d + at);
        v[u] = load8<CT, true>(a.c.v, from * d + at);
        if constexpr (kScaled) {
          ks[u] = a.c.ks[from];
          vs[u] = a.c.vs[from];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int x = x0 + 32 * u;
      if (x >= all) break;
      float y[kPer];
      values8<CT>(k[u], ks[u], y);
      store8<OT>(a.k_out, out + x * kPer, y);
      values8<CT>(v[u], vs[u], y);
      store8<OT>(a.v_out, out + x * kPer, y);
    }
  }
}

template <int ST, bool VEC, bool COMMIT>
void launch_write(const WriteArgs& a, int ct, int64_t rows, cudaStream_t s) {
  const unsigned grid = (unsigned)((rows + kKvThreads / 32 - 1) / (kKvThreads / 32));
  switch (ct) {
    case DT_F32: kv_write_kernel<ST, DT_F32, VEC, COMMIT><<<grid, kKvThreads, 0, s>>>(a); break;
    case DT_BF16: kv_write_kernel<ST, DT_BF16, VEC, COMMIT><<<grid, kKvThreads, 0, s>>>(a); break;
    case DT_E4M3: kv_write_kernel<ST, DT_E4M3, VEC, COMMIT><<<grid, kKvThreads, 0, s>>>(a); break;
    default: kv_write_kernel<ST, DT_I8, VEC, COMMIT><<<grid, kKvThreads, 0, s>>>(a);
  }
}

template <bool COMMIT>
dt_status run_write(const WriteArgs& a, int st, int ct, int64_t rows, cudaStream_t s) {
  if (rows == 0) return DT_OK;
  // 16-byte loads where every row of every head starts on 16 bytes
  const int es = kv_code_bytes(st);
  const bool vec = (((uintptr_t)a.k | (uintptr_t)a.v) & 15) == 0 && (a.ld_k * es) % 16 == 0 &&
                   (a.ld_v * es) % 16 == 0;
  ProfileScope ps(DT_K_KV, s);
  if (st == DT_F32)
    vec ? launch_write<DT_F32, true, COMMIT>(a, ct, rows, s)
        : launch_write<DT_F32, false, COMMIT>(a, ct, rows, s);
  else
    vec ? launch_write<DT_BF16, true, COMMIT>(a, ct, rows, s)
        : launch_write<DT_BF16, false, COMMIT>(a, ct, rows, s);
  return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ECUDA;
}

template <int OT>
void launch_read(const ReadArgs& a, int ct, unsigned grid, cudaStream_t s) {
  switch (ct) {
    case DT_F32: kv_read_kernel<DT_F32, OT><<<grid, kKvThreads, 0, s>>>(a); break;
    case DT_BF16: kv_read_kernel<DT_BF16, OT><<<grid, kKvThreads, 0, s>>>(a); break;
    case DT_E4M3: kv_read_kernel<DT_E4M3, OT><<<grid, kKvThreads, 0, s>>>(a); break;
    default: kv_read_kernel<DT_I8, OT><<<grid, kKvThreads, 0, s>>>(a);
  }
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" {

size_t dt_kv_workspace_bytes(void) { return kWsHeader; }

dt_status dt_kv_write(const void* d_k, const void* d_v, int64_t ld_k, int64_t ld_v, dt_dtype dt,
                      const int32_t* d_row_start, const int32_t* d_pos,
                      const int32_t* d_page_table, int max_pages, int batch, int total_rows,
                      const dt_kv_cache* cache, void* ws, size_t ws_bytes, dt_stream stream) {
  dt_status ok = check_cache(cache, d_page_table, max_pages, batch);
  if (ok != DT_OK) return ok;
  if (!d_k || !d_v || !d_row_start || !d_pos || total_rows < 0) return DT_EINVAL;
  if (dt != DT_F32 && dt != DT_BF16) return DT_EINVAL;
  if (((uintptr_t)d_k | (uintptr_t)d_v) & (dt == DT_F32 ? 3 : 1)) return DT_EINVAL;
  const int64_t row = (int64_t)cache->Hkv * cache->d;
  if (ld_k < row || ld_v < row) return DT_EINVAL;
  if ((ok = check_ws(ws, ws_bytes, kWsHeader)) != DT_OK) return ok;
  WriteArgs a = {};
  a.k = d_k;
  a.v = d_v;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.row_start = d_row_start;
  a.pos = d_pos;
  a.batch = batch;
  a.total_rows = total_rows;
  a.d = cache->d;
  a.c = kv_view(cache, d_page_table, max_pages);
  a.status = (int32_t*)ws;
  return run_write<false>(a, dt, cache->dt, total_rows, (cudaStream_t)stream);
}

dt_status dt_kv_commit(const void* d_k_tree, const void* d_v_tree, dt_dtype dt,
                       const int32_t* d_acc_nodes, const int32_t* d_n_acc, int Bk, int Nmax,
                       const int32_t* d_pos, const int32_t* d_page_table, int max_pages,
                       int batch, const dt_kv_cache* cache, void* ws, size_t ws_bytes,
                       dt_stream stream) {
  dt_status ok = check_cache(cache, d_page_table, max_pages, batch);
  if (ok != DT_OK) return ok;
  if (!d_k_tree || !d_v_tree || !d_acc_nodes || !d_n_acc || !d_pos) return DT_EINVAL;
  if (dt != DT_F32 && dt != DT_BF16) return DT_EINVAL;
  if (((uintptr_t)d_k_tree | (uintptr_t)d_v_tree) & (dt == DT_F32 ? 3 : 1)) return DT_EINVAL;
  if (Bk < 1 || Nmax < 1) return DT_EINVAL;
  if (Bk > 64 || Nmax > 64) return DT_EUNSUPPORTED;
  if ((ok = check_ws(ws, ws_bytes, kWsHeader)) != DT_OK) return ok;
  WriteArgs a = {};
  a.k = d_k_tree;
  a.v = d_v_tree;
  a.ld_k = a.ld_v = (int64_t)cache->Hkv * cache->d;
  a.acc = d_acc_nodes;
  a.n_acc = d_n_acc;
  a.pos = d_pos;
  a.batch = batch;
  a.Bk = Bk;
  a.Nmax = Nmax;
  a.d = cache->d;
  a.c = kv_view(cache, d_page_table, max_pages);
  a.status = (int32_t*)ws;
  return run_write<true>(a, dt, cache->dt, (int64_t)batch * (Bk + 1), (cudaStream_t)stream);
}

dt_status dt_kv_read(const dt_kv_cache* cache, const int32_t* d_page_table, int max_pages,
                     const int32_t* d_row_start, const int32_t* d_pos, int batch, int total_rows,
                     dt_dtype dt, void* d_k_out, void* d_v_out, void* ws, size_t ws_bytes,
                     dt_stream stream) {
  dt_status ok = check_cache(cache, d_page_table, max_pages, batch);
  if (ok != DT_OK) return ok;
  if (!d_row_start || !d_pos || !d_k_out || !d_v_out || total_rows < 0) return DT_EINVAL;
  if (dt != DT_F32 && dt != DT_BF16) return DT_EINVAL;
  if (((uintptr_t)d_k_out | (uintptr_t)d_v_out) & 15) return DT_EINVAL;
  if ((ok = check_ws(ws, ws_bytes, kWsHeader)) != DT_OK) return ok;
  const int64_t blocks = ((int64_t)total_rows + kKvThreads / 32 - 1) / (kKvThreads / 32);
  if (total_rows == 0) return DT_OK;
  ReadArgs a;
  a.c = kv_view(cache, d_page_table, max_pages);
  a.row_start = d_row_start;
  a.pos = d_pos;
  a.batch = batch;
  a.total_rows = total_rows;
  a.d = cache->d;
  a.k_out = d_k_out;
  a.v_out = d_v_out;
  a.status = (int32_t*)ws;
  cudaStream_t s = (cudaStream_t)stream;
  ProfileScope ps(DT_K_KV, s);
  if (dt == DT_F32)
    launch_read<DT_F32>(a, cache->dt, (unsigned)blocks, s);
  else
    launch_read<DT_BF16>(a, cache->dt, (unsigned)blocks, s);
  return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ECUDA;
}

}  // extern "C"
