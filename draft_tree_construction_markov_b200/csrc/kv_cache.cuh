// The paged KV cache as the kernels see it: addresses of a position's rows,
// checks of the caller's description, conversion of stored codes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <limits.h>

#include "common.cuh"

namespace dt {

constexpr int kMaxKvBatch = 1024;

// Device-side view of a dt_kv_cache and a batch's page table.
struct KvView {
  void* k;
  void* v;
  float* ks;  // null where the type has no scales
  float* vs;
  const int32_t* table;
  int max_pages, n_pages, page_shift, Hkv;

  // Slot of (head 0, position p) in units of head rows, or -1; head h is
  // page_size rows further on.  p >= 0.
  __device__ __forceinline__ int64_t slot(int b, int p, int32_t* status) const {
    const int pi = p >> page_shift;
    int page = -1;
    if (pi < max_pages) page = table[(int64_t)b * max_pages + pi];
    if (page < 0 || page >= n_pages) {
      set_status(status, DT_EDEVICE);
      return -1;
    }
    return (((int64_t)page * Hkv) << page_shift) + (p & ((1 << page_shift) - 1));
  }
};

inline int kv_code_bytes(int dt) { return dt == DT_F32 ? 4 : dt == DT_BF16 ? 2 : 1; }

// Host-side checks shared by the calls on a cache (null tables are the
// caller's to check).
inline dt_status check_cache(const dt_kv_cache* c, const int32_t* table, int max_pages, int batch) {
  if (!c || !c->d_k || !c->d_v || !table) return DT_EINVAL;
  if (c->dt != DT_F32 && c->dt != DT_BF16 && c->dt != DT_E4M3 && c->dt != DT_I8) return DT_EINVAL;
  const bool scaled = c->dt == DT_E4M3 || c->dt == DT_I8;
  if (scaled && (!c->d_k_scale || !c->d_v_scale)) return DT_EINVAL;
  if (c->n_pages < 1 || c->page_size < 1 || c->Hkv < 1 || max_pages < 1 || batch < 1)
    return DT_EINVAL;
  if (((uintptr_t)c->d_k | (uintptr_t)c->d_v) & 15) return DT_EINVAL;
  if (((uintptr_t)c->d_k_scale | (uintptr_t)c->d_v_scale) & 15) return DT_EINVAL;
  if (c->page_size & (c->page_size - 1)) return DT_EUNSUPPORTED;
  if (c->page_size < 8 || c->page_size > 256) return DT_EUNSUPPORTED;
  if ((c->d != 64 && c->d != 128) || c->Hkv > 1024 || batch > kMaxKvBatch) return DT_EUNSUPPORTED;
  if ((int64_t)c->n_pages * c->Hkv * c->page_size >= (int64_t)1 << 31) return DT_EUNSUPPORTED;
  if ((int64_t)max_pages * c->page_size >= (int64_t)1 << 30) return DT_EUNSUPPORTED;
  return DT_OK;
}

inline KvView kv_view(const dt_kv_cache* c, const int32_t* table, int max_pages) {
  KvView v;
  v.k = c->d_k;
  v.v = c->d_v;
  const bool scaled = c->dt == DT_E4M3 || c->dt == DT_I8;
  v.ks = scaled ? c->d_k_scale : nullptr;
  v.vs = scaled ? c->d_v_scale : nullptr;
  v.table = table;
  v.max_pages = max_pages;
  v.n_pages = c->n_pages;
  v.page_shift = __builtin_ctz((unsigned)c->page_size);
  v.Hkv = c->Hkv;
  return v;
}

// Request of packed row r: the last b with start[b] <= r, or -1 when the row
// is in no request's range.  start holds batch + 1 entries.
__device__ __forceinline__ int row_request(const int32_t* start, int batch, int r) {
  if (r < start[0] || r >= start[batch]) return -1;
  int lo = 0, hi = batch;  // start[lo] <= r < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The same by a whole warp, and the row's position: pos[b] + r - start[b].  Up
// to 31 requests take one look, in which the positions come along.
__device__ __forceinline__ int row_request_warp(const int32_t* start, const int32_t* pos, int batch,
                                                int r, int64_t& p) {
  const int lane = threadIdx.x & 31;
  if (batch < 32) {
    const int s = lane <= batch ? start[lane] : INT_MAX, q = lane < batch ? pos[lane] : 0;
    // the last start that is not behind r
    const int b = __popc(__ballot_sync(0xffffffffu, s <= r)) - 1;
    if (b < 0 || b >= batch) return -1;
    p = (int64_t)__shfl_sync(0xffffffffu, q, b) + (r - __shfl_sync(0xffffffffu, s, b));
    return b;
  }
  if (r < start[0] || r >= start[batch]) return -1;
  int lo = 0, hi = batch;  // start[lo] <= r < start[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (1 + lane) * step;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && start[min(at, hi)] <= r));
    lo += n * step;
    hi = min(lo + step, hi);
  }
  p = (int64_t)pos[lo] + (r - start[lo]);
  return lo;
}

// Stored code -> fp32.
template <int CT>
struct Code;
template <>
struct Code<DT_F32> {
  using T = float;
  static __device__ __forceinline__ float get(T x) { return x; }
};
template <>
struct Code<DT_BF16> {
  using T = uint16_t;
  static __device__ __forceinline__ float get(T x) { return bf16_to_f32(x); }
};
template <>
struct Code<DT_E4M3> {
  using T = uint8_t;
  static __device__ __forceinline__ float get(T x) {
    __nv_fp8_e4m3 f;
    f.__x = x;
    return (float)f;
  }
};
template <>
struct Code<DT_I8> {
  using T = int8_t;
  static __device__ __forceinline__ float get(T x) { return (float)x; }
};

}  // namespace dt
