// Attention over a paged KV cache: a chunk of new tokens (causal, optionally a
// sliding window with a few first tokens kept), or a draft tree's rows.
//
// This file holds the C entry points and the plain kernel, one warp per (row,
// head): 32 keys at a time a lane takes one key's score, the warp keeps the
// running maximum and sum, and then lanes own head-dim columns of the output.
#include "paged_attn.cuh"

namespace dt {
namespace {

constexpr int kPlainWarps = 4;
constexpr int kMaxWindow = 1 << 30;  // no request is longer; keeps position - window in 32 bits

template <int CT>
__device__ __forceinline__ float dot_row(const void* base, int64_t at, int d, const float* q) {
  const typename Code<CT>::T* p = (const typename Code<CT>::T*)base + at;
  float s = 0.f;
  for (int e = 0; e < d; ++e) s = fmaf(Code<CT>::get(p[e]), q[e], s);
  return s;
}

// grid (total rows, ceil(Hq / 4))
template <int CT, int DT>
__global__ void __launch_bounds__(32 * kPlainWarps) paged_plain_kernel(PagedArgs a) {
  __shared__ float sq[kPlainWarps][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.x, h = blockIdx.y * kPlainWarps + warp;
  int b, i;
  if (a.row_start) {
    b = row_request(a.row_start, a.batch, r);
    if (b < 0) return;
    i = r - a.row_start[b];
  } else {
    b = r / (a.Nmax + 1);
    i = r % (a.Nmax + 1);
  }
  const PagedRequest rq = paged_request(a, b);
  if (i >= rq.n || h >= a.Hq) return;
  const int kvh = h / a.G;
  const typename Code<DT>::T* q = (const typename Code<DT>::T*)a.q + r * a.ld_q + (int64_t)h * a.d;
  for (int e = lane; e < a.d; e += 32) sq[warp][e] = Code<DT>::get(q[e]);
  __syncwarp();

  const int per = a.d / 32;  // output columns of a lane: lane * per ...
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  // 32 keys: this lane's score s (ok: it is visible), then every lane's value row
  auto step = [&](bool ok, float s, auto value) {
    const float top = fmaxf(m, warp_max(ok ? s : -INFINITY));
    const float keep = m == top ? 1.f : expf(m - top);
    // all scores so far -infinity: weights of 0
    const float p = !ok || s == -INFINITY ? 0.f : expf(s - top);
    l = l * keep + warp_sum(p);
    m = top;
    for (int x = 0; x < per; ++x) o[x] *= keep;
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
      float s = 0.f;
      if (ok) {
        slot = a.c.slot(b, j, a.status);
        if (slot >= 0) {
          slot += (int64_t)kvh << a.c.page_shift;
          s = dot_row<CT>(a.c.k, slot * a.d, a.d, sq[warp]) * (a.c.ks ? a.c.ks[slot] : 1.f);
        }
        s *= a.scale;
      }
      step(ok, s, [&](int k, float p) {
        const int64_t at = __shfl_sync(0xffffffffu, slot, k);
        if (at < 0) return;
        const typename Code<CT>::T* v = (const typename Code<CT>::T*)a.c.v + at * a.d + lane * per;
        if (a.c.vs) p *= a.c.vs[at];
        for (int x = 0; x < per; ++x) o[x] = fmaf(p, Code<CT>::get(v[x]), o[x]);
      });
    }
  }
  if (a.kt) {
    const uint64_t anc = i ? a.anc[(int64_t)b * a.Nmax + i - 1] : 0ull;
    for (int j0 = 0; j0 < rq.n; j0 += 32) {
      const int j = j0 + lane;
      const bool ok = j < rq.n && tree_sees(anc, i, j);
      const int64_t row0 = ((int64_t)rq.r0 * a.c.Hkv + kvh) * a.d;
      const int64_t ld = (int64_t)a.c.Hkv * a.d;
      const float s = ok ? dot_row<DT>(a.kt, row0 + j * ld, a.d, sq[warp]) * a.scale : 0.f;
      step(ok, s, [&](int k, float p) {
        const typename Code<DT>::T* v =
            (const typename Code<DT>::T*)a.vt + row0 + (j0 + k) * ld + lane * per;
        for (int x = 0; x < per; ++x) o[x] = fmaf(p, Code<DT>::get(v[x]), o[x]);
      });
    }
  }
  const bool any = a.kt || vis.sink > 0 || vis.last > vis.first;
  const float inv = any ? 1.f / l : 0.f;
  const int64_t at = ((int64_t)r * a.Hq + h) * a.d + lane * per;
  for (int x = 0; x < per; ++x) {
    const float y = any ? o[x] * inv : 0.f;
    if constexpr (DT == DT_F32)
      ((float*)a.out)[at + x] = y;
    else
      ((__nv_bfloat16*)a.out)[at + x] = __float2bfloat16_rn(y);
  }
}

template <int DT>
void launch_plain(const PagedArgs& a, int ct, dim3 grid, cudaStream_t s) {
  switch (ct) {
    case DT_F32: paged_plain_kernel<DT_F32, DT><<<grid, 32 * kPlainWarps, 0, s>>>(a); break;
    case DT_BF16: paged_plain_kernel<DT_BF16, DT><<<grid, 32 * kPlainWarps, 0, s>>>(a); break;
    case DT_E4M3: paged_plain_kernel<DT_E4M3, DT><<<grid, 32 * kPlainWarps, 0, s>>>(a); break;
    default: paged_plain_kernel<DT_I8, DT><<<grid, 32 * kPlainWarps, 0, s>>>(a);
  }
}

dt_status run_paged(const PagedArgs& a, int ct, int dt, cudaStream_t s) {
  if (a.total_rows == 0) return DT_OK;
  ProfileScope ps(DT_K_ATTN, s);
  const dim3 grid(a.total_rows, (a.Hq + kPlainWarps - 1) / kPlainWarps);
  if (dt == DT_F32)
    launch_plain<DT_F32>(a, ct, grid, s);
  else
    launch_plain<DT_BF16>(a, ct, grid, s);
  return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ECUDA;
}

size_t paged_workspace(int64_t total_rows, int Hq, int Hkv, int d) {
  return kWsHeader;
}

// checks that both entry points share, after the cache's own
dt_status check_paged(const dt_kv_cache* c, const void* q, const void* out, int Hq, float scale,
                      int window, int n_sink, dt_dtype dt) {
  if (!q || !out || (dt != DT_F32 && dt != DT_BF16)) return DT_EINVAL;
  if (Hq < 1 || Hq % c->Hkv || !(scale > 0.f) || window < 0 || n_sink < 0) return DT_EINVAL;
  if (((uintptr_t)q | (uintptr_t)out) & 15) return DT_EINVAL;
  if (dt == DT_BF16 && c->dt == DT_F32) return DT_EUNSUPPORTED;
  if (Hq > 65535) return DT_EUNSUPPORTED;
  return DT_OK;
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" {

size_t dt_paged_attn_workspace_bytes(int batch, int total_rows, int Hq, int Hkv, int d) {
  if (batch < 1 || total_rows < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || d < 1) return 0;
  return paged_workspace(total_rows, Hq, Hkv, d);
}

dt_status dt_paged_attn(const void* d_q, int64_t ld_q, const int32_t* d_row_start,
                        const dt_kv_cache* cache, const int32_t* d_page_table, int max_pages,
                        const int32_t* d_kv_len, int batch, int total_rows, int max_rows, int Hq,
                        float scale, int window, int n_sink, dt_dtype dt, void* d_out, void* ws,
                        size_t ws_bytes, dt_stream stream) {
  dt_status ok = check_cache(cache, d_page_table, max_pages, batch);
  if (ok != DT_OK) return ok;
  ok = check_paged(cache, d_q, d_out, Hq, scale, window, n_sink, dt);
  if (ok != DT_OK) return ok;
  if (!d_row_start || !d_kv_len || total_rows < 0 || max_rows < 1) return DT_EINVAL;
  if (ld_q < (int64_t)Hq * cache->d || (ld_q * (dt == DT_F32 ? 4 : 2)) % 16) return DT_EINVAL;
  if ((int64_t)total_rows * Hq >= (int64_t)1 << 30) return DT_EUNSUPPORTED;
  if (!ws || ws_bytes < paged_workspace(total_rows, Hq, cache->Hkv, cache->d))
    return DT_EWORKSPACE;
  PagedArgs a = {};
  a.q = d_q;
  a.ld_q = ld_q;
  a.row_start = d_row_start;
  a.kv_len = d_kv_len;
  a.c = kv_view(cache, d_page_table, max_pages);
  a.batch = batch;
  a.total_rows = total_rows;
  a.max_rows = max_rows;
  a.Hq = Hq;
  a.G = Hq / cache->Hkv;
  a.d = cache->d;
  a.scale = scale;
  a.window = min(window, kMaxWindow);
  a.n_sink = n_sink;
  a.out = d_out;
  a.status = (int32_t*)ws;
  return run_paged(a, cache->dt, dt, (cudaStream_t)stream);
}

size_t dt_tree_verify_attn_paged_workspace_bytes(int batch, int Nmax, int Hq, int Hkv, int d) {
  if (batch < 1 || Nmax < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || d < 1) return 0;
  return paged_workspace((int64_t)batch * (Nmax + 1), Hq, Hkv, d);
}

dt_status dt_tree_verify_attn_paged(const void* d_q, const dt_kv_cache* cache,
                                    const int32_t* d_page_table, int max_pages,
                                    const int32_t* d_prefix_len, const void* d_k_tree,
                                    const void* d_v_tree, const uint64_t* d_anc,
                                    const int32_t* d_depths, const int32_t* d_n_nodes, int batch,
                                    int Nmax, int Hq, float scale, int window, int n_sink,
                                    dt_dtype dt, void* d_out, void* ws, size_t ws_bytes,
                                    dt_stream stream) {
  dt_status ok = check_cache(cache, d_page_table, max_pages, batch);
  if (ok != DT_OK) return ok;
  ok = check_paged(cache, d_q, d_out, Hq, scale, window, n_sink, dt);
  if (ok != DT_OK) return ok;
  if (!d_prefix_len || !d_k_tree || !d_v_tree || !d_anc || !d_n_nodes || Nmax < 1)
    return DT_EINVAL;
  if (((uintptr_t)d_k_tree | (uintptr_t)d_v_tree) & 15) return DT_EINVAL;
  if (window && !d_depths) return DT_EINVAL;
  if (Nmax > 64 || (window && window <= Nmax)) return DT_EUNSUPPORTED;
  const int rows = batch * (Nmax + 1);
  if ((int64_t)rows * Hq >= (int64_t)1 << 30) return DT_EUNSUPPORTED;
  if (!ws || ws_bytes < paged_workspace(rows, Hq, cache->Hkv, cache->d)) return DT_EWORKSPACE;
  PagedArgs a = {};
  a.q = d_q;
  a.ld_q = (int64_t)Hq * cache->d;
  a.kv_len = d_prefix_len;
  a.c = kv_view(cache, d_page_table, max_pages);
  a.batch = batch;
  a.total_rows = rows;
  a.max_rows = Nmax + 1;
  a.Hq = Hq;
  a.G = Hq / cache->Hkv;
  a.d = cache->d;
  a.scale = scale;
  a.window = min(window, kMaxWindow);
  a.n_sink = n_sink;
  a.kt = d_k_tree;
  a.vt = d_v_tree;
  a.anc = d_anc;
  a.depths = d_depths;
  a.n_nodes = d_n_nodes;
  a.Nmax = Nmax;
  a.out = d_out;
  a.status = (int32_t*)ws;
  return run_paged(a, cache->dt, dt, (cudaStream_t)stream);
}

}  // extern "C"
