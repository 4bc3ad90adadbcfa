// Attention over a paged KV cache: a chunk of new tokens (causal, optionally a
// sliding window with a few first tokens kept), or a draft tree's rows.
//
// This file holds the C entry points and the kernel of fp32 queries, one warp
// per (row, head) and key by key, for checks and small sizes: it is bound by
// latency, about 1 us a position (one token over 4096 positions, e4m3: 4.0 ms
// against 42 us; 512 rows over 4096, bf16: 36 ms against 77 us).  bf16 queries take
// the tiled kernels.
#include <algorithm>

#include "paged_attn.cuh"

namespace dt {
namespace {

constexpr int kPlainWarps = 4;
constexpr int kMaxWindow = 1 << 30;  // no request is longer; keeps position - window in 32 bits

// grid (total rows, ceil(Hq / 4))
template <int CT, int DT>
__global__ void __launch_bounds__(32 * kPlainWarps) paged_plain_kernel(PagedArgs a) {
  const int r = blockIdx.x, h = blockIdx.y * kPlainWarps + (threadIdx.x >> 5);
  int b, i;
  if (a.row_start) {
    b = row_request(a.row_start, a.batch, r);
    if (b < 0) return;
    i = r - a.row_start[b];
  } else {
    b = r / (a.Nmax + 1);
    i = r % (a.Nmax + 1);
  }
  if (i < paged_request(a, b).n && h < a.Hq) paged_row<CT, DT>(a, b, i, h);
}

// Rows that worker `me` finished and that came out infinite or NaN: again, key by
// key (see paged_row), where that can give anything else.  It can where a value that
// the row does not see may be the cause (hides_odd), and where an output is infinite:
// weights may be 2^8 over the maximum in use, and a sum may have passed fp32 for that
// alone.  (A NaN scale that all rows see would otherwise cost every later call of its
// request a repeat of all rows: 5.7 ms instead of 0.07 ms for a token over 8000
// positions.)
template <int CT>
__device__ __noinline__ void join_redo(const PagedArgs& a, Cut cut, int me, int most) {
  __shared__ int64_t sums[kMaxKvBatch + 1];
  const int64_t all = count_units(a, sums, cut);
  const int workers = (int)min((int64_t)most, all);
  if (me >= workers) return;
  const int64_t u0 = first_unit(all, me, workers);
  int64_t left = first_unit(all, me + 1, workers) - u0;
  const int lane = threadIdx.x & 31;
  Cursor c;
  for (c.seek(a, sums, u0, cut);; c.next_tile(a, cut)) {
    if (c.u == 0 && c.t.units <= left) {
      for (int r = threadIdx.x >> 5; r < c.t.live; r += kJoinWarps) {
        const int i = (c.t.m0 + r) / a.G, h = c.kvh * a.G + (c.t.m0 + r) % a.G;
        const uint16_t* out = (const uint16_t*)a.out + (((int64_t)c.rq.r0 + i) * a.Hq + h) * a.d;
        bool odd = false, infinite = false;
        for (int e = lane; e < a.d; e += 32) {
          odd |= (out[e] & 0x7f80u) == 0x7f80u;
          infinite |= (out[e] & 0x7fffu) == 0x7f80u;
        }
        if (!__any_sync(0xffffffffu, odd)) continue;
        if (__any_sync(0xffffffffu, infinite) ||
            hides_odd<CT>(a, c.rq, c.t, c.b, c.kvh, c.t.m0 + r))
          paged_row<CT, DT_BF16>(a, c.b, i, h);
      }
    }
    left -= c.t.units - c.u;
    if (left <= 0) break;
  }
  __syncthreads();
}

// Joins the shares of row tiles.  The tasks of all workers are a list that the
// blocks share out (most workers have few or none, one may have hundreds); every
// block adds the list up for itself.  A warp has its row's statistics and the
// first parts' sums on the way together, its lanes four columns each.
template <int CT>
__global__ void __launch_bounds__(32 * kJoinWarps)
    paged_join_kernel(const __grid_constant__ PagedArgs a, Cut cut, int workers) {
  __shared__ float4 sums[kJoinWarps][32];
  static_assert(kDecodeWorkers >= 2 * kPagedSms);
  __shared__ int before[kDecodeWorkers + 1];  // tasks before worker w
  __shared__ int carry[kJoinWarps];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool redo = false;
  constexpr int kPer = (kDecodeWorkers + 32 * kJoinWarps - 1) / (32 * kJoinWarps);
  {
    int t[kPer], sum = 0;
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int w = threadIdx.x * kPer + y;
      t[y] = w < workers ? a.tasks[w] : 0;
      redo |= w < workers && a.redo[w];
    }
#pragma unroll
    for (int y = 0; y < kPer; ++y) sum += t[y];
    int x = sum;
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += v;
    }
    if (lane == 31) carry[warp] = x;
    redo = __syncthreads_or(redo);
    int at = x - sum;
    for (int y = 0; y < warp; ++y) at += carry[y];
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int w = threadIdx.x * kPer + y;
      if (w <= workers) before[w] = at;
      at += t[y];
    }
    __syncthreads();
  }
  if (redo)
    for (int w = blockIdx.x; w < workers; w += gridDim.x)
      if (a.redo[w]) join_redo<CT>(a, cut, w, workers);
  const bool col = lane * 4 < a.d;
  for (int task = blockIdx.x; task < before[workers]; task += gridDim.x) {
    int lo = 0, hi = workers;  // before[lo] <= task < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= task)
        lo = mid;
      else
        hi = mid;
    }
    const PagedSplit sp = a.split[lo];
    const int share = join_share(sp.parts), mine = warp % share;
    const int r = (task - before[lo]) * (kJoinWarps / share) + warp / share;
    const bool there = r < sp.live;
    // part 0: the second slot of the worker before; part k: the first slot of worker + k - 1
    auto at = [&](int k) {
      const int64_t slot = k ? 2 * ((int64_t)lo + k - 1) : 2 * (int64_t)lo - 1;
      return slot * a.part_rows + r;
    };
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (there) {
      constexpr int kAhead = 6;  // parts on their way
      float w[kAhead];
      float4 x[kAhead];
      auto ask = [&](int k0) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const int k = k0 + y * share;
          w[y] = -INFINITY;
          x[y] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < sp.parts) {
            w[y] = a.part_ml[at(k)].x;
            if (col) x[y] = *(const float4*)(a.part_o + at(k) * a.d + lane * 4);
          }
        }
      };
      ask(mine);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < sp.parts) ml = a.part_ml[at(lane)];
      m = ml.x;
      for (int k = 32 + lane; k < sp.parts; k += 32) m = fmaxf(m, a.part_ml[at(k)].x);
      m = warp_max(m);
      auto weigh = [&](float2 p) {  // (a NaN sum stays one)
        l += p.x == -INFINITY ? p.y : ex2(p.x - m) * p.y;
      };
      weigh(ml);
      for (int k = 32 + lane; k < sp.parts; k += 32) weigh(a.part_ml[at(k)]);
      l = warp_sum(l);
      for (int k0 = mine; k0 < sp.parts; k0 += kAhead * share) {
        if (k0 != mine) ask(k0);
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const float f = w[y] == -INFINITY ? 0.f : ex2(w[y] - m);
          o.x = fmaf(f, x[y].x, o.x);
          o.y = fmaf(f, x[y].y, o.y);
          o.z = fmaf(f, x[y].z, o.z);
          o.w = fmaf(f, x[y].w, o.w);
        }
      }
    }
    if (share > 1) {
      __syncthreads();
      sums[warp][lane] = o;
      __syncthreads();
      for (int y = 1; mine == 0 && y < share; ++y) {
        const float4 x = sums[warp + y][lane];
        o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
      }
    }
    if (!there || mine) continue;
    const int i = (sp.m0 + r) / a.G, h = sp.kvh * a.G + (sp.m0 + r) % a.G;
    const bool sees = !(l < 0.f);
    const float inv = row_factor(l, sees);
    if (col)
      *(uint2*)((uint16_t*)a.out + (((int64_t)sp.r0 + i) * a.Hq + h) * a.d + lane * 4) =
          sees ? make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv))
               : make_uint2(0u, 0u);
    const float odd = o.x * 0.f + o.y * 0.f + o.z * 0.f + o.w * 0.f;
    if (__any_sync(0xffffffffu, sees && odd != 0.f && l - l == 0.f)) {  // (as in join_redo)
      const PagedRequest rq = paged_request(a, sp.b);
      const float most = fmaxf(fmaxf(fabsf(o.x), fabsf(o.y)), fmaxf(fabsf(o.z), fabsf(o.w)));
      if (__any_sync(0xffffffffu, most == INFINITY) ||
          hides_odd<CT>(a, rq, row_tile(a, rq, sp.m0 / cut.per, cut), sp.b, sp.kvh, sp.m0 + r))
        paged_row<CT, DT_BF16>(a, sp.b, i, h);
    }
  }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeFn) nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// Records, fp32 sums and statistics of the row tiles that shares cut, two per
// worker; `all`: (row, head) pairs of a KV head that a row tile can have at most.
struct PartPlan {
  size_t redo, tasks, sums, stats, bytes;  // offsets behind the header, and all
};
PartPlan part_plan(int64_t workers, int64_t rows, int d) {
  PartPlan p;
  p.redo = (workers * sizeof(PagedSplit) + 15) & ~(size_t)15;
  p.tasks = p.redo + workers * 4;
  p.sums = p.redo + ((workers * 8 + 15) & ~(size_t)15);
  p.stats = p.sums + 2 * workers * rows * d * 4;
  p.bytes = kWsHeader + p.stats + 2 * workers * rows * sizeof(float2);
  return p;
}
// (two row tiles a CTA take half the workers, so no more); trees never take the kernel of few rows
size_t tree_workspace(int64_t all, int d) {
  return part_plan(2 * kPagedSms, std::min<int64_t>(all, 128), d).bytes;
}
size_t chunk_workspace(int64_t all, int d) {
  return std::max(tree_workspace(all, d),
                  part_plan(kDecodeWorkers, std::min<int64_t>(all, kDecodePairs), d).bytes);
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

dt_status run_paged(PagedArgs a, const dt_kv_cache* cache, int dt, void* ws, cudaStream_t s) {
  if (a.total_rows == 0) return DT_OK;
  const int ct = cache->dt;
  if (dt == DT_F32) {
    ProfileScope ps(DT_K_ATTN, s);
    const dim3 grid(a.total_rows, (a.Hq + kPlainWarps - 1) / kPlainWarps);
    launch_plain<DT_F32>(a, ct, grid, s);
    return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ECUDA;
  }
  const int64_t pairs = (int64_t)a.max_rows * a.G;  // of a request, for one KV head
  const int64_t all = (int64_t)(a.kt ? a.Nmax + 1 : a.total_rows) * a.G;
  // Few rows: a 128-row tile would be almost empty (64 single tokens over an e4m3
  // cache: 110 us against 231 us with tiles).
  const bool few = !a.kt && pairs <= kDecodePairs;
  // Two row tiles share a CTA's keys where a request has more than one.  Trees up
  // to 256 pairs keep one: their node counts vary, only the device knows them, and most do not
  // reach the second.  64 trees of 8 to 32 nodes, 4 heads: 234 us over e4m3 and 155 over bf16
  // pages with one tile, 282 and 182 with two; of 32 nodes each (132 pairs, four over a
  // tile): 360 and 235 with one, 320 and 205 with two.  One tree of 64 nodes, 260
  // pairs: 34 us with two, 39 us with one.
  const int tiles = pairs > (a.kt ? 256 : 128) ? 2 : 1;
  a.part_rows = (int)std::min<int64_t>(all, few ? kDecodePairs : 128 * tiles);
  const PartPlan p = part_plan(few ? kDecodeWorkers : 2 * kPagedSms / tiles, a.part_rows, a.d);
  uint8_t* w = (uint8_t*)ws + kWsHeader;
  a.split = (PagedSplit*)w;
  a.redo = (int*)(w + p.redo);
  a.tasks = (int*)(w + p.tasks);
  a.part_o = (float*)(w + p.sums);
  a.part_ml = (float2*)(w + p.stats);
  const cudaError_t e = few ? launch_paged_decode(a, ct, cache, (int)pairs, s)
                            : launch_paged_tc(a, ct, cache, tiles, s);
  return e == cudaSuccess ? DT_OK : DT_ECUDA;
}

// Has [p, p + n) a byte in common with any of `rows` pieces of w bytes that lie ld bytes
// apart from q on?  (A row that is done again reads its query once more after rows of the
// output were written, and other CTAs read theirs at any time.)
bool meets(const void* out, size_t n, const void* in, int64_t rows, size_t ld, size_t w) {
  const uintptr_t p = (uintptr_t)out, q = (uintptr_t)in;
  const int64_t i = p < q + w ? 0 : (int64_t)((p - q - w) / ld) + 1;  // first that ends behind p
  return n && i < rows && q + i * ld < p + n;
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

namespace dt {

bool paged_map(CUtensorMap* m, const void* base, int bytes, uint64_t cols, uint64_t rows,
               uint32_t box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * bytes};
  const uint32_t width = (uint32_t)std::min<uint64_t>(cols * bytes, 128);
  const cuuint32_t boxes[2] = {width / bytes, box}, one[2] = {1, 1};
  return fn(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
            const_cast<void*>(base), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_paged_join(const PagedArgs& a, int ct, Cut cut, int workers, cudaStream_t s) {
  ProfileScope ps(DT_K_ATTN_COMBINE, s);
  const dim3 grid(std::min(4 * dt_num_sms(), std::max(workers, 1) * a.part_rows));
  auto kern = ct == DT_BF16   ? paged_join_kernel<DT_BF16>
              : ct == DT_E4M3 ? paged_join_kernel<DT_E4M3>
                              : paged_join_kernel<DT_I8>;
  const cudaError_t e = launch_pdl(kern, grid, dim3(32 * kJoinWarps), 0, s, a, cut, workers);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace dt

using namespace dt;

extern "C" {

size_t dt_paged_attn_workspace_bytes(int batch, int total_rows, int Hq, int Hkv, int d) {
  if (batch < 1 || total_rows < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || d < 1) return 0;
  return chunk_workspace((int64_t)total_rows * (Hq / Hkv), d);
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
  ok = check_ws(ws, ws_bytes, chunk_workspace((int64_t)total_rows * (Hq / cache->Hkv), cache->d));
  if (ok != DT_OK) return ok;
  const size_t es = dt == DT_F32 ? 4 : 2, row = (size_t)Hq * cache->d * es;
  if (meets(d_out, total_rows * row, d_q, total_rows, ld_q * es, row)) return DT_EINVAL;
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
  return run_paged(a, cache, dt, ws, (cudaStream_t)stream);
}

size_t dt_tree_verify_attn_paged_workspace_bytes(int batch, int Nmax, int Hq, int Hkv, int d) {
  if (batch < 1 || Nmax < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || d < 1) return 0;
  return tree_workspace((int64_t)(Nmax + 1) * (Hq / Hkv), d);
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
  ok = check_ws(ws, ws_bytes, tree_workspace((int64_t)(Nmax + 1) * (Hq / cache->Hkv), cache->d));
  if (ok != DT_OK) return ok;
  const size_t one = (size_t)rows * cache->d * (dt == DT_F32 ? 4 : 2);  // bytes of a head of all rows
  const size_t all = one * Hq, own = one * cache->Hkv;
  if (meets(d_out, all, d_q, 1, all, all) || meets(d_out, all, d_k_tree, 1, own, own) ||
      meets(d_out, all, d_v_tree, 1, own, own))
    return DT_EINVAL;
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
  return run_paged(a, cache, dt, ws, (cudaStream_t)stream);
}

}  // extern "C"
