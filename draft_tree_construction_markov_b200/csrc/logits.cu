// Penalties for repeated tokens, biases and grammar masks on target logits.
//
// A CTA owns a slice of the vocabulary for one request and some of its rows.
// It first counts the request's history into a shared-memory table of its
// slice (one word per token: generated count, prompt flag), together with the
// slice's bias entries and the tree nodes whose token falls in it, and lists the
// tokens that any of these touch.  Then it streams the rows with their masks, a
// thread taking 8 neighbouring tokens (one 16-byte load of bf16), several rows
// on their way at once; groups that the mask forbids whole are written without
// being read, and in place a group without a forbidden token is not touched at
// all.  At last the threads share the listed tokens of all rows out among
// themselves and settle them one by one: common tokens are neighbours in the
// vocabulary, and left to the threads that stream them they would make a few
// threads of one slice do all of the work.  A token's count on a path is the
// table's plus the bits that the row's ancestor word and the word of the nodes
// that hold the token have in common.
//
// Bound: memory, each live row read and written once; the history is re-read
// by every slice of its request, from L2.
// Measured (B200): 16 trees of up to 32 nodes, V = 151936, bf16, histories of 256
// to 8192 tokens, 64 biases and a mask a node: 213 MB in 83 us (2.6 TB/s).  What
// is left over the copy is each CTA's table (counted anew for every slice and
// group of rows) and the last CTAs of the largest trees.
#include <limits.h>

#include "common.cuh"

namespace dt {
namespace {

constexpr int kLgThreads = 256;
constexpr int kLgSlice = 4096;                 // tokens per CTA
constexpr int kLgTab = kLgSlice + 8;           // rows start up to 7 tokens into a group of 8
constexpr int kLgGroups = kLgSlice / 8 / kLgThreads;  // groups per thread and row
template <bool BF16>
constexpr int kLgRows = BF16 ? 2 : 1;                 // rows at a time

struct LogitsArgs {
  const void* in;
  void* out;
  const int32_t* tokens;
  const uint64_t* anc;
  const int32_t* n_nodes;
  int batch, Nmax, V;
  const int32_t* hist;
  const int32_t* hist_start;
  const int32_t* n_prompt;
  int n_hist;
  const float* rep;
  const float* pres;
  const float* freq;
  const int32_t* bias_start;
  const int32_t* bias_token;
  const float* bias_value;
  int n_bias;
  const uint32_t* mask;
  const int32_t* mask_row;
  int n_mask_rows;
  int32_t* status;
};

// bits t .. t + 7 of a bit array of nw words; bits outside it are 0
__device__ __forceinline__ uint32_t bits8(const uint32_t* p, int t, int nw) {
  const int w = t >> 5, sh = t & 31;
  const uint32_t lo = (w >= 0 && w < nw) ? p[w] : 0u;
  const uint32_t hi = (sh > 24 && w + 1 < nw) ? p[w + 1] : 0u;
  return __funnelshift_r(lo, hi, sh) & 0xffu;
}

// the range [s, e) of request b in a list of n entries; an impossible one is
// recorded and empty
__device__ __forceinline__ int2 list_range(const int32_t* start, int b, int n, int32_t* status) {
  const int s = start[b], e = start[b + 1];
  if (s < 0 || e < s || e > n) {
    set_status(status, DT_EDEVICE);
    return make_int2(0, 0);
  }
  return make_int2(s, e);
}

// grid (slices, batch, row groups)
template <bool BF16, bool INPLACE>
__global__ void __launch_bounds__(kLgThreads, 5) logits_kernel(LogitsArgs a) {
  constexpr int W = BF16 ? 4 : 8;  // 32-bit words of a group of 8 tokens
  __shared__ uint32_t cnt[kLgTab];
  __shared__ uint32_t bidx[kLgTab];
  __shared__ uint16_t listed[kLgTab];            // table entries that something touches
  __shared__ int node_tok[64], node_id[64];
  __shared__ int n_nodes_here, n_listed;
  __shared__ int row_mask[65];                   // mask row of row i, -1: everything allowed
  __shared__ uint64_t row_path[65];              // its ancestor word
  const int tid = threadIdx.x, b = blockIdx.y;
  const int base = blockIdx.x * kLgSlice - 8;  // token of table entry 0
  int n = 0;
  if (a.n_nodes) {
    n = a.n_nodes[b];
    if (n < 0 || n > a.Nmax) {
      if (tid == 0) set_status(a.status, DT_EDEVICE);
      n = min(max(n, 0), a.Nmax);
    }
  }
  if ((int)blockIdx.z > n) return;  // uniform: none of this CTA's rows is live

  // ---- the slice's table
  for (int i = tid; i < kLgTab; i += kLgThreads) cnt[i] = bidx[i] = 0;
  if (tid == 0) n_nodes_here = n_listed = 0;
  if (tid <= n) {
    const int64_t row = (int64_t)b * (a.Nmax + 1) + tid;
    int m = -1;
    if (a.mask) {
      m = a.mask_row ? a.mask_row[row] : (int)min(row, (int64_t)INT_MAX);
      if (m < -1 || m >= a.n_mask_rows) {
        set_status(a.status, DT_EDEVICE);
        m = -1;
      }
    }
    row_mask[tid] = m;
    row_path[tid] = tid ? a.anc[row - b - 1] : 0ull;  // b * Nmax + tid - 1
  }
  __syncthreads();
  if (a.hist) {
    const int2 r = list_range(a.hist_start, b, a.n_hist, a.status);
    int np = a.n_prompt ? a.n_prompt[b] : 0;
    if (np < 0 || np > r.y - r.x) {
      set_status(a.status, DT_EDEVICE);
      np = min(max(np, 0), r.y - r.x);
    }
    for (int i0 = r.x + tid; i0 < r.y; i0 += 4 * kLgThreads) {
      int x4[4];  // (four loads on their way)
#pragma unroll
      for (int k = 0; k < 4; ++k) x4[k] = i0 + k * kLgThreads < r.y ? a.hist[i0 + k * kLgThreads] : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kLgThreads, x = x4[k];
        if (i >= r.y) break;
        if (x < 0 || x >= a.V) {
          set_status(a.status, DT_EDEVICE);
        } else if ((uint32_t)(x - base) < (uint32_t)kLgTab) {
          if (i - r.x < np)
            atomicOr(&cnt[x - base], 0x80000000u);
          else
            atomicAdd(&cnt[x - base], 1u);
        }
      }
    }
  }
  int2 br = make_int2(0, 0);
  if (a.bias_start) {
    br = list_range(a.bias_start, b, a.n_bias, a.status);
    for (int i = br.x + tid; i < br.y; i += kLgThreads) {
      const int x = a.bias_token[i];
      if (x < 0 || x >= a.V)
        set_status(a.status, DT_EDEVICE);
      else if ((uint32_t)(x - base) < (uint32_t)kLgTab)
        atomicMax(&bidx[x - base], (uint32_t)(i - br.x + 1));  // the last entry counts
    }
  }
  if (tid < n) {
    const int x = a.tokens[(int64_t)b * a.Nmax + tid];
    if (x < 0 || x >= a.V) {
      set_status(a.status, DT_EDEVICE);
    } else if ((uint32_t)(x - base) < (uint32_t)kLgTab) {
      const int k = atomicAdd(&n_nodes_here, 1);
      node_tok[k] = x - base;
      node_id[k] = tid;
      atomicOr(&cnt[x - base], 0x40000000u);  // a node holds it
    }
  }
  __syncthreads();
  for (int i0 = 0; i0 < kLgTab; i0 += kLgThreads) {
    const int i = i0 + tid;
    const bool t = i < kLgTab && (cnt[i] | bidx[i]);
    const uint32_t w = __ballot_sync(0xffffffffu, t);
    int at = 0;
    if ((tid & 31) == 0 && w) at = atomicAdd(&n_listed, __popc(w));
    at = __shfl_sync(0xffffffffu, at, 0);
    // (their order does not matter: every token is settled by itself)
    if (t) listed[at + __popc(w & ((1u << (tid & 31)) - 1))] = (uint16_t)i;
  }
  __syncthreads();
  const int nl = n_nodes_here, n_touched = n_listed;
  const float rep = a.rep ? a.rep[b] : 1.f, pres = a.pres ? a.pres[b] : 0.f,
              freq = a.freq ? a.freq[b] : 0.f;
  const int nw = (a.V + 31) / 32;

  // ---- the rows
  constexpr int RB = kLgRows<BF16>;
  for (int i0 = blockIdx.z; i0 <= n; i0 += RB * gridDim.z) {
    int64_t R[RB];            // first element of row k
    const uint32_t* mask[RB];
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      const int i = min(i0 + k * (int)gridDim.z, n);
      R[k] = ((int64_t)b * (a.Nmax + 1) + i) * a.V;
      mask[k] = row_mask[i] >= 0 ? a.mask + (int64_t)row_mask[i] * nw : nullptr;
    }
    uint32_t u[RB][kLgGroups][W];
    uint32_t mb[RB][kLgGroups];
    auto first = [&](int k, int j) {  // first token of the thread's group j of row k
      return (blockIdx.x * (kLgSlice / 8) + j * kLgThreads + tid) * 8 - (int)(R[k] & 7);
    };
#pragma unroll
    for (int k = 0; k < RB; ++k)
#pragma unroll
      for (int j = 0; j < kLgGroups; ++j)
        mb[k][j] = mask[k] ? bits8(mask[k], first(k, j), nw) : 0xffu;
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      const bool live = i0 + k * (int)gridDim.z <= n;
#pragma unroll
      for (int j = 0; j < kLgGroups; ++j) {
        const int t0 = first(k, j);
#pragma unroll
        for (int w = 0; w < W; ++w) u[k][j][w] = 0;
        if (live && t0 >= 0 && t0 + 8 <= a.V && mb[k][j] != 0 && !(INPLACE && mb[k][j] == 0xffu)) {
          const uint4* p = (const uint4*)((const uint8_t*)a.in + (R[k] + t0) * (BF16 ? 2 : 4));
#pragma unroll
          for (int w = 0; w < W / 4; ++w) {
            const uint4 q = p[w];
            u[k][j][4 * w] = q.x, u[k][j][4 * w + 1] = q.y;
            u[k][j][4 * w + 2] = q.z, u[k][j][4 * w + 3] = q.w;
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      if (i0 + k * (int)gridDim.z > n) break;
#pragma unroll
      for (int j = 0; j < kLgGroups; ++j) {
        const int t0 = first(k, j);
        uint32_t(&v)[W] = u[k][j];
        const uint32_t m = mb[k][j];
        if (INPLACE && m == 0xffu) continue;
        if (t0 >= 0 && t0 + 8 <= a.V) {
          if (m != 0xffu) {
#pragma unroll
            for (int w = 0; w < W; ++w) {
              if (BF16) {
                const uint32_t keep = (m >> (2 * w) & 1u) * 0xffffu | (m >> (2 * w + 1) & 1u) * 0xffff0000u;
                v[w] = (v[w] & keep) | (0xff80ff80u & ~keep);
              } else if (!((m >> w) & 1u)) {
                v[w] = 0xff800000u;
              }
            }
          }
          uint4* p = (uint4*)((uint8_t*)a.out + (R[k] + t0) * (BF16 ? 2 : 4));
#pragma unroll
          for (int w = 0; w < W / 4; ++w)
            p[w] = make_uint4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
        } else if (t0 + 8 > 0 && t0 < a.V) {
          // a group cut by the row's start or end: token by token
          for (int e = 0; e < 8; ++e) {
            const int x = t0 + e;
            if (x < 0 || x >= a.V) continue;
            const bool ok = (m >> e) & 1u;
            if (BF16)
              ((uint16_t*)a.out)[R[k] + x] = ok ? ((const uint16_t*)a.in)[R[k] + x] : 0xff80u;
            else
              ((uint32_t*)a.out)[R[k] + x] = ok ? ((const uint32_t*)a.in)[R[k] + x] : 0xff800000u;
          }
        }
      }
    }
  }

  // ---- the listed tokens: `lanes` threads a token, each with its share of the rows
  __syncthreads();
  if (n_touched == 0) return;
  const int rows = (n - (int)blockIdx.z) / (int)gridDim.z + 1;  // of this CTA
  const int lanes = min(max(kLgThreads / n_touched, 1), rows);
  for (int k = tid; k < n_touched * lanes; k += kLgThreads) {
    const int entry = listed[k % n_touched], x = base + entry;
    const uint32_t c = cnt[entry], bi = bidx[entry];
    const float bias = bi ? a.bias_value[br.x + bi - 1] : 0.f;
    uint64_t nodes = 0;  // that hold this token
    if (c & 0x40000000u)
      for (int y = 0; y < nl; ++y)
        if (node_tok[y] == entry) nodes |= 1ull << node_id[y];
    // (rows four at a time: their masks and logits are on their way together)
    for (int q0 = k / n_touched; q0 < rows; q0 += 4 * lanes) {
      float z4[4];
      bool ok[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int q = q0 + y * lanes, i = blockIdx.z + min(q, rows - 1) * gridDim.z;
        const int64_t R = ((int64_t)b * (a.Nmax + 1) + i) * a.V;
        // groups begin up to 7 tokens before the row: the token may be another slice's
        const int group = (x + (int)(R & 7)) >> 3;
        ok[y] = q < rows && group / (kLgSlice / 8) == (int)blockIdx.x;
        z4[y] = 0.f;
        if (ok[y]) {
          const int m = row_mask[i];
          const uint32_t word = m >= 0 ? a.mask[(int64_t)m * nw + (x >> 5)] : 0xffffffffu;
          z4[y] = BF16 ? bf16_to_f32(((const uint16_t*)a.in)[R + x]) : ((const float*)a.in)[R + x];
          ok[y] = (word >> (x & 31)) & 1u;
        }
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if (!ok[y]) continue;
        const int i = blockIdx.z + (q0 + y * lanes) * gridDim.z;
        const int64_t at = ((int64_t)b * (a.Nmax + 1) + i) * a.V + x;
        const uint32_t made = (c & 0x3fffffffu) + __popcll(row_path[i] & nodes);
        float z = z4[y];
        if (made || (c >> 31)) z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
        if (made) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)made)), pres);
        if (bi) z = __fadd_rn(z, bias);
        if (BF16) {
          uint32_t r;
          asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(z));
          ((uint16_t*)a.out)[at] = (uint16_t)r;
        } else {
          ((float*)a.out)[at] = z;
        }
      }
    }
  }
}

}  // namespace
}  // namespace dt

using namespace dt;

extern "C" {

size_t dt_logits_workspace_bytes(void) { return kWsHeader; }

dt_status dt_logits_process(const void* d_logits, dt_dtype dt, const int32_t* d_tokens,
                            const uint64_t* d_anc, const int32_t* d_n_nodes, int batch, int Nmax,
                            int V, const int32_t* d_history, const int32_t* d_hist_start,
                            const int32_t* d_n_prompt, int n_history, const float* d_repetition,
                            const float* d_presence, const float* d_frequency,
                            const int32_t* d_bias_start, const int32_t* d_bias_token,
                            const float* d_bias_value, int n_bias, const uint32_t* d_mask,
                            const int32_t* d_mask_row, int n_mask_rows, void* d_out, void* ws,
                            size_t ws_bytes, dt_stream stream) {
  if (!d_logits || !d_out || (dt != DT_F32 && dt != DT_BF16)) return DT_EINVAL;
  if (batch < 1 || Nmax < 0 || V < 1 || n_history < 0 || n_bias < 0 || n_mask_rows < 0)
    return DT_EINVAL;
  const bool tree = d_tokens && d_anc && d_n_nodes;
  if (Nmax > 0 ? !tree : (d_tokens || d_anc || d_n_nodes)) return DT_EINVAL;
  if (!d_history != !d_hist_start || (d_n_prompt && !d_history)) return DT_EINVAL;
  if (!d_bias_start != !d_bias_token || !d_bias_start != !d_bias_value) return DT_EINVAL;
  if (d_mask_row && !d_mask) return DT_EINVAL;
  if (((uintptr_t)d_logits | (uintptr_t)d_out) & 15) return DT_EINVAL;
  if (Nmax > 64 || batch > 1024 || V >= 1 << 24) return DT_EUNSUPPORTED;
  const size_t bytes = (size_t)batch * (Nmax + 1) * V * (dt == DT_BF16 ? 2 : 4);
  const uintptr_t x = (uintptr_t)d_logits, y = (uintptr_t)d_out;
  if (x != y && x < y + bytes && y < x + bytes) return DT_EINVAL;  // partial overlap
  const dt_status ok = check_ws(ws, ws_bytes, kWsHeader);
  if (ok != DT_OK) return ok;
  LogitsArgs a;
  a.in = d_logits;
  a.out = d_out;
  a.tokens = d_tokens;
  a.anc = d_anc;
  a.n_nodes = d_n_nodes;
  a.batch = batch;
  a.Nmax = Nmax;
  a.V = V;
  a.hist = d_history;
  a.hist_start = d_hist_start;
  a.n_prompt = d_n_prompt;
  a.n_hist = n_history;
  a.rep = d_repetition;
  a.pres = d_presence;
  a.freq = d_frequency;
  a.bias_start = d_bias_start;
  a.bias_token = d_bias_token;
  a.bias_value = d_bias_value;
  a.n_bias = n_bias;
  a.mask = d_mask;
  a.mask_row = d_mask_row;
  a.n_mask_rows = n_mask_rows;
  a.status = (int32_t*)ws;
  // a row may start 7 tokens into its first group of 8
  const int slices = (V + 7 + kLgSlice - 1) / kLgSlice;
  const int rows = Nmax + 1;
  // Rows are split over CTAs until there are about 16 per SM: trees differ in
  // size, and the rows of the largest are what the call waits for.  Against that
  // every CTA of a slice counts the history anew.
  const int want = (16 * dt_num_sms() + slices * batch - 1) / (slices * batch);
  const int z = want < 1 ? 1 : want > rows ? rows : want;
  const dim3 grid(slices, batch, z);
  cudaStream_t s = (cudaStream_t)stream;
  ProfileScope ps(DT_K_LOGITS, s);
  const bool in_place = d_logits == d_out;
  if (dt == DT_BF16)
    in_place ? logits_kernel<true, true><<<grid, kLgThreads, 0, s>>>(a)
             : logits_kernel<true, false><<<grid, kLgThreads, 0, s>>>(a);
  else
    in_place ? logits_kernel<false, true><<<grid, kLgThreads, 0, s>>>(a)
             : logits_kernel<false, false><<<grid, kLgThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DT_OK : DT_ECUDA;
}

}  // extern "C"
