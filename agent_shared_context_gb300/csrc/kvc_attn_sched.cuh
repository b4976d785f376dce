// kvc_attn_sched.cuh -- how the paged-attention kernels divide their work, and
// how the parts of a divided row tile are joined.
//
// The lengths of the requests live on the device, so the host cannot size the
// work.  A *tile* is a fixed run of key rows (kTile of them at most), an *item*
// is one (request, KV head, run of query tokens) and costs as many units as it
// has key tiles in sight.  The units of all items, in the order request, head,
// query run, are cut into equal shares, one per CTA of a persistent grid: a
// single long decode, a batch of ragged ones and a dense prefill all fill the
// GPU, with no work list to build first.  Every CTA adds the units up for
// itself (R lengths from L2) and walks its share.  An item that spans several
// shares leaves un-normalised partial rows (O, m, l) in the workspace; the CTA
// that arrives last at the item's counter joins them in the order of their
// key tiles, so the result does not depend on who was last.
#pragma once

#include <cstdint>

#include "kvc_internal.h"

namespace kvc {
namespace attn {

// Everything a kernel needs to divide the work (by value, all host-checked).
struct SchedArgs {
  const int32_t* q_start;   // [R + 1]
  const int32_t* kv_lens;   // [R]
  int32_t R, H, N;          // requests, KV heads, query tokens
  int32_t kv_cap;           // max_blocks * page_size
  int32_t causal, window;
  int32_t tok_item;         // query tokens per item
  int32_t group_tok;        // key tokens of a tile group (a page or several, below)
  int32_t group_tiles;      // tiles per group
  int32_t tile_tok;         // key tokens per tile inside a group
};

struct Request {
  int32_t q0, nq, kv, pos0;   // first query token, their number, keys, position of the first
};

// Table values come from the device: whatever they hold, rows stay in [0, N)
// and keys in [0, kv_cap].
__device__ __forceinline__ Request load_request(const SchedArgs& a, int r) {
  Request q;
  const int s0 = a.q_start[r], s1 = a.q_start[r + 1];
  q.q0 = min(max(s0, 0), a.N);
  q.nq = min(max(s1, q.q0), a.N) - q.q0;
  q.kv = min(max(a.kv_lens[r], 0), a.kv_cap);
  q.pos0 = q.kv - q.nq;
  return q;
}

__device__ __forceinline__ bool request_out_of_range(const SchedArgs& a, int r) {
  const int s0 = a.q_start[r], s1 = a.q_start[r + 1], n = a.kv_lens[r];
  return s0 < 0 || s1 < s0 || s1 > a.N || n < 0 || n > a.kv_cap;
}

__device__ __forceinline__ int tile_of(const SchedArgs& a, int tok) {
  const int g = tok / a.group_tok;
  return g * a.group_tiles + (tok - g * a.group_tok) / a.tile_tok;
}

// Key tiles [lo, hi) that query tokens [t0, t1) of the request can see.  An
// item that sees nothing keeps one (fully masked) tile: its rows are written.
__device__ __forceinline__ void item_tiles(const SchedArgs& a, const Request& q, int t0, int t1,
                                           int* lo, int* hi) {
  const int k1 = a.causal ? min(q.kv, q.pos0 + t1) : q.kv;
  const int k0 = a.window > 0 ? max(0, q.pos0 + t0 - a.window + 1) : 0;
  if (k1 <= k0) {
    *lo = 0;
    *hi = 1;
    return;
  }
  *lo = tile_of(a, k0);
  *hi = tile_of(a, k1 - 1) + 1;
}

__device__ __forceinline__ int n_items(const SchedArgs& a, const Request& q) {
  return (q.nq + a.tok_item - 1) / a.tok_item;
}

// Units of one KV head of a request.
__device__ __forceinline__ int64_t head_units(const SchedArgs& a, const Request& q) {
  int64_t u = 0;
  const int n = n_items(a, q);
  for (int i = 0; i < n; ++i) {
    int lo, hi;
    item_tiles(a, q, i * a.tok_item, min(q.nq, (i + 1) * a.tok_item), &lo, &hi);
    u += hi - lo;
  }
  return u;
}

// One CTA's part of one item.
struct Item {
  int32_t r, h, t0, nt;        // request, KV head, first query token in the request, their number
  int32_t q0, kv, pos0;        // global row of token t0, keys, position of token t0
  int32_t tile0, ntiles;       // key tiles of this part
  int32_t part, nparts, cta0;  // this part among the item's, the first part's CTA
};

struct Shared {
  int64_t warp_sum[32];
  int64_t total;
  int64_t begin_off;   // units of the start request before the share's first unit
  int32_t begin_r;
};

// CTA that owns unit u when U units are cut into n shares [c U / n, (c+1) U / n).
__device__ __forceinline__ int owner_of(int64_t u, int64_t U, int n) {
  return static_cast<int>(((u + 1) * n - 1) / U);
}

// Walks the share of one CTA.  All threads that walk hold the same state.
struct Walker {
  int64_t U, u, u1;            // all units, the next one, the end of the share
  int32_t r, h, i;             // where the next unit lies
  int64_t item_u0;             // first unit of that item
  Request q;
  int32_t n;                   // items of request r
  int32_t grid;

  // Next part of the share; false at its end.
  __device__ __forceinline__ bool next(const SchedArgs& a, Item* out) {
    if (u >= u1) return false;
    for (;;) {
      if (i < n) {
        const int t0 = i * a.tok_item, t1 = min(q.nq, t0 + a.tok_item);
        int lo, hi;
        item_tiles(a, q, t0, t1, &lo, &hi);
        const int64_t end = item_u0 + (hi - lo);
        if (u < end) {
          const int64_t stop = end < u1 ? end : u1;
          out->r = r;
          out->h = h;
          out->t0 = t0;
          out->nt = t1 - t0;
          out->q0 = q.q0 + t0;
          out->kv = q.kv;
          out->pos0 = q.pos0 + t0;
          out->tile0 = lo + static_cast<int>(u - item_u0);
          out->ntiles = static_cast<int>(stop - u);
          const int c0 = owner_of(item_u0, U, grid);
          out->cta0 = c0;
          out->part = static_cast<int>(blockIdx.x) - c0;
          out->nparts = owner_of(end - 1, U, grid) - c0 + 1;
          u = stop;
          return true;
        }
        item_u0 = end;
        ++i;
      } else if (n > 0 && h + 1 < a.H) {
        ++h;
        i = 0;
      } else {
        ++r;
        if (r >= a.R) return false;
        h = 0;
        i = 0;
        q = load_request(a, r);
        n = n_items(a, q);
      }
    }
  }
};

template <int THREADS>
__device__ __forceinline__ int64_t block_inclusive(int64_t v, Shared* sh, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == 31) sh->warp_sum[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t x = sh->warp_sum[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return v + before;
}

// Called by every thread of the CTA; the same walker in all of them.
template <int THREADS>
__device__ Walker walker_begin(const SchedArgs& a, Shared* sh, int32_t* dev_status) {
  const int tid = threadIdx.x;
  int64_t U = 0, mine = 0, incl = 0;
  bool bad = false;
  for (int base = 0; base < a.R; base += THREADS) {
    const int r = base + tid;
    mine = 0;
    if (r < a.R) {
      bad |= request_out_of_range(a, r);
      mine = head_units(a, load_request(a, r)) * a.H;
    }
    int64_t total;
    incl = block_inclusive<THREADS>(mine, sh, &total);
    U += total;
  }
  if (bad && blockIdx.x == 0) atomicCAS(dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
  // no empty shares between others: an item's parts are consecutive CTAs
  const int n = static_cast<int>(U < gridDim.x ? U : gridDim.x);
  const bool idle = static_cast<int>(blockIdx.x) >= n;
  const int64_t u0 = idle ? U : U * blockIdx.x / n;
  if (tid == 0) {
    sh->begin_r = a.R;
    sh->begin_off = 0;
  }
  __syncthreads();
  int64_t before = 0;
  for (int base = 0; base < a.R; base += THREADS) {
    const int r = base + tid;
    int64_t total = U;
    if (a.R > THREADS) {             // one chunk: the first pass's sums still stand
      mine = r < a.R ? head_units(a, load_request(a, r)) * a.H : 0;
      incl = block_inclusive<THREADS>(mine, sh, &total);
    }
    if (before + incl > u0 && before + incl - mine <= u0) {   // one thread at most
      sh->begin_r = r;
      sh->begin_off = u0 - (before + incl - mine);
    }
    before += total;
    if (before > u0) break;
  }
  __syncthreads();
  Walker w;
  w.U = U;
  w.u = u0;
  w.u1 = idle ? U : U * (blockIdx.x + 1) / n;
  w.grid = n;
  w.r = sh->begin_r;
  w.h = 0;
  w.i = 0;
  w.n = 0;
  w.item_u0 = u0;
  w.q = Request{0, 0, 0, 0};
  if (w.u < w.u1) {
    w.q = load_request(a, w.r);
    w.n = n_items(a, w.q);
    const int64_t hu = head_units(a, w.q);
    w.h = static_cast<int>(sh->begin_off / hu);
    w.item_u0 = u0 - (sh->begin_off - w.h * hu);
  }
  return w;
}

// ------------------------------------------------------------ joining parts
// A share leaves at most two parts of divided items: the end of an item that
// an earlier share began (slot 0) and the beginning of one that a later share
// goes on with (slot 1); an item that covers the whole share takes slot 0.
// A slot holds O [rows][d], m [rows] and l [rows] in fp32 with m in units of
// log2: the rows' softmax is sum exp2(x - m) = l and O = sum exp2(x - m) v.
__host__ __device__ inline size_t slot_floats(int rows, int d) {
  return static_cast<size_t>(rows) * (d + 2);
}

__device__ __forceinline__ int slot_of(int part) { return part == 0 ? 1 : 0; }

// exp2(m - M) for a part's weight, 0 for a part that saw nothing.
__device__ __forceinline__ float part_weight(float m, float l, float M) {
  return l == 0.0f ? 0.0f : exp2f(m - M);
}

}  // namespace attn
}  // namespace kvc
