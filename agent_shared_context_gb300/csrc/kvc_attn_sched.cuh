// kvc_attn_sched.cuh -- how the paged-attention kernels divide their work, and
// how the parts of a divided row tile are joined.
//
// The lengths of the requests live on the device, so the host cannot size the
// work.  A *tile* is a fixed run of key rows (kTile of them at most), an *item*
// is one (request, KV head, run of query tokens) and costs as many units as it
// has key tiles in sight, and some for itself.  The units of all items, in the order request, head,
// query run, are cut into equal shares, one per CTA of a persistent grid: a
// single long decode, a batch of ragged ones and a dense prefill all fill the
// GPU, with no work list to build first.  An item's beginning and end cost as
// much as some tiles; it counts that many units more, before its first tile.
// Every CTA adds the units up for itself (R lengths from L2) and walks its
// share.  An item that spans several shares leaves un-normalised partial rows
// (O, m, l) in the workspace; the CTA that arrives last at the item's counter
// joins them in the order of their key tiles, so the result does not depend on
// who was last.
#pragma once

#include <cstdint>

#include "kvc_internal.h"

namespace kvc {
namespace attn {

// Division by a divisor that a call fixes (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): exact for 0 <= n < 2^31.
struct FastDiv {
  uint32_t mul, shift;
  int32_t d;
};

inline FastDiv make_fastdiv(int32_t d) {
  FastDiv f{0, 0, d};
  while ((int64_t(1) << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
  return f;
}

__device__ __forceinline__ int fast_div(int n, const FastDiv& f) {
  const uint32_t u = static_cast<uint32_t>(n);
  return static_cast<int>((__umulhi(u, f.mul) + u) >> f.shift);
}

// Everything a kernel needs to divide the work (by value, all host-checked).
struct SchedArgs {
  const int32_t* q_start;   // [R + 1]
  const int32_t* kv_lens;   // [R]
  int32_t R, H, N;          // requests, KV heads, query tokens
  int32_t kv_cap;           // max_blocks * page_size
  int32_t causal, window;
  FastDiv item;             // query tokens per item
  FastDiv group;            // key tokens of a tile group (a page or several, below)
  FastDiv tile;             // key tokens per tile inside a group
  int32_t group_tiles;      // tiles per group
  int32_t overhead;         // units of an item besides its tiles
  int32_t even;             // tile t holds the tokens [t tile, (t + 1) tile)
};

struct Request {
  int32_t q0, nq, kv, pos0;   // first query token, their number, keys, position of the first
};

// Table values come from the device: whatever they hold, rows stay in [0, N)
// and keys in [0, kv_cap].
__device__ __forceinline__ Request load_request(const SchedArgs& a, int r, bool* bad = nullptr) {
  Request q;
  const int s0 = a.q_start[r], s1 = a.q_start[r + 1], n = a.kv_lens[r];
  q.q0 = min(max(s0, 0), a.N);
  q.nq = min(max(s1, q.q0), a.N) - q.q0;
  q.kv = min(max(n, 0), a.kv_cap);
  q.pos0 = q.kv - q.nq;
  if (bad != nullptr) *bad |= s0 < 0 || s1 < s0 || s1 > a.N || n < 0 || n > a.kv_cap;
  return q;
}

__device__ __forceinline__ int tile_of(const SchedArgs& a, int tok) {
  if (a.even) return fast_div(tok, a.tile);
  const int g = fast_div(tok, a.group);
  return g * a.group_tiles + fast_div(tok - g * a.group.d, a.tile);
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

__device__ __forceinline__ int item_units(const SchedArgs& a, const Request& q, int i) {
  int lo, hi;
  item_tiles(a, q, i * a.item.d, min(q.nq, (i + 1) * a.item.d), &lo, &hi);
  return hi - lo + a.overhead;
}

__device__ __forceinline__ int n_items(const SchedArgs& a, const Request& q) {
  return fast_div(q.nq + a.item.d - 1, a.item);
}

// sum over 0 <= i < n of floor((a i + b) / m): the lattice points under a line (on sums
// of floors: Graham, Knuth and Patashnik, "Concrete Mathematics", 3.5).  The whole parts
// of a / m and b / m are summed in closed form; of what is left the points are counted
// by rows in place of columns, a sum of the same kind with a and m exchanged, so that
// (a, m) goes the way of Euclid's algorithm.
static __device__ __noinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t s = 0;
  while (n > 0) {
    if (a >= m) {
      s += static_cast<int64_t>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += static_cast<int64_t>(n) * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return s;
}

// Units of the request's first `n` items of one KV head.  A causal chunk on tiles
// that are full has a closed form: item i sees the tiles before
// ceil((pos0 + (i + 1) item) / tile), with a window those from
// floor((pos0 + i item - window + 1) / tile) on, where that is not negative.  (700
// windowed tokens added up item by item took 3 us more.)
static __device__ __noinline__ int64_t first_units(const SchedArgs& a, const Request& q, int n) {
  if (n <= 0) return 0;
  if (a.even && n > 2) {
    const int64_t last = item_units(a, q, n - 1);      // the last may be shorter than an item
    if (!a.causal) return last * n;
    if (q.pos0 >= 0) {
      int64_t u = last + static_cast<int64_t>(n - 1) * a.overhead +
                  floor_sum(n - 1, a.tile.d, a.item.d, q.pos0 + a.item.d + a.tile.d - 1);
      if (a.window > 0) {
        const int64_t past = static_cast<int64_t>(q.pos0) - a.window + 1;   // of item 0
        const int64_t i0 = past >= 0 ? 0 : fast_div(static_cast<int>(min(
            -past + a.item.d - 1, int64_t(0x7fffffff))), a.item);
        if (i0 < n - 1)
          u -= floor_sum(static_cast<uint32_t>(n - 1 - i0), a.tile.d, a.item.d,
                         static_cast<uint32_t>(past + i0 * a.item.d));
      }
      return u;
    }
  }
  int64_t u = 0;
  for (int i = 0; i < n; ++i) u += item_units(a, q, i);
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
  int64_t off;         // units before the share's first in what is searched
  int32_t r, h, i;     // where the share begins
  int32_t item_off;    // units of that item before the share
};

// Calls, not copies: the kernels' instruction footprint is a cost of its own
// (their first pass through the code misses every cache).
static __device__ __noinline__ int64_t div64(int64_t x, int64_t y) {
  if (x < (int64_t(1) << 32) && y < (int64_t(1) << 32))
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// U units cut into n shares [c U / n, (c + 1) U / n).
struct Shares {
  int64_t U;
  int32_t n;

  __device__ __forceinline__ int64_t start(int c) const {
    const int64_t x = c * U;
    if (x < (int64_t(1) << 32)) return static_cast<uint32_t>(x) / static_cast<uint32_t>(n);
    return x / n;
  }
  __device__ __forceinline__ int owner(int64_t u) const {
    const int64_t x = (u + 1) * n - 1;
    if ((x | U) < (int64_t(1) << 32))
      return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(U));
    return static_cast<int>(x / U);
  }
};

// Walks the share of one CTA.  All threads that walk hold the same state.
struct Walker {
  Shares sh;
  int64_t u, u1;               // the next unit, the end of the share
  int32_t r, h, i;             // where the next unit lies
  int64_t item_u0;             // first unit of that item
  Request q;
  int32_t n;                   // items of request r
  int64_t item_first, item_end;   // units of the last part's item, and whether it is all
  bool begins, ends;              // here: what parts() goes by

  // Next part of the share; false at its end.
  __device__ __forceinline__ bool next(const SchedArgs& a, Item* out) {
    if (u >= u1) return false;
    for (;;) {
      if (i < n) {
        const int t0 = i * a.item.d, t1 = min(q.nq, t0 + a.item.d);
        int lo, hi;
        item_tiles(a, q, t0, t1, &lo, &hi);
        const int64_t first = item_u0 + a.overhead, end = first + (hi - lo);
        if (u < first) u = first < u1 ? first : u1;
        if (u >= u1) return false;
        if (u < end) {
          const int64_t stop = end < u1 ? end : u1;
          out->r = r;
          out->h = h;
          out->t0 = t0;
          out->nt = t1 - t0;
          out->q0 = q.q0 + t0;
          out->kv = q.kv;
          out->pos0 = q.pos0 + t0;
          out->tile0 = lo + static_cast<int>(u - first);
          out->ntiles = static_cast<int>(stop - u);
          begins = u == first;
          ends = end <= u1;
          item_first = first;
          item_end = end;
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

// The part that next() gave among its item's.
__device__ __forceinline__ void parts(const Walker& w, Item* it) {
  const int me = blockIdx.x;
  it->cta0 = w.begins ? me : w.sh.owner(w.item_first);
  it->part = me - it->cta0;
  it->nparts = (w.ends ? me : w.sh.owner(w.item_end - 1)) - it->cta0 + 1;
}

template <int THREADS>
__device__ __noinline__ int64_t block_inclusive(int64_t v, Shared* sh, int64_t* total) {
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
#pragma unroll 4
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t x = sh->warp_sum[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return v + before;
}

__device__ __forceinline__ Walker walker_empty(const SchedArgs& a, int64_t U) {
  Walker w;
  w.sh.U = U;
  // no empty shares between others: an item's parts are consecutive CTAs
  w.sh.n = static_cast<int>(U < gridDim.x ? U : gridDim.x);
  w.u = w.u1 = w.item_u0 = U;
  w.r = a.R;
  w.h = w.i = w.n = 0;
  w.q = Request{0, 0, 0, 0};
  w.item_first = w.item_end = 0;
  w.begins = w.ends = true;
  return w;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
  return __shfl_sync(0xffffffffu, v, lane);
}

// Up to 32 requests: a lane has one, and every warp finds the share by itself.
static __device__ __noinline__ Walker walker_lanes(const SchedArgs& a, int32_t* dev_status) {
  const int lane = threadIdx.x & 31;
  Request q{0, 0, 0, 0};
  int n = 0;
  int64_t units = 0;
  bool bad = false;
  if (lane < a.R) {
    q = load_request(a, lane, &bad);
    n = n_items(a, q);
    units = n == 1 ? item_units(a, q, 0) : first_units(a, q, n);
  }
  if (bad && blockIdx.x == 0) atomicCAS(dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
  const int64_t mine = units * a.H;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  Walker w = walker_empty(a, shfl64(incl, 31));
  if (static_cast<int>(blockIdx.x) >= w.sh.n) return w;
  w.u = w.sh.start(blockIdx.x);
  w.u1 = w.sh.start(blockIdx.x + 1);
  w.r = __ffs(__ballot_sync(0xffffffffu, incl > w.u)) - 1;
  int64_t off = w.u - shfl64(incl - mine, w.r);
  const int64_t hu = shfl64(units, w.r);
  w.h = static_cast<int>(div64(off, hu));
  off -= w.h * hu;
  w.q.q0 = __shfl_sync(0xffffffffu, q.q0, w.r);
  w.q.nq = __shfl_sync(0xffffffffu, q.nq, w.r);
  w.q.kv = __shfl_sync(0xffffffffu, q.kv, w.r);
  w.q.pos0 = __shfl_sync(0xffffffffu, q.pos0, w.r);
  w.n = __shfl_sync(0xffffffffu, n, w.r);
  w.item_u0 = w.u - off;
  if (w.n > 1) {
    // the last item that begins at or before `off`
#pragma unroll 1
    for (int base = 0; base < w.n; base += 32) {
      const int64_t p = first_units(a, w.q, min(base + lane, w.n - 1));
      const uint32_t before = __ballot_sync(0xffffffffu, base + lane < w.n && p <= off);
      if (before == 0) break;
      const int last = 31 - __clz(before);
      w.i = base + last;
      w.item_u0 = w.u - off + shfl64(p, last);
    }
  }
  return w;
}

// More requests: a thread has one at a time.
template <int THREADS>
__device__ __noinline__ Walker walker_block(const SchedArgs& a, Shared* sh, int32_t* dev_status) {
  const int tid = threadIdx.x;
  int64_t U = 0, mine = 0, incl = 0;
  bool bad = false;
  for (int base = 0; base < a.R; base += THREADS) {
    const int r = base + tid;
    mine = 0;
    if (r < a.R) {
      const Request q = load_request(a, r, &bad);
      mine = first_units(a, q, n_items(a, q)) * a.H;
    }
    int64_t total;
    incl = block_inclusive<THREADS>(mine, sh, &total);
    U += total;
  }
  if (bad && blockIdx.x == 0) atomicCAS(dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
  Walker w = walker_empty(a, U);
  if (static_cast<int>(blockIdx.x) >= w.sh.n) return w;
  w.u = w.sh.start(blockIdx.x);
  w.u1 = w.sh.start(blockIdx.x + 1);
  // the request of unit u ...
  int64_t before = 0;
  for (int base = 0; base < a.R; base += THREADS) {
    const int r = base + tid;
    int64_t total = U;
    if (a.R > THREADS) {             // one chunk: the first pass's sums still stand
      mine = 0;
      if (r < a.R) {
        const Request q = load_request(a, r);
        mine = first_units(a, q, n_items(a, q)) * a.H;
      }
      incl = block_inclusive<THREADS>(mine, sh, &total);
    }
    if (before + incl > w.u && before + incl - mine <= w.u) {   // one thread
      const int64_t off = w.u - (before + incl - mine);
      const int64_t hu = div64(mine, a.H);
      sh->r = r;
      sh->h = static_cast<int>(div64(off, hu));
      sh->off = off - sh->h * hu;
    }
    before += total;
    if (before > w.u) break;
  }
  __syncthreads();
  w.r = sh->r;
  w.h = sh->h;
  w.q = load_request(a, w.r);
  w.n = n_items(a, w.q);
  // ... and its item
  const int64_t off = sh->off;
  if (w.n == 1) {
    w.item_u0 = w.u - off;
  } else {
    for (int i = tid; i < w.n; i += THREADS) {
      const int64_t p = first_units(a, w.q, i);
      if (p <= off && off < p + item_units(a, w.q, i)) {        // one thread
        sh->i = i;
        sh->item_off = static_cast<int>(off - p);
      }
      if (p > off) break;
    }
    __syncthreads();
    w.i = sh->i;
    w.item_u0 = w.u - sh->item_off;
  }
  return w;
}

// Called by every thread of the CTA; the same walker in all of them.
template <int THREADS>
__device__ __forceinline__ Walker walker_begin(const SchedArgs& a, Shared* sh,
                                               int32_t* dev_status) {
  if (a.R <= 32) return walker_lanes(a, dev_status);
  return walker_block<THREADS>(a, sh, dev_status);
}

// ------------------------------------------------------------ joining parts
// A share leaves at most two parts of divided items: the end of an item that
// an earlier share began (slot 0) and the beginning of one that a later share
// goes on with (slot 1); an item that covers the whole share takes slot 0.
// A slot holds O, m and l of its rows in fp32, with m in units of log2: the
// row's softmax is sum exp2(x - m) = l and O = sum exp2(x - m) v.  O lies as
// [d / 4][rows] groups of four columns, so that threads that each have a row
// write and read neighbouring 16 bytes.
__host__ __device__ inline size_t slot_floats(int rows, int d) {
  return static_cast<size_t>(rows) * (d + 2);
}

__device__ __forceinline__ int slot_of(int part) { return part == 0 ? 1 : 0; }

// exp2(m - M) for a part's weight, 0 for a part that saw nothing.
__device__ __forceinline__ float part_weight(float m, float l, float M) {
  return l == 0.0f ? 0.0f : exp2f(m - M);
}

__device__ __forceinline__ void scale(float4& x, float f) {
  x.x *= f;
  x.y *= f;
  x.z *= f;
  x.w *= f;
}

__device__ __forceinline__ void add_scaled(float4& x, float4 v, float f) {
  x.x = fmaf(v.x, f, x.x);
  x.y = fmaf(v.y, f, x.y);
  x.z = fmaf(v.z, f, x.z);
  x.w = fmaf(v.w, f, x.w);
}

// One of `n_threads` threads joins the parts of rows [0, rows) of an item and
// hands (row, first column, four values of O / l, lse in nats) to `store`.
// Part p lies in slot slot_of(p) of CTA cta0 + p, `slot_rows` rows with row0
// the first.  Parts are added in the order of their keys; the loads of kP of them
// are in flight at a time, which takes registers.
template <int kP, int kC, typename Store>
__device__ __forceinline__ void join_parts(const float* slots, size_t slot_n, int slot_rows,
                                           int row0, int d, const Item& it, int rows, int tid,
                                           int n_threads, Store store) {
  // threads over rows first, then over groups of columns; a thread keeps its row
  int span = 1;
  while (span < rows) span <<= 1;
  if (span > n_threads) span = n_threads;
  const int d4 = d / 4, step = n_threads / span;
  const float* base = slots + static_cast<size_t>(it.cta0) * 2 * slot_n;
#pragma unroll 1
  for (int row = tid & (span - 1); row < rows; row += span) {
    auto part = [&](int p) { return base + (static_cast<size_t>(p) * 2 + slot_of(p)) * slot_n; };
#pragma unroll 1
    for (int c0 = tid / span; c0 < d4; c0 += kC * step) {
      float4 acc[kC];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int p0 = 0; p0 < it.nparts; p0 += kP) {
        float pm[kP], pl[kP];
        float4 v[kP][kC];
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          const float* ps = part(p0 + p);
          const bool has = p0 + p < it.nparts;
          pm[p] = has ? __ldcg(ps + slot_rows * d + row0 + row) : -INFINITY;
          pl[p] = has ? __ldcg(ps + slot_rows * d + slot_rows + row0 + row) : 0.f;
#pragma unroll
          for (int c = 0; c < kC; ++c)
            if (has && c0 + c * step < d4)
              v[p][c] = __ldcg(reinterpret_cast<const float4*>(ps) + (c0 + c * step) * slot_rows +
                               row0 + row);
        }
        float top = M;
#pragma unroll
        for (int p = 0; p < kP; ++p) top = fmaxf(top, pm[p]);
        const float f0 = part_weight(M, L, top);
        M = top;
        L *= f0;
#pragma unroll
        for (int c = 0; c < kC; ++c) scale(acc[c], f0);
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          if (pl[p] == 0.f) continue;
          const float f = part_weight(pm[p], pl[p], M);
          L = fmaf(pl[p], f, L);
#pragma unroll
          for (int c = 0; c < kC; ++c)
            if (c0 + c * step < d4) add_scaled(acc[c], v[p][c], f);
        }
      }
      const float inv = 1.f / L;
      const float lse = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (c0 + c * step < d4)
          store(row, (c0 + c * step) * 4,
                L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                         : make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv,
                                       acc[c].w * inv),
                lse);
    }
  }
}

}  // namespace attn
}  // namespace kvc
