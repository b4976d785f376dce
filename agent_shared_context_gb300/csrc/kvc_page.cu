// kvc_page.cu -- the bookkeeping of a paged cache on the GPU: the plan of a
// step (block tables, slots and positions from the requests' lengths) and the
// write of K and V rows into their pages.
//
// Plan.  Request r holds c_r tokens and brings n_r (-1: it is finished).  With
// exclusive sums over the requests in order,
//   need_r = ceil((c_r + n_r) / B) - ceil(c_r / B)   pages to take,
//   back_r = ceil(c_r / B) if finished               pages to return,
// the stack is free_pages[0 .. F) followed by the returned pages, and the i-th
// page taken in (request, block) order is the i-th from its top.  Nothing
// depends on another request but through these sums, so every CTA adds them up
// for itself in shared memory (R lengths from L2) and then fills its own slice
// of the new table entries, the returned pages and the tokens; one launch, no
// order between CTAs.  The state comes out in other buffers than it went in by
// (kv_lens, n_free); table rows and stack entries that the call reads are not
// those that it writes, so repeating the call repeats its result.
//
// Bound by launch and L2 latency for a step of a few requests, by the 12 bytes
// written per token for large admissions.  Measured: 16 requests with a token each
// 5.5 us, most of it the host's; 1,024 requests of which 100 end and the rest bring
// up to 1,024 tokens each, 465,000 in all, 8.8 us (5.8 MB: 0.86 us of HBM time; the
// sums over the requests and the search of each run of tokens are the rest).
#include "kvc_attn_sched.cuh"
#include "kvc_paged_internal.h"

namespace kvc {
namespace {

using attn::FastDiv;
using attn::fast_div;

constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 4;                // consecutive tokens of a thread
constexpr int kPlanWarps = kPlanThreads / 32;

// Sums stop at this instead of running over: nothing that large can be served.
constexpr uint32_t kMost = 0x7fffffffu;

__device__ __forceinline__ uint32_t add(uint32_t x, uint32_t y) { return min(x + y, kMost); }

// Replaces two numbers per thread by their sums over the threads before, and gives the
// totals.
__device__ __forceinline__ void block_sums(uint32_t* x, uint32_t* y, uint2* warp_sum,
                                           uint32_t* all_x, uint32_t* all_y) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, *x, o), v = __shfl_up_sync(0xffffffffu, *y, o);
    if (lane >= o) {
      *x = add(*x, u);
      *y = add(*y, v);
    }
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = make_uint2(*x, *y);
  __syncthreads();
  // every warp adds the warps up by itself
  uint2 t = lane < kPlanWarps ? warp_sum[lane] : make_uint2(0, 0);
#pragma unroll
  for (int o = 1; o < kPlanWarps; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, t.x, o), v = __shfl_up_sync(0xffffffffu, t.y, o);
    if (lane >= o) {
      t.x = add(t.x, u);
      t.y = add(t.y, v);
    }
  }
  *x = __shfl_up_sync(0xffffffffu, *x, 1);
  *y = __shfl_up_sync(0xffffffffu, *y, 1);
  if (lane == 0) *x = *y = 0;
  *all_x = __shfl_sync(0xffffffffu, t.x, kPlanWarps - 1);
  *all_y = __shfl_sync(0xffffffffu, t.y, kPlanWarps - 1);
  const uint32_t bx = __shfl_sync(0xffffffffu, t.x, warp > 0 ? warp - 1 : 0);
  const uint32_t by = __shfl_sync(0xffffffffu, t.y, warp > 0 ? warp - 1 : 0);
  if (warp > 0) {
    *x = add(*x, bx);
    *y = add(*y, by);
  }
}

// First index in [0, n) with end[index] > x (end is non-decreasing); n if none.
__device__ __forceinline__ int find_after(const int32_t* end, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

struct PlanShared {
  uint2 warp_sum[kPlanWarps];
  int32_t taken;
};

// Bytes of shared memory per request.
constexpr int kPlanBytes = 5 * 4 + 1;

// VEC: four consecutive tokens per thread.
template <bool VEC>
__global__ void __launch_bounds__(kPlanThreads)
    page_plan_kernel(const PlanArgs a, const FastDiv page) {
  extern __shared__ int32_t plan_smem[];
  __shared__ PlanShared sh;
  int32_t* tok_end = plan_smem;                 // [R] inclusive sums
  int32_t* need_end = tok_end + a.R;
  int32_t* back_end = need_end + a.R;
  int32_t* kv = back_end + a.R;                 // the lengths, and the new ones of good requests
  int32_t* fresh = kv + a.R;
  uint8_t* status = reinterpret_cast<uint8_t*>(fresh + a.R);
  const int tid = threadIdx.x;
  const int cap = a.width * a.B;                // <= 2^30
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  grid_wait();
  const int F = min(max(a.n_free_in[0], 0), a.P);
  auto blocks = [&](int n) { return fast_div(n + a.B - 1, page); };

  // tokens and returned pages
  uint32_t toks = 0, back = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = a.new_lens[r], c = a.kv_in[r];
    const bool bad = n < -1 || c < 0 || c > cap;
    kv[r] = c;
    fresh[r] = bad ? 0 : n;
    status[r] = bad ? KVC_PLAN_INVALID : KVC_PLAN_OK;
    toks = add(toks, bad || n < 0 ? 0 : n);
    back = add(back, !bad && n == -1 ? blocks(c) : 0);
  }
  uint32_t all_toks, all_back;
  block_sums(&toks, &back, sh.warp_sum, &all_toks, &all_back);
  // the pages asked for
  uint32_t need = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = fresh[r], c = kv[r];
    toks = add(toks, n > 0 ? n : 0);
    back = add(back, n == -1 ? blocks(c) : 0);
    tok_end[r] = static_cast<int>(toks);
    back_end[r] = static_cast<int>(back);
    if (n > 0) {
      if (static_cast<uint32_t>(c) + n > static_cast<uint32_t>(cap))
        status[r] = KVC_PLAN_ROW_FULL;
      else if (toks > static_cast<uint32_t>(a.max_tokens))
        status[r] = KVC_PLAN_TOKENS;
      else
        need = add(need, blocks(c + n) - blocks(c));
    }
  }
  if (tid == 0) sh.taken = 0;
  uint32_t unused = 0, all_need, none;
  block_sums(&need, &unused, sh.warp_sum, &all_need, &none);
  const uint32_t avail = add(F, all_back);
  uint32_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = fresh[r], c = kv[r];
    uint32_t k = 0;
    if (status[r] == KVC_PLAN_OK && n > 0) k = blocks(c + n) - blocks(c);
    need = add(need, k);
    if (k > 0 && need > avail)
      status[r] = KVC_PLAN_NO_PAGES;
    else if (k > 0)
      mine = need;
    need_end[r] = static_cast<int>(need);
  }
  if (mine > 0) atomicMax(&sh.taken, static_cast<int>(mine));
  __syncthreads();
  const int taken = sh.taken;
  const int left = static_cast<int>(avail) - taken;   // pages on the stack afterwards
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;

  // entry i of the returned pages, in (request, block) order
  auto returned = [&](int i) -> int {
    const int r = find_after(back_end, a.R, i);
    return a.table[static_cast<int64_t>(r) * a.width + (i - (r > 0 ? back_end[r - 1] : 0))];
  };
  // page of the i-th allocation
  auto pop = [&](int i) -> int {
    const int q = static_cast<int>(avail) - 1 - i;
    return q < F ? a.free_pages[q] : returned(q - F);
  };
  // returned pages that stay on the stack
  for (int64_t q = F + first; q < left && q < a.P; q += step)
    a.free_pages[q] = returned(static_cast<int>(q) - F);
  // new table entries
  for (int64_t i = first; i < taken; i += step) {
    const int r = find_after(need_end, a.R, static_cast<int>(i));
    const int before = r > 0 ? need_end[r - 1] : 0;
    a.table[static_cast<int64_t>(r) * a.width + blocks(kv[r]) + (static_cast<int>(i) - before)] =
        pop(static_cast<int>(i));
  }
  // tokens: a thread walks on from the request of its first one
  constexpr int kT = VEC ? kPlanTokens : 1;
  for (int64_t i0 = first * kT; i0 < a.max_tokens; i0 += step * kT) {
    int64_t slot[kT];
    int pos[kT];
    int r = i0 < all_toks ? find_after(tok_end, a.R, static_cast<int>(i0)) : a.R;
    int seen_blk = -1, seen_r = -1, page_id = 0;
#pragma unroll
    for (int j = 0; j < kT; ++j) {
      const int64_t i = i0 + j;
      slot[j] = -1;
      pos[j] = -1;
      if (i >= all_toks || i >= a.max_tokens) continue;
      while (tok_end[r] <= i) ++r;
      if (status[r] != KVC_PLAN_OK) continue;
      const int c = kv[r];
      pos[j] = c + static_cast<int>(i) - (r > 0 ? tok_end[r - 1] : 0);
      const int blk = fast_div(pos[j], page), held = blocks(c);
      if (blk != seen_blk || r != seen_r) {
        page_id = blk < held ? a.table[static_cast<int64_t>(r) * a.width + blk]
                             : pop((r > 0 ? need_end[r - 1] : 0) + blk - held);
        seen_blk = blk;
        seen_r = r;
      }
      slot[j] = static_cast<int64_t>(page_id) * a.B + (pos[j] - blk * a.B);
    }
    if (VEC && i0 + kT <= a.max_tokens) {
      longlong2* s2 = reinterpret_cast<longlong2*>(a.slots + i0);
#pragma unroll
      for (int j = 0; j + 1 < kT; j += 2) s2[j / 2] = make_longlong2(slot[j], slot[j + 1]);
      if (VEC)
        *reinterpret_cast<int4*>(a.positions + i0) =
            make_int4(pos[0], pos[1 % kT], pos[2 % kT], pos[3 % kT]);
    } else {
#pragma unroll
      for (int j = 0; j < kT; ++j)
        if (i0 + j < a.max_tokens) {
          a.slots[i0 + j] = slot[j];
          a.positions[i0 + j] = pos[j];
        }
    }
  }
  // the requests' own values
  for (int64_t r = first; r < a.R; r += step) {
    const int n = fresh[r], c = kv[r], st = status[r];
    a.status[r] = st;
    a.kv_out[r] = st != KVC_PLAN_OK ? c : (n == -1 ? 0 : c + n);
    a.q_start[r + 1] = min(tok_end[r], a.max_tokens);
  }
  if (first == 0) {
    a.q_start[0] = 0;
    a.n_free_out[0] = left;
  }
}

// ------------------------------------------------------------------- write
constexpr int kWriteThreads = 256;
constexpr int kWriteVecs = 4;                    // vectors per thread, all in flight

// One CTA copies a run of rows of one (layer, head) of K or V.  Bound by HBM:
// each 16-byte vector is read once and written once, past the caches.  BIG: row
// or slot numbers beyond 31 bits (64-bit divisions made the copy wait for
// arithmetic: two trajectories of 10,240 tokens took 1,051 us with them; they take
// 746 us now, 5.37 GB at 7.2 TB/s, 1.06 of a device copy's rate).  A step's rows of
// one layer, 16 tokens or 2,048, take 7 to 8.5 us, most of it the host's.
template <bool BIG>
__global__ void __launch_bounds__(kWriteThreads)
    page_write_kernel(const WriteArgs a, const FastDiv per_src, const FastDiv per_page,
                      const FastDiv per_row) {
  const int kv = blockIdx.z;
  const int l = blockIdx.y / a.H, h = blockIdx.y - l * a.H;
  const int rows_cta = kWriteThreads * kWriteVecs / a.vec_row;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_cta;
  const int64_t e = a.elem;
  const char* src = static_cast<const char*>(a.src[kv].base) +
                    (l * a.src[kv].s_layer + h * a.src[kv].s_head) * e;
  char* pool = static_cast<char*>(a.pool[kv].base) +
               ((a.L0 + l) * a.pool[kv].s_layer + h * a.pool[kv].s_head) * e;
  grid_wait();
  uint4 v[kWriteVecs];
  int64_t slot[kWriteVecs];
  int col[kWriteVecs];
#pragma unroll
  for (int k = 0; k < kWriteVecs; ++k) {
    const int i = threadIdx.x + k * kWriteThreads;
    const int row = fast_div(i, per_row);
    col[k] = (i - row * a.vec_row) * 16;
    const int64_t n = row0 + row;
    slot[k] = -1;
    if (row < rows_cta && n < a.rows) {
      slot[k] = a.slots[n];
      const int64_t r = BIG ? n / a.T : fast_div(static_cast<int>(n), per_src);
      v[k] = __ldcs(reinterpret_cast<const uint4*>(
          src + (r * a.src[kv].s_req + (n - r * a.T) * a.src[kv].s_tok) * e + col[k]));
    }
  }
#pragma unroll
  for (int k = 0; k < kWriteVecs; ++k) {
    if (slot[k] < 0 || slot[k] >= a.n_slots) continue;
    const int64_t page = BIG ? slot[k] / a.B : fast_div(static_cast<int>(slot[k]), per_page);
    __stcs(reinterpret_cast<uint4*>(
               pool + (page * a.pool[kv].s_req + (slot[k] - page * a.B) * a.pool[kv].s_tok) * e +
               col[k]),
           v[k]);
  }
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const size_t smem = static_cast<size_t>(a.R) * kPlanBytes;
  // Four tokens to a thread, with 16-byte stores, once every thread of the GPU has more
  // than one: in a replayed graph 4.1 against 3.4 us for 16 tokens, 8.8 against 10.4 us
  // for 465,000.
  const bool vec = a.max_tokens > di.sm_count * kPlanThreads &&
                   (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0 &&
                   (reinterpret_cast<uintptr_t>(a.positions) & 15) == 0;
  auto* fn = vec ? page_plan_kernel<true> : page_plan_kernel<false>;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int64_t per = vec ? kPlanTokens : 1;
  const int64_t runs = (a.max_tokens + per - 1) / per;
  int64_t grid = ((runs > a.R ? runs : a.R) + kPlanThreads - 1) / kPlanThreads;
  if (grid > di.sm_count) grid = di.sm_count;
  if (grid < 1) grid = 1;
  return launch_early(fn, dim3(static_cast<unsigned>(grid)), kPlanThreads, smem, stream, a,
                      attn::make_fastdiv(a.B));
}

cudaError_t launch_page_write(const WriteArgs& a, cudaStream_t stream) {
  const int64_t rows_cta = kWriteThreads * kWriteVecs / a.vec_row;
  const dim3 grid(static_cast<unsigned>((a.rows + rows_cta - 1) / rows_cta),
                  static_cast<unsigned>(a.nl * a.H), 2);
  const int64_t most = int64_t(1) << 31;
  auto* fn =
      a.rows >= most || a.n_slots >= most ? page_write_kernel<true> : page_write_kernel<false>;
  return launch_early(fn, grid, kWriteThreads, 0, stream, a, attn::make_fastdiv(a.T),
                      attn::make_fastdiv(a.B), attn::make_fastdiv(a.vec_row));
}

}  // namespace kvc
