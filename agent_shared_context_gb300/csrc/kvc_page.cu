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
// written per token for large admissions.
#include "kvc_paged_internal.h"

namespace kvc {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;

// Inclusive sum over the CTA of one int64 per thread; *total is the sum of all.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* warp_sum, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    const int64_t x = warp_sum[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return v + before;
}

__device__ __forceinline__ int clamp_int(int64_t v) {
  return v > 0x7fffffff ? 0x7fffffff : static_cast<int>(v);
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
  int64_t warp_sum[kPlanWarps];
  int32_t taken;
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  __shared__ PlanShared sh;
  int32_t* tok_end = plan_smem;                 // [R] inclusive sums
  int32_t* need_end = tok_end + a.R;
  int32_t* back_end = need_end + a.R;
  uint8_t* status = reinterpret_cast<uint8_t*>(back_end + a.R);
  const int tid = threadIdx.x;
  const int64_t cap = static_cast<int64_t>(a.width) * a.B;
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  const int F = min(max(a.n_free_in[0], 0), a.P);

  // tokens and returned pages
  int64_t toks = 0, back = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = a.new_lens[r], c = a.kv_in[r];
    const bool bad = n < -1 || c < 0 || c > cap;
    toks += bad || n < 0 ? 0 : n;
    back += !bad && n == -1 ? (c + a.B - 1) / a.B : 0;
  }
  int64_t all_toks, all_back, all_need;
  int64_t t = block_sum(toks, sh.warp_sum, &all_toks) - toks;
  int64_t b = block_sum(back, sh.warp_sum, &all_back) - back;
  // status before pages run short, and the pages asked for
  int64_t need = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = a.new_lens[r], c = a.kv_in[r];
    const bool bad = n < -1 || c < 0 || c > cap;
    const int64_t nn = bad || n < 0 ? 0 : n;
    t += nn;
    b += !bad && n == -1 ? (c + a.B - 1) / a.B : 0;
    int st = KVC_PLAN_OK;
    if (bad)
      st = KVC_PLAN_INVALID;
    else if (c + nn > cap)
      st = KVC_PLAN_ROW_FULL;
    else if (n > 0 && t > a.max_tokens)
      st = KVC_PLAN_TOKENS;
    else if (n > 0)
      need += (c + nn + a.B - 1) / a.B - (c + a.B - 1) / a.B;
    tok_end[r] = clamp_int(t);
    back_end[r] = clamp_int(b);
    status[r] = static_cast<uint8_t>(st);
  }
  int64_t e = block_sum(need, sh.warp_sum, &all_need) - need;
  const int64_t avail = F + all_back;
  if (tid == 0) sh.taken = 0;
  __syncthreads();
  int taken = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = a.new_lens[r], c = a.kv_in[r];
    int64_t k = 0;
    if (status[r] == KVC_PLAN_OK && n > 0)
      k = (c + static_cast<int64_t>(n) + a.B - 1) / a.B - (c + a.B - 1) / a.B;
    e += k;
    if (k > 0 && e > avail)
      status[r] = KVC_PLAN_NO_PAGES;
    else if (k > 0)
      taken = clamp_int(e);
    need_end[r] = clamp_int(e);
  }
  if (taken > 0) atomicMax(&sh.taken, taken);
  __syncthreads();
  taken = sh.taken;
  const int64_t left = avail - taken;           // pages on the stack afterwards
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;

  // page of the i-th allocation
  auto pop = [&](int i) -> int {
    const int64_t p = avail - 1 - i;
    if (p < F) return a.free_pages[p];
    const int k = static_cast<int>(p - F);
    const int r = find_after(back_end, a.R, k);
    const int before = r > 0 ? back_end[r - 1] : 0;
    return a.table[static_cast<int64_t>(r) * a.width + (k - before)];
  };
  // returned pages that stay on the stack
  for (int64_t p = F + first; p < left && p < a.P; p += step) {
    const int k = static_cast<int>(p - F);
    const int r = find_after(back_end, a.R, k);
    const int before = r > 0 ? back_end[r - 1] : 0;
    a.free_pages[p] = a.table[static_cast<int64_t>(r) * a.width + (k - before)];
  }
  // new table entries
  for (int64_t i = first; i < taken; i += step) {
    const int r = find_after(need_end, a.R, static_cast<int>(i));
    const int before = r > 0 ? need_end[r - 1] : 0;
    const int held = (a.kv_in[r] + a.B - 1) / a.B;
    a.table[static_cast<int64_t>(r) * a.width + held + (static_cast<int>(i) - before)] =
        pop(static_cast<int>(i));
  }
  // tokens
  for (int64_t i = first; i < a.max_tokens; i += step) {
    int64_t slot = -1;
    int pos = -1;
    if (i < all_toks) {
      const int r = find_after(tok_end, a.R, static_cast<int>(i));
      if (status[r] == KVC_PLAN_OK) {
        const int c = a.kv_in[r];
        pos = c + static_cast<int>(i) - (r > 0 ? tok_end[r - 1] : 0);
        const int blk = pos / a.B, held = (c + a.B - 1) / a.B;
        const int page = blk < held ? a.table[static_cast<int64_t>(r) * a.width + blk]
                                    : pop((r > 0 ? need_end[r - 1] : 0) + blk - held);
        slot = static_cast<int64_t>(page) * a.B + (pos - blk * a.B);
      }
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  // the requests' own values
  for (int64_t r = first; r < a.R; r += step) {
    const int n = a.new_lens[r], c = a.kv_in[r], st = status[r];
    a.status[r] = st;
    a.kv_out[r] = st != KVC_PLAN_OK ? c : (n == -1 ? 0 : c + n);
    a.q_start[r + 1] = min(tok_end[r], a.max_tokens);
  }
  if (first == 0) {
    a.q_start[0] = 0;
    a.n_free_out[0] = clamp_int(left);
  }
}

// ------------------------------------------------------------------- write
constexpr int kWriteThreads = 256;
constexpr int kWriteVecs = 4;                    // vectors per thread, all in flight

// One CTA copies a run of rows of one (layer, head) of K or V.  Bound by HBM:
// each 16-byte vector is read once and written once.
__global__ void __launch_bounds__(kWriteThreads) page_write_kernel(const WriteArgs a) {
  const int kv = blockIdx.z;
  const int l = blockIdx.y / a.H, h = blockIdx.y - l * a.H;
  const int64_t rows_cta = kWriteThreads * kWriteVecs / a.vec_row;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_cta;
  const int64_t e = a.elem;
  const char* src = static_cast<const char*>(a.src[kv].base) +
                    (l * a.src[kv].s_layer + h * a.src[kv].s_head) * e;
  char* pool = static_cast<char*>(a.pool[kv].base) +
               ((a.L0 + l) * a.pool[kv].s_layer + h * a.pool[kv].s_head) * e;
  uint4 v[kWriteVecs];
  int64_t at[kWriteVecs];
#pragma unroll
  for (int k = 0; k < kWriteVecs; ++k) {
    const int i = threadIdx.x + k * kWriteThreads;
    const int row = i / a.vec_row, c = i - row * a.vec_row;
    const int64_t n = row0 + row;
    at[k] = -1;
    if (row < rows_cta && n < a.rows) {
      const int64_t slot = a.slots[n];
      if (slot >= 0 && slot < a.n_slots) {
        const int64_t r = n / a.T, t = n - r * a.T;
        v[k] = *reinterpret_cast<const uint4*>(
            src + (r * a.src[kv].s_req + t * a.src[kv].s_tok) * e + c * 16);
        const int64_t page = slot / a.B;
        at[k] = (page * a.pool[kv].s_req + (slot - page * a.B) * a.pool[kv].s_tok) * e + c * 16;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kWriteVecs; ++k)
    if (at[k] >= 0) *reinterpret_cast<uint4*>(pool + at[k]) = v[k];
}

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const size_t smem = static_cast<size_t>(a.R) * 13;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int64_t most = a.max_tokens > a.R ? a.max_tokens : a.R;
  int64_t grid = (most + kPlanThreads - 1) / kPlanThreads;
  if (grid > di.sm_count) grid = di.sm_count;
  if (grid < 1) grid = 1;
  page_plan_kernel<<<static_cast<int>(grid), kPlanThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_page_write(const WriteArgs& a, cudaStream_t stream) {
  const int64_t rows_cta = kWriteThreads * kWriteVecs / a.vec_row;
  const dim3 grid(static_cast<unsigned>((a.rows + rows_cta - 1) / rows_cta),
                  static_cast<unsigned>(a.nl * a.H), 2);
  page_write_kernel<<<grid, kWriteThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
