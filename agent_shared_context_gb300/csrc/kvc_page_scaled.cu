// kvc_page_scaled.cu -- K and V rows into pages of 8-bit numbers (kvc_page_write_scaled).
//
// A block of rows of one layer and head shares a power of two 2^e: with m its largest
// finite magnitude, e is the least with m <= 448 2^e, and a number is x 2^-e rounded to
// e4m3 (4 bits of exponent, 3 of mantissa), to nearest and ties to even.  The product
// is exact, so there is one rounding.  A block that takes on a larger e divides its
// numbers by a power of two: that too is exact but for those that leave the normal
// range.
//
// One CTA has a window of 128 tokens of one (layer, head) of K or V.  Each warp holds
// 16 rows in registers from the first load to the store, so a row is read once.  In
// shared memory: the tokens' slots, from which every token finds the first one of its
// block in the call (its leader), and the blocks' largest magnitudes at their leaders.
// A block belongs to the window of its leader: that CTA also reads its rows behind the
// window (127 at most), and leaves those of the window before alone.
//
// Bound by HBM: 2 bytes read and 1 written per element.  Rows are read past L1 and
// written as whole 32-byte sectors.  Measured: two trajectories of 10,240 tokens, 32
// layers, 8 heads of 128, blocks of 32, 582 us, 6.9 TB/s (with a maximum, a slot and an
// address worked out for each row by itself 1,074 us: three of four cycles issued an
// instruction).  That is for rows in step with their blocks, 16 of which lie in one block;
// others are still worked out row by row.  With 16 layers: blocks of 16 in step 288 us, 7.0
// TB/s; from rows 5 and 42 on 511 us, 3.9; of 10,250 tokens, one trajectory of two in step, 393 us.
// One layer, in a replayed graph: a step's 16 tokens 6.1 us, 2,048 tokens 11.2 (a chain of
// slots, leaders, maxima, exponents and stores, with barriers between); by itself a call
// is the host's 15 to 18.
#include <cuda_bf16.h>

#include "kvc_attn_sched.cuh"
#include "kvc_paged_internal.h"
#include "kvc_scaled.cuh"

namespace kvc {
namespace {

using attn::FastDiv;
using attn::fast_div;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWarpRows = 16;
constexpr int kWindow = kWarps * kWarpRows;
constexpr int kHalo = kMaxScaleBlock - 1;      // tokens of a block before and after one

struct ScaledWrite {
  WriteArgs w;
  uint8_t* exps[2];
  int64_t e_page, e_layer, e_head;
  int32_t block, keep;
  FastDiv per_src, per_page, per_block;
};

// Bits of 2^-e, -100 <= e <= 119.
__device__ __forceinline__ float pow2_neg(int e) { return __int_as_float((127 - e) << 23); }

// Least exponent for a largest magnitude given as bf16 bits (finite).
__device__ __forceinline__ int exponent_for(uint32_t bits) {
  if (bits < 0x0080u) return kScaleExpMin;                // zero or below 2^-126
  // m = 1.f 2^k; 448 = 1.75 2^8
  const int k = static_cast<int>(bits >> 7) - 127;
  const int e = k - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
  return min(max(e, kScaleExpMin), kScaleExpMax);
}

// Eight bf16 numbers times f as e4m3; with `odd`, infinities become NaN.
__device__ __forceinline__ uint2 quantize8(uint4 v, float f, bool odd) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(x[i] << 16) * f, hi = __uint_as_float(x[i] & 0xffff0000u) * f;
    q[i] = pack_e4m3(lo, hi);
    if (odd) {
      if ((x[i] & 0x7f80u) == 0x7f80u) q[i] |= 0x007fu;
      if ((x[i] & 0x7f800000u) == 0x7f800000u) q[i] |= 0x7f00u;
    }
  }
  return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}

template <int D, bool BIG>
__global__ void __launch_bounds__(kThreads) page_write_scaled_kernel(const __grid_constant__ ScaledWrite p) {
  constexpr int kLanes = D / 8;                    // of a row, 16 bytes each
  constexpr int kAtOnce = 32 / kLanes;             // rows of a warp's load
  constexpr int kLoads = kWarpRows / kAtOnce;
  constexpr int kSpan = kHalo + kWindow + kHalo;
  __shared__ int64_t slot_of[kSpan];               // token n0 - kHalo + i
  __shared__ int64_t to_of[kSpan];                 // byte offset of its row in the pool
  __shared__ uint8_t row_of[kSpan];                // row in its block
  __shared__ uint32_t top[kWindow];                // at the leaders: largest magnitude,
  __shared__ int32_t exp_new[kWindow];             // the block's exponent
  __shared__ int32_t exp_up[kWindow];              // and by how much it grew (-1: began anew)
  __shared__ int16_t leader[kWindow + kHalo];      // of the window's tokens and those behind
  __shared__ uint8_t odd_row[kWindow + kHalo];

  const WriteArgs& a = p.w;
  const int kv = blockIdx.z;
  const int l = blockIdx.y / a.H, h = blockIdx.y - l * a.H;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kWindow;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / kLanes, col = lane % kLanes;
  const char* src = static_cast<const char*>(a.src[kv].base) +
                    (l * a.src[kv].s_layer + h * a.src[kv].s_head) * 2 + col * 16;
  uint8_t* pool = static_cast<uint8_t*>(a.pool[kv].base) + (a.L0 + l) * a.pool[kv].s_layer +
                  h * a.pool[kv].s_head;
  uint8_t* exps = p.exps[kv] + (a.L0 + l) * p.e_layer + h * p.e_head;

  auto row_at = [&](int64_t n) -> const uint4* {
    const int64_t r = BIG ? n / a.T : fast_div(static_cast<int>(n), p.per_src);
    return reinterpret_cast<const uint4*>(src + (r * a.src[kv].s_req +
                                                 (n - r * a.T) * a.src[kv].s_tok) * 2);
  };
  auto page_of = [&](int64_t s) -> int64_t {
    return BIG ? s / a.B : fast_div(static_cast<int>(s), p.per_page);
  };
  // largest magnitude of a row over its lanes, bits of infinities and NaNs included
  auto row_top = [&](const uint4& v) -> uint32_t {
    uint32_t m = max_abs2(max_abs2(max_abs2(max_abs2(0, v.x), v.y), v.z), v.w);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m & 0xffffu, m >> 16);
  };
  // the same without infinities and NaNs, where there are any
  auto finite_top = [&](const uint4& v) -> uint32_t {
    uint32_t m = 0;
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = x[i] & 0x7fffu, hi = (x[i] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) m = max(m, lo);
      if (hi < 0x7f80u) m = max(m, hi);
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  };

  grid_wait();
  uint4 v[kLoads];
  const int64_t first = n0 + warp * kWarpRows;
  const int64_t r0 = BIG ? first / a.T : fast_div(static_cast<int>(first), p.per_src);
  if (first + kWarpRows <= a.rows && first - r0 * a.T + kWarpRows <= a.T) {
    // all of one source: the addresses are a step apart
    const char* from = src + (r0 * a.src[kv].s_req + (first - r0 * a.T + sub) * a.src[kv].s_tok) * 2;
    const int64_t step = kAtOnce * a.src[kv].s_tok * 2;
#pragma unroll
    for (int j = 0; j < kLoads; ++j, from += step) v[j] = __ldcs(reinterpret_cast<const uint4*>(from));
  } else {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int64_t n = first + j * kAtOnce + sub;
      v[j] = n < a.rows ? __ldcs(row_at(n)) : make_uint4(0, 0, 0, 0);
    }
  }
  // the tokens that share a block with one of the window's
  const int reach = p.block - 1;
  for (int i = kHalo - reach + threadIdx.x; i < kHalo + kWindow + reach; i += kThreads) {
    const int64_t n = n0 - kHalo + i;
    int64_t s = n >= 0 && n < a.rows ? a.slots[n] : -1;
    if (s >= a.n_slots) s = -1;
    int row = 0;
    if (s >= 0) {
      const int64_t page = page_of(s);
      const int in_page = static_cast<int>(s - page * a.B);
      row = in_page - fast_div(in_page, p.per_block) * p.block;
      to_of[i] = page * a.pool[kv].s_req + in_page * a.pool[kv].s_tok;
    }
    slot_of[i] = s < 0 ? -1 : s;
    row_of[i] = static_cast<uint8_t>(row);
  }
  if (threadIdx.x < kWindow) top[threadIdx.x] = 0;
  __syncthreads();

  // Every token's leader: the first token of the call in its block, which lie as the rows do.
  for (int i = threadIdx.x; i < kWindow + reach; i += kThreads) {
    const int at = i + kHalo;
    const int64_t s = slot_of[at];
    int lead = -1;
    if (s >= 0) {
      int m = at - row_of[at];
      while (slot_of[m] != s - (at - m)) ++m;      // ends at `at`
      lead = m - kHalo;
      if (lead >= kWindow) lead = -1;
    }
    leader[i] = static_cast<int16_t>(lead < 0 ? -1 : lead);    // -1: another window's, or none
  }
  __syncthreads();

  // Where a warp's rows are all of one block, as in a long source whose 16 rows begin where
  // blocks (of a multiple of 16 rows) do, they have one maximum, one exponent and no place of their own to look up but the pool's.
  const int mine = leader[warp * kWarpRows + (lane & (kWarpRows - 1))];
  const int lead0 = __shfl_sync(0xffffffffu, mine, 0);
  const bool together = __all_sync(0xffffffffu, mine == lead0 && mine >= 0);
  bool odd_any = false;
  if (together) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      m = max_abs2(max_abs2(max_abs2(max_abs2(m, v[j].x), v[j].y), v[j].z), v[j].w);
    m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    odd_any = m >= 0x7f80u;
    if (!odd_any && lane == 0) atomicMax(&top[lead0], m);
  }
  if (!together || odd_any) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = warp * kWarpRows + j * kAtOnce + sub;
      uint32_t m = row_top(v[j]);
      const bool odd = m >= 0x7f80u;
      if (__any_sync(0xffffffffu, odd)) {
        const uint32_t f = finite_top(v[j]);
        if (odd) m = f;
      }
      if (col == 0) {
        odd_row[i] = odd;
        if (leader[i] >= 0) atomicMax(&top[leader[i]], m);
      }
    }
  }
  // rows behind the window (its last block's): few, looked at now and read again below
  for (int i0 = kWindow + warp * kAtOnce; i0 < kWindow + p.block - 1; i0 += kWarps * kAtOnce) {
    const int i = i0 + sub;
    const bool mine = i < kWindow + p.block - 1 && leader[i] >= 0;
    if (!__any_sync(0xffffffffu, mine)) continue;
    const uint4 x = mine ? *row_at(n0 + i) : make_uint4(0, 0, 0, 0);
    uint32_t m = row_top(x);
    const bool odd = m >= 0x7f80u;
    if (__any_sync(0xffffffffu, odd)) {
      const uint32_t f = finite_top(x);
      if (odd) m = f;
    }
    if (mine && col == 0) {
      odd_row[i] = odd;
      atomicMax(&top[leader[i]], m);
    }
  }
  __syncthreads();

  // the blocks' exponents
  int grown = 0;
  if (threadIdx.x < kWindow && leader[threadIdx.x] == static_cast<int>(threadIdx.x)) {
    const int at = threadIdx.x + kHalo;
    const int64_t s = slot_of[at], page = page_of(s);
    const int in_page = static_cast<int>(s - page * a.B);
    uint8_t* where = exps + page * p.e_page + fast_div(in_page, p.per_block);
    int e = exponent_for(top[threadIdx.x]), up = -1;
    if (p.keep || row_of[at] != 0) {
      const int old = min(static_cast<int>(*where) - 127, kScaleExpMax);
      e = max(e, old);
      up = e - old;
    }
    exp_new[threadIdx.x] = e;
    exp_up[threadIdx.x] = up;
    *where = static_cast<uint8_t>(e + 127);
    grown = up > 0;
  }
  grown = __syncthreads_or(grown);

  uint8_t* to = pool + col * 8;
  auto store = [&](int i, const uint4& x) {
    if (leader[i] < 0) return;
    const uint2 q = quantize8(x, pow2_neg(exp_new[leader[i]]), odd_row[i] != 0);
    __stcs(reinterpret_cast<uint2*>(to + to_of[i + kHalo]), q);
  };
  if (together && !odd_any) {
    const float f = pow2_neg(exp_new[lead0]);
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      __stcs(reinterpret_cast<uint2*>(to + to_of[kHalo + warp * kWarpRows + j * kAtOnce + sub]),
             quantize8(v[j], f, false));
  } else {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) store(warp * kWarpRows + j * kAtOnce + sub, v[j]);
  }
  for (int i = kWindow + warp * kAtOnce + sub; i < kWindow + p.block - 1; i += kWarps * kAtOnce)
    if (leader[i] >= 0) store(i, *row_at(n0 + i));

  if (!grown) return;
  // the other rows of blocks whose exponent grew
  for (int i = warp; i < kWindow; i += kWarps) {
    if (leader[i] != i || exp_up[i] <= 0) continue;
    const int at = i + kHalo;
    const int64_t s = slot_of[at], page = page_of(s);
    const int in_page = static_cast<int>(s - page * a.B);
    const int first = in_page - row_of[at];        // the block's first row in the page
    const int rows = min(p.block, a.B - first);
    // numbers times 2^-up; beyond 2^-24 all of them are zero (or NaN)
    const float f = pow2_neg(min(exp_up[i], 100));
    for (int j = sub; j < rows; j += kAtOnce) {
      const int m = at - row_of[at] + j;           // the token that this row would be
      if (m >= kHalo - reach && m < kHalo + kWindow + reach && slot_of[m] == s - row_of[at] + j)
        continue;
      uint2* where = reinterpret_cast<uint2*>(pool + page * a.pool[kv].s_req +
                                              (first + j) * a.pool[kv].s_tok + col * 8);
      const uint2 old = *where;
      *where = make_uint2(rescale4(old.x, f), rescale4(old.y, f));
    }
  }
}

}  // namespace

cudaError_t launch_page_write_scaled(const WriteArgs& w, const ScaleArgs& sc, bool keep,
                                     cudaStream_t stream) {
  ScaledWrite p{};
  p.w = w;
  for (int i = 0; i < 2; ++i) p.exps[i] = sc.exps[i];
  p.e_page = sc.s_page;
  p.e_layer = sc.s_layer;
  p.e_head = sc.s_head;
  p.block = sc.block;
  p.keep = keep;
  p.per_src = attn::make_fastdiv(w.T);
  p.per_page = attn::make_fastdiv(w.B);
  p.per_block = attn::make_fastdiv(sc.block);
  const dim3 grid(static_cast<unsigned>((w.rows + kWindow - 1) / kWindow),
                  static_cast<unsigned>(w.nl * w.H), 2);
  const int64_t most = int64_t(1) << 31;
  const bool big = w.rows >= most || w.n_slots >= most;
  auto* fn = w.vec_row == 4 ? (big ? page_write_scaled_kernel<64, true> : page_write_scaled_kernel<64, false>)
                            : (big ? page_write_scaled_kernel<128, true> : page_write_scaled_kernel<128, false>);
  return launch_early(fn, grid, kThreads, 0, stream, p);
}

}  // namespace kvc
