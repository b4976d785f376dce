// kvc_attn_decode.cu -- attention of single new tokens over a paged cache
// (bf16, d = 64 or 128, up to 16 query heads per KV head).
//
// Decoding reads every key and value once and computes little with them: it is
// bound by HBM, and a small batch by latency.  A row tile of 128 rows and a
// pipeline of roles would be idle for the most part, so here a row tile has the
// 8 rows (16 where the group needs them) that a warp-level MMA (m16n8k16) takes
// as its N, keys and columns of d being its M, and every warp is on its own: it
// copies its 32 keys of a 128-key tile into its own ring in shared memory
// (cp.async, three stages, no barrier with the other warps), forms S^T = K Q^T
// with Q^T in registers and O^T += V^T P^T, and keeps the running maximum, sum
// and output of its keys.  The four warps' results are joined at the end of an
// item.
//
// The mathematics is that of kvc_attn_f32.cu, P enters the product with V as two
// numbers (cut_bf16 and the rest of it): the tensor core has time for both.
//
// Rows of keys beyond the request's, or out of all rows' sight, are filled with
// zeros instead of being read, so what a page holds there cannot reach a sum.
// A tile that only some of the rows see (several new tokens) is looked through
// for infinities and NaNs; with one in it the product with V goes element by
// element and skips what a row does not see.
//
// The work is divided over a persistent grid as kvc_attn_sched.cuh says.
//
// Measured, 32 query heads on 8 of 128: 16 requests of 10,240 keys 109 us, 671 MB at
// 6.2 TB/s (asymptotically 7.2 TB/s and some 10 us of launch, division of the work,
// first loads and joining); one request of 131,072 keys 87 us, 6.1 TB/s; one of 777
// keys 9.0 us, all of it latency.  Of 64: 16 requests of 10,240 keys 61 us, 5.5 TB/s.
// Where the chunk kernel would be faster: launch rules below.
#include <cuda_bf16.h>

#include "kvc_attn_sched.cuh"
#include "kvc_attn_warp.cuh"
#include "kvc_paged_internal.h"
#include "kvc_ptx.cuh"

namespace kvc {
namespace {

using namespace attn;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;                  // keys of a warp's step
constexpr int kG = kKeys / 16;             // groups of 16, the MMA's M
constexpr int kTile = kKeys * kWarps;
constexpr int kSlotRows = 16;              // rows of a partial result
constexpr int kStages = 3;
constexpr int kMaxCtas = 320;
constexpr int kItemCost = 2;

struct DecodeArgs {
  AttnArgs a;
  SchedArgs s;
  FastDiv page;
};

template <int D, int NQ = 1>
struct Cfg {
  static constexpr int kRows = 8 * NQ;                            // rows of a tile
  static constexpr int kRowBytes = D * 2;
  static constexpr int kHalfStage = kKeys * kRowBytes;            // K or V of a step
  static constexpr int kWarpBytes = kStages * 2 * kHalfStage;
  static constexpr int kJoin = kWarps * kRows * (D + 2) * 4;      // O, m, l of every warp
  static constexpr int kSmem = kWarps * kWarpBytes + kJoin;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte unit `u` of key row `n`: the rows of a unit lie in
// different banks.
template <int D>
__device__ __forceinline__ uint32_t at(int n, int u) {
  return static_cast<uint32_t>(n * Cfg<D>::kRowBytes + ((u ^ (n & 7)) << 4));
}

// NQ: groups of eight rows of an item.
template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, D == 128 ? 1 : 2)
    attn_decode_kernel(const __grid_constant__ DecodeArgs p) {
  using C = Cfg<D, NQ>;
  constexpr int kRows = C::kRows;
  constexpr int kUnits = D / 8;                    // 16-byte units of a row
  constexpr int kRowsAtOnce = 32 / kUnits;         // rows of a warp's 32 units
  static_assert(kKeys <= 32 && kKeys % 16 == 0, "a lane looks up a key's page");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sched;
  __shared__ int32_t last;
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::kWarpBytes;
  float* join = reinterpret_cast<float*>(smem + kWarps * C::kWarpBytes);
  const int gr = lane >> 2, qc = lane & 3;         // row and pair of columns of a fragment

  grid_wait();
  Walker w = walker_begin<kThreads>(p.s, &sched, a.dev_status);
  int32_t* counters = static_cast<int32_t*>(a.workspace);
  float* slots = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kAttnCounterBytes);
  const size_t slot_n = slot_floats(kSlotRows, D);
  const __nv_bfloat16* pools[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
    pools[kv] = static_cast<const __nv_bfloat16*>(a.pool[kv].base) + a.layer * a.pool[kv].s_layer;
  bool bad_page = false;

  Item it;
  while (w.next(p.s, &it)) {
    const int rows = it.nt * a.G;
    const int any_hi = a.causal ? min(it.kv, it.pos0 + it.nt) : it.kv;
    const int any_lo = a.window > 0 ? max(0, it.pos0 + 1 - a.window) : 0;
    const int all_hi = a.causal ? min(it.kv, it.pos0 + 1) : it.kv;
    const int all_lo = a.window > 0 ? max(0, it.pos0 + it.nt - a.window) : 0;
    const int32_t* table = a.table + static_cast<int64_t>(it.r) * a.width;
    const __nv_bfloat16* src[2] = {pools[0] + it.h * a.pool[0].s_head,
                                   pools[1] + it.h * a.pool[1].s_head};

    // page of the lane's key of step t (-1: not to be read)
    auto page_of = [&](int t) -> int {
      const int tok = (it.tile0 + t) * kTile + warp * kKeys + lane;
      return t < it.ntiles && lane < kKeys && tok >= any_lo && tok < any_hi
                 ? table[fast_div(tok, p.page)]
                 : -1;
    };
    auto issue = [&](int t, int page) {
      if (t < it.ntiles) {
        const int tok = (it.tile0 + t) * kTile + warp * kKeys + lane;
        const bool seen = lane < kKeys && tok >= any_lo && tok < any_hi;
        if (seen && (page < 0 || page >= a.P)) {
          bad_page = true;
          page = -1;
        }
        const int in_page = tok - fast_div(tok, p.page) * a.B;
        const uint32_t dst = ring + (t % kStages) * 2 * C::kHalfStage;
#pragma unroll
        for (int j = 0; j < kKeys / kRowsAtOnce; ++j) {
          const int n = j * kRowsAtOnce + lane / kUnits, u = lane % kUnits;
          const int pg = __shfl_sync(0xffffffffu, page, n);
          const int64_t row = __shfl_sync(0xffffffffu, in_page, n);
          const bool real = pg >= 0;
          const int64_t pg64 = real ? pg : 0;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv)
            cp_async16(dst + kv * C::kHalfStage + at<D>(n, u),
                       real ? src[kv] + pg64 * a.pool[kv].s_req + row * a.pool[kv].s_tok + u * 8
                            : src[kv],
                       real);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };

    int pages = page_of(0);
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) {
      const int next = page_of(t + 1);
      issue(t, pages);
      pages = next;
    }

    // Q^T as the B operand: row gr of each eight, two columns of each 8
    uint32_t q[NQ][D / 16][2];
#pragma unroll
    for (int g8 = 0; g8 < NQ; ++g8) {
      const int row = g8 * 8 + gr, tok = row / a.G, g = row - tok * a.G;
      const bool has = row < rows;
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) +
                                (has ? (it.q0 + tok) * a.q_tok + (it.h * a.G + g) * a.q_head : 0);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          q[g8][k][c] =
              has ? *reinterpret_cast<const uint32_t*>(qr + k * 16 + c * 8 + qc * 2) : 0u;
    }
    // of the rows 8 g8 + 2 qc and the next, which the lane's results belong to
    float m[NQ][2], l[NQ][2];
    int key_lo[NQ][2], key_hi[NQ][2];
#pragma unroll
    for (int g8 = 0; g8 < NQ; ++g8)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pos = it.pos0 + min((g8 * 8 + qc * 2 + i) / a.G, it.nt - 1);
        key_hi[g8][i] = a.causal ? min(it.kv, pos + 1) : it.kv;
        key_lo[g8][i] = a.window > 0 ? max(0, pos - a.window + 1) : 0;
        m[g8][i] = -INFINITY;
        l[g8][i] = 0.f;
      }
    float o[NQ][D / 16][4];
#pragma unroll
    for (int g8 = 0; g8 < NQ; ++g8)
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[g8][n][c] = 0.f;

#pragma unroll 1
    for (int t = 0; t < it.ntiles; ++t) {
      const int next = page_of(t + kStages);
      issue(t + kStages - 1, pages);
      pages = next;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const int k0 = (it.tile0 + t) * kTile + warp * kKeys;
      const uint32_t sK = ring + (t % kStages) * 2 * C::kHalfStage, sV = sK + C::kHalfStage;
      if (k0 < any_hi && k0 + kKeys > any_lo) {
        // S^T = K Q^T
        float s[NQ][kG][4];
#pragma unroll
        for (int g8 = 0; g8 < NQ; ++g8)
#pragma unroll
          for (int n = 0; n < kG; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[g8][n][c] = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int n = 0; n < kG; ++n) {
            uint32_t f[4];       // keys 0-7, 8-15 with columns 0-7, then with columns 8-15
            ldmatrix4(sK + at<D>(n * 16 + (lane & 15), 2 * k + (lane >> 4)), f);
#pragma unroll
            for (int g8 = 0; g8 < NQ; ++g8) mma16816(s[g8][n], f, q[g8][k][0], q[g8][k][1]);
          }
        const bool whole = k0 >= all_lo && k0 + kKeys <= all_hi;
        uint32_t ph[NQ][kG][2], pl[NQ][kG][2];       // P^T and its remainder as B operands
#pragma unroll
        for (int g8 = 0; g8 < NQ; ++g8) {
          if (!whole) {
#pragma unroll
            for (int n = 0; n < kG; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int tok = k0 + n * 16 + (c >> 1) * 8 + gr, i = c & 1;
                if (tok < key_lo[g8][i] || tok >= key_hi[g8][i]) s[g8][n][c] = -INFINITY;
              }
          }
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(s[g8][0][i], s[g8][0][i + 2]);
#pragma unroll
            for (int n = 1; n < kG; ++n) top = fmaxf(top, fmaxf(s[g8][n][i], s[g8][n][i + 2]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float m_new = fmaxf(m[g8][i], top * a.scale_log2);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            f[i] = exp2_fast(m[g8][i] - ref);
            m[g8][i] = m_new;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < kG; ++n)
#pragma unroll
              for (int c = i; c < 4; c += 2) {
                s[g8][n][c] = exp2_fast(fmaf(s[g8][n][c], a.scale_log2, -ref));
                sum += s[g8][n][c];
              }
            l[g8][i] = l[g8][i] * f[i] + sum;
          }
#pragma unroll
          for (int n = 0; n < kG; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t p2 = ptx::pack_f32x2(__float_as_uint(s[g8][n][2 * h]),
                                                  __float_as_uint(s[g8][n][2 * h + 1]));
              const uint32_t u = ptx::cut_bf16(p2);
              ph[g8][n][h] = transpose8x8(u);
              pl[g8][n][h] = transpose8x8(ptx::rest_bf16(p2, u));
            }
          if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c) o[g8][n][c] *= f[c & 1];
          }
        }
        // value rows that some rows see and others do not
        bool odd = false;
        if (!whole && it.nt > 1) {
#pragma unroll 1
          for (int j = 0; j < kKeys / kRowsAtOnce; ++j) {
            const int n = j * kRowsAtOnce + lane / kUnits;
            uint4 v;
            const uint32_t addr = sV + at<D>(n, lane % kUnits);
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(addr));
            auto ones = [](uint32_t x) {
              return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
            };
            odd = odd || ones(v.x) || ones(v.y) || ones(v.z) || ones(v.w);
          }
          odd = __any_sync(0xffffffffu, odd);
        }
        if (!odd) {
          // O^T += V^T P^T
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int half = 0; half < kG; ++half) {
              uint32_t f[4];     // columns 0-7, 8-15 with keys 0-7, then with keys 8-15
              ldmatrix4_trans(
                  sV + at<D>(half * 16 + (lane & 7) + (lane >> 4) * 8, 2 * n + ((lane >> 3) & 1)), f);
#pragma unroll
              for (int g8 = 0; g8 < NQ; ++g8) {
                mma16816(o[g8][n], f, ph[g8][half][0], ph[g8][half][1]);
                mma16816(o[g8][n], f, pl[g8][half][0], pl[g8][half][1]);
              }
            }
        } else {
#pragma unroll 1
          for (int key = 0; key < kKeys; ++key) {
            const int from = (key & 7) * 4 + qc, tok = k0 + key;   // the lane with the key's P
#pragma unroll
            for (int g8 = 0; g8 < NQ; ++g8) {
              float pk[2] = {0.f, 0.f};
#pragma unroll
              for (int n = 0; n < kG; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const float x = __shfl_sync(0xffffffffu, s[g8][n][c], from);
                  if (n * 2 + (c >> 1) == (key >> 3)) pk[c & 1] = x;
                }
#pragma unroll
              for (int n = 0; n < D / 16; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint16_t v;
                  asm volatile("ld.shared.b16 %0, [%1];"
                               : "=h"(v)
                               : "r"(sV + at<D>(key, 2 * n + h) + gr * 2));
                  const float x = __uint_as_float(static_cast<uint32_t>(v) << 16);
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (tok >= key_lo[g8][i] && tok < key_hi[g8][i])
                      o[g8][n][2 * h + i] = fmaf(pk[i], x, o[g8][n][2 * h + i]);
                }
            }
          }
        }
      }
      __syncwarp();                                // the stage may be filled again
    }

    // the four warps' rows
#pragma unroll
    for (int g8 = 0; g8 < NQ; ++g8)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[g8][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = g8 * 8 + qc * 2 + i;
        if (row < rows) {
          float* mine = join + warp * kRows * (D + 2);
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) mine[row * D + n * 16 + h * 8 + gr] = o[g8][n][2 * h + i];
          if (gr == 0) {
            mine[kRows * D + row] = m[g8][i];
            mine[kRows * D + kRows + row] = sum;
          }
        }
      }
    parts(w, &it);
    __syncthreads();
    const bool whole_item = it.nparts == 1;
    float* part = slots + (static_cast<size_t>(blockIdx.x) * 2 + slot_of(it.part)) * slot_n;
    for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
      const int row = e / (D / 4), c4 = e - row * (D / 4);
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) M = fmaxf(M, join[v * kRows * (D + 2) + kRows * D + row]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float* from = join + v * kRows * (D + 2);
        const float lv = from[kRows * D + kRows + row];
        if (lv == 0.f) continue;
        const float f = part_weight(from[kRows * D + row], lv, M);
        const float4 x = *reinterpret_cast<const float4*>(from + row * D + c4 * 4);
        L = fmaf(lv, f, L);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
      if (whole_item) {
        const float inv = 1.f / L;
        const int tok = row / a.G, head = it.h * a.G + row - tok * a.G;
        const int64_t orow = it.q0 + tok;
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * a.o_tok +
                                  head * a.o_head + c4 * 4) =
            L == 0.f ? make_uint2(0, 0)
                     : make_uint2(pack_bf16(acc.x * inv, acc.y * inv),
                                  pack_bf16(acc.z * inv, acc.w * inv));
        if (a.lse != nullptr && c4 == 0)
          a.lse[orow * (a.H * a.G) + head] =
              L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4*>(part + (c4 * kSlotRows + row) * 4) = acc;
        if (c4 == 0) {
          part[kSlotRows * D + row] = M;
          part[kSlotRows * D + kSlotRows + row] = L;
        }
      }
    }
    if (!whole_item) {
      // a divided item: join the parts if all others have left theirs
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) last = atomicAdd(counters + it.cta0, 1) == it.nparts - 1;
      __syncthreads();
      if (last) {
        __threadfence();
        if (threadIdx.x == 0) counters[it.cta0] = 0;
        join_parts<8, 1>(slots, slot_n, kSlotRows, 0, D, it, rows, threadIdx.x, kThreads,
                   [&](int row, int col, float4 v, float lse) {
                     const int tok = row / a.G, head = it.h * a.G + row - tok * a.G;
                     const int64_t orow = it.q0 + tok;
                     *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                                               orow * a.o_tok + head * a.o_head + col) =
                         make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
                     if (a.lse != nullptr && col == 0) a.lse[orow * (a.H * a.G) + head] = lse;
                   });
      }
    }
    __syncthreads();                               // the joining buffer may be filled again
  }
  if (bad_page) atomicCAS(a.dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
}

template <int D, int NQ>
cudaError_t launch_decode(const AttnArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  DecodeArgs p{};
  p.a = a;
  p.page = make_fastdiv(a.B);
  SchedArgs& s = p.s;
  s.q_start = a.q_start;
  s.kv_lens = a.kv_lens;
  s.R = a.R;
  s.H = a.H;
  s.N = a.N;
  s.kv_cap = a.width * a.B;
  s.causal = a.causal;
  s.window = a.window;
  s.item = make_fastdiv(Cfg<D, NQ>::kRows / a.G);
  s.group = s.tile = make_fastdiv(kTile);
  s.group_tiles = 1;
  s.overhead = kItemCost;
  s.even = 1;
  e = cudaFuncSetAttribute(attn_decode_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<D, NQ>::kSmem);
  if (e != cudaSuccess) return e;
  const int most = di.sm_count * (D == 128 ? 1 : 2);
  return launch_early(attn_decode_kernel<D, NQ>, dim3(most < kMaxCtas ? most : kMaxCtas), kThreads,
                      Cfg<D, NQ>::kSmem, stream, p);
}

}  // namespace

// At most one new token per request on average, all query heads of a KV head in
// one row tile.
// No more tokens than requests, and few: the host does not know the lengths, and one
// request may have all of the tokens, which then read its keys once for each 8 or 16
// rows.  With 32 query heads on 8 of 128, decoding here against the chunk kernel: 2
// requests of 1,000 keys 11.9 us (23.6), 16 of 4,000 54 (59), 32 of 1,000 38 (44), 64 of
// 4,000 181 (179); all tokens one request's, 10,240 keys: 8 of them 40 us (48), 16 65
// (50), 32 114 (52), 64 214 (61).
// Scaled pools go by the same rule, whose border is not theirs: the chunk kernel converts
// whole tiles for the few rows.  There 32 requests of 4,000 keys take 59 us, and 64, of 256
// rows, 310 where the decoding kernel would take 109; 128 of them 600 (211); 64 of 10,240
// 673 (260); heads of 64, 64 of 4,000 253 (78); all tokens one request's, 10,240 keys: 8
// of them 30 us, 16 41, 32 69, 64 73 (122).
bool attn_decode_fits(const AttnArgs& a) {
  return a.N <= a.R && a.G <= 16 && static_cast<int64_t>(a.N) * a.G <= 128;
}

cudaError_t launch_attn_decode(const AttnArgs& a, cudaStream_t stream) {
  if (a.d == 128)
    return a.G <= 8 ? launch_decode<128, 1>(a, stream) : launch_decode<128, 2>(a, stream);
  return a.G <= 8 ? launch_decode<64, 1>(a, stream) : launch_decode<64, 2>(a, stream);
}

}  // namespace kvc
