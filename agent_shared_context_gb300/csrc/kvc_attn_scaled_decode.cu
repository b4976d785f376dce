// kvc_attn_scaled_decode.cu -- attention of single new tokens over pages of 8-bit numbers
// (e4m3 with a power of two for each block of tokens and head; d = 64 or 128, up to 16
// query heads per KV head).
//
// The division of the work and the roles are those of kvc_attn_decode.cu: eight rows (or
// sixteen) of queries are the N of a warp-level MMA (m16n8k16), keys and columns of d its
// M; each of four warps copies its 32 keys of a 128-key tile into its own ring
// (cp.async) and keeps the running maximum, sum and output of its keys.
//
// Half the bytes of bf16 leave half the time for the same arithmetic, so the numbers go
// to the tensor core as fp16, which one instruction makes of two e4m3 numbers, exactly,
// and not as scaled elements, which would take six.  With k8, v8 the numbers and a_j,
// b_j the exponents of key j's blocks:
//   x_j = scale log2(e) 2^(a_j + u) (q 2^-u) . k8_j,   u such that q 2^-u fits fp16,
//   l   = sum_j 2^(x_j - m),            m = max x_j,
//   O   = sum_j 2^(x_j + b_j - r) v8_j, r = max (x_j + b_j) - 14,
//   out = O 2^(r - m) / l.
// The largest 2^(x_j + b_j - r) is 2^14, whatever the blocks' exponents are; as fp16 each
// is off by 2^-11 of itself, or by 2^-39 of the row's largest.  The first is little beside
// the output's rounding to bf16 (2^-8), and the second wherever the largest term has a part
// in the output's element.  q 2^-u has its largest element in [2^14, 2^15): all of bf16's
// bits remain but for elements 2^28 times smaller.
//
// An 8 x 16-byte matrix comes out of shared memory by ldmatrix as if its elements had 16
// bits: a lane gets four neighbouring columns of a key, so K's columns enter the MMA in
// another order, in which Q is loaded as well; of V, transposed by 16-bit units, two
// columns of two keys, which are the MMA's rows gr and gr + 8: column 2 gr + h of a unit
// of 16 is row gr + 8 h of the product.
//
// Measured, 32 query heads on 8 of 128: 16 requests of 10,240 keys, blocks of 16, 69.7 us,
// 341 MB at 4.9 TB/s (bf16 pools 109 us, twice the bytes); one request of 131,072 keys 62
// us (87); one of 777 keys 9.0 us; heads of 64: 51, 46 and 8.6 us.  Of this some 10 us are
// beginning and end; the rest is bound by the latency of a step (some 900 instructions for
// 32 keys, from ldmatrix through conversion, product, maximum and exponentials to the
// second product), which two warps in each quarter of the SM do not hide: 37% of the
// cycles issue one.  Three CTAs of fewer registers (spills) 73 us, two stages instead of
// three 71.
//
// Keys that no row sees are filled with zeros.  A tile of which only some rows see a part
// is looked through for NaNs in V (there are no infinities); with one in it the product
// with V goes element by element and skips what a row does not see.
#include <cuda_bf16.h>

#include "kvc_attn_sched.cuh"
#include "kvc_attn_warp.cuh"
#include "kvc_paged_internal.h"
#include "kvc_ptx.cuh"
#include "kvc_scaled.cuh"

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
constexpr int kCtas = 2;                   // resident on an SM
constexpr int kMaxCtas = 320;
constexpr int kItemCost = 2;
constexpr float kHead = 14.f;              // log2 of the largest weight of a value

struct DecodeArgs {
  AttnArgs a;
  ScaleArgs sc;
  SchedArgs s;
  FastDiv page, block;
};

template <int D, int NQ>
struct Cfg {
  static constexpr int kRows = 8 * NQ;                            // rows of a tile
  static constexpr int kHalfStage = kKeys * D;                    // K or V of a step
  static constexpr int kWarpBytes = kStages * 2 * kHalfStage;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static_assert(kRows * (D + 2) * 4 <= kWarpBytes, "a warp's result takes its ring's place");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte unit `u` of key row `n`: the rows of a unit lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t at(int n, int u) {
  return D == 128 ? static_cast<uint32_t>(n * 128 + ((u ^ (n & 7)) << 4))
                  : static_cast<uint32_t>(n * 64 + ((u ^ ((n >> 1) & 3)) << 4));
}

// NQ: groups of eight rows of an item.
template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, kCtas)
    scaled_decode_kernel(const __grid_constant__ DecodeArgs p) {
  using C = Cfg<D, NQ>;
  constexpr int kRows = C::kRows;
  constexpr int kUnits = D / 16;                   // 16-byte units of a row
  constexpr int kRowsAtOnce = 32 / kUnits;         // rows of a warp's 32 units
  static_assert(kKeys == 32, "a lane looks up a key's page");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared sched;
  __shared__ int32_t last;
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = ptx::smem_u32(smem) + warp * C::kWarpBytes;
  const int gr = lane >> 2, qc = lane & 3;         // row and pair of columns of a fragment

  grid_wait();
  Walker w = walker_begin<kThreads>(p.s, &sched, a.dev_status);
  int32_t* counters = static_cast<int32_t*>(a.workspace);
  float* slots = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kAttnCounterBytes);
  const size_t slot_n = slot_floats(kSlotRows, D);
  const uint8_t *pools[2], *scales[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    pools[kv] = static_cast<const uint8_t*>(a.pool[kv].base) + a.layer * a.pool[kv].s_layer;
    scales[kv] = p.sc.exps[kv] + a.layer * p.sc.s_layer;
  }
  const bool alike = a.pool[0].s_req == a.pool[1].s_req && a.pool[0].s_tok == a.pool[1].s_tok;
  bool bad_page = false;

  Item it;
  while (w.next(p.s, &it)) {
    const int rows = it.nt * a.G;
    const int any_hi = a.causal ? min(it.kv, it.pos0 + it.nt) : it.kv;
    const int any_lo = a.window > 0 ? max(0, it.pos0 + 1 - a.window) : 0;
    const int all_hi = a.causal ? min(it.kv, it.pos0 + 1) : it.kv;
    const int all_lo = a.window > 0 ? max(0, it.pos0 + it.nt - a.window) : 0;
    const int32_t* table = a.table + static_cast<int64_t>(it.r) * a.width;
    const uint8_t* src[2] = {pools[0] + it.h * a.pool[0].s_head + lane % kUnits * 16,
                             pools[1] + it.h * a.pool[1].s_head + lane % kUnits * 16};
    const int64_t head_scale = it.h * p.sc.s_head;

    // page of the lane's key of step t (-1: not to be read)
    auto page_of = [&](int t) -> int {
      const int tok = (it.tile0 + t) * kTile + warp * kKeys + lane;
      return t < it.ntiles && tok >= any_lo && tok < any_hi ? table[fast_div(tok, p.page)] : -1;
    };
    // starts the copy of step t; the lane's key's exponent bytes, K's below V's
    auto issue = [&](int t, int page) -> int {
      int e = 127 | 127 << 8;
      if (t < it.ntiles) {
        const int tok = (it.tile0 + t) * kTile + warp * kKeys + lane;
        const bool seen = tok >= any_lo && tok < any_hi;
        if (seen && (page < 0 || page >= a.P)) {
          bad_page = true;
          page = -1;
        }
        const int in_page = tok - fast_div(tok, p.page) * a.B;
        const bool has = seen && page >= 0;
        const uint32_t rows = __ballot_sync(0xffffffffu, has);
        // the lane's row, which the lanes that copy it ask for; none is not read anywhere
        int64_t off[2] = {0, 0};
        if (has) {
          const int64_t where = page * p.sc.s_page + head_scale + fast_div(in_page, p.block);
          e = scales[0][where] | scales[1][where] << 8;
          off[0] = page * a.pool[0].s_req + in_page * a.pool[0].s_tok;
          if (!alike) off[1] = page * a.pool[1].s_req + in_page * a.pool[1].s_tok;
        }
        const uint32_t dst = ring + (t % kStages) * 2 * C::kHalfStage;
#pragma unroll
        for (int j = 0; j < kKeys / kRowsAtOnce; ++j) {
          const int n = j * kRowsAtOnce + lane / kUnits;
          const uint32_t to = dst + at<D>(n, lane % kUnits);
          const bool real = (rows >> n) & 1u;
          const int64_t k = __shfl_sync(0xffffffffu, off[0], n);
          cp_async16(to, src[0] + k, real);
          const int64_t v = alike ? k : __shfl_sync(0xffffffffu, off[1], n);
          cp_async16(to + C::kHalfStage, src[1] + v, real);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return e;
    };

    int exps[kStages];                             // of steps t, t + 1, ...
    int pages = page_of(0);
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) {
      const int next = page_of(t + 1);
      exps[t] = issue(t, pages);
      pages = next;
    }

    // Q^T as the B operand: row gr of each eight, columns 4 qc .. 4 qc + 3 of each 16
    uint32_t q[NQ][D / 16][2];
    float row_scale[NQ][2];                        // of the rows below
#pragma unroll
    for (int g8 = 0; g8 < NQ; ++g8) {
      const int row = g8 * 8 + gr, tok = row / a.G, g = row - tok * a.G;
      const bool has = row < rows;
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) +
                                (has ? (it.q0 + tok) * a.q_tok + (it.h * a.G + g) * a.q_head : 0);
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint2 x = has ? *reinterpret_cast<const uint2*>(qr + k * 16 + qc * 4) : make_uint2(0, 0);
        q[g8][k][0] = x.x;
        q[g8][k][1] = x.y;
        top = max_abs2(max_abs2(top, x.x), x.y);
      }
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int up = f16_up(top);
      const float f = pow2_of(127 + up), back = a.scale_log2 * pow2_of(127 - up);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) q[g8][k][c] = bf16x2_f16x2(q[g8][k][c], f);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        row_scale[g8][i] = __shfl_sync(0xffffffffu, back, (qc * 2 + i) * 4);
    }
    // of the rows 8 g8 + 2 qc and the next, which the lane's results belong to
    float m[NQ][2], r[NQ][2], l[NQ][2];
    int key_lo[NQ][2], key_hi[NQ][2];
#pragma unroll
    for (int g8 = 0; g8 < NQ; ++g8)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pos = it.pos0 + min((g8 * 8 + qc * 2 + i) / a.G, it.nt - 1);
        key_hi[g8][i] = a.causal ? min(it.kv, pos + 1) : it.kv;
        key_lo[g8][i] = a.window > 0 ? max(0, pos - a.window + 1) : 0;
        m[g8][i] = r[g8][i] = -INFINITY;
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
      exps[kStages - 1] = issue(t + kStages - 1, pages);
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
        for (int k = 0; k < kUnits; k += 2)
#pragma unroll
          for (int n = 0; n < kG; ++n) {
            uint32_t f[4];       // unit k of keys 0-7, of keys 8-15, then unit k + 1
            ldmatrix4(sK + at<D>(n * 16 + (lane & 15), k + (lane >> 4)), f);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t a0, a1, a2, a3;
              e4m3_f16x4(f[2 * j], a0, a2);
              e4m3_f16x4(f[2 * j + 1], a1, a3);
#pragma unroll
              for (int g8 = 0; g8 < NQ; ++g8)
                mma_f16(s[g8][n], a0, a1, a2, a3, q[g8][k + j][0], q[g8][k + j][1]);
            }
          }
        // the blocks' exponents, of keys gr and gr + 8 of each group
        float k_scale[kG][2], v_exp[kG][2];
#pragma unroll
        for (int n = 0; n < kG; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int e = __shfl_sync(0xffffffffu, exps[0], n * 16 + h * 8 + gr);
            k_scale[n][h] = pow2_of(e & 0xff);
            v_exp[n][h] = static_cast<float>((e >> 8) - 127);
          }
        const bool whole = k0 >= all_lo && k0 + kKeys <= all_hi;
        uint32_t ph[NQ][kG][2];                    // the values' weights as B operands
#pragma unroll
        for (int g8 = 0; g8 < NQ; ++g8) {
#pragma unroll
          for (int n = 0; n < kG; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)      // no infinity times 0
              s[g8][n][c] *= fminf(k_scale[n][c >> 1] * row_scale[g8][c & 1], 8.507059e37f);
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
            float top = -INFINITY, vtop = -INFINITY;
#pragma unroll
            for (int n = 0; n < kG; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                top = fmaxf(top, s[g8][n][2 * h + i]);
                vtop = fmaxf(vtop, s[g8][n][2 * h + i] + v_exp[n][h]);
              }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, x));
            }
            const float m_new = fmaxf(m[g8][i], top), r_new = fmaxf(r[g8][i], vtop - kHead);
            const float m_ref = m_new == -INFINITY ? 0.f : m_new;
            const float r_ref = r_new == -INFINITY ? 0.f : r_new;
            f[i] = exp2_fast(r[g8][i] - r_ref);
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < kG; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float& x = s[g8][n][2 * h + i];
                sum += exp2_fast(x - m_ref);
                x = exp2_fast(x + (v_exp[n][h] - r_ref));
              }
            l[g8][i] = l[g8][i] * exp2_fast(m[g8][i] - m_ref) + sum;
            m[g8][i] = m_new;
            r[g8][i] = r_new;
          }
#pragma unroll
          for (int n = 0; n < kG; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              ph[g8][n][h] = transpose8x8(pack_f16(s[g8][n][2 * h], s[g8][n][2 * h + 1]));
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
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(sV + at<D>(j * kRowsAtOnce + lane / kUnits, lane % kUnits)));
            odd = odd || has_nan_e4m3(v.x) || has_nan_e4m3(v.y) || has_nan_e4m3(v.z) ||
                  has_nan_e4m3(v.w);
          }
          odd = __any_sync(0xffffffffu, odd);
        }
        if (!odd) {
          // O^T += V^T P^T
#pragma unroll
          for (int n = 0; n < kUnits; n += 2)
#pragma unroll
            for (int half = 0; half < kG; ++half) {
              uint32_t f[4];     // unit n of keys 0-7, of keys 8-15, then unit n + 1
              ldmatrix4_trans(sV + at<D>(half * 16 + (lane & 15), n + (lane >> 4)), f);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                // columns 2 gr of both keys below columns 2 gr + 1
                const uint32_t x = __byte_perm(f[2 * j], 0, 0x3120);
                const uint32_t y = __byte_perm(f[2 * j + 1], 0, 0x3120);
                uint32_t a0, a1, a2, a3;
                e4m3_f16x4(x, a0, a1);
                e4m3_f16x4(y, a2, a3);
#pragma unroll
                for (int g8 = 0; g8 < NQ; ++g8)
                  mma_f16(o[g8][n + j], a0, a1, a2, a3, ph[g8][half][0], ph[g8][half][1]);
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
              for (int n = 0; n < kUnits; ++n) {
                uint16_t v;                        // columns 2 gr and 2 gr + 1 of the unit
                asm volatile("ld.shared.b16 %0, [%1];"
                             : "=h"(v)
                             : "r"(sV + at<D>(key, n) + gr * 2));
                float x[2];
                f16x2_f32(e4m3_f16x2(v), x[0], x[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (tok >= key_lo[g8][i] && tok < key_hi[g8][i])
                      o[g8][n][2 * h + i] = fmaf(pk[i], x[h], o[g8][n][2 * h + i]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int j = 0; j + 1 < kStages; ++j) exps[j] = exps[j + 1];
      __syncwarp();                                // the stage may be filled again
    }

    // the four warps' rows, each in its ring's place (no copy is in flight any more)
    float* mine = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
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
          // O beside l, relative to 2^m
          const float f = m[g8][i] == -INFINITY ? 0.f : exp2f(r[g8][i] - m[g8][i]);
#pragma unroll
          for (int n = 0; n < D / 16; ++n)
            *reinterpret_cast<float2*>(mine + row * D + n * 16 + 2 * gr) =
                make_float2(o[g8][n][i] * f, o[g8][n][2 + i] * f);
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
      auto of_warp = [&](int v) { return reinterpret_cast<const float*>(smem + v * C::kWarpBytes); };
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) M = fmaxf(M, of_warp(v)[kRows * D + row]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float lv = of_warp(v)[kRows * D + kRows + row];
        if (lv == 0.f) continue;
        const float f = part_weight(of_warp(v)[kRows * D + row], lv, M);
        L = fmaf(lv, f, L);
        add_scaled(acc, *reinterpret_cast<const float4*>(of_warp(v) + row * D + c4 * 4), f);
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
    __syncthreads();                               // the rings may be filled again
  }
  if (bad_page) atomicCAS(a.dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
}

template <int D, int NQ>
cudaError_t launch_decode(const AttnArgs& a, const ScaleArgs& sc, cudaStream_t stream) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  DecodeArgs p{};
  p.a = a;
  p.sc = sc;
  p.page = make_fastdiv(a.B);
  p.block = make_fastdiv(sc.block);
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
  e = cudaFuncSetAttribute(scaled_decode_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<D, NQ>::kSmem);
  if (e != cudaSuccess) return e;
  const int most = di.sm_count * kCtas;
  return launch_early(scaled_decode_kernel<D, NQ>, dim3(most < kMaxCtas ? most : kMaxCtas), kThreads,
                      Cfg<D, NQ>::kSmem, stream, p);
}

}  // namespace

size_t attn_scaled_workspace_bytes(int d) {
  const size_t mine =
      kAttnCounterBytes + kMaxCtas * 2 * slot_floats(kSlotRows, d) * sizeof(float);
  const size_t tc = attn_tc_workspace_bytes(d);
  return mine > tc ? mine : tc;
}

cudaError_t launch_attn_scaled_decode(const AttnArgs& a, const ScaleArgs& sc, cudaStream_t stream) {
  if (a.d == 128)
    return a.G <= 8 ? launch_decode<128, 1>(a, sc, stream) : launch_decode<128, 2>(a, sc, stream);
  return a.G <= 8 ? launch_decode<64, 1>(a, sc, stream) : launch_decode<64, 2>(a, sc, stream);
}

}  // namespace kvc
