// kvc_attn_simt.cu -- attention of a chunk of new tokens over a paged cache of
// f32 keys and values, in FP32 arithmetic.
//
// One pass over the keys with the running maximum and sum of the softmax: with
// x_j = scale log2(e) q.k_j, a row keeps m = max x_j, l = sum exp2(x_j - m) and
// O = sum exp2(x_j - m) v_j, and scales l and O by exp2(m_old - m_new) when a
// tile raises m.  out = O / l and lse = ln(2) (m + log2 l); a row that sees no
// key keeps m = -inf, l = 0 and gives out = 0, lse = -inf.
//
// A tile is 64 keys.  The rows of an item are (token, query head of the KV
// head's group), so that K and V are read once for the whole group.  256 threads
// have 4 rows x 4 keys of the scores and 4 rows x 4 columns (per 64 of d) of the
// output each, which asks shared memory for one 16-byte word per 8 FMAs.  The
// next tile is copied (cp.async) while one is worked on, where d leaves room for
// two; the pages of its rows are looked up a tile ahead of that.
#include "kvc_attn_sched.cuh"
#include "kvc_paged_internal.h"
#include "kvc_ptx.cuh"

namespace kvc {
namespace {

using namespace attn;

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr int kSlotRows = 64;
constexpr int kMaxCtas = 320;

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

__device__ __forceinline__ uint64_t twice(float x) {
  return ptx::pack_f32x2(__float_as_uint(x), __float_as_uint(x));
}

__device__ __forceinline__ float4 as_float4(uint64_t lo, uint64_t hi) {
  float4 v;
  ptx::unpack_f32x2(lo, v.x, v.y);
  ptx::unpack_f32x2(hi, v.z, v.w);
  return v;
}

struct Smem {
  Shared sched;
  int32_t last;
  int64_t off[2][2][kTile];        // [parity][K or V][key]: element offset in its pool, -1: none
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool real) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  const int bytes = real ? 16 : 0;         // the rest is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes)
               : "memory");
}

// RPT: rows per thread; an item has 16 * RPT rows.  DC: 64-column groups of d per
// thread.  ST: tiles in shared memory.
template <int RPT, int DC, int ST>
__global__ void __launch_bounds__(kThreads)
    attn_simt_kernel(const AttnArgs a, const SchedArgs sa, const FastDiv per_page,
                     const FastDiv per_row) {
  extern __shared__ float4 smem4[];
  __shared__ Smem sh;
  constexpr int kRows = 16 * RPT;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int d = a.d, dp = d + 4, dv = d >> 2;
  float* Qs = reinterpret_cast<float*>(smem4);      // [kRows][dp]
  float* Kt = Qs + kRows * dp;                      // [ST][kTile][dp]
  float* Vt = Kt + ST * kTile * dp;                 // [ST][kTile][d]
  float* Ps = Vt + ST * kTile * d;                  // [kRows][kTile + 4]
  constexpr int kPp = kTile + 4;

  grid_wait();
  Walker w = walker_begin<kThreads>(sa, &sh.sched, a.dev_status);
  int32_t* counters = static_cast<int32_t*>(a.workspace);
  float* slots = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kAttnCounterBytes);
  const size_t slot_n = slot_floats(kSlotRows, d);
  const float* poolK = static_cast<const float*>(a.pool[0].base) + a.layer * a.pool[0].s_layer;
  const float* poolV = static_cast<const float*>(a.pool[1].base) + a.layer * a.pool[1].s_layer;

  Item it;
  while (w.next(sa, &it)) {
    parts(w, &it);
    const int rows = it.nt * a.G;
    // the item's query rows; rows past the item are zero
    for (int i = tid; i < kRows * dv; i += kThreads) {
      const int row = fast_div(i, per_row), c = (i - row * dv) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows) {
        const int tok = row / a.G, g = row - tok * a.G;
        v = load4(static_cast<const float*>(a.q) + (it.q0 + tok) * a.q_tok +
                  (it.h * a.G + g) * a.q_head + c);
      }
      *reinterpret_cast<float4*>(Qs + row * dp + c) = v;
    }
    const int all_hi = a.causal ? min(it.kv, it.pos0 + 1) : it.kv;      // keys that all rows see
    const int all_lo = a.window > 0 ? max(0, it.pos0 + it.nt - a.window) : 0;
    float m[RPT], l[RPT];
    int key_lo[RPT], key_hi[RPT];              // keys in sight of the thread's rows
    uint64_t o[RPT][DC][2];                    // four columns in two pairs
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = ty * RPT + i;
      const int pos = it.pos0 + row / a.G;
      key_hi[i] = row < rows ? (a.causal ? min(it.kv, pos + 1) : it.kv) : 0;
      key_lo[i] = a.window > 0 ? pos - a.window + 1 : 0;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < DC; ++c) o[i][c][0] = o[i][c][1] = 0;
    }

    const int32_t* table = a.table + static_cast<int64_t>(it.r) * a.width;
    // where the rows of tile t lie
    auto locate = [&](int t) {
      const int n = tid & (kTile - 1), kv = tid / kTile;      // the first 128 threads
      if (kv > 1 || t >= it.ntiles) return;
      const int tok = (it.tile0 + t) * kTile + n;
      int64_t off = -1;
      if (tok < it.kv) {
        const int blk = fast_div(tok, per_page);
        const int page = table[blk];
        if (page >= 0 && page < a.P)
          off = page * a.pool[kv].s_req + it.h * a.pool[kv].s_head +
                static_cast<int64_t>(tok - blk * a.B) * a.pool[kv].s_tok;
        else
          atomicCAS(a.dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
      }
      sh.off[t & 1][kv][n] = off;
    };
    auto copy = [&](int t) {
      if (t < it.ntiles) {
        float* Ks = Kt + (t % ST) * kTile * dp;
        float* Vs = Vt + (t % ST) * kTile * d;
        for (int i = tid; i < kTile * dv; i += kThreads) {
          const int n = fast_div(i, per_row), c = (i - n * dv) * 4;
          const int64_t ok = sh.off[t & 1][0][n], ov = sh.off[t & 1][1][n];
          cp_async16(Ks + n * dp + c, poolK + (ok < 0 ? 0 : ok + c), ok >= 0);
          cp_async16(Vs + n * d + c, poolV + (ov < 0 ? 0 : ov + c), ov >= 0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    locate(0);
    if (ST > 1) {
      locate(1);
      __syncthreads();
      copy(0);
    }
    for (int t = 0; t < it.ntiles; ++t) {
      const int k0 = (it.tile0 + t) * kTile;
      const float* Ks = Kt + (t % ST) * kTile * dp;
      const float* Vs = Vt + (t % ST) * kTile * d;
      __syncthreads();                          // the previous tile has been read
      copy(ST > 1 ? t + 1 : t);
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
      __syncthreads();
      locate(t + ST);

      // two columns of d at a time (fma.f32x2): even and odd ones add up apart
      uint64_t s2[RPT][4];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = 0;
#pragma unroll 2
      for (int c = 0; c < d; c += 4) {
        ulonglong2 kq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          kq[j] = *reinterpret_cast<const ulonglong2*>(Ks + (tx + 16 * j) * dp + c);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(Qs + (ty * RPT + i) * dp + c);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s2[i][j] = ptx::fma_f32x2(q.y, kq[j].y, ptx::fma_f32x2(q.x, kq[j].x, s2[i][j]));
        }
      }
      float s[RPT][4];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float even, uneven;
          ptx::unpack_f32x2(s2[i][j], even, uneven);
          s[i][j] = even + uneven;
        }
      // A tile that some rows do not see whole: an infinity or a NaN among its values must
      // not meet the zeros of those rows.
      bool odd = false;
      if (k0 < all_lo || k0 + kTile > all_hi) {
        for (int i = tid; i < kTile * dv; i += kThreads) {
          const float4 v = *reinterpret_cast<const float4*>(Vs + i * 4);
          // 0 times each is 0, or NaN
          odd = odd || (v.x * 0.f + v.y * 0.f) + (v.z * 0.f + v.w * 0.f) != 0.f;
        }
        odd = __syncthreads_or(odd);
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int tok = k0 + tx + 16 * j;
          const bool see = tok >= key_lo[i] && tok < key_hi[i];
          s[i][j] = see ? s[i][j] * a.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int b = 8; b > 0; b >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, b));
        const float m_new = fmaxf(m[i], mx);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float f = exp2f(m[i] - ref);      // 0 while nothing was seen
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - ref);
          sum += p;
          Ps[(ty * RPT + i) * kPp + tx + 16 * j] = p;
        }
#pragma unroll
        for (int b = 8; b > 0; b >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
        l[i] = l[i] * f + sum;
        m[i] = m_new;
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const uint64_t f2 = twice(f);
          o[i][c][0] = ptx::mul_f32x2(o[i][c][0], f2);
          o[i][c][1] = ptx::mul_f32x2(o[i][c][1], f2);
        }
      }
      __syncwarp();                             // a warp reads the P rows it wrote
      if (!odd) {
        for (int n = 0; n < kTile; n += 4) {
          float4 p[RPT];
#pragma unroll
          for (int i = 0; i < RPT; ++i)
            p[i] = *reinterpret_cast<const float4*>(Ps + (ty * RPT + i) * kPp + n);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < DC; ++c) {
              const int col = tx * 4 + c * 64;
              if (col < d) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(Vs + (n + j) * d + col);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                  const uint64_t q =
                      twice(j == 0 ? p[i].x : j == 1 ? p[i].y : j == 2 ? p[i].z : p[i].w);
                  o[i][c][0] = ptx::fma_f32x2(q, v.x, o[i][c][0]);
                  o[i][c][1] = ptx::fma_f32x2(q, v.y, o[i][c][1]);
                }
              }
            }
        }
      } else {
        for (int n = 0; n < kTile; ++n) {
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            // a key out of a row's sight adds nothing, whatever its value row holds
            if (!(k0 + n >= key_lo[i] && k0 + n < key_hi[i])) continue;
            const float q = Ps[(ty * RPT + i) * kPp + n];
#pragma unroll
            for (int c = 0; c < DC; ++c) {
              const int col = tx * 4 + c * 64;
              if (col < d) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(Vs + n * d + col);
                o[i][c][0] = ptx::fma_f32x2(twice(q), v.x, o[i][c][0]);
                o[i][c][1] = ptx::fma_f32x2(twice(q), v.y, o[i][c][1]);
              }
            }
          }
        }
      }
      __syncwarp();
    }

    if (it.nparts == 1) {
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int row = ty * RPT + i;
        if (row >= rows) continue;
        const int tok = row / a.G, head = it.h * a.G + row - tok * a.G;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const int col = tx * 4 + c * 64;
          if (col < d)
            store4(static_cast<float*>(a.out) + (it.q0 + tok) * a.o_tok + head * a.o_head + col,
                   as_float4(ptx::mul_f32x2(o[i][c][0], twice(inv)),
                             ptx::mul_f32x2(o[i][c][1], twice(inv))));
        }
        if (a.lse != nullptr && tx == 0)
          a.lse[static_cast<int64_t>(it.q0 + tok) * (a.H * a.G) + head] =
              l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
      }
      continue;
    }

    // a divided item: leave the partial rows, and join them if all others have
    float* slot = slots + (static_cast<size_t>(blockIdx.x) * 2 + slot_of(it.part)) * slot_n;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = ty * RPT + i;
      if (row >= rows) continue;
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        const int col = tx * 4 + c * 64;
        if (col < d) store4(slot + (col / 4 * kSlotRows + row) * 4, as_float4(o[i][c][0], o[i][c][1]));
      }
      if (tx == 0) {
        slot[kSlotRows * d + row] = m[i];
        slot[kSlotRows * d + kSlotRows + row] = l[i];
      }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) sh.last = atomicAdd(counters + it.cta0, 1) == it.nparts - 1;
    __syncthreads();
    if (!sh.last) continue;
    __threadfence();
    if (tid == 0) counters[it.cta0] = 0;
    join_parts<4>(slots, slot_n, kSlotRows, 0, d, it, rows, tid, kThreads,
               [&](int row, int col, float4 v, float lse) {
                 const int tok = row / a.G, head = it.h * a.G + row - tok * a.G;
                 store4(static_cast<float*>(a.out) + (it.q0 + tok) * a.o_tok + head * a.o_head + col,
                        v);
                 if (a.lse != nullptr && col == 0)
                   a.lse[static_cast<int64_t>(it.q0 + tok) * (a.H * a.G) + head] = lse;
               });
  }
}

size_t smem_bytes(int rows, int d, int tiles) {
  return sizeof(float) * (static_cast<size_t>(rows) * (d + 4) +
                          static_cast<size_t>(tiles) * kTile * (2 * d + 4) + rows * (kTile + 4));
}

template <int RPT, int DC, int ST>
cudaError_t launch_one(const AttnArgs& a, const DeviceInfo& di, cudaStream_t stream) {
  const int rows = 16 * RPT;
  const size_t smem = smem_bytes(rows, a.d, ST);
  auto* fn = attn_simt_kernel<RPT, DC, ST>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  SchedArgs s{};
  s.q_start = a.q_start;
  s.kv_lens = a.kv_lens;
  s.R = a.R;
  s.H = a.H;
  s.N = a.N;
  s.kv_cap = a.width * a.B;
  s.causal = a.causal;
  s.window = a.window;
  s.item = make_fastdiv(rows / a.G);
  s.group = s.tile = make_fastdiv(kTile);
  s.group_tiles = 1;
  s.even = 1;
  s.overhead = 1;
  const int per_sm = 2 * (smem + sizeof(Smem) + 1024) <= static_cast<size_t>(di.smem_per_sm) ? 2 : 1;
  const int grid = di.sm_count * per_sm < kMaxCtas ? di.sm_count * per_sm : kMaxCtas;
  return launch_early(fn, dim3(grid), kThreads, smem, stream, a, s, make_fastdiv(a.B),
                      make_fastdiv(a.d / 4));
}

// Two tiles where they fit in shared memory.
template <int RPT, int DC>
cudaError_t launch_st(const AttnArgs& a, cudaStream_t stream) {
  DeviceInfo di;
  const cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  if (smem_bytes(16 * RPT, a.d, 2) + sizeof(Smem) + 1024 <= static_cast<size_t>(di.max_smem_optin))
    return launch_one<RPT, DC, 2>(a, di, stream);
  return launch_one<RPT, DC, 1>(a, di, stream);
}

template <int RPT>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t stream) {
  switch ((a.d + 63) / 64) {
    case 1: return launch_st<RPT, 1>(a, stream);
    case 2: return launch_st<RPT, 2>(a, stream);
    case 3: return launch_st<RPT, 3>(a, stream);
    default: return launch_st<RPT, 4>(a, stream);
  }
}

}  // namespace

size_t attn_simt_workspace_bytes(int d) {
  return kAttnCounterBytes + kMaxCtas * 2 * slot_floats(kSlotRows, d) * sizeof(float);
}

cudaError_t launch_attn_simt(const AttnArgs& a, cudaStream_t stream) {
  return launch_d<4>(a, stream);
}

}  // namespace kvc
