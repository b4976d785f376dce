// kvc_attn_f32.cu -- attention of new tokens over a paged cache of f32 keys and
// values.
//
// One pass over the keys with the running maximum and sum of the softmax: with
// x_j = scale log2(e) q.k_j, a row keeps m = max x_j, l = sum exp2(x_j - m) and
// O = sum exp2(x_j - m) v_j, and scales l and O by exp2(m_old - m_new) when a
// tile raises m.  out = O / l and lse = ln(2) (m + log2 l); a row that sees no
// key keeps m = -inf, l = 0 and gives out = 0, lse = -inf.
//
// Both products run on the tensor cores with each f32 factor as the sum of two
// tf32 numbers of 11 bits: x = h + e with h = tf32(x) rounded and e = x - h cut,
// and x y = h h' + h e' + e h' up to 5 2^-22 |x y| (the cut 2^-21 of each, and
// e e').  The tensor core's sums may drop bits where an FMA would round, so no
// sum of theirs is longer than a tile: a tile's P V is added to O by an FMA.
// Numbers from 2^-126 to 2^-115 keep the 11 bits of h alone (e is below the smallest
// normal number), smaller ones may count as zeros.
//
// A row is (token, query head of the KV head's group), so that K and V are read
// once for the whole group.  Eight warps: RB groups of rows, of MB blocks of 16,
// times 8 / RB runs of the tile's keys.  A warp keeps m, l and O of its rows and
// keys by itself; the runs are joined at the end of an item.  The order of the
// columns of d in the first product and of the keys in the second is free as long
// as both factors have the same one: a lane takes four consecutive columns of a
// key for two steps of 8, and the scores that it has are the factors of P V that
// it needs.  Units of 16 bytes are placed so that the lanes of a load are in banks
// of their own.  The next tiles are copied (cp.async) while one is worked on.
//
// An infinity or a NaN cannot be split, and a key out of a row's sight must add
// nothing even if its values are infinite: a tile that has one is worked through
// element by element in FP32.
//
// Measured, in us, with FP32 FMAs in place of the tensor cores in brackets: four
// chunks of 300 tokens over 4,000 keys, 8 on 2 heads, of 64: 239 (338), 40 TFLOP/s
// of the 9.5 GFLOP that count; of 128: 417 (685); decoding 16 requests of 5,000
// keys with heads of 128: 67 (199), 2.4 TB/s; six ragged chunks of up to 65 tokens
// over 2,000 keys, heads of 64: 27 (41).  (FMAs were bound by their rate and by
// shared memory.)  The tensor cores alone would take 95 us for the first: there is
// room for two warps a scheduler, 255 registers each, and they wait for one
// another's chains (issue slots 43%, tensor pipe 40% busy).  Two blocks of 16 rows
// in a warp share the splitting of K and V: with one block, 16 warps an SM, the
// first took 271 us.  Decoding has two tiles of copies in flight, and the next ones
// start when all warps have searched a tile and met: 0.36 of HBM's rate.
#include "kvc_attn_sched.cuh"
#include "kvc_paged_internal.h"

namespace kvc {
namespace {

using namespace attn;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlotRows = 64;
constexpr int kMaxCtas = 320;
constexpr uint32_t kAll = 0xffffffffu;

// DC: groups of 32 columns.  RB: groups of rows.  MB: blocks of 16 rows in each.
template <int DC, int RB, int MB>
struct Cfg {
  static constexpr int kRows = 16 * RB * MB;
  static constexpr int kPitch = 32 * DC;
  static constexpr int kRuns = kWarps / RB;                 // of a tile's keys
  static constexpr int kTile = DC > 4 ? 32 : 64;
  static constexpr int kSteps = kTile / kRuns / 8;          // of 8 keys in a run
  static constexpr int kStages = RB == 1 ? 3 : 2;
  static constexpr int kCtasSm = DC <= 2 && MB == 1 ? 2 : 1;
  static constexpr bool kSplitQ = DC <= 4;                  // Q is kept as h and e
  static constexpr int kStage = 2 * kTile * kPitch;         // floats of K and V of a tile
  static constexpr int kQ = kRows * kPitch;
  static constexpr int kJoin = kRuns * kRows * (kPitch + 2);
  static constexpr int kFloats = kStages * kStage + (kSplitQ ? 2 : 1) * kQ;
  static constexpr int kSmem = 4 * kFloats;
  static_assert(kSteps >= 1 && kJoin <= kFloats, "the runs are joined over tiles and Q");
};

struct Smem {
  Shared sched;
  Walker walker;                   // thread 0 walks the share
  Item it;
  int32_t more, last;
  int64_t off[2][2][64];           // [parity][K or V][key]: element offset in its pool, -1: none
};

// Float index of 16-byte unit `u` of a row: K and Q are read by 8 rows x 4
// consecutive units, V by 4 pairs of rows x 8 consecutive units.
template <int PITCH>
__device__ __forceinline__ int at_k(int n, int u) {
  return n * PITCH + ((u ^ ((n & 1) << 2)) << 2);
}
template <int PITCH>
__device__ __forceinline__ int at_v(int n, int u) {
  return n * PITCH + ((u ^ (((n >> 1) & 3) << 1)) << 2);
}

__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

__device__ __forceinline__ float part4(float4 v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// x = h + e; of e the tensor core ignores the lower 13 bits.
__device__ __forceinline__ void split(float x, uint32_t& h, uint32_t& e) {
  h = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  e = __float_as_uint(x - __uint_as_float(h));
}

// The larger of x and the components' magnitudes, NaN if one is.
__device__ __forceinline__ float size_of(float4 v, float x) {
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(x) : "f"(fabsf(v.x)), "f"(fabsf(v.y)));
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(x) : "f"(fabsf(v.z)), "f"(fabsf(v.w)));
  return x;
}
constexpr float kTooLarge = 3.39e38f;      // h might be infinite

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool real) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  const int bytes = real ? 16 : 0;         // the rest is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes)
               : "memory");
}

template <int DC, int RB, int MB>
__global__ void __launch_bounds__(kThreads, Cfg<DC, RB, MB>::kCtasSm)
    attn_f32_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ SchedArgs sa,
                    const FastDiv per_page) {
  using C = Cfg<DC, RB, MB>;
  constexpr int kPitch = C::kPitch, kTile = C::kTile, kStages = C::kStages, kSteps = C::kSteps;
  constexpr int kRows = C::kRows, kUnroll = RB == 1 ? 2 : 1;
  constexpr int kUnits = kPitch / 4, kCopies = 4;
  extern __shared__ float4 smem4[];
  __shared__ Smem sh;
  float* smem = reinterpret_cast<float*>(smem4);    // [stage][K, V][key][pitch]
  float* Qh = smem + kStages * C::kStage;           // [row][pitch]: h, or Q itself
  float* Qe = Qh + C::kQ;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;           // row and columns of a fragment
  const int rb = warp % RB, run = warp / RB;
  const int row0 = rb * 16 * MB + g;                // the thread's rows: row0 + 8 i
  const int d = a.d, d16 = (d + 15) / 16, dq = d16 * 4;

  grid_wait();
  {
    const Walker w = walker_begin<kThreads>(sa, &sh.sched, a.dev_status);
    if (tid == 0) sh.walker = w;
  }
  int32_t* counters = static_cast<int32_t*>(a.workspace);
  float* slots = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kAttnCounterBytes);
  const size_t slot_n = slot_floats(kSlotRows, d);
  const float* pools[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
    pools[kv] = static_cast<const float*>(a.pool[kv].base) + a.layer * a.pool[kv].s_layer;

  for (;;) {
    __syncthreads();                            // the last item is done with
    if (tid == 0) {
      Item next;
      sh.more = sh.walker.next(sa, &next);
      if (sh.more) {
        parts(sh.walker, &next);
        sh.it = next;
      }
    }
    __syncthreads();
    if (!sh.more) break;
    const Item& it = sh.it;
    const int rows = it.nt * a.G;
    const int all_hi = a.causal ? min(it.kv, it.pos0 + 1) : it.kv;      // keys that all rows see
    const int all_lo = a.window > 0 ? max(0, it.pos0 + it.nt - a.window) : 0;

    const int32_t* table = a.table + static_cast<int64_t>(it.r) * a.width;
    // where the rows of tile t lie
    auto locate = [&](int t) {
      const int n = tid % kTile, kv = tid / kTile;
      if (kv > 1 || t >= it.ntiles) return;
      const int tok = (it.tile0 + t) * kTile + n;
      int64_t off = -1;
      // keys that some row sees: others' pages may not be the request's any more
      if (tok < (a.causal ? min(it.kv, it.pos0 + it.nt) : it.kv) &&
          (a.window == 0 || tok > it.pos0 - a.window)) {
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
        float* Ks = smem + (t % kStages) * C::kStage;
        float* Vs = Ks + kTile * kPitch;
#pragma unroll kCopies
        for (int i = tid; i < kTile * kUnits; i += kThreads) {
          const int n = i / kUnits, u = i % kUnits;
          if (u >= dq) continue;
          const int64_t ok = sh.off[t & 1][0][n], ov = sh.off[t & 1][1][n];
          const bool in = u * 4 < d;
          cp_async16(Ks + at_k<kPitch>(n, u), pools[0] + (in && ok >= 0 ? ok + u * 4 : 0),
                     in && ok >= 0);
          cp_async16(Vs + at_v<kPitch>(n, u), pools[1] + (in && ov >= 0 ? ov + u * 4 : 0),
                     in && ov >= 0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) locate(t);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) copy(t);
    if (kStages > 2) __syncthreads();           // two tiles' offsets are kept
    locate(kStages - 1);

    // the item's query rows; rows past the item and columns past d are zero
    bool q_odd = false;
    for (int i = tid; i < kRows * kUnits; i += kThreads) {
      const int row = i / kUnits, u = i % kUnits;
      if (u >= dq) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows && u * 4 < d) {
        const int tok = row / a.G;
        v = load4(static_cast<const float*>(a.q) + (it.q0 + tok) * a.q_tok +
                  (it.h * a.G + row - tok * a.G) * a.q_head + u * 4);
      }
      q_odd |= !(size_of(v, 0.f) < kTooLarge);
      const int at = at_k<kPitch>(row, u);
      if (C::kSplitQ) {
        uint4 h, e;
        split(v.x, h.x, e.x);
        split(v.y, h.y, e.y);
        split(v.z, h.z, e.z);
        split(v.w, h.w, e.w);
        *reinterpret_cast<uint4*>(Qh + at) = h;
        *reinterpret_cast<uint4*>(Qe + at) = e;
      } else {
        store4(Qh + at, v);
      }
    }

    int key_lo[2 * MB], key_hi[2 * MB];         // keys in sight of the thread's rows
    float m[2 * MB], l[2 * MB];                 // l: of the thread's own keys
    float o[MB][DC][4][4];                      // [columns 32 c + 4 n + j][j][fragment]
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i) {
      const int row = row0 + 8 * i, pos = it.pos0 + row / a.G;
      key_hi[i] = row < rows ? (a.causal ? min(it.kv, pos + 1) : it.kv) : 0;
      key_lo[i] = a.window > 0 ? pos - a.window + 1 : 0;
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < DC; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[b][c][j][i] = 0.f;

    for (int t = 0; t < it.ntiles; ++t) {
      const float* Ks = smem + (t % kStages) * C::kStage;
      const float* Vs = Ks + kTile * kPitch;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      // what the thread has copied itself is there
      float size = 0.f;
#pragma unroll kCopies
      for (int i = tid; i < kTile * kUnits; i += kThreads) {
        const int n = i / kUnits, u = i % kUnits;
        if (u >= dq) continue;
        size = size_of(load4(Ks + at_k<kPitch>(n, u)), size);
        size = size_of(load4(Vs + at_v<kPitch>(n, u)), size);
      }
      // every tile landed, and every reader of the last one done
      const bool odd = __syncthreads_or(!(size < kTooLarge) || q_odd);
      copy(t + kStages - 1);
      locate(t + kStages);

      const int key0 = run * (kTile / C::kRuns);            // of the warp, in the tile
      const int tok0 = (it.tile0 + t) * kTile + key0;
      float s[MB][kSteps][4];
      if (!odd) {
        float x[MB][kSteps][4];                 // h e' + e h'
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int n = 0; n < kSteps; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][n][i] = x[b][n][i] = 0.f;
#pragma unroll kUnroll
        for (int c = 0; c < d16; ++c) {
          uint32_t h[MB][2][4], e[MB][2][4];    // of two steps of 8 columns
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            const int at0 = at_k<kPitch>(row0 + 16 * b, 4 * c + t4);
            const int at1 = at_k<kPitch>(row0 + 16 * b + 8, 4 * c + t4);
            if (C::kSplitQ) {
              const uint4 h0 = *reinterpret_cast<const uint4*>(Qh + at0);
              const uint4 h1 = *reinterpret_cast<const uint4*>(Qh + at1);
              const uint4 e0 = *reinterpret_cast<const uint4*>(Qe + at0);
              const uint4 e1 = *reinterpret_cast<const uint4*>(Qe + at1);
              h[b][0][0] = h0.x, h[b][0][1] = h1.x, h[b][0][2] = h0.y, h[b][0][3] = h1.y;
              h[b][1][0] = h0.z, h[b][1][1] = h1.z, h[b][1][2] = h0.w, h[b][1][3] = h1.w;
              e[b][0][0] = e0.x, e[b][0][1] = e1.x, e[b][0][2] = e0.y, e[b][0][3] = e1.y;
              e[b][1][0] = e0.z, e[b][1][1] = e1.z, e[b][1][2] = e0.w, e[b][1][3] = e1.w;
            } else {
              const float4 q0 = load4(Qh + at0), q1 = load4(Qh + at1);
              split(q0.x, h[b][0][0], e[b][0][0]), split(q1.x, h[b][0][1], e[b][0][1]);
              split(q0.y, h[b][0][2], e[b][0][2]), split(q1.y, h[b][0][3], e[b][0][3]);
              split(q0.z, h[b][1][0], e[b][1][0]), split(q1.z, h[b][1][1], e[b][1][1]);
              split(q0.w, h[b][1][2], e[b][1][2]), split(q1.w, h[b][1][3], e[b][1][3]);
            }
          }
#pragma unroll
          for (int n = 0; n < kSteps; ++n) {
            const float4 k = load4(Ks + at_k<kPitch>(key0 + n * 8 + g, 4 * c + t4));
            uint32_t kh[4], ke[4];
            split(k.x, kh[0], ke[0]);
            split(k.y, kh[1], ke[1]);
            split(k.z, kh[2], ke[2]);
            split(k.w, kh[3], ke[3]);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
              mma(s[b][n], h[b][0], kh[0], kh[1]);
              mma(x[b][n], h[b][0], ke[0], ke[1]);
              mma(s[b][n], h[b][1], kh[2], kh[3]);
              mma(x[b][n], e[b][0], kh[0], kh[1]);
              mma(x[b][n], h[b][1], ke[2], ke[3]);
              mma(x[b][n], e[b][1], kh[2], kh[3]);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int n = 0; n < kSteps; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[b][n][i] += x[b][n][i];
      } else {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int n = 0; n < kSteps; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = min(row0 + 16 * b + 8 * (i >> 1), rows - 1), tok = row / a.G;
              const float* q = static_cast<const float*>(a.q) + (it.q0 + tok) * a.q_tok +
                               (it.h * a.G + row - tok * a.G) * a.q_head;
              const int key = key0 + n * 8 + 2 * t4 + (i & 1);
              float sum = 0.f;
#pragma unroll 1
              for (int c = 0; c < d; ++c)
                sum = fmaf(q[c], Ks[at_k<kPitch>(key, c >> 2) + (c & 3)], sum);
              s[b][n][i] = sum;
            }
      }

      const bool whole = tok0 >= all_lo && tok0 + kTile / C::kRuns <= all_hi;
      float f[2 * MB];
#pragma unroll
      for (int b = 0; b < MB; ++b) {
#pragma unroll
        for (int n = 0; n < kSteps; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[b][n][i] *= a.scale_log2;
            if (!whole) {
              const int tok = tok0 + n * 8 + 2 * t4 + (i & 1);
              if (tok < key_lo[2 * b + (i >> 1)] || tok >= key_hi[2 * b + (i >> 1)])
                s[b][n][i] = -INFINITY;
            }
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = fmaxf(s[b][0][2 * i], s[b][0][2 * i + 1]);
#pragma unroll
          for (int n = 1; n < kSteps; ++n)
            mx = fmaxf(mx, fmaxf(s[b][n][2 * i], s[b][n][2 * i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
          const int r = 2 * b + i;
          const float m_new = fmaxf(m[r], mx);
          const float ref = m_new == -INFINITY ? 0.f : m_new;
          f[r] = exp2f(m[r] - ref);             // 0 while nothing was seen
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < kSteps; ++n)
#pragma unroll
            for (int j = 2 * i; j < 2 * i + 2; ++j) {
              s[b][n][j] = exp2f(s[b][n][j] - ref);
              sum += s[b][n][j];
            }
          l[r] = fmaf(l[r], f[r], sum);
          m[r] = m_new;
        }
      }

      if (!odd) {
        uint32_t ph[MB][kSteps][4], pe[MB][kSteps][4];   // keys 2 t4, 2 t4 + 1 of each step
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int n = 0; n < kSteps; ++n) {
            split(s[b][n][0], ph[b][n][0], pe[b][n][0]);
            split(s[b][n][2], ph[b][n][1], pe[b][n][1]);
            split(s[b][n][1], ph[b][n][2], pe[b][n][2]);
            split(s[b][n][3], ph[b][n][3], pe[b][n][3]);
          }
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          float y[MB][4][4];
#pragma unroll
          for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) y[b][j][i] = 0.f;
#pragma unroll
          for (int n = 0; n < kSteps; ++n) {
            const int key = key0 + n * 8 + 2 * t4;
            const float4 v0 = load4(Vs + at_v<kPitch>(key, 8 * c + g));
            const float4 v1 = load4(Vs + at_v<kPitch>(key + 1, 8 * c + g));
            uint32_t h0[4], e0[4], h1[4], e1[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              split(part4(v0, j), h0[j], e0[j]);
              split(part4(v1, j), h1[j], e1[j]);
            }
#pragma unroll
            for (int b = 0; b < MB; ++b) {
#pragma unroll
              for (int j = 0; j < 4; ++j) mma(y[b][j], pe[b][n], h0[j], h1[j]);
#pragma unroll
              for (int j = 0; j < 4; ++j) mma(y[b][j], ph[b][n], e0[j], e1[j]);
#pragma unroll
              for (int j = 0; j < 4; ++j) mma(y[b][j], ph[b][n], h0[j], h1[j]);
            }
          }
#pragma unroll
          for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                o[b][c][j][i] = fmaf(o[b][c][j][i], f[2 * b + (i >> 1)], y[b][j][i]);
        }
      } else {
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int c = 0; c < DC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[b][c][j][i] *= f[2 * b + (i >> 1)];
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
          for (int n = 0; n < kSteps; ++n)
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const int key = n * 8 + k, from = (lane & ~3) + (k >> 1);
              float p[2];                       // of the thread's rows
              bool see[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float even = __shfl_sync(kAll, s[b][n][2 * i], from);
                const float uneven = __shfl_sync(kAll, s[b][n][2 * i + 1], from);
                p[i] = (k & 1) ? uneven : even;
                // a key out of a row's sight adds nothing, whatever its value row holds
                see[i] = tok0 + key >= key_lo[2 * b + i] && tok0 + key < key_hi[2 * b + i];
              }
#pragma unroll
              for (int c = 0; c < DC; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  if (32 * c + 8 * t4 + 4 * e >= d) continue;
                  const float4 v = load4(Vs + at_v<kPitch>(key0 + key, 8 * c + 2 * t4 + e));
#pragma unroll
                  for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                      if (see[i])
                        o[b][c][j][2 * i + e] = fmaf(p[i], part4(v, j), o[b][c][j][2 * i + e]);
                }
            }
      }
    }

    // the runs of keys are joined, over the tiles and Q
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* mine = smem + run * kRows * (kPitch + 2);
#pragma unroll
    for (int i = 0; i < 2 * MB; ++i) {
      float sum = l[i];
      sum += __shfl_xor_sync(kAll, sum, 1);
      sum += __shfl_xor_sync(kAll, sum, 2);
      const int row = row0 + 8 * i;
#pragma unroll
      for (int c = 0; c < DC; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          store4(mine + row * kPitch + 32 * c + 8 * t4 + 4 * e,
                 make_float4(o[i / 2][c][0][2 * (i % 2) + e], o[i / 2][c][1][2 * (i % 2) + e],
                             o[i / 2][c][2][2 * (i % 2) + e], o[i / 2][c][3][2 * (i % 2) + e]));
      if (t4 == 0) {
        mine[kRows * kPitch + row] = m[i];
        mine[kRows * kPitch + kRows + row] = sum;
      }
    }
    __syncthreads();
    const bool whole_item = it.nparts == 1;
    float* part = slots + (static_cast<size_t>(blockIdx.x) * 2 + slot_of(it.part)) * slot_n;
    const int d4 = d / 4;
    for (int e = tid; e < rows * DC * 8; e += kThreads) {
      const int row = e / (DC * 8), c4 = e - row * (DC * 8);
      if (c4 >= d4) continue;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int v = 0; v < C::kRuns; ++v)
        M = fmaxf(M, smem[v * kRows * (kPitch + 2) + kRows * kPitch + row]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < C::kRuns; ++v) {
        const float* from = smem + v * kRows * (kPitch + 2);
        const float lv = from[kRows * kPitch + kRows + row];
        if (lv == 0.f) continue;
        const float f = part_weight(from[kRows * kPitch + row], lv, M);
        const float4 x = load4(from + row * kPitch + c4 * 4);
        L = fmaf(lv, f, L);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
      if (whole_item) {
        const int tok = row / a.G, head = it.h * a.G + row - tok * a.G;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        store4(static_cast<float*>(a.out) + (it.q0 + tok) * a.o_tok + head * a.o_head + c4 * 4,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (a.lse != nullptr && c4 == 0)
          a.lse[static_cast<int64_t>(it.q0 + tok) * (a.H * a.G) + head] =
              L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      } else {
        store4(part + (c4 * kSlotRows + row) * 4, acc);
        if (c4 == 0) {
          part[kSlotRows * d + row] = M;
          part[kSlotRows * d + kSlotRows + row] = L;
        }
      }
    }
    if (whole_item) continue;
    // a divided item: join the parts if all others have left theirs
    __threadfence();
    __syncthreads();
    if (tid == 0) sh.last = atomicAdd(counters + it.cta0, 1) == it.nparts - 1;
    __syncthreads();
    if (!sh.last) continue;
    __threadfence();
    if (tid == 0) counters[it.cta0] = 0;
    constexpr int kWide = DC * MB <= 4 && C::kCtasSm == 1 ? 4 : 2;   // as registers allow
    join_parts<4, kWide>(slots, slot_n, kSlotRows, 0, d, it, rows, tid, kThreads,
                  [&](int row, int col, float4 v, float lse) {
                    const int tok = row / a.G, head = it.h * a.G + row - tok * a.G;
                    store4(static_cast<float*>(a.out) + (it.q0 + tok) * a.o_tok +
                               head * a.o_head + col,
                           v);
                    if (a.lse != nullptr && col == 0)
                      a.lse[static_cast<int64_t>(it.q0 + tok) * (a.H * a.G) + head] = lse;
                  });
  }
}

template <int DC, int RB, int MB>
cudaError_t launch_one(const AttnArgs& a, cudaStream_t stream) {
  using C = Cfg<DC, RB, MB>;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  auto* fn = attn_f32_kernel<DC, RB, MB>;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
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
  s.item = make_fastdiv(C::kRows / a.G);
  s.group = s.tile = make_fastdiv(C::kTile);
  s.group_tiles = 1;
  s.even = 1;
  s.overhead = 1;
  const int most = di.sm_count * C::kCtasSm;
  return launch_early(fn, dim3(most < kMaxCtas ? most : kMaxCtas), kThreads, C::kSmem, stream, a, s,
                      make_fastdiv(a.B));
}

// 16 rows where the requests have no more on average, since 64 would be idle for the
// most part (decoding as above 124 us with them); not beyond 256 in all, which could be
// one request's and would read its keys 16 times.
template <int DC>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.N) * a.G;
  if (a.G <= 16 && rows <= static_cast<int64_t>(a.R) * 16 && rows <= 256)
    return launch_one<DC, 1, 1>(a, stream);
  return launch_one<DC, 2, 2>(a, stream);
}

}  // namespace

size_t attn_f32_workspace_bytes(int d) {
  return kAttnCounterBytes + kMaxCtas * 2 * slot_floats(kSlotRows, d) * sizeof(float);
}

cudaError_t launch_attn_f32(const AttnArgs& a, cudaStream_t stream) {
  switch ((a.d + 31) / 32) {
    case 1: return launch_rows<1>(a, stream);
    case 2: return launch_rows<2>(a, stream);
    case 3: return launch_rows<3>(a, stream);
    case 4: return launch_rows<4>(a, stream);
    case 5:
    case 6: return launch_one<6, 4, 1>(a, stream);
    default: return launch_one<8, 4, 1>(a, stream);
  }
}

}  // namespace kvc
