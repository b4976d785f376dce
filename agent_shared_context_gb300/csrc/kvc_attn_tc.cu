// kvc_attn_tc.cu -- attention of a chunk of new tokens over a paged cache on
// tcgen05 tensor cores (bf16, d = 64 or 128).
//
// The mathematics is that of kvc_attn_f32.cu: one pass over the keys with the
// running maximum m and sum l of each row's softmax.  Any reference value that
// keeps exp2(x - m) in range gives the same O / l, so m follows the maximum
// only when a tile raises it by more than 8 (log2): P then stays below 2^8,
// and O, which lives in TMEM, is rescaled in few tiles only.
//
// A row of the MMA is (token, query head of the KV head's group), so K and V
// are read once for the whole group; a row tile holds floor(128 / G) tokens,
// which one TMA box of Q fetches.  Two *streams* share a CTA, each with a row
// tile's scores S (fp32, 128 columns) and output O in TMEM and a warpgroup for
// its softmax, so the tensor core works for one while the other exponentiates:
//   pair mode    (an item with more tokens than one row tile): the streams are
//                two row tiles over the same key tiles;
//   single mode  (decoding, the end of a chunk): both streams have the same
//                rows and take every other key tile; stream 0 joins them.
// Which mode an item takes is its own affair, so one launch serves batches
// that mix decoding with chunks.  The work is divided over a persistent grid
// as kvc_attn_sched.cuh says.
//
//   warps 0-3, 4-7  softmax of stream 0 and 1: scores from TMEM (thread = row),
//                   running maximum, exp2, P to TMEM as bf16 (over S); the
//                   output at the end of an item;
//   warp 8          walks the share, hands the items to the others through a
//                   ring, looks the pages up and issues the TMA loads of Q, K
//                   and V;
//   warps 9, 11     issue stream 0's and 1's S = Q K^T (both K-major in shared
//                   memory) and O += P V (P in TMEM, V as the MN-major operand
//                   it is);
//   warp 10         only holds its place in its warpgroup.
//
// A key tile is 128 keys, copied in runs that divide it and the page: pages of
// a multiple of 16 rows fill every tile.  Of others a tile holds as many whole
// ones (rounded up to 8 rows) as fit, or 128 rows of one, and leaves holes that
// are masked (launch_tc says when).  Where a tile is not in sight of all its rows the scores are
// masked, and the softmax warps look through the value rows that are not in
// sight of all: 0 times an infinity or a NaN, which a page may hold there, is not
// 0.  Where they find one they clear it, and if some rows do see it those add its
// products from memory.
//
// The product with V takes P as bf16 (its sum l stays fp32).  Roundings of up to
// 2^-8 average out over many keys of like weight but not where few carry a
// row, so in the steps of 16 keys in which some row has a key with more than 1/8
// of its sum so far (1/16 in single mode, which waits for memory anyway) P enters
// as two numbers, cut_bf16 and the rest of it: few steps of a long context.  S
// leaves room for the rest in TMEM, beside P.
//
// Error against 64 bits (root of the mean square), beside that of f32 arithmetic
// rounded once: the dense prefill below 2.50e-4 (2.25e-4), the sixteen chunks 1.41e-4
// (1.13e-4).  Two numbers from 1/16 on would give 2.39e-4 and 1.33e-4 and take 1,026
// and 335 us; in every step the error in brackets, and 1,241 and 405 us.
//
// Measured: dense prefill of two contexts of 8,192 tokens, 32 query heads on 8 of 128,
// 0.96 to 0.97 ms, 1.14 PFLOP/s or 0.60 of the library's matrix products; sixteen chunks
// of 128 tokens over 10,368 keys 320 us, 1.08 PFLOP/s (heads of 64: 253 us, 0.68
// PFLOP/s); five ragged ones of up to 700 tokens, 28 on 4 heads, a window of 4,096, pages
// of 48: 104 us, 0.59 PFLOP/s.  A pair of row tiles takes some 3,800 cycles per 128 keys.
// A loop of its MMAs alone takes 2,960 of these: a step of 16 columns of S for 64 keys
// 60 cycles, hardly less than the 65 that one for 128 keys takes, since both read all of
// Q's columns out of shared memory (with Q in TMEM 48); a step of P V 64.  At the full
// rate the MMAs would need 2,050.  The rest is the hand-over: each half of a tile waits
// for the softmax's and the MMA's signals.  An item costs some 10,000 cycles besides
// (masked tiles, the output), a CTA 5 us to its first tile, a divided item's end 8 us.
//
// Scaled pools (F8): pages of e4m3 numbers, a power of two for each block of tokens and
// head.  Tiles in shared memory are the numbers as fp16 (exact, one instruction for two;
// bf16 elements take six, and 568 us where this took 454), so Q, P and V are fp16 too.
//   warps 12-15     copy 32 rows of every tile each (cp.async, two tiles ahead) into a
//                   stage and write them as fp16 into a slot, where TMA would have; and
//                   make Q fp16 in place, times a power of two for each row.
// 32 neighbouring keys share one exponent of K, which goes into their scores, and one of
// V, which goes into the exponents of P: nothing is multiplied key by key unless exponents
// of K are more than 15 apart or those of V more than 10.  P is fp16 relative to the
// largest term of O, not of l; its 11 bits need no second number.  With a shared exponent a
// term may look larger than it is by as much as V's exponents differ, so where m is set the
// largest is 2^5 times that, for the true one to be 2^5 at least; it may grow to 2^15.  With
// 2^12 (terms good to 2^-37 of the largest, not 2^-30) O is rescaled oftener, 454 us.
// Measured: sixteen chunks of 128 tokens over 10,368 keys, blocks of 16, 438 us, 0.79
// PFLOP/s (bf16 pools 323); five ragged ones, a window of 4,096, pages of 48, 132 us (105).
// Without regard to how far V's exponents differ 428 and 128 us, and terms good to 2^-15 of
// the largest only.
// A pair of row tiles takes some 6,000 cycles for 128 keys, a half 3,000: 420 to its
// first scores, 560 for their largest, 1,120 for P, the rest rescales and waits.  512
// threads leave it 128 registers and a fourth warp in each quarter of the SM: 3,300
// instructions per quarter and tile pair (bf16 1,750), 52% of the cycles issue one.
// Tried: two converting warps of 168 registers 689 us; one warp that copies and looks up
// for all four 590 to 633; bulk copies for runs of rows 445, as fast but with more
// roles; 64 scores at once in registers (spills) 565; registers moved between warpgroups
// (setmaxnreg): ptxas has no allocation with calls in the kernel, without them 965 and
// more.  Without the conversion's loop 347.
//
// Every wait is bounded: one that expires stores KVC_ERR_DEVICE_TIMEOUT into
// *dev_status and raises the CTA's abort flag; the roles stop, copies and MMAs
// in flight are waited for (with the limit again), TMEM is freed.
#include <cuda_bf16.h>

#include <cstring>
#include <type_traits>

#include "kvc_attn_sched.cuh"
#include "kvc_attn_warp.cuh"
#include "kvc_paged_internal.h"
#include "kvc_ptx.cuh"
#include "kvc_scaled.cuh"

namespace kvc {
namespace {

using namespace ptx;
using namespace attn;

constexpr int kTcThreads = 384;              // 12 warps (roles above)
constexpr int kThreadsScaled = 512;        // and four that convert scaled pools' numbers
constexpr int kRowsM = 128;                // rows of a stream (MMA M)
constexpr int kTile = 128;                 // keys of a tile
constexpr int kHalf = kTile / 2;           // keys of a step of a stream
constexpr int kSubBytes = kTile * 128;     // 128 rows x 64 bf16
constexpr int kSlotRows = 256;             // rows of a partial result
constexpr int kMaxCtas = 160;
constexpr int kItems = 4;                  // depth of the item ring
constexpr int kNoPage = INT32_MIN;         // no key there: read as zeros
constexpr int kItemCost = 6;               // tiles that an item's beginning and end cost
constexpr float kLag = 8.0f;               // log2 by which m may lag behind
constexpr float kRoom = 15.0f;             // log2 of P's largest value as fp16
constexpr float kTop = 5.0f;               // and of that of the largest term when m is set
constexpr int kSpanK = 15, kSpanV = 10;    // most by which exponents of 32 keys with one differ
constexpr uint32_t kOwn = 0x80;            // ScaledInfo: keys with exponents of their own
static_assert(kTop + kSpanV <= kRoom, "the largest term when m is set fits P");
constexpr float kApart = 60.0f;            // exponents of V that are looked at key by key
constexpr float kFar = 90.0f;              // log2 from where a larger score counts all others out
constexpr float kHeavyPair = 0.125f;       // share of a row's sum that makes a key heavy
constexpr float kHeavySingle = 0.0625f;

// F8: the pools are scaled ones.
template <int D, bool F8>
struct Cfg {
  static constexpr int kSub = D / 64;
  static constexpr int kSlotBytes = kSub * kSubBytes;
  static constexpr int kSlots = (D == 128 ? 5 : 10) - (F8 ? D == 128 ? 1 : 2 : 0);
  static constexpr int kQBytes = 2 * kSlotBytes;
  // Tiles of numbers on their way, each converting warp's 32 rows of them together.  Two and
  // no more: a converting warp asks for the item of the tile kStages further while it has yet
  // to convert this one, and an item is handed out once Q of the one before is under way,
  // that is once all of K of the one before that is converted.  An item has two tiles of K
  // and V at least, so two further is the next item at most; four further than an item's K
  // could be the one after it, and each would wait for the other.
  static constexpr int kStages = F8 ? 2 : 0;
  static constexpr int kStageBytes = 32 * D;
  // (the rest of a scaled pool's shared memory, Bars, is added where that is known)
  static constexpr int kTiles = kQBytes + kSlots * kSlotBytes + 4 * kStages * kStageBytes;
  static constexpr int kThreads = F8 ? kThreadsScaled : kvc::kTcThreads;
};

struct TcMaps {
  CUtensorMap q, k, v;
};

struct TcArgs {
  AttnArgs a;
  SchedArgs s;
  FastDiv page, rows, tiles;   // by B, by run_rows, by the tiles of a group
  int32_t tok_tile;        // tokens of a row tile, floor(128 / G)
  int32_t runs;            // a tile is copied in runs of tokens of one page,
  int32_t run_tokens;      // so many each,
  int32_t run_rows;        // and so many rows in shared memory
  uint32_t holes[4];       // columns of a tile that never hold a key (pages < 128 rows)
  int32_t has_holes;
  int32_t ragged;          // some tiles hold fewer than 128 keys
  int32_t out32;           // output rows are 32-byte aligned
  ScaleArgs sc;            // of scaled pools
  FastDiv block;
};

struct ItemSlot {
  Item it;
  int32_t ring0;           // ring position of the item's first K tile
  int32_t edge_lo, edge_hi;  // key tiles below and from which not every row sees all keys
};

// What a stream's softmax tells its MMA warp along with P.
struct alignas(8) Told {
  uint32_t heavy;          // MMA steps of 16 keys with P as two numbers, a byte per warp
  int32_t o_init;          // O holds something before the first P V
};

template <int A, int B>
constexpr int kMost = A > B ? A : B;

// What the converting warps say of scaled pools' tiles and queries.
template <int DEPTH>
struct ScaledInfo {
  // Of each 32 keys of a tile, at the ring position of its K modulo DEPTH (twice the slots:
  // a stream looks at it before it gives the tile's V back): K's power of two, the exponent
  // of V's and that power's inverse, and by how much V's exponents differ, or kOwn.
  struct alignas(8) Tile {
    float k[4], v_exp[4], v_inv[4];
    uint8_t span[4];
  } tile[DEPTH];
  int8_t q_up[2][2 * kRowsM];      // rows of Q are times 2^q_up, of this item and the next
  uint64_t q_ready;                // Q is fp16
};
template <>
struct ScaledInfo<0> {
  uint64_t q_ready;
};

template <int NS, int STAGES, bool F8>
struct Bars {
  uint64_t kv_full[NS], kv_empty[NS];
  uint64_t q_full, q_empty;
  uint64_t s_full[2][2], p_full[2][2];   // [stream][half of the tile's keys]
  uint64_t o_seen[2];              // the stream's warps know that an item's O is complete
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t ml_full, ml_empty;      // stream 1's row statistics for stream 0
  uint64_t wg[2];                  // the four warps of a stream
  uint64_t drain[2];
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t last[2];
  Told told[2][2];
  ScaledInfo<F8 ? 2 * NS : 0> scaled;
  int32_t landed[2];               // value tiles that each stream's MMA warp has seen land
  uint32_t poison[NS][4];          // value rows with an infinity or NaN that some rows see
  float ml[kRowsM][2];
  ItemSlot items[kItems];
  Shared sched;
};

// The waits.  What the first poll does not end goes on in a call, so that the
// roles' loops stay small: an instruction cache holds them all.
//
// Counts the polls of a wait: every 4,096 of them it looks at the timer, which
// costs hundreds of cycles, and at the abort flag, which it raises at the limit.
struct Patience {
  uint64_t t0 = 0;
  uint32_t polls = 0;
  __device__ __forceinline__ bool out(volatile int32_t* flag) {
    if ((++polls & 4095u) != 0u) return false;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > kWaitLimitNs) *flag = 1;
    return *flag != 0;
  }
};

__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int32_t* abort) {
  Patience p;
  bool ok = true;
#pragma unroll 1
  while (ok && !mbar_try_wait(bar, parity)) ok = !p.out(abort);
  return __all_sync(0xffffffffu, ok);
}

// A whole warp waits for a phase: all lanes give up together.
template <int NS, int STAGES, bool F8>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars<NS, STAGES, F8>* b) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_on(bar, parity, &b->abort_flag);
}

// A count that one thread raises after it has seen something land, and that others
// wait for: what was visible to the one that raised it is visible to them.
__device__ __forceinline__ void raise_count(int32_t* count) {
  const uint32_t at = smem_u32(count);
  asm volatile(
      "{\n\t.reg .b32 n;\n\t"
      "ld.relaxed.cta.shared::cta.b32 n, [%0];\n\t"
      "add.s32 n, n, 1;\n\t"
      "st.release.cta.shared::cta.b32 [%0], n;\n\t}" ::"r"(at)
      : "memory");
}

__device__ __forceinline__ int32_t read_count(const int32_t* count) {
  int32_t n;
  asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(n) : "r"(smem_u32(count)) : "memory");
  return n;
}

// A whole warp waits until *count has reached `want`.
__device__ __noinline__ bool warp_wait_count(const int32_t* count, int32_t want,
                                             volatile int32_t* abort) {
  Patience p;
  bool ok = true;
#pragma unroll 1
  while (ok && read_count(count) - want < 0) ok = !p.out(abort);
  return __all_sync(0xffffffffu, ok);
}

// A value that all lanes hold, in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }

// ------------------------------------------------------------ tile geometry
// Ring positions, relative to the item's first: the order in which the MMAs
// consume the tiles.
__device__ __forceinline__ int ring_k(bool pair, int i) {
  return pair ? 2 * i : (i < 2 ? i : 2 * i - 1);
}
__device__ __forceinline__ int ring_v(bool pair, int n, int i) {
  return pair ? 2 * i + 1 : (i == n - 1 ? 2 * n - 1 : 2 + 2 * i);
}

struct TileSpan {
  int tok0, cnt;           // first key token and tokens of the tile
};

__device__ __forceinline__ TileSpan tile_span(const TcArgs& p, int tile) {
  TileSpan t;
  if (p.s.even) {
    t.tok0 = tile * p.s.tile.d;
    t.cnt = p.s.tile.d;
  } else {
    const int g = fast_div(tile, p.tiles), sub = tile - g * p.s.group_tiles;
    t.tok0 = g * p.s.group.d + sub * p.s.tile.d;
    t.cnt = min(p.s.tile.d, p.s.group.d - sub * p.s.tile.d);
  }
  return t;
}

// Column of the tile at which token `tok` lies or would lie: the keys before it
// are exactly the key columns below.
__device__ __forceinline__ int tile_col(const TcArgs& p, const TileSpan& t, int tok) {
  const int rel = tok - t.tok0;
  if (rel <= 0) return 0;
  if (rel >= t.cnt) return kTile;
  if (!p.has_holes) return rel;
  const int pg = fast_div(rel, p.page);
  return pg * p.run_rows + (rel - pg * p.a.B);
}

// Token of a key column (not of a hole).
__device__ __forceinline__ int tile_tok(const TcArgs& p, const TileSpan& t, int col) {
  if (!p.has_holes) return t.tok0 + col;
  const int pg = fast_div(col, p.rows);
  return t.tok0 + pg * p.a.B + (col - pg * p.run_rows);
}

// Keys that every row of tokens [pos0, pos0 + nt) sees, and that any sees.
struct Sight {
  int all_lo, all_hi, any_lo, any_hi;
};

__device__ __forceinline__ Sight sight(const AttnArgs& a, int kv, int pos0, int nt) {
  Sight s;
  s.all_hi = a.causal ? min(kv, pos0 + 1) : kv;
  s.any_hi = a.causal ? min(kv, pos0 + nt) : kv;
  s.all_lo = a.window > 0 ? max(0, pos0 + nt - a.window) : 0;
  s.any_lo = a.window > 0 ? max(0, pos0 + 1 - a.window) : 0;
  return s;
}

// Key tiles that not every row sees whole: below *lo and from *hi on.
__device__ __forceinline__ void edges(const SchedArgs& a, const Sight& s, int* lo, int* hi) {
  *lo = s.all_lo > 0 ? tile_of(a, s.all_lo - 1) + 1 : 0;
  *hi = s.all_hi > 0 ? tile_of(a, s.all_hi) : 0;
}

__device__ __forceinline__ uint32_t bits_below(int n) {      // n lowest bits
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// Joins the parts of one row in the order of their keys, 4 kC columns at a time with the
// loads of kP parts in flight.  A warp's rows lie side by side.  This is at the end of
// most CTAs' work, and its time is that of the loads one after another: with 16 columns
// of one part in flight it took 15 us, so that five ragged chunks took 120 us for 108.
template <int D, int kC, int kP>
__device__ __forceinline__ void join_row(const float* slots, size_t slot_n, int nparts, int row,
                                         __nv_bfloat16* out, bool out32, float* lse) {
  auto part = [&](int n) { return slots + (static_cast<size_t>(n) * 2 + slot_of(n)) * slot_n; };
  float M = -INFINITY, L = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < D / 4; c0 += kC) {
    float4 acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    M = -INFINITY;
    L = 0.f;
#pragma unroll 1
    for (int n0 = 0; n0 < nparts; n0 += kP) {
      float4 v[kP][kC];
      float pm[kP], pl[kP];
#pragma unroll
      for (int n = 0; n < kP; ++n) {
        const float* from = part(min(n0 + n, nparts - 1));
        pm[n] = __ldcg(from + kSlotRows * D + row);
        pl[n] = n0 + n < nparts ? __ldcg(from + kSlotRows * D + kSlotRows + row) : 0.f;
        const float4* o = reinterpret_cast<const float4*>(from) + c0 * kSlotRows + row;
#pragma unroll
        for (int c = 0; c < kC; ++c) v[n][c] = __ldcg(o + c * kSlotRows);
      }
      float top = M;
#pragma unroll
      for (int n = 0; n < kP; ++n) top = fmaxf(top, pm[n]);
      const float f0 = part_weight(M, L, top);
      M = top;
      L *= f0;
#pragma unroll
      for (int c = 0; c < kC; ++c) scale(acc[c], f0);
#pragma unroll
      for (int n = 0; n < kP; ++n) {
        if (pl[n] == 0.f) continue;              // nothing seen, or no such part
        const float f = part_weight(pm[n], pl[n], M);
        L = fmaf(pl[n], f, L);
#pragma unroll
        for (int c = 0; c < kC; ++c) add_scaled(acc[c], v[n][c], f);
      }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t u[2 * kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      u[2 * c] = pack_bf16(acc[c].x * inv, acc[c].y * inv);
      u[2 * c + 1] = pack_bf16(acc[c].z * inv, acc[c].w * inv);
    }
    __nv_bfloat16* to = out + c0 * 4;
    if (out32) {
#pragma unroll
      for (int c = 0; c < kC; c += 4) st_global_32(to + c * 4, u + 2 * c);
    } else {
#pragma unroll
      for (int c = 0; c < kC; c += 2)
        *reinterpret_cast<uint4*>(to + c * 4) =
            make_uint4(u[2 * c], u[2 * c + 1], u[2 * c + 2], u[2 * c + 3]);
    }
  }
  if (lse != nullptr)
    *lse = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// ----------------------------------------------------------------- scaled pools
// Scores of a row of Q times 2^up with keys of one exponent byte, as exponents of 2.  What
// would leave the range of fp32 is beyond any use as a score.
__device__ __forceinline__ float score_scale(float row_scale, float k) {
  return fminf(fmaxf(row_scale * k, 1.1754944e-38f), 8.507059e37f);
}

// The exponent byte of a power of two.
__device__ __forceinline__ int exp_byte(float x) { return __float_as_int(x) >> 23; }

// The largest exponent byte of a warp's keys (a lane has one, those in `rows` count), and by
// how much another one of at least `from` is below.
__device__ __forceinline__ int group_exp(int exp, uint32_t rows, int from, int* span) {
  const bool has = (rows >> (threadIdx.x & 31)) & 1u;
  const uint32_t top = __reduce_max_sync(0xffffffffu, has ? static_cast<uint32_t>(exp) : 0u);
  const uint32_t low =
      __reduce_min_sync(0xffffffffu, has && exp >= from ? static_cast<uint32_t>(exp) : 255u);
  *span = max(static_cast<int>(top) - static_cast<int>(low), 0);
  return static_cast<int>(top);
}

// *p, or `other` where there is nothing to load: the loaded register itself, so that nothing
// waits for it before it is used.
__device__ __forceinline__ int load_if(bool has, const int32_t* p, int other) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "mov.b32 %0, %3;\n\t"
      "@p ld.global.b32 %0, [%1];\n\t}"
      : "=&r"(x)
      : "l"(p), "r"(static_cast<int>(has)), "r"(other)
      : "memory");
  return x;
}
__device__ __forceinline__ int load_if(bool has, const uint8_t* p, int other) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "mov.b32 %0, %3;\n\t"
      "@p ld.global.u8 %0, [%1];\n\t}"
      : "=&r"(x)
      : "l"(p), "r"(static_cast<int>(has)), "r"(other)
      : "memory");
  return x;
}

// 2^-n in both halves, exactly; 0 beyond 2^-15.
__device__ __forceinline__ uint32_t f16x2_down(int n) {
  const uint32_t h = n <= 0 ? 0x3c00u : n < 15 ? static_cast<uint32_t>(15 - n) << 10 : n == 15 ? 0x200u : 0u;
  return h | h << 16;
}

// Exponent bytes of a key, V's above K's; 127 where no row sees it.
__device__ __noinline__ int exps_of(const TcArgs& p, const Item& it, const Sight& see, int tok) {
  const AttnArgs& a = p.a;
  if (tok < see.any_lo || tok >= see.any_hi) return 127 | 127 << 8;
  const int blk = fast_div(tok, p.page);
  const int page = a.table[static_cast<int64_t>(it.r) * a.width + blk];
  if (page < 0 || page >= a.P) return 127 | 127 << 8;
  const int64_t where = page * p.sc.s_page + a.layer * p.sc.s_layer + it.h * p.sc.s_head +
                        fast_div(tok - blk * a.B, p.block);
  return p.sc.exps[0][where] | p.sc.exps[1][where] << 8;
}

template <int D, bool F8>
__global__ void __launch_bounds__(F8 ? kThreadsScaled : kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs p) {
  using C = Cfg<D, F8>;
  constexpr int kThreads = C::kThreads;
  constexpr int NS = C::kSlots;
  using B = Bars<NS, C::kStages, F8>;
  constexpr uint32_t kIdescS = F8 ? idesc_f16_f32(kRowsM, kHalf) : idesc_bf16_f32(kRowsM, kHalf);
  constexpr uint32_t kIdescO =
      (F8 ? idesc_f16_f32(kRowsM, D) : idesc_bf16_f32(kRowsM, D)) | kIdescBMnMajor;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  B* b;
  if constexpr (F8) {
    // no room to align them in: all of it is dynamic, and begins where it should
    b = reinterpret_cast<B*>(smem + C::kTiles);
    if ((smem_u32(smem) & 1023u) != 0) {
      if (threadIdx.x == 0) atomicCAS(p.a.dev_status, 0, static_cast<int32_t>(KVC_ERR_CUDA));
      return;
    }
  } else {
    __shared__ B bars_mem;
    b = &bars_mem;
    smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  }
  uint8_t* q_smem = smem;
  uint8_t* kv_smem = smem + C::kQBytes;
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&b->kv_full[i], F8 ? 4 : 1);
      mbar_init(&b->kv_empty[i], 2);       // one MMA warp for each stream
    }
    mbar_init(&b->scaled.q_ready, 4);
    mbar_init(&b->q_full, 1);
    mbar_init(&b->q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&b->s_full[i][h], 1);
        mbar_init(&b->p_full[i][h], 4);
      }
      mbar_init(&b->o_seen[i], 4);
      mbar_init(&b->wg[i], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&b->item_full[i], 1);
      mbar_init(&b->item_empty[i], F8 ? 14 : 10);    // 8 softmax, 2 MMA, 4 converting warps
    }
    mbar_init(&b->ml_full, 4);
    mbar_init(&b->ml_empty, 4);
    mbar_init(&b->drain[0], 1);
    mbar_init(&b->drain[1], 1);
    b->abort_flag = 0;
    b->landed[0] = b->landed[1] = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc<512>(&b->tmem_base);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    if (!F8) {
      tma_prefetch_desc(&maps.k);
      tma_prefetch_desc(&maps.v);
    }
  }
  if (!F8 && p.runs * p.run_rows < kTile) {
    // rows that no load ever writes: 0, so that P V is 0 there
    uint4* z = reinterpret_cast<uint4*>(kv_smem);
    for (int i = threadIdx.x; i < NS * C::kSlotBytes / 16; i += kThreads)
      z[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  grid_wait();
  Walker w = walker_begin<kThreads>(p.s, &b->sched, a.dev_status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b->tmem_base;
  const uint32_t tS[2] = {tmem, tmem + 128};
  const uint32_t tO[2] = {tmem + 256, tmem + 256 + D};
  if (warp == 8) {
    // ------------------------------------------------------------ producer
    int ring = 0, n_items = 0;
    int s = 0;                                    // ring % NS
    uint32_t wrap = 1;                            // parity of kv_empty[s] to wait for
    bool ok = true;
    const int boxes = p.runs * C::kSub;
    const int my_run = lane / C::kSub, my_sub = lane - my_run * C::kSub;
    const uint32_t tile_bytes = static_cast<uint32_t>(p.runs * p.run_rows) * 128 * C::kSub;
    uint8_t* my_dst = kv_smem + my_sub * kSubBytes + my_run * p.run_rows * 128;
    bool bad_page = false;

    for (;;) {
      Item it;
      const bool more = w.next(p.s, &it);
      const int slot = n_items % kItems;
      ok = warp_wait(&b->item_empty[slot], ((n_items / kItems) & 1) ^ 1, b);
      if (!ok) break;
      if (more)
        parts(w, &it);
      else
        it.ntiles = 0;
      int edge_lo = 0, edge_hi = 0;
      Sight see{};
      if (more) {
        see = sight(a, it.kv, it.pos0, it.nt);
        edges(p.s, see, &edge_lo, &edge_hi);
      }
      if (lane == 0) {
        b->items[slot].it = it;
        b->items[slot].ring0 = ring;
        b->items[slot].edge_lo = edge_lo;
        b->items[slot].edge_hi = edge_hi;
        mbar_arrive(&b->item_full[slot]);
      }
      __syncwarp();
      if (!more) break;
      const bool pair = it.nt > p.tok_tile;

      // Page and first row in it of the lane's box of key tiles 0, 1, ... in order,
      // looked up one tile ahead.  A box beyond the pool (page P) is filled with 0, as is
      // one that no row sees: its page may not be the request's any more.
      const int32_t* table = a.table + static_cast<int64_t>(it.r) * a.width;
      struct Box {
        int page, row;
      };
      auto fetch = [&](int tile) -> Box {
        const int tok = tile_span(p, tile).tok0 + my_run * p.run_tokens;
        if (lane >= boxes || tok >= see.any_hi || tok + p.run_tokens <= see.any_lo)
          return Box{kNoPage, 0};
        const int blk = fast_div(tok, p.page);
        return Box{table[blk], tok - blk * a.B};
      };
      Box ahead{0, 0}, now{0, 0}, before{0, 0};    // of the next, the last two K tiles
      if (!F8) ahead = fetch(it.tile0);

      // Q: one box per row tile and 64 columns
      ok = warp_wait(&b->q_empty, (n_items & 1) ^ 1, b);
      if (!ok) break;
      if (lane == 0) {
        const int tiles = pair ? 2 : 1;
        mbar_arrive_expect_tx(&b->q_full,
                              static_cast<uint32_t>(tiles * C::kSub * a.G * p.tok_tile) * 128);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < C::kSub; ++c)
            tma_load_3d(q_smem + (t * C::kSub + c) * kSubBytes, &maps.q, &b->q_full, c * 64,
                        it.h * a.G, it.q0 + t * p.tok_tile);
      }
      ++n_items;

      const int n = it.ntiles;
      if (F8) {                                    // the converting warps fetch the tiles
        ring += 2 * n;
        continue;
      }
      int i_k = 0, i_v = 0;                        // next tiles
#pragma unroll 1
      for (int pos = 0; pos < 2 * n; ++pos) {
        // the order in which the MMAs take them: ring_k, ring_v
        const bool is_v = pos == 2 * n - 1 || (pair ? (pos & 1) : pos >= 2 && !(pos & 1));
        Box use;
        if (is_v) {
          use = i_v + 1 == i_k ? now : before;
          ++i_v;
        } else {
          before = now;
          now = ahead;
          ++i_k;
          ahead = fetch(it.tile0 + i_k);
          if (now.page < 0 || now.page >= a.P) {
            bad_page |= now.page != kNoPage;
            now.page = a.P;
          }
          use = now;
        }
        uint64_t* bar = &b->kv_full[s];
        ok = warp_wait(&b->kv_empty[s], wrap, b);
        if (!ok) break;
        if (is_v && lane < 4) b->poison[s][lane] = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar, tile_bytes);
        __syncwarp();
        if (lane < boxes)
          tma_load_5d(my_dst + s * C::kSlotBytes, is_v ? &maps.v : &maps.k, bar, my_sub * 64,
                      use.row, it.h, a.layer, use.page);
        ++ring;
        if (++s == NS) {
          s = 0;
          wrap ^= 1;
        }
      }
      if (!ok) break;
    }
    if (bad_page) atomicCAS(a.dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
    if (!ok) {
      // the copies in flight write to this CTA's shared memory: let them land
      for (int i = ring - 1; !F8 && i >= 0 && i >= ring - NS; --i)
        mbar_wait_bounded(&b->kv_full[i % NS], (i / NS) & 1, kWaitLimitNs);
      if (n_items > 0) mbar_wait_bounded(&b->q_full, (n_items - 1) & 1, kWaitLimitNs);
    }
  } else if (warp == 9 || warp == 11) {
    // ------------------------------------------------- MMAs of one stream
    // Values that every MMA needs come out of a warp reduction: the compiler then
    // knows that they are uniform and keeps the descriptors in uniform registers.
    const int st = uniform(warp == 9 ? 0 : 1);
    const uint32_t base = uniform(tmem);
    const uint32_t dS = base + st * 128, dO = base + 256 + st * D;
    // low words of the shared-memory descriptors
    const uint64_t desc_q = desc_kmajor_sw128(uniform(smem_u32(q_smem)));
    const uint64_t desc_k = desc_kmajor_sw128(uniform(smem_u32(kv_smem)));
    const uint64_t desc_v = desc_mnmajor_sw128(uniform(smem_u32(kv_smem)), kSubBytes);
    uint32_t ph_p = 0, ph_o = 0;
    bool ended = false;                            // an item's O may not be seen yet
    bool ok = true;
    for (int n_items = 0; ok; ++n_items) {
      const int slot = n_items % kItems;
      ok = warp_wait(&b->item_full[slot], (n_items / kItems) & 1, b);
      if (!ok) break;
      const int n = uniform(b->items[slot].it.ntiles);
      if (n == 0) break;
      const bool pair = uniform(b->items[slot].it.nt) > p.tok_tile;
      const int ring0 = uniform(b->items[slot].ring0);
      if (lane == 0) mbar_arrive(&b->item_empty[slot]);
      __syncwarp();
      const int first = pair ? 0 : st, step = pair ? 1 : 2;
      const uint64_t dq = desc_q + static_cast<uint64_t>((pair ? st : 0) * (C::kSlotBytes >> 4));

      // Both MMA warps see every tile of the ring pass, in its order, and both free
      // every slot: a wait on a parity is only good for the next phase.
      auto full = [&](int pos) {
        return warp_wait(&b->kv_full[pos % NS], (pos / NS) & 1, b);
      };
      int seen = ring0;                            // single mode: next position not seen
      auto pass_to = [&](int pos) {                // tiles of the other stream
        for (; seen < pos; ++seen) {
          if (!full(seen)) return false;
          if (lane == 0) mbar_arrive(&b->kv_empty[seen % NS]);
          __syncwarp();
        }
        return true;
      };
      auto own = [&](int pos) {
        if (!pair && !pass_to(pos)) return false;
        seen = pos + 1;
        return full(pos);
      };
      ok = warp_wait(F8 ? &b->scaled.q_ready : &b->q_full, n_items & 1, b);
      if (!ok) break;
      if (first >= n) {                            // single mode, one tile: none for stream 1
        if (lane == 0) mbar_arrive(&b->q_empty);
        __syncwarp();
        ok = pass_to(ring0 + 2 * n);
        continue;
      }
      // the next phase of s_full must not complete before the last one was seen
      if (ended) {
        ok = warp_wait(&b->o_seen[st], ph_o, b);
        if (!ok) break;
        ph_o ^= 1;
      }
      ended = true;
      // For each half of the keys: O += P V of the tile before, then S of tile i, so
      // that a half's scores are made while the other half's are exponentiated.
#pragma unroll 1
      for (int i = first;; i += step) {
        const bool pv = i > first, more = i < n;
        const int v_at = ring0 + ring_v(pair, n, i - step), k_at = ring0 + ring_k(pair, i);
        if (pv) {
          ok = own(v_at);
          if (!ok) break;
          if (lane == 0) raise_count(&b->landed[st]);
        }
        if (more) ok = own(k_at);
        if (!ok) break;
        const uint64_t dv = desc_v + static_cast<uint64_t>(v_at % NS * (C::kSlotBytes >> 4));
        const uint64_t dk = desc_k + static_cast<uint64_t>(k_at % NS * (C::kSlotBytes >> 4));
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t tS_h = dS + h * kHalf;
          if (pv) {
            ok = warp_wait(&b->p_full[st][h], ph_p, b);
            if (!ok) break;
            tc_fence_after();
            const volatile Told* told = &b->told[st][h];
            const uint32_t heavy = uniform(told->heavy);
            const uint32_t acc = i > first + step || h > 0 ? 1u : uniform(told->o_init);
            const uint64_t dvh = dv + h * (kHalf * 128 >> 4);
            static_assert(kHalf == 64, "four steps of 16 keys");
            mma_bf16_ts_x4(dO, tS_h, dvh, kIdescO, acc);
            if (!F8 && heavy != 0) {
              // the rest of P, for the warps that have one in the step
#pragma unroll 1
              for (int k = 0; k < kHalf / 16; ++k) {
                const uint32_t who = (heavy >> k) & 0x01010101u;
                if (who == 0) continue;
                const uint32_t off[4] = {(who & 1u) - 1u, ((who >> 8) & 1u) - 1u,
                                         ((who >> 16) & 1u) - 1u, ((who >> 24) & 1u) - 1u};
                mma_bf16_ts_lanes(dO, tS_h + kHalf / 2 + k * 8, dvh + k * (2048 >> 4), kIdescO,
                                       off);
              }
            }
          }
          if (more) {
            const uint64_t dkh = dk + h * (kHalf * 128 >> 4);
            // 64 columns of d in each 128-byte row
            mma_bf16_ss_x4(tS_h, dq, dkh, kIdescS, 0);
            if (D == 128)
              mma_bf16_ss_x4(tS_h, dq + (kSubBytes >> 4), dkh + (kSubBytes >> 4), kIdescS, 1);
          }
          mma_commit_elect(&b->s_full[st][h]);
        }
        if (!ok) break;
        if (pv) {
          ph_p ^= 1;
          mma_commit_elect(&b->kv_empty[v_at % NS]);
        }
        if (!more) break;
        mma_commit_elect(&b->kv_empty[k_at % NS]);
        if (i + step >= n) mma_commit_elect(&b->q_empty);
      }
      if (ok && !pair) ok = pass_to(ring0 + 2 * n);
    }
    if (!ok) {
      mma_commit_elect(&b->drain[st]);
      mbar_wait_bounded(&b->drain[st], 0, kWaitLimitNs);
      __syncwarp();
    }
  } else if (warp < 8) {
    // -------------------------------------------------------------- softmax
    const int st = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;    // lane 32 w in bits 31-16
    const uint32_t sS = tS[st] + lane_base, sO = tO[st] + lane_base;
    const int row_tok = row / a.G, row_g = row - row_tok * a.G;
    const bool row_in_tile = row_tok < p.tok_tile;
    uint32_t ph_s = 0, ph_wg = 0, ph_ml = 0;
    int32_t n_tiles = 0;                          // tiles of the stream in earlier items
    int32_t* counters = static_cast<int32_t*>(a.workspace);
    float* slots =
        reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kAttnCounterBytes);
    const size_t slot_n = slot_floats(kSlotRows, D);
    bool ok = true;
    // the four warps of the stream meet
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->wg[st]);
      const bool met = warp_wait(&b->wg[st], ph_wg, b);
      ph_wg ^= 1;
      return met;
    };

    for (int n_items = 0; ok; ++n_items) {
      const int slot = n_items % kItems;
      ok = warp_wait(&b->item_full[slot], (n_items / kItems) & 1, b);
      if (!ok) break;
      // (Scaled pools: the item stays where it is until the next one, for the registers.)
      using Kept = std::conditional_t<F8, const ItemSlot&, const ItemSlot>;
      Kept kept = b->items[slot];
      const Item& it = kept.it;
      const int ring0 = kept.ring0;
      const int edge_lo = kept.edge_lo, edge_hi = kept.edge_hi;
      __syncwarp();
      if (it.ntiles == 0) break;
      const int give = F8 ? (n_items + kItems - 1) % kItems : slot;
      if (lane == 0 && (!F8 || n_items > 0)) mbar_arrive(&b->item_empty[give]);
      const bool pair = it.nt > p.tok_tile;
      const int n_st = pair ? it.ntiles : (it.ntiles + 1 - st) >> 1;
      const int tok_off = pair ? st * p.tok_tile : 0;       // first token of the stream's rows
      const int n_tok = min(p.tok_tile, it.nt - tok_off);
      const bool valid = row_in_tile && row_tok < n_tok;
      const bool busy = (warp & 3) * 32 < n_tok * a.G;      // any valid row in the warp
      const int pos = it.pos0 + tok_off + min(row_tok, n_tok - 1);
      const int key_hi = a.causal ? min(it.kv, pos + 1) : it.kv;
      const int key_lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      float m = -INFINITY, l = 0.f;
      float row_scale = a.scale_log2;                       // of the row's scores
      [[maybe_unused]] float v_top = -INFINITY;             // largest exponent of V so far

      for (int kh = 0; kh < 2 * n_st; ++kh) {               // halves of the stream's tiles
        const int k = kh >> 1, half = kh & 1;
        const int i = pair ? k : 2 * k + st;                // key tile of the item
        const bool edge = it.tile0 + i < edge_lo || it.tile0 + i >= edge_hi;
        const uint32_t sH = sS + half * kHalf;
        const uint32_t* bad = nullptr;                      // value rows that are added from memory
        if (edge) {
          // The count says that the barrier's phase is the tile's (a wait on a parity alone
          // could pass one phase early); it stays so until the tile is given back, after
          // these rows' P.  The wait itself then makes the copy's bytes visible here.
          const int ring_pos = ring0 + ring_v(pair, it.ntiles, i), slot_v = ring_pos % NS;
          ok = warp_wait_count(&b->landed[st], n_tiles + k + 1, &b->abort_flag) &&
               warp_wait(&b->kv_full[slot_v], (ring_pos / NS) & 1, b);
          if (!ok) break;
          const TileSpan t = tile_span(p, it.tile0 + i);
          const Sight see = sight(a, it.kv, it.pos0, it.nt);
          const int c0 = tile_col(p, t, see.any_lo), c3 = tile_col(p, t, see.any_hi);
          const int c1 = tile_col(p, t, see.all_lo), c2 = tile_col(p, t, see.all_hi);
          if (half * kHalf < c1 || half * kHalf + kHalf > c2) {   // not seen by all rows
            uint8_t* rows = kv_smem + slot_v * C::kSlotBytes + half * kHalf * 128;
            // 16 bytes at a time, neighbouring threads neighbouring bytes
            auto at = [&](int j, int* n) {
              const int u = row + 128 * j;
              *n = half * kHalf + ((u >> 3) & (kHalf - 1));
              return reinterpret_cast<uint4*>(rows + (u / (8 * kHalf)) * kSubBytes +
                                              ((u >> 3) & (kHalf - 1)) * 128 + (u & 7) * 16);
            };
            auto odd = [](uint32_t u) {                       // an exponent of all ones
              constexpr uint32_t ones = F8 ? 0x7c00u : 0x7f80u;
              return (u & ones) == ones || (u & ones << 16) == ones << 16;
            };
            auto fma2 = [](uint32_t x, uint32_t z) {
              return F8 ? fma_f16x2(x, 0, z) : fma_bf16x2(x, 0, z);
            };
            // 0 times each is 0, or NaN
            uint32_t z0 = 0, z1 = 0;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              int n;
              const uint4 v = *at(j, &n);
              z0 = fma2(v.x, z0);
              z1 = fma2(v.y, z1);
              z0 = fma2(v.z, z0);
              z1 = fma2(v.w, z1);
            }
            if ((z0 | z1) != 0) {
#pragma unroll 1
              for (int j = 0; j < D / 16; ++j) {
                int n;
                uint4* q = at(j, &n);
                if (n >= c1 && n < c2) continue;
                const uint4 v = *q;
                if (!(odd(v.x) || odd(v.y) || odd(v.z) || odd(v.w))) continue;
                if (n >= c0 && n < c3) {
                  atomicOr(&b->poison[slot_v][n >> 5], 1u << (n & 31));
                } else {
                  *q = make_uint4(0, 0, 0, 0);                  // no row sees it
                  fence_proxy_async_smem();
                }
              }
            }
            ok = meet();
            if (!ok) break;
            bad = &b->poison[slot_v][2 * half];
            if ((bad[0] | bad[1]) != 0) {
#pragma unroll 1
              for (int j = 0; j < D / 16; ++j) {
                int n;
                uint4* q = at(j, &n);
                if ((bad[(n >> 5) & 1] >> (n & 31)) & 1u) *q = make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              ok = meet();
              if (!ok) break;
            } else {
              bad = nullptr;
            }
          }
        }
        ok = warp_wait(&b->s_full[st][half], ph_s, b);
        if (!ok) break;
        if (busy) {
          tc_fence_after();
          // O may be touched once the product of the half before is in it: that half's next
          // scores (or the end of the item) are signalled after it
          auto settle = [&]() {
            const bool there = warp_wait(&b->s_full[st][half ^ 1], ph_s ^ (half ? 1u : 0u), b);
            tc_fence_after();
            return there;
          };
          [[maybe_unused]] uint32_t heavy = 0;               // steps with P as two numbers
          if constexpr (F8) {
            // Scaled pools.  32 keys at a time, which share an exponent of K and one of V, and
            // twice over the scores (their largest, then P): the registers of 512 threads hold
            // no more.  m follows the largest exponent of a value's term, x + e of its block,
            // or a score by far, so that P as fp16 is good to 2^-30 of the largest term.
            if (kh == 0)
              row_scale =
                  a.scale_log2 *
                  pow2_of(127 - b->scaled.q_up[n_items & 1][(pair ? st * kRowsM : 0) + row]);
            const auto& info = b->scaled.tile[(ring0 + ring_k(pair, i)) % (2 * NS)];
            uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
            if (edge) {
              const TileSpan t = tile_span(p, it.tile0 + i);
              const int lo = tile_col(p, t, key_lo) - half * kHalf;
              const int hi = tile_col(p, t, key_hi) - half * kHalf;
              keep0 = bits_below(hi) & ~bits_below(lo);
              keep1 = bits_below(hi - 32) & ~bits_below(lo - 32);
            }
            // Keys with exponents of their own, or so far apart that sums of the smaller terms
            // would not be seen by those of the weights, are taken one by one.
            const float2 v_exp = *reinterpret_cast<const float2*>(&info.v_exp[2 * half]);
            auto spans = [&]() -> uint32_t {
              return *reinterpret_cast<const uint16_t*>(&info.span[2 * half]);
            };
            v_top = max3(v_top, v_exp.x, v_exp.y);
            const bool apart = (fminf(v_exp.x, v_exp.y) < v_top - kApart) |
                               ((spans() & (kOwn | kOwn << 8)) != 0);
            uint32_t x[32];
            auto scores = [&](int g) {
              tmem_ld_32x32b_x32(sH + 32 * g, x);
              tmem_ld_wait();
              const uint32_t keep = g ? keep1 : keep0;
              if (__any_sync(0xffffffffu, keep != 0xffffffffu)) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!((keep >> j) & 1u)) x[j] = 0xff800000u;               // -inf
              }
            };
            auto sc = [&](int j) { return __uint_as_float(x[j]); };
            // exponent bytes of key `lane` of group g, V's above K's
            auto own_exps = [&](int g) {
              if (info.span[2 * half + g] != kOwn)
                return exp_byte(info.k[2 * half + g]) |
                       static_cast<int>(info.v_exp[2 * half + g] + 127.f) << 8;
              return exps_of(p, it, sight(a, it.kv, it.pos0, it.nt),
                             tile_span(p, it.tile0 + i).tok0 + half * kHalf + 32 * g + lane);
            };
            float top = -INFINITY;
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
              scores(g);
              float t, far;
              if (!apart) {
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = max3(sc(8 * c), sc(8 * c + 1), sc(8 * c + 2));
#pragma unroll
                for (int j = 3; j < 7; j += 2)
#pragma unroll
                  for (int c = 0; c < 4; ++c) mx[c] = max3(mx[c], sc(8 * c + j), sc(8 * c + j + 1));
#pragma unroll
                for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], sc(8 * c + 7));
                far = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) *
                      score_scale(row_scale, info.k[2 * half + g]);
                t = far + info.v_exp[2 * half + g];
              } else {
                const int own = own_exps(g);
                t = far = -INFINITY;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const int e = __shfl_sync(0xffffffffu, own, j);
                  const float y = sc(j) * score_scale(row_scale, pow2_of(e & 255));
                  far = fmaxf(far, y);
                  t = fmaxf(t, y + static_cast<float>((e >> 8) - 127));
                }
              }
              top = max3(top, t, far - kFar);
            }
            const bool raise = top > m + kRoom || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, raise)) {
              // a term may be smaller than `top` says by its group's span
              const uint32_t two = spans();
              const uint32_t span = max(two & (kOwn - 1), (two >> 8) & (kOwn - 1));
              const float m_new = raise ? top - (kTop + static_cast<float>(span)) : m;
              const float f = raise ? exp2_fast(m - m_new) : 1.f;            // 0 from m = -inf
              // l may have what m lacks: in two steps
              const float h = raise ? exp2_fast(0.5f * (m - m_new)) : 1.f;
              l = l * h * h;
              m = m_new;
              if (kh > 0) {
                ok = settle();
                if (!ok) break;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  tmem_ld_32x32b_x32(sO + c, x);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                  tmem_st_32x32b_x32(sO + c, x);
                }
              }
            }
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
              scores(g);
              uint64_t sum[2] = {0, 0};
              float v_inv = 1.f;
              if (!apart) {
                const uint32_t sc_bits =
                    __float_as_uint(score_scale(row_scale, info.k[2 * half + g]));
                const uint32_t ref_bits = __float_as_uint(info.v_exp[2 * half + g] - ref);
                const uint64_t scale2 = pack_f32x2(sc_bits, sc_bits);
                const uint64_t ref2 = pack_f32x2(ref_bits, ref_bits);
                v_inv = info.v_inv[2 * half + g];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  float p0, p1;
                  unpack_f32x2(fma_f32x2(pack_f32x2(x[j], x[j + 1]), scale2, ref2), p0, p1);
                  p0 = exp2_fast(p0);
                  p1 = exp2_fast(p1);
                  sum[(j >> 1) & 1] = add_f32x2(
                      sum[(j >> 1) & 1], pack_f32x2(__float_as_uint(p0), __float_as_uint(p1)));
                  x[j >> 1] = pack_f16(p0, p1);
                }
              } else {
                const int own = own_exps(g);
                float s0 = 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  float q[2];
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const int e = __shfl_sync(0xffffffffu, own, j + c);
                    const float y = sc(j + c) * score_scale(row_scale, pow2_of(e & 255));
                    s0 += exp2_fast(y - ref);
                    q[c] = exp2_fast(y + (static_cast<float>((e >> 8) - 127) - ref));
                  }
                  x[j >> 1] = pack_f16(q[0], q[1]);
                }
                sum[0] = pack_f32x2(__float_as_uint(s0), 0);
              }
              tmem_st_32x32b_x16(sH + 16 * g, x);
              float s0, s1;
              unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
              l = fmaf(s0 + s1, v_inv, l);
            }
          } else {
            uint32_t x[kHalf];
            tmem_ld_32x32b_x32(sH, x);
            tmem_ld_32x32b_x32(sH + 32, x + 32);
            tmem_ld_wait();
            if (edge || p.ragged) {
              const TileSpan t = tile_span(p, it.tile0 + i);
              const int lo = tile_col(p, t, key_lo) - half * kHalf;
              const int hi = min(tile_col(p, t, key_hi), p.has_holes ? kTile : t.cnt) - half * kHalf;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t keep = bits_below(hi - 32 * c) & ~bits_below(lo - 32 * c) &
                                      ~(half == 0 ? p.holes[c] : p.holes[2 + c]);
                if (__any_sync(0xffffffffu, keep != 0xffffffffu)) {
#pragma unroll
                  for (int j = 0; j < 32; ++j)
                    if (!((keep >> j) & 1u)) x[32 * c + j] = 0xff800000u;    // -inf
                }
              }
            }
            auto sc = [&](int j) { return __uint_as_float(x[j]); };
            float mx[4];                                       // of each 16 keys
#pragma unroll
            for (int g = 0; g < 4; ++g) mx[g] = max3(sc(16 * g), sc(16 * g + 1), sc(16 * g + 2));
#pragma unroll
            for (int j = 3; j < 15; j += 2)
#pragma unroll
              for (int g = 0; g < 4; ++g) mx[g] = max3(mx[g], sc(16 * g + j), sc(16 * g + j + 1));
#pragma unroll
            for (int g = 0; g < 4; ++g) mx[g] = fmaxf(mx[g], sc(16 * g + 15));
            const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale_log2;
            const bool raise = top > m + kLag || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, raise)) {
              const float f = raise ? exp2_fast(m - top) : 1.f;              // 0 from m = -inf
              if (raise) m = top;
              l *= f;
              if (kh > 0) {
                ok = settle();
                if (!ok) break;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  uint32_t o[32];
                  tmem_ld_32x32b_x32(sO + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                  tmem_st_32x32b_x32(sO + c, o);
                }
              }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const uint32_t sc_bits = __float_as_uint(a.scale_log2), ref_bits = __float_as_uint(-ref);
            const uint64_t scale2 = pack_f32x2(sc_bits, sc_bits);
            const uint64_t ref2 = pack_f32x2(ref_bits, ref_bits);
            // steps of 16 keys in which one has more than a share of the row's sum so far
            const float p_top = exp2_fast(top - ref);
            const float least = (pair ? kHeavyPair : kHeavySingle) * (l + p_top);
            if (__any_sync(0xffffffffu, valid && p_top > least)) {
#pragma unroll
              for (int g = 0; g < 4; ++g)
                if (__any_sync(0xffffffffu,
                               valid && exp2_fast(fmaf(mx[g], a.scale_log2, -ref)) > least))
                  heavy |= 1u << g;
            }
            // P, in passes without branches, so that the exponentials of many keys are in
            // flight: 64 where no step needs two numbers, 16 elsewhere
            uint64_t sum[2] = {0, 0};
            auto two = [&](int j) {                            // keys j, j + 1
              float p0, p1;
              unpack_f32x2(fma_f32x2(pack_f32x2(x[j], x[j + 1]), scale2, ref2), p0, p1);
              const uint64_t p2 =
                  pack_f32x2(__float_as_uint(exp2_fast(p0)), __float_as_uint(exp2_fast(p1)));
              sum[(j >> 1) & 1] = add_f32x2(sum[(j >> 1) & 1], p2);
              unpack_f32x2(p2, p0, p1);
              x[j >> 1] = pack_bf16(p0, p1);
              return p2;
            };
            if (heavy == 0) {
#pragma unroll
              for (int j = 0; j < kHalf; j += 2) two(j);
            } else {
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                if (((heavy >> g) & 1u) == 0) {
#pragma unroll
                  for (int j = 16 * g; j < 16 * g + 16; j += 2) two(j);
                  continue;
                }
                uint32_t rest[8];
#pragma unroll
                for (int j = 16 * g; j < 16 * g + 16; j += 2) {
                  const uint64_t p2 = two(j);
                  x[j >> 1] = cut_bf16(p2);
                  rest[(j >> 1) & 7] = rest_bf16(p2, x[j >> 1]);
                }
                tmem_st_32x32b_x8(sH + kHalf / 2 + 8 * g, rest);
              }
            }
            tmem_st_32x32b_x32(sH, x);
            {
              float s0, s1;
              unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
              l += s0 + s1;
            }
          }
          if (lane == 0)
            reinterpret_cast<volatile uint8_t*>(&b->told[st][half].heavy)[warp & 3] = heavy;
          tmem_st_wait();

          bool init = false;
          if (bad != nullptr) {
            if (kh > 0) {
              ok = settle();
              if (!ok) break;
            }
#pragma unroll 1
            for (int n = 0; n < kHalf; ++n) {
              if (!((bad[n >> 5] >> (n & 31)) & 1u)) {
                if ((bad[n >> 5] >> (n & 31)) == 0) n |= 31;      // none left in the word
                continue;
              }
              const TileSpan t = tile_span(p, it.tile0 + i);
              const int tok = tile_tok(p, t, n + half * kHalf), blk = fast_div(tok, p.page);
              const int page = a.table[static_cast<int64_t>(it.r) * a.width + blk];
              auto half_of = [&](uint32_t two_p) {
                if (F8) {
                  float p0, p1;
                  f16x2_f32(two_p, p0, p1);
                  return (n & 1) ? p1 : p0;
                }
                return __uint_as_float((n & 1) ? two_p & 0xffff0000u : two_p << 16);
              };
              const uint32_t two_p = tmem_ld_32x32b_x1(sH + (n >> 1));
              const uint32_t two_r = tmem_ld_32x32b_x1(sH + kHalf / 2 + (n >> 1));
              tmem_ld_wait();
              const float pr =
                  half_of(two_p) + ((heavy >> (n >> 4)) & 1u ? half_of(two_r) : 0.f);
              const int64_t v = page * a.pool[1].s_req + a.layer * a.pool[1].s_layer +
                                it.h * a.pool[1].s_head +
                                static_cast<int64_t>(tok - blk * a.B) * a.pool[1].s_tok;
              // (fp16 has no number for weights that a NaN still has to show in)
              const bool sees = tok >= key_lo && tok < key_hi;
              float v_scale = 1.f;                           // beside the group's, which P has
              if constexpr (F8) {
                const auto& info = b->scaled.tile[(ring0 + ring_k(pair, i)) % (2 * NS)];
                const int g = 2 * half + (n >> 5);
                const int e = p.sc.exps[1][page * p.sc.s_page + a.layer * p.sc.s_layer +
                                           it.h * p.sc.s_head + fast_div(tok - blk * a.B, p.block)];
                if (info.span[g] != kOwn)
                  v_scale = pow2_of(max(e - static_cast<int>(info.v_exp[g]), 0));
              }
              auto value = [&](int c) {
                if (F8)
                  return e4m3_f32(static_cast<const uint8_t*>(a.pool[1].base)[v + c]) * v_scale;
                return __bfloat162float(static_cast<const __nv_bfloat16*>(a.pool[1].base)[v + c]);
              };
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(sO + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const float old = kh > 0 || init ? __uint_as_float(o[j]) : 0.f;
                  const float add = (F8 ? sees : pr != 0.f) ? pr * value(c + j) : 0.f;
                  o[j] = __float_as_uint(old + add);
                }
                tmem_st_32x32b_x32(sO + c, o);
                tmem_st_wait();
              }
              init = true;
            }
          }
          if (kh == 0 && (warp & 3) == 0 && lane == 0) b->told[st][0].o_init = init ? 1 : 0;
          tc_fence_before();
        } else if (lane == 0) {
          reinterpret_cast<volatile uint8_t*>(&b->told[st][half].heavy)[warp & 3] = 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->p_full[st][half]);
        ph_s ^= half;                                        // both halves' phases are alike
      }
      if (!ok) break;
      n_tiles += n_st;
      if (n_st > 0) {
        // O is complete
        ok = warp_wait(&b->s_full[st][0], ph_s, b) && warp_wait(&b->s_full[st][1], ph_s, b);
        if (!ok) break;
        ph_s ^= 1;
        tc_fence_after();
        if (lane == 0) mbar_arrive(&b->o_seen[st]);
        __syncwarp();
      }

      // single mode: stream 0 joins the two streams' rows
      float f0 = 1.f, f1 = 0.f;
      if (F8) {
        // m follows the values' terms: O / l, and m that of the scores
        f0 = l == 0.f ? 0.f : 1.f / l;
        m = l == 0.f ? -INFINITY : m + log2f(l);
        l = l == 0.f ? 0.f : 1.f;
      }
      const bool join = !pair && it.ntiles > 1;
      if (join) {
        if (st == 1) {
          b->ml[row][0] = m;
          b->ml[row][1] = F8 ? f0 : l;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->ml_full);
          ok = warp_wait(&b->ml_empty, ph_ml, b);
          if (!ok) break;
          ph_ml ^= 1;
          continue;
        }
        ok = warp_wait(&b->ml_full, ph_ml, b);
        if (!ok) break;
        ph_ml ^= 1;
        tc_fence_after();
        const float m1 = b->ml[row][0], l1 = b->ml[row][1];
        const float top = fmaxf(m, m1);
        const float w0 = part_weight(m, l, top), w1 = part_weight(m1, l1, top);
        if (F8) {
          l = w0 + w1;
          f0 *= w0;
          f1 = l1 * w1;
        } else {
          f0 = w0;
          f1 = w1;
          l = l * f0 + l1 * f1;
        }
        m = top;
      } else if (!pair && st == 1) {
        continue;
      }
      const bool whole_item = it.nparts == 1;
      const float inv = whole_item ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const int head = it.h * a.G + row_g;
      const int64_t q_row = it.q0 + tok_off + row_tok;
      const int slot_row = (pair ? st * kRowsM : 0) + row;
      float* part = slots + (static_cast<size_t>(blockIdx.x) * 2 + slot_of(it.part)) * slot_n;
      if (busy) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + q_row * a.o_tok + head * a.o_head;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(sO + c, o);
          tmem_ld_wait();
          if (join) {
            uint32_t o1[32];
            tmem_ld_32x32b_x32(tO[1] + lane_base + c, o1);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float u = f0 == 0.f ? 0.f : __uint_as_float(o[j]) * f0;
              const float v = f1 == 0.f ? 0.f : __uint_as_float(o1[j]) * f1;
              o[j] = __float_as_uint(u + v);
            }
          } else if (F8) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = f0 == 0.f ? 0u : __float_as_uint(__uint_as_float(o[j]) * f0);
          }
          if (valid && whole_item) {
            uint32_t u[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              u[j] = l == 0.f ? 0u
                              : pack_bf16(__uint_as_float(o[2 * j]) * inv,
                                          __uint_as_float(o[2 * j + 1]) * inv);
            if (p.out32) {                         // whole sectors, half the requests
              st_global_32(out + c, u);
              st_global_32(out + c + 16, u + 8);
            } else {
#pragma unroll
              for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<uint4*>(out + c + 2 * j) =
                    make_uint4(u[j], u[j + 1], u[j + 2], u[j + 3]);
            }
          } else if (valid) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(part + ((c + j) / 4 * kSlotRows + slot_row) * 4) =
                  make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
        tc_fence_before();
        if (valid && whole_item && a.lse != nullptr)
          a.lse[q_row * (a.H * a.G) + head] =
              l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        if (valid && !whole_item) {
          part[kSlotRows * D + slot_row] = m;
          part[kSlotRows * D + kSlotRows + slot_row] = l;
        }
      }
      __syncwarp();
      if (join && lane == 0) mbar_arrive(&b->ml_empty);
      if (whole_item) continue;

      // a divided item: join the parts if all others have left theirs
      __threadfence();
      ok = meet();
      if (!ok) break;
      if (row == 0) {
        __threadfence();
        b->last[st] = atomicAdd(counters + 2 * it.cta0 + st, 1) == it.nparts - 1;
      }
      ok = meet();
      if (!ok) break;
      if (!b->last[st]) continue;
      __threadfence();
      if (row == 0) counters[2 * it.cta0 + st] = 0;
      if (valid)
        join_row<D, 8, 2>(slots + static_cast<size_t>(it.cta0) * 2 * slot_n, slot_n, it.nparts,
                          slot_row,
                          static_cast<__nv_bfloat16*>(a.out) + q_row * a.o_tok + head * a.o_head,
                          p.out32, a.lse == nullptr ? nullptr : a.lse + q_row * (a.H * a.G) + head);
    }
  } else if (warp >= 12) {
    if constexpr (F8) {
      // --------------------------- numbers of scaled pools: fetched, and made fp16 tiles
      // Each warp has 32 keys of every tile, copies their rows some tiles ahead of what it
      // converts, and shares nothing with the other three but the slots' barriers.  One warp's
      // time for a tile is all latency: nothing below is waited for where it is loaded.
      constexpr int kUnits = D / 16;               // 16-byte units of a row
      constexpr int kAtOnce = 32 / kUnits;         // rows of a warp's 32 units
      const int row0 = (warp - 12) * 32;
      uint8_t* stages = kv_smem + NS * C::kSlotBytes + (warp - 12) * C::kStages * C::kStageBytes;
      // Row and unit of a lane among the kAtOnce rows of a load: eight lanes have units of two
      // neighbouring rows such that neither their reads nor their writes share a bank.
      const int unit = lane % kUnits;
      const int sub = D == 128 ? (lane >> 4) * 2 + (((lane >> 2) ^ (lane >> 3)) & 1) : lane / kUnits;
      bool ok = true, more = true, bad_page = false;
      int n_items = 0, pos = 0, end = 0, i_k = 0, tile0 = 0;
      bool pair = false;
      Sight see{};
      const int32_t* table = a.table;
      const uint8_t *src[2] = {nullptr, nullptr}, *exps[2] = {nullptr, nullptr};
      int ahead = 0;                               // page of the lane's key of the next K tile
      // what a V tile takes over from its K
      struct Keys {
        int64_t off;                               // of the lane's row
        int page, row;
        uint32_t rows;                             // lanes that have one
      } now{}, before{};
      const bool alike = a.pool[0].s_req == a.pool[1].s_req && a.pool[0].s_tok == a.pool[1].s_tok;
      auto page_of = [&](int tile) -> int {
        const int tok = tile * kTile + row0 + lane;
        const bool seen = tok >= see.any_lo && tok < see.any_hi;
        return load_if(seen, table + (seen ? fast_div(tok, p.page) : 0), kNoPage);
      };
      struct Staged {
        int kind;                                  // 0: nothing, 1: K, 2: V; with the item's first
                                                   // tile kFirst, and kPair if it has two row tiles;
                                                   // kOld: V of the K before the last
        uint32_t rows;                             // that are there; the others are zeros
        int exp_k, exp_v;                          // exponent bytes of the lane's key
      };
      constexpr int kFirst = 4, kPair = 8, kOld = 16;
      // Starts the copy of the next tile into stage `st`.
      auto issue = [&](int st) -> Staged {
        if (more && pos == end) {
          const int slot = n_items % kItems;
          ok = warp_wait(&b->item_full[slot], (n_items / kItems) & 1, b);
          more = ok;
          if (ok) {
            const Item it = b->items[slot].it;
            __syncwarp();
            if (lane == 0) mbar_arrive(&b->item_empty[slot]);
            ++n_items;
            more = it.ntiles > 0;
            if (more) {
              pos = i_k = 0;
              end = 2 * it.ntiles;
              tile0 = it.tile0;
              pair = it.nt > p.tok_tile;
              see = sight(a, it.kv, it.pos0, it.nt);
              table = a.table + static_cast<int64_t>(it.r) * a.width;
#pragma unroll
              for (int kv = 0; kv < 2; ++kv) {
                src[kv] = static_cast<const uint8_t*>(a.pool[kv].base) +
                          a.layer * a.pool[kv].s_layer + it.h * a.pool[kv].s_head;
                exps[kv] = p.sc.exps[kv] + a.layer * p.sc.s_layer + it.h * p.sc.s_head;
              }
              ahead = page_of(tile0);
            }
          }
        }
        if (!more) {
          asm volatile("cp.async.commit_group;" ::: "memory");
          return Staged{0, 0, 0, 0};
        }
        const bool is_v = pos == end - 1 || (pair ? (pos & 1) : pos >= 2 && !(pos & 1));
        bool old = false;
        Staged next{is_v ? 2 : 1, 0, 0, 0};
        if (is_v) {
          // of the last K tile, or of the one before it
          old = !(pair || pos == end - 1);
          if (!alike) {
            Keys& keys = old ? before : now;
            keys.off = keys.page * a.pool[1].s_req + keys.row * a.pool[1].s_tok;
          }
        } else {
          const int tile = tile0 + i_k;
          before = now;
          now.page = ahead;
          ahead = page_of(tile + 1);
          if (now.page < 0 || now.page >= a.P) {
            bad_page |= now.page != kNoPage;
            now.page = -1;
          }
          ++i_k;
          const bool has = now.page >= 0;
          const int tok = tile * kTile + row0 + lane;
          now.row = tok - fast_div(tok, p.page) * a.B;
          now.rows = __ballot_sync(0xffffffffu, has);
          now.off = now.page * a.pool[0].s_req + now.row * a.pool[0].s_tok;
          const int64_t where = has ? now.page * p.sc.s_page + fast_div(now.row, p.block) : 0;
          next.exp_k = load_if(has, exps[0] + where, 127);
          next.exp_v = load_if(has, exps[1] + where, 127);
        }
        ++pos;
        if (pos == 1) next.kind |= kFirst | (pair ? kPair : 0);
        if (old) next.kind |= kOld;
        next.rows = old ? before.rows : now.rows;
        const int64_t off = old ? before.off : now.off;
        const uint8_t* base = src[is_v ? 1 : 0] + unit * 16;
        const uint32_t dst = smem_u32(stages + st * C::kStageBytes) + sub * D + unit * 16;
#pragma unroll
        for (int j = 0; j < 32 / kAtOnce; ++j) {
          const int n = j * kAtOnce + sub;
          const int64_t at = __shfl_sync(0xffffffffu, off, n);
          const bool real = (next.rows >> n) & 1u;
          cp_async16(dst + j * 512, real ? base + at : base, real);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return next;
      };
      Staged staged[kMost<C::kStages, 1>] = {};    // of the tiles in the stages
      int s = 0, st = 0, empty = C::kStages, ring = 0, n_q = 0;
      int group_k = 127, group_v = 127, span_v = 0;
      bool wide = false;
      uint32_t down_v = 0, down_before = 0;        // multipliers of V's rows
      uint32_t wrap = 1;
#pragma unroll 1
      while (ok) {
        // The next tile's numbers leave the stage for registers, so that the copy of the one
        // after those in the stages begins before they are converted.
        const Staged now_in = staged[0];
        const bool tile_there = empty == 0;
        if (!tile_there)
          --empty;                                 // the first copies
        else if (now_in.kind == 0)
          break;
        const bool is_v = (now_in.kind & 3) == 2, is_k = (now_in.kind & 3) == 1;
        // The 32 keys get one exponent, the largest of theirs, and the numbers of the others
        // are divided by what is between: exact in fp16 up to 2^15.  With more between all stay
        // as they are and say so; of K, the least exponents (of zeros or next to it) aside, and
        // of V from 2^10 on, for m's sake.
        uint32_t down = now_in.kind & kOld ? down_before : down_v;
        if (is_k) {
          span_v = 0;
          wide = false;
          if (now_in.rows != 0) {                  // (none: as the keys before)
            int span_k;
            group_k = group_exp(now_in.exp_k, now_in.rows, kScaleExpMin + 128, &span_k);
            group_v = group_exp(now_in.exp_v, now_in.rows, 0, &span_v);
            wide = span_k > kSpanK || span_v > kSpanV;
          }
          down_before = down_v;
          down_v = f16x2_down(wide ? 0 : group_v - now_in.exp_v);
          down = f16x2_down(wide ? 0 : group_k - now_in.exp_k);
        }
        uint4 x[32 / kAtOnce];
        if (tile_there) {
          // a lane reads what it copied
          asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
          const uint8_t* from = stages + st * C::kStageBytes + sub * D + unit * 16;
#pragma unroll
          for (int j = 0; j < 32 / kAtOnce; ++j)
            x[j] = *reinterpret_cast<const uint4*>(from + j * 512);
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i + 1 < C::kStages; ++i) staged[i] = staged[i + 1];
        staged[kMost<C::kStages, 1> - 1] = issue(st);
        if (++st == C::kStages) st = 0;
        if (!tile_there) continue;
        ok = ok && warp_wait(&b->kv_empty[s], wrap, b);
        if (!ok) break;
        if (warp == 12 && lane < 4 && is_v) b->poison[s][lane] = 0;
        if (is_k && lane == 0) {
          auto& info = b->scaled.tile[ring % (2 * NS)];
          info.k[warp - 12] = pow2_of(group_k);
          info.v_exp[warp - 12] = static_cast<float>(group_v - 127);
          info.v_inv[warp - 12] = pow2_of(254 - group_v);
          info.span[warp - 12] = static_cast<uint8_t>(wide ? kOwn : span_v);
        }
        // 64 columns to a swizzled tile
        const int half = unit >> 2, c = (unit & 3) * 2;
        uint8_t* to = kv_smem + s * C::kSlotBytes + half * kSubBytes + (row0 + sub) * 128;
#pragma unroll
        for (int j = 0; j < 32 / kAtOnce; ++j) {
          const int n = j * kAtOnce + sub;
          const uint32_t f = __shfl_sync(0xffffffffu, down, n);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t lo = k ? x[j].z : x[j].x, hi = k ? x[j].w : x[j].y;
            uint4 y;
            e4m3_f16x4(lo, y.x, y.y);
            e4m3_f16x4(hi, y.z, y.w);
            y = make_uint4(mul_f16x2(y.x, f), mul_f16x2(y.y, f), mul_f16x2(y.z, f), mul_f16x2(y.w, f));
            *reinterpret_cast<uint4*>(to + j * kAtOnce * 128 + (((c + k) ^ (n & 7)) << 4)) = y;
          }
        }
        fence_proxy_async_smem();                  // for the MMAs
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->kv_full[s]);
        ++ring;
        if (++s == NS) {
          s = 0;
          wrap ^= 1;
        }
        if (now_in.kind & kFirst) {
          // Q, in place: a thread has a row of each row tile
          ok = warp_wait(&b->q_full, n_q & 1, b);
          if (!ok) break;
          const int row = threadIdx.x & 127;
#pragma unroll 1
          for (int t = 0; t < (now_in.kind & kPair ? 2 : 1); ++t) {
            uint8_t* line = q_smem + t * C::kSlotBytes + row * 128;
            auto at = [&](int u) {
              return reinterpret_cast<uint4*>(line + (u >> 3) * kSubBytes + (((u ^ row) & 7) << 4));
            };
            uint32_t top = 0;
#pragma unroll 4
            for (int u = 0; u < D / 8; ++u) {
              const uint4 x = *at(u);
              top = max_abs2(max_abs2(max_abs2(max_abs2(top, x.x), x.y), x.z), x.w);
            }
            const int up = f16_up(top);
            const float f = pow2_of(127 + up);
#pragma unroll 2
            for (int u = 0; u < D / 8; ++u) {
              const uint4 x = *at(u);
              *at(u) = make_uint4(bf16x2_f16x2(x.x, f), bf16x2_f16x2(x.y, f), bf16x2_f16x2(x.z, f),
                                  bf16x2_f16x2(x.w, f));
            }
            b->scaled.q_up[n_q & 1][t * kRowsM + row] = static_cast<int8_t>(up);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b->scaled.q_ready);
          ++n_q;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (bad_page) atomicCAS(a.dev_status, 0, static_cast<int32_t>(KVC_ERR_SHAPE));
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc<512>(tmem);
  if (threadIdx.x == 0 && b->abort_flag != 0)
    atomicCAS(a.dev_status, 0, static_cast<int32_t>(KVC_ERR_DEVICE_TIMEOUT));
}

cudaError_t encode_pool(CUtensorMap* map, const AttnArgs& a, int kv, int rows) {
  const View& v = a.pool[kv];
  const int64_t ext[4] = {a.B, a.H, a.L, a.P};
  const int64_t str[4] = {v.s_tok, v.s_head, v.s_layer, v.s_req};
  uint64_t dims[5] = {static_cast<uint64_t>(a.d), 0, 0, 0, 0}, strides[4];
  for (int i = 0; i < 4; ++i) {
    dims[i + 1] = static_cast<uint64_t>(ext[i]);
    strides[i] = static_cast<uint64_t>(ext[i] > 1 ? str[i] : a.d) * 2;   // unused where 1 long
  }
  const uint32_t box[5] = {64, static_cast<uint32_t>(rows), 1, 1, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, v.base, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

// `sc`: of scaled pools.
template <int D, bool F8>
cudaError_t launch_tc(const AttnArgs& a, const ScaleArgs* sc, cudaStream_t stream) {
  using C = Cfg<D, F8>;
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  TcArgs p;
  std::memset(&p, 0, sizeof(p));
  p.a = a;
  p.tok_tile = kRowsM / a.G;
  // Where a run of 16 rows or more divides both page and tile, tiles are full whatever
  // the page.  Otherwise a tile has whole pages, or a page whole tiles, and masked
  // columns.  Runs of 8 rows fill them too, but their many copies cost as much as
  // tiles of 100 keys: they are taken where fewer would be in one.  (Eight chunks of
  // 256 tokens over 8,000 keys, 32 on 8 heads of 128: full tiles by runs of 16 and more
  // 260 us, of 8 rows 346 us; masked tiles of 125 keys 286 us, 120 298, 112 310, 104
  // 330, 100 346, 72 468.)
  int fit = kTile;
  while (a.B % fit != 0) fit /= 2;
  const int padded = (a.B + 7) / 8 * 8, tiles_page = (a.B + kTile - 1) / kTile;
  const int filled = a.B < kTile ? kTile / padded * a.B : a.B / tiles_page;   // keys of a tile
  // Scaled pools are copied row by row: tiles are full whatever the page.
  const bool full = F8 || fit >= 16 || (fit == 8 && filled < 100);
  const bool small = !full && a.B < kTile;
  p.run_rows = F8 ? kTile : full ? fit : small ? padded : kTile;
  p.run_tokens = small ? a.B : p.run_rows;
  p.runs = kTile / p.run_rows;
  if (small)
    for (int n = 0; n < kTile; ++n)
      if (n / p.run_rows >= p.runs || n % p.run_rows >= a.B) p.holes[n >> 5] |= 1u << (n & 31);
  p.has_holes = (p.holes[0] | p.holes[1] | p.holes[2] | p.holes[3]) != 0;
  SchedArgs& s = p.s;
  s.q_start = a.q_start;
  s.kv_lens = a.kv_lens;
  s.R = a.R;
  s.H = a.H;
  s.N = a.N;
  s.kv_cap = a.width * a.B;
  s.causal = a.causal;
  s.window = a.window;
  const int group = full ? kTile : small ? p.runs * a.B : a.B;
  s.item = make_fastdiv(2 * p.tok_tile);
  s.group = make_fastdiv(group);
  s.group_tiles = (group + kTile - 1) / kTile;
  s.tile = make_fastdiv(group < kTile ? group : kTile);
  s.even = s.group_tiles == 1;
  s.overhead = kItemCost;
  p.out32 = (reinterpret_cast<uintptr_t>(a.out) % 32 == 0) && (a.o_tok * 2) % 32 == 0 &&
            (a.o_head * 2) % 32 == 0;
  p.ragged = p.has_holes || !s.even;
  p.page = make_fastdiv(a.B);
  p.rows = make_fastdiv(p.run_rows);
  p.tiles = make_fastdiv(s.group_tiles);

  TcMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  {
    const int hq = a.H * a.G;
    const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(hq),
                              static_cast<uint64_t>(a.N)};
    const uint64_t strides[2] = {static_cast<uint64_t>(hq > 1 ? a.q_head : D) * 2,
                                 static_cast<uint64_t>(a.N > 1 ? a.q_tok : D) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(p.tok_tile)};
    e = encode_tiled(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims,
                     strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  if (F8) {
    p.sc = *sc;
    p.block = make_fastdiv(sc->block);
  } else {
    e = encode_pool(&maps.k, a, 0, p.run_rows);
    if (e != cudaSuccess) return e;
    e = encode_pool(&maps.v, a, 1, p.run_rows);
    if (e != cudaSuccess) return e;
  }
  constexpr int smem = F8 ? C::kTiles + static_cast<int>(sizeof(Bars<C::kSlots, C::kStages, F8>))
                          : 1024 + C::kTiles;
  static_assert(smem + (F8 ? 0 : sizeof(Bars<C::kSlots, C::kStages, F8>)) <= 227 * 1024,
                "shared memory of a CTA");
  e = cudaFuncSetAttribute(attn_tc_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  const int grid = di.sm_count < kMaxCtas ? di.sm_count : kMaxCtas;
  return launch_early(attn_tc_kernel<D, F8>, dim3(grid), C::kThreads, smem, stream, maps, p);
}

}  // namespace

size_t attn_tc_workspace_bytes(int d) {
  return kAttnCounterBytes + kMaxCtas * 2 * slot_floats(kSlotRows, d) * sizeof(float);
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t stream) {
  return a.d == 128 ? launch_tc<128, false>(a, nullptr, stream)
                    : launch_tc<64, false>(a, nullptr, stream);
}

cudaError_t launch_attn_scaled_tc(const AttnArgs& a, const ScaleArgs& sc, cudaStream_t stream) {
  return a.d == 128 ? launch_tc<128, true>(a, &sc, stream) : launch_tc<64, true>(a, &sc, stream);
}

}  // namespace kvc
