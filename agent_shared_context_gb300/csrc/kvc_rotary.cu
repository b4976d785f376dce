// kvc_rotary.cu -- norms of the query and key heads and their rotation by position
// (kvc_rotate_heads), and the table of frequencies that it goes by (kvc_rotary_turns).
//
// Pair i of a head turns by the angle p f_i at position p, f_i in radians per
// position.  p f_i passes 10^6 in a long context, where 32 bits leave nothing of the
// angle, and 64-bit arithmetic is slow here.  But only the angle's part of a turn
// matters, and that is an integer product: with F_i = f_i / (2 pi) in units of 2^-64
// turns, p F_i mod 2^64 is the angle as a fraction of a turn, exact but for F's own
// error, a few 2^-53 of p F_i.  Its upper 32 bits, as fp32 off by 2^-26 of a turn, go
// through sincospi.
//
// One CTA has a token: its pairs' cosines and sines are made once, in shared memory,
// while the heads' values are on their way, and serve all heads.  A row (one head) lies
// in a group of lanes, two vectors of 16 bytes to a lane that hold both halves of their
// pairs, so a row's sum of squares is a few shuffles and a rotation needs no exchange;
// where a part of the head is rotated the rest goes along in the same lanes.  Heads whose
// pairs do not lie in such vectors (an odd part of the head, odd strides) go by single
// pairs.  All arithmetic is fp32, rounded once at the end.  Each lane reads what it
// writes before it writes it: in place is fine.
//
// Bound by HBM, and by launch and latency for a step's few tokens.  Measured: two
// contexts of 8,192 tokens, 28 heads on 4 of 128, 56.3 us, 4.8 TB/s: CTAs of a token live for
// little more than two latencies, and 48 registers leave five of them on an SM.  (CTAs that
// stay and load a token ahead, with a barrier for each: 69 us; two or four rows to a thread
// 63 and 85.)  2,048 tokens of 32 on 8 heads with norms 14.1 us, 16 tokens 4.2 us.
#include <cuda_bf16.h>

#include <cmath>

#include "kvc_check.h"
#include "kvc_paged_internal.h"

namespace kvc {
namespace {

constexpr int kMaxPairs = 128;             // d <= 256
constexpr int kMaxThreads = 512;

struct Rows {
  const char* in;
  char* out;
  int64_t in_tok, in_head, out_tok, out_head;    // bytes
  const void* w;
};

struct RotaryArgs {
  Rows q, k;
  const int32_t* positions;
  const uint64_t* turns;
  int32_t Hq, rows;          // query heads, all heads
  int32_t d, half;           // head dim, rotated pairs
  int32_t lanes;             // of a row, a power of two
  int32_t norm;
  float eps, inv_d, amplitude;
};

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T x[V];
};

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = x * c - y * s;
  b = y * c + x * s;
}

// What a lane has of a row: the vectors at elements `a` and `b`.
struct Place {
  int a, b;                  // -1: none
  int pair;                  // first pair of the two
};

// V elements to a vector, P pairs of vectors to a lane.
template <typename T, int V, int P, bool INTER, bool NORM>
__global__ void __launch_bounds__(kMaxThreads) rotate_kernel(const RotaryArgs p) {
  __shared__ alignas(32) float cs[kMaxPairs], sn[kMaxPairs];
  const int64_t tok = blockIdx.x;
  const int lane = threadIdx.x & (p.lanes - 1);
  const int group = threadIdx.x / p.lanes, groups = blockDim.x / p.lanes;

  Place at[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int u = lane + i * p.lanes;
    if (INTER) {
      at[i] = Place{2 * u * V, (2 * u + 1) * V, u * V};
    } else {
      const int h = p.half / V;
      // rotated vectors pair up with those half a rotated part away, the rest by twos
      at[i] = u < h ? Place{u * V, u * V + p.half, u * V}
                    : Place{2 * p.half + 2 * (u - h) * V, 2 * p.half + (2 * (u - h) + 1) * V, p.half};
    }
    if (at[i].a >= p.d) at[i].a = -1;
    if (at[i].b >= p.d) at[i].b = -1;
  }

  // The position, the table and the first rows are on their way before any of them is
  // waited for: one latency, not three.
  grid_wait();
  const int pos = p.positions[tok], tid = threadIdx.x;
  const uint64_t my_turns = tid < p.half ? p.turns[tid] : 0;
  using W = Vec<T, V>;
  // the token's rows, the same for all threads
  const char* const in[2] = {p.q.in + tok * p.q.in_tok, p.k.in + tok * p.k.in_tok};
  char* const out[2] = {p.q.out + tok * p.q.out_tok, p.k.out + tok * p.k.out_tok};
  for (int first = 0; first < p.rows; first += groups) {
    const int row = first + group;
    const bool is_q = row < p.Hq;
    const int head = is_q ? row : row - p.Hq;
    W a[P], b[P];
    if (row < p.rows) {
      const T* src = reinterpret_cast<const T*>((is_q ? in[0] : in[1]) +
                                                head * (is_q ? p.q.in_head : p.k.in_head));
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (at[i].a >= 0) a[i] = *reinterpret_cast<const W*>(src + at[i].a);
        if (at[i].b >= 0) b[i] = *reinterpret_cast<const W*>(src + at[i].b);
      }
    }
    if (first == 0) {
      if (pos < 0) return;                      // the whole CTA: no row of this token
      for (int i = tid; i < p.half; i += blockDim.x) {
        const uint64_t turn = static_cast<uint64_t>(static_cast<uint32_t>(pos)) *
                              (i == tid ? my_turns : p.turns[i]);
        float s, c;
        // the upper 32 bits as a signed number of half turns
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f,
                  &s, &c);
        cs[i] = c * p.amplitude;
        sn[i] = s * p.amplitude;
      }
      __syncthreads();
    }
    float f = 1.f;
    if (NORM) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float x = to_f32<T>(a[i].x[j]), y = to_f32<T>(b[i].x[j]);
          if (row < p.rows && at[i].a >= 0) sum = fmaf(x, x, sum);
          if (row < p.rows && at[i].b >= 0) sum = fmaf(y, y, sum);
        }
      for (int o = p.lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      f = rsqrtf(fmaf(sum, p.inv_d, p.eps));
    }
    if (row >= p.rows) continue;
    T* dst = reinterpret_cast<T*>((is_q ? out[0] : out[1]) +
                                  head * (is_q ? p.q.out_head : p.k.out_head));
    const T* w = static_cast<const T*>(is_q ? p.q.w : p.k.w);
    // A few elements at a time: with all of a lane's in fp32 the registers would leave room
    // for half as many rows on their way.
    constexpr int C = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int j0 = 0; j0 < V; j0 += C) {
        float x[C], y[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
          x[j] = to_f32<T>(a[i].x[j0 + j]);
          y[j] = to_f32<T>(b[i].x[j0 + j]);
        }
        if (NORM) {
          using WC = Vec<T, C>;
          WC wa, wb;
          if (w != nullptr && at[i].a >= 0) wa = *reinterpret_cast<const WC*>(w + at[i].a + j0);
          if (w != nullptr && at[i].b >= 0) wb = *reinterpret_cast<const WC*>(w + at[i].b + j0);
#pragma unroll
          for (int j = 0; j < C; ++j) {
            x[j] *= f;
            y[j] *= f;
            if (w != nullptr) {
              x[j] *= to_f32<T>(wa.x[j]);
              y[j] *= to_f32<T>(wb.x[j]);
            }
          }
        }
        if constexpr (INTER && V > 1) {
          // pairs of a's neighbours, then of b's
          const int n = at[i].pair + j0 / 2, m = n + V / 2;
          const auto ca = *reinterpret_cast<const Vec<float, C / 2>*>(cs + n);
          const auto sa = *reinterpret_cast<const Vec<float, C / 2>*>(sn + n);
          const auto cb = *reinterpret_cast<const Vec<float, C / 2>*>(cs + m);
          const auto sb = *reinterpret_cast<const Vec<float, C / 2>*>(sn + m);
#pragma unroll
          for (int j = 0; j + 1 < C; j += 2) {
            if (n + j / 2 < p.half) turn(x[j], x[j + 1], ca.x[j / 2], sa.x[j / 2]);
            if (m + j / 2 < p.half) turn(y[j], y[j + 1], cb.x[j / 2], sb.x[j / 2]);
          }
        } else if (at[i].pair < p.half) {
          const auto c = *reinterpret_cast<const Vec<float, C>*>(cs + at[i].pair + j0);
          const auto s = *reinterpret_cast<const Vec<float, C>*>(sn + at[i].pair + j0);
#pragma unroll
          for (int j = 0; j < C; ++j) turn(x[j], y[j], c.x[j], s.x[j]);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
          a[i].x[j0 + j] = from_f32<T>(x[j]);
          b[i].x[j0 + j] = from_f32<T>(y[j]);
        }
      }
      if (at[i].a >= 0) *reinterpret_cast<W*>(dst + at[i].a) = a[i];
      if (at[i].b >= 0) *reinterpret_cast<W*>(dst + at[i].b) = b[i];
    }
  }
}

template <typename T, int V, int P>
cudaError_t launch(const RotaryArgs& a, int64_t N, bool inter, cudaStream_t stream) {
  // a group of lanes for each row, in as few turns as threads allow
  const int need = a.rows * a.lanes, turns = (need + kMaxThreads - 1) / kMaxThreads;
  const int threads = ((need + turns - 1) / turns + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(N));
  auto* fn = inter ? (a.norm ? rotate_kernel<T, V, P, true, true>
                             : rotate_kernel<T, V, P, true, false>)
                   : (a.norm ? rotate_kernel<T, V, P, false, true>
                             : rotate_kernel<T, V, P, false, false>);
  return launch_early(fn, grid, threads, 0, stream, a);
}

// The bytes of [N, heads, d] rows, `step` bytes from a token (0) or head (1) to the next.
struct Extent {
  Span s;
  int64_t row, step[2], count[2];
  // from the first to the last byte of what one token (head) has
  int64_t foot(int dim) const { return (count[1 - dim] - 1) * step[1 - dim] + row; }
};

Extent extent(const void* p, int64_t N, int64_t heads, int64_t s_tok, int64_t s_head, int64_t d,
              int64_t e) {
  return Extent{span(p, ((N - 1) * s_tok + (heads - 1) * s_head + d) * e), d * e,
                {s_tok * e, s_head * e}, {N, heads}};
}

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }    // b > 0

// Whether rows at 0, sa, .. (na of them) and at off, off + sb, .. (nb) share a byte.
bool rows_share(int64_t off, int64_t sa, int64_t na, int64_t sb, int64_t nb, int64_t row) {
  if (na == 1) sa = sb;
  if (nb == 1) sb = sa;
  if (na == 1 && nb == 1) return off < row && off > -row;
  // rows i and j share one where off + j sb - i sa lies within a row's size
  auto meets = [&](int64_t at, int64_t s, int64_t lo, int64_t hi) {      // at - m s, lo <= m <= hi
    const int64_t m = floor_div(at, s);
    return (m >= lo && m <= hi && at - m * s < row) ||
           (m + 1 >= lo && m + 1 <= hi && (m + 1) * s - at < row);
  };
  if (sa == sb) return meets(off, sa, 1 - nb, na - 1);
  if (nb > 65535) return true;                     // not looked at one by one
  for (int64_t j = 0; j < nb; ++j)
    if (meets(off + j * sb, sa, 0, na - 1)) return true;
  return false;
}

// Whether two rows of it share a byte.
bool folded(const Extent& x) {
  for (int out = 0; out < 2; ++out)
    if (x.count[out] == 1 || x.foot(out) <= x.step[out]) return false;
  // neither nests in the other: the heads' distances beside the tokens'
  for (int64_t h = 1; h < x.count[1]; ++h)
    if (rows_share(h * x.step[1], x.step[0], x.count[0], x.step[0], 1, x.row)) return true;
  return false;
}

// Whether two of them share a byte.  The parts of one projection's rows do not, be they
// beside each other in every token or alternating head by head.  Strides that are not told
// apart here count as shared.
bool share(const Extent& a, const Extent& b) {
  if (!overlap(a.s, b.s)) return false;
  const int64_t off = static_cast<int64_t>(b.s.lo) - static_cast<int64_t>(a.s.lo);
  for (int out = 0; out < 2; ++out) {              // tokens outermost, or heads
    const int in = 1 - out;
    const bool am = a.count[out] > 1, bm = b.count[out] > 1;
    if (am && bm && a.step[out] != b.step[out]) continue;
    const int64_t t = am ? a.step[out] : b.step[out];
    auto at = [&](int64_t o) {
      return rows_share(o, a.step[in], a.count[in], b.step[in], b.count[in], a.row);
    };
    if (!am && !bm) return at(off);
    if (a.foot(out) > t || b.foot(out) > t) continue;
    // only those of a and b can meet that begin less than t apart
    const int64_t m = floor_div(off, t), lo = 1 - b.count[out], hi = a.count[out] - 1;
    return (m >= lo && m <= hi && at(off - m * t)) ||
           (m + 1 >= lo && m + 1 <= hi && at(off - (m + 1) * t));
  }
  return true;
}

kvc_status check_heads(const kvc_rotary_params* rp, const void* p, int32_t heads, int64_t s_tok,
                       int64_t s_head, const char* name) {
  const int64_t e = rp->dtype == KVC_BF16 ? 2 : 4, lim = (int64_t(1) << 40) / e;
  KVC_TRY(check_ptr(p, name, static_cast<unsigned>(e)));
  if (s_tok < 0 || s_head < 0 || (heads > 1 && s_head < rp->d) ||
      (rp->n_tokens > 1 && s_tok < rp->d))
    return fail(KVC_ERR_SHAPE, "%s: strides must be >= d", name);
  if (s_tok >= lim || s_head >= lim)
    return fail(KVC_ERR_UNSUPPORTED, "%s: byte strides must be < 2^40", name);
  return KVC_OK;
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

kvc_status kvc_rotary_turns(const kvc_rotary_scaling* sc, double base, int32_t rot_dim,
                            int64_t* turns, float* amplitude) {
  if (rot_dim < 0 || rot_dim > 2 * kMaxPairs || rot_dim % 2 != 0)
    return fail(KVC_ERR_UNSUPPORTED, "rot_dim = %d is no even number in [0, %d]", rot_dim,
                2 * kMaxPairs);
  if (!(base > 1.0) || !std::isfinite(base))
    return fail(KVC_ERR_INVALID_ARGUMENT, "base must be finite and > 1");
  if ((turns == nullptr && rot_dim > 0) || amplitude == nullptr)
    return fail(KVC_ERR_INVALID_ARGUMENT, "turns or amplitude is NULL");
  const int mode = sc == nullptr ? KVC_ROTARY_PLAIN : sc->mode;
  if (mode != KVC_ROTARY_PLAIN && mode != KVC_ROTARY_LINEAR && mode != KVC_ROTARY_BANDS &&
      mode != KVC_ROTARY_RAMP)
    return fail(KVC_ERR_INVALID_ARGUMENT, "unknown scaling mode %d", mode);
  if (mode != KVC_ROTARY_PLAIN && !(sc->factor >= 1.0 && std::isfinite(sc->factor)))
    return fail(KVC_ERR_INVALID_ARGUMENT, "factor must be finite and >= 1");
  if ((mode == KVC_ROTARY_BANDS || mode == KVC_ROTARY_RAMP) &&
      !(sc->low > 0.0 && sc->high > sc->low && std::isfinite(sc->high) && sc->original >= 1.0 &&
        std::isfinite(sc->original)))
    return fail(KVC_ERR_INVALID_ARGUMENT, "0 < low < high and original >= 1 are needed");
  const double two_pi = 6.283185307179586476925;
  double from = 0.0, to = 0.0;
  if (mode == KVC_ROTARY_RAMP) {
    auto at = [&](double t) {
      return rot_dim * std::log(sc->original / (t * two_pi)) / (2.0 * std::log(base));
    };
    from = std::fmax(std::floor(at(sc->high)), 0.0);
    to = std::fmin(std::ceil(at(sc->low)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim), keep = 1.0;
    if (mode == KVC_ROTARY_LINEAR) {
      keep = 0.0;
    } else if (mode == KVC_ROTARY_BANDS) {
      keep = (sc->original * f / two_pi - sc->low) / (sc->high - sc->low);
    } else if (mode == KVC_ROTARY_RAMP) {
      keep = 1.0 - (i - from) / std::fmax(to - from, 0.001);
    }
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    if (keep < 1.0) f = f * keep + f * (1.0 - keep) / sc->factor;
    // f <= 1: less than 2^62
    turns[i] = static_cast<int64_t>(std::nearbyint(std::ldexp(f / two_pi, 64)));
  }
  *amplitude = mode == KVC_ROTARY_RAMP ? static_cast<float>(0.1 * std::log(sc->factor) + 1.0) : 1.0f;
  return KVC_OK;
}

kvc_status kvc_rotate_heads(const kvc_rotary_params* rp, const void* q, const void* k,
                            const void* w_q, const void* w_k, const int32_t* positions,
                            const int64_t* turns, void* q_out, void* k_out, cudaStream_t stream) {
  if (rp == nullptr) return fail(KVC_ERR_INVALID_ARGUMENT, "rotary descriptor is NULL");
  if (rp->dtype != KVC_BF16 && rp->dtype != KVC_F32)
    return fail(KVC_ERR_DTYPE, "unknown dtype %d", static_cast<int>(rp->dtype));
  if (rp->n_tokens < 0 || rp->n_tokens > (1 << 30))
    return fail(KVC_ERR_SHAPE, "n_tokens = %d outside [0, 2^30]", rp->n_tokens);
  if (rp->n_q_heads < 0 || rp->n_kv_heads < 0 || rp->n_q_heads > 65535 || rp->n_kv_heads > 65535 ||
      rp->n_q_heads + rp->n_kv_heads < 1)
    return fail(KVC_ERR_SHAPE, "n_q_heads = %d, n_kv_heads = %d: each in [0, 65535], one at least",
                rp->n_q_heads, rp->n_kv_heads);
  if (rp->d < 2 || rp->d > 2 * kMaxPairs || rp->d % 2 != 0)
    return fail(KVC_ERR_UNSUPPORTED, "head dim must be even and in [2, %d] (got %d)", 2 * kMaxPairs,
                rp->d);
  if (rp->rot_dim < 0 || rp->rot_dim > rp->d || rp->rot_dim % 2 != 0)
    return fail(KVC_ERR_SHAPE, "rot_dim = %d is no even number in [0, d]", rp->rot_dim);
  if ((rp->interleaved != 0 && rp->interleaved != 1) || (rp->norm != 0 && rp->norm != 1))
    return fail(KVC_ERR_INVALID_ARGUMENT, "interleaved and norm are 0 or 1");
  if (rp->norm && !(rp->eps >= 0.0f && std::isfinite(rp->eps)))
    return fail(KVC_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (!std::isfinite(rp->amplitude))
    return fail(KVC_ERR_INVALID_ARGUMENT, "amplitude must be finite");
  if (!rp->norm && (w_q != nullptr || w_k != nullptr))
    return fail(KVC_ERR_INVALID_ARGUMENT, "weights are those of the norm: norm is 0");
  if (rp->n_tokens == 0) return KVC_OK;
  const unsigned e = rp->dtype == KVC_BF16 ? 2 : 4;
  const int64_t N = rp->n_tokens, d = rp->d;
  KVC_TRY(check_ptr(positions, "positions", 4));
  if (rp->rot_dim > 0) KVC_TRY(check_ptr(turns, "turns", 8));
  if (w_q != nullptr) KVC_TRY(check_ptr(w_q, "w_q", e));
  if (w_k != nullptr) KVC_TRY(check_ptr(w_k, "w_k", e));
  const struct {
    const char *in_name, *out_name;
    const void* in;
    void* out;
    int32_t heads;
    int64_t in_tok, in_head, out_tok, out_head;
  } part[2] = {{"q", "q_out", q, q_out, rp->n_q_heads, rp->q_s_tok, rp->q_s_head, rp->q_out_s_tok,
                rp->q_out_s_head},
               {"k", "k_out", k, k_out, rp->n_kv_heads, rp->k_s_tok, rp->k_s_head, rp->k_out_s_tok,
                rp->k_out_s_head}};
  const Span fixed[] = {span(positions, 4 * N), span(turns, 4 * int64_t(rp->rot_dim)),
                        span(w_q, w_q == nullptr ? 0 : d * e), span(w_k, w_k == nullptr ? 0 : d * e)};
  Extent in[2], out[2];
  bool whole = true;         // vectors of 16 bytes throughout
  const auto in16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  for (int i = 0; i < 2; ++i) {
    if (part[i].heads == 0) continue;
    KVC_TRY(check_heads(rp, part[i].in, part[i].heads, part[i].in_tok, part[i].in_head,
                        part[i].in_name));
    KVC_TRY(check_heads(rp, part[i].out, part[i].heads, part[i].out_tok, part[i].out_head,
                        part[i].out_name));
    in[i] = extent(part[i].in, N, part[i].heads, part[i].in_tok, part[i].in_head, d, e);
    out[i] = extent(part[i].out, N, part[i].heads, part[i].out_tok, part[i].out_head, d, e);
    if (folded(out[i]))
      return fail(KVC_ERR_ALIAS, "%s: rows overlap one another", part[i].out_name);
    for (const Span& s : fixed)
      if (s.lo != 0 && overlap(out[i].s, s))
        return fail(KVC_ERR_ALIAS, "%s overlaps positions, turns or weights", part[i].out_name);
    whole = whole && in16(part[i].in) && in16(part[i].out) && part[i].in_tok * e % 16 == 0 &&
            part[i].in_head * e % 16 == 0 && part[i].out_tok * e % 16 == 0 &&
            part[i].out_head * e % 16 == 0;
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j) {
      if (part[i].heads == 0 || part[j].heads == 0) continue;
      const bool in_place = i == j && part[i].in == part[i].out &&
                            part[i].in_tok == part[i].out_tok && part[i].in_head == part[i].out_head;
      if (!in_place && share(out[i], in[j]))
        return fail(KVC_ERR_ALIAS, "%s overlaps %s and is not the same rows", part[i].out_name,
                    part[j].in_name);
      if (i < j && share(out[i], out[j]))
        return fail(KVC_ERR_ALIAS, "q_out and k_out overlap");
    }
  RotaryArgs a{};
  for (int i = 0; i < 2; ++i) {
    Rows& r = i == 0 ? a.q : a.k;
    r.in = static_cast<const char*>(part[i].in);
    r.out = static_cast<char*>(part[i].out);
    r.in_tok = part[i].in_tok * e;
    r.in_head = part[i].in_head * e;
    r.out_tok = part[i].out_tok * e;
    r.out_head = part[i].out_head * e;
    r.w = i == 0 ? w_q : w_k;
  }
  a.positions = positions;
  a.turns = reinterpret_cast<const uint64_t*>(turns);
  a.Hq = rp->n_q_heads;
  a.rows = rp->n_q_heads + rp->n_kv_heads;
  a.d = rp->d;
  a.half = rp->rot_dim / 2;
  a.norm = rp->norm;
  a.eps = rp->eps;
  a.inv_d = 1.0f / rp->d;
  a.amplitude = rp->amplitude;
  const int v = 16 / static_cast<int>(e);
  whole = whole && rp->d % v == 0 && (rp->interleaved || a.half % v == 0) && in16(w_q) && in16(w_k);
  a.lanes = 1;
  const int pairs = whole ? (rp->d / v + 1) / 2 : rp->d / 2;
  while (a.lanes < pairs && a.lanes < 32) a.lanes *= 2;
  cudaError_t err;
  if (rp->dtype == KVC_BF16)
    err = whole ? launch<__nv_bfloat16, 8, 1>(a, N, rp->interleaved, stream)
                : launch<__nv_bfloat16, 1, 4>(a, N, rp->interleaved, stream);
  else
    err = whole ? launch<float, 4, 1>(a, N, rp->interleaved, stream)
                : launch<float, 1, 4>(a, N, rp->interleaved, stream);
  if (err != cudaSuccess) return cuda_fail(err, "kvc_rotate_heads launch");
  return KVC_OK;
}

}  // extern "C"
