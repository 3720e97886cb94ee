// Rotary positions of query and key heads, optionally after a root-mean-square
// norm of each head, in one pass over the projections.
//
//   y = R(pos) (w * x / sqrt(mean(x^2) + eps)),
// where R turns the pair (a, b) number i of the first rotary_dim dimensions by
// the angle pos * f_i:
//   a' = m (a cos - b sin),  b' = m (b cos + a sin),
// and copies the others. Pairs are (i, i + rotary_dim / 2) in the half layout
// and (2i, 2i + 1) in the interleaved one; m is the scaling's magnitude factor.
//
// Angles. f_i is kept as a fraction of a turn a position in 64-bit fixed point,
// F_i = f_i / (2 pi) * 2^64 mod 2^64, right to 2^-55 of a turn (f_i comes from
// fp64). The product pos * F_i mod 2^64 is then the angle modulo one turn, off by
// |pos| * 2^-55 turns, 2^-24 at the last 32-bit position, where a 32-bit float
// product would be off by a radian from positions of a few million on. Its top 32
// bits go to sincospif as a float, which rounds them to 2^-26 of a turn.
//
// The kernel reads and writes every value once and is bound by HBM; the sines of
// a token are computed once per warp and used for every head that the warp
// takes. All arithmetic is fp32; the one rounding is that of the output type.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/confkv.h"
#include "common.cuh"
#include "kernels.h"

namespace confkv {

namespace {

constexpr int kMaxPairs = CONFKV_ROPE_MAX_PAIRS;
constexpr double kPi = 3.14159265358979323846;

struct RopeSide {
  const void* x;
  void* y;
  const float* w;
  int heads;
  long long xb, xt, xh, yb, yt, yh;   // strides in elements
};

struct RopeArgs {
  RopeSide side[2];
  const int32_t* pos;
  int batch, tokens, heads;   // heads of both sides
  int D, rd;
  int hsplit;                 // warps that share one token's heads
  float eps, mag;
  unsigned long long turns[kMaxPairs];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight consecutive values as one or two 16-byte words.
template <class T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f(e[i]);
  }
};

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  uint4 w[sizeof(T) / 2];
  T* e = reinterpret_cast<T*>(w);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f<T>(v[i]);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
}

// cos and sin of pos * F turns, times the magnitude.
__device__ __forceinline__ void angle(int pos, unsigned long long F, float mag, float* c, float* s) {
  const unsigned long long ph = (unsigned long long)(long long)pos * F;
  const float half_turns = (float)(int)(ph >> 32) * 0x1p-31f;   // [-1, 1]
  float sn, cs;
  sincospif(half_turns, &sn, &cs);
  *c = cs * mag;
  *s = sn * mag;
}

// Vector form: head_dim 32, 64, 128 or 256, rows on 16-byte boundaries, and in the
// half layout rotary_dim a multiple of 16. LPR = D / 16 lanes hold one row, two groups of eight
// values each: rotary lane j has the pairs 8j..8j+7 whichever the layout. A
// warp takes one token and 32 / LPR heads at a time, U rounds in flight; the
// loads wait as they came, so that 32 warps an SM fit and cover the trip to HBM.
template <class X, class Y, bool HALF, bool NORM, int LPR>
__global__ void __launch_bounds__(128, NORM ? 6 : 8) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ unsigned long long turns[kMaxPairs];
  for (int i = threadIdx.x; i < a.rd / 2; i += 128) turns[i] = a.turns[i];
  chain_enter();
  __syncthreads();
  constexpr int SLOTS = 32 / LPR, U = sizeof(X) == 2 ? 2 : 1;
  const int lane = threadIdx.x & 31;
  const long long warp = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int part = (int)(warp % a.hsplit);
  const long long tok = warp / a.hsplit;
  if (tok >= (long long)a.batch * a.tokens) return;
  const int b = (int)(tok / a.tokens), t = (int)(tok % a.tokens);
  const int j = lane % LPR, slot = lane / LPR;
  const int turned = min(8, a.rd / 2 - 8 * j);   // of this lane's eight pairs (half layout: all or none)
  const bool rot = turned > 0;
  const int o0 = rot && HALF ? 8 * j : 16 * j;
  const int o1 = rot && HALF ? a.rd / 2 + 8 * j : 16 * j + 8;
  // the slots of a warp share a token: each computes its part of the eight angles
  float cs[8], sn[8];
  {
    constexpr int OWN = SLOTS >= 8 ? 1 : 8 / SLOTS;
    float c[OWN], s[OWN];
    const int pos = a.pos[tok];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      const int f = 8 * j + (slot * OWN + i) % 8;
      angle(pos, f < a.rd / 2 ? turns[f] : 0, a.mag, &c[i], &s[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, c[i % OWN], i / OWN * LPR + j);
      sn[i] = __shfl_sync(0xffffffffu, s[i % OWN], i / OWN * LPR + j);
    }
  }
  const float inv_d = 1.0f / (float)(16 * LPR);
  // The heads of both sides are dealt in one sequence: this slot takes numbers
  // g0, g0 + step, ... The count of rounds is the same for the whole warp, so
  // that the norm's shuffles find every lane; a slot without a head in a round
  // neither loads nor stores.
  const int g0 = part * SLOTS + slot, step = a.hsplit * SLOTS;
#pragma unroll 1
  for (int sd = 0; sd < 2; ++sd) {
    const RopeSide& r = a.side[sd];
    if (r.heads == 0) break;
    const int base = sd ? a.side[0].heads : 0;
    const int first = g0 >= base ? g0 - base : (step - (base - g0) % step) % step;
    float w0[8], w1[8];
    if (NORM && r.w) {
      Raw8<float> t;
      t.load(r.w + o0);
      t.get(w0);
      t.load(r.w + o1);
      t.get(w1);
    }
    const X* xr = static_cast<const X*>(r.x) + b * r.xb + t * r.xt;
    Y* yr = static_cast<Y*>(r.y) + b * r.yb + t * r.yt;
    const int rounds = (r.heads + step - 1) / step;
    for (int k = 0; k < rounds; k += U) {
      Raw8<X> v[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = first + (k + u) * step;
        if (h < r.heads) {
          v[u][0].load(xr + h * r.xh + o0);
          v[u][1].load(xr + h * r.xh + o1);
        } else {
          v[u][0].zero();
          v[u][1].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = first + (k + u) * step;
        float p[8], q[8];
        v[u][0].get(p);
        v[u][1].get(q);
        if (NORM && r.w) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(p[i], p[i], fmaf(q[i], q[i], ss));
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float sc = rsqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            p[i] *= sc * w0[i];
            q[i] *= sc * w1[i];
          }
        }
        if (rot) {
          if constexpr (HALF) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x0 = p[i], x1 = q[i];
              p[i] = fmaf(x0, cs[i], -x1 * sn[i]);
              q[i] = fmaf(x1, cs[i], x0 * sn[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x0 = p[2 * i], x1 = p[2 * i + 1], z0 = q[2 * i], z1 = q[2 * i + 1];
              if (i < turned) {
                p[2 * i] = fmaf(x0, cs[i], -x1 * sn[i]);
                p[2 * i + 1] = fmaf(x1, cs[i], x0 * sn[i]);
              }
              if (4 + i < turned) {
                q[2 * i] = fmaf(z0, cs[4 + i], -z1 * sn[4 + i]);
                q[2 * i + 1] = fmaf(z1, cs[4 + i], z0 * sn[4 + i]);
              }
            }
          }
        }
        if (h < r.heads) {
          store8(yr + h * r.yh + o0, p);
          store8(yr + h * r.yh + o1, q);
        }
      }
    }
  }
}

// Any even head_dim up to 64 NS, any rotary_dim, strides and alignment: one warp
// per row, each lane the pairs lane, lane + 32, ... and the plain dimensions past
// them. A warp keeps its token's sines for the heads it takes, two rows in flight.
// Bound by instructions: 16384 tokens x 40 heads of 128 in fp16, 102 dimensions
// rotated in the half layout, 146 us (the vector form, at 96: 56); with the sines
// computed for every row it was 393. Two pairs a lane at a time gained nothing.
template <class X, class Y, int NS>
__global__ void __launch_bounds__(128) rope_any_kernel(const __grid_constant__ RopeArgs a, int half) {
  __shared__ unsigned long long turns[kMaxPairs];
  for (int i = threadIdx.x; i < a.rd / 2; i += 128) turns[i] = a.turns[i];
  chain_enter();
  __syncthreads();
  constexpr int U = 2;   // rows in flight
  const int lane = threadIdx.x & 31;
  const long long warp = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int part = (int)(warp % a.hsplit);
  const long long tok = warp / a.hsplit;
  if (tok >= (long long)a.batch * a.tokens) return;
  const int b = (int)(tok / a.tokens), t = (int)(tok % a.tokens);
  const int np = a.rd / 2, D = a.D;
  const int pos = np ? a.pos[tok] : 0;
  float cs[NS], sn[NS];
#pragma unroll
  for (int u = 0; u < NS; ++u) {
    const int i = lane + 32 * u;
    cs[u] = sn[u] = 0.0f;
    if (i < np) angle(pos, turns[i], a.mag, &cs[u], &sn[u]);
  }
  const int st = half ? 1 : 2, mate = half ? np : 1;   // pair i: dimensions st i and st i + mate
  // the token's first row of either side
  const X* x0 = static_cast<const X*>(a.side[0].x) + b * a.side[0].xb + t * a.side[0].xt;
  const X* x1 = static_cast<const X*>(a.side[1].x) + b * a.side[1].xb + t * a.side[1].xt;
  Y* y0 = static_cast<Y*>(a.side[0].y) + b * a.side[0].yb + t * a.side[0].yt;
  Y* y1 = static_cast<Y*>(a.side[1].y) + b * a.side[1].yb + t * a.side[1].yt;
  for (int h0 = part; h0 < a.heads; h0 += U * a.hsplit) {
    // a row as the lane's slots, unconverted: pair members first, then the rest
    X p[U][NS], q[U][NS], z[U][2 * NS];
    Y* yr[U];
    const float* w[U];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int g = h0 + v * a.hsplit, g1 = g - a.side[0].heads;
      yr[v] = nullptr;
      w[v] = nullptr;
      if (g >= a.heads) break;
      const X* xr = g1 < 0 ? x0 + g * a.side[0].xh : x1 + g1 * a.side[1].xh;
      yr[v] = g1 < 0 ? y0 + g * a.side[0].yh : y1 + g1 * a.side[1].yh;
      w[v] = g1 < 0 ? a.side[0].w : a.side[1].w;
      auto get = [&](int d, bool in) { return in ? xr[d] : from_f<X>(0.0f); };
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const int i = lane + 32 * u;
        p[v][u] = get(st * i, i < np);
        q[v][u] = get(st * i + mate, i < np);
      }
#pragma unroll
      for (int u = 0; u < 2 * NS; ++u) {
        const int d = a.rd + lane + 32 * u;
        z[v][u] = get(d, d < D);
      }
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      if (!yr[v]) break;   // (the same in the whole warp)
      float sc = 1.0f;
      if (w[v]) {
        float ss = 0.0f;
#pragma unroll
        for (int u = 0; u < NS; ++u) {
          const float e0 = to_f(p[v][u]), e1 = to_f(q[v][u]);
          ss = fmaf(e0, e0, fmaf(e1, e1, ss));
        }
#pragma unroll
        for (int u = 0; u < 2 * NS; ++u) ss = fmaf(to_f(z[v][u]), to_f(z[v][u]), ss);
        sc = rsqrtf(warp_sum(ss) / (float)D + a.eps);
      }
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const int i = lane + 32 * u;
        if (i >= np) continue;
        const int d0 = st * i, d1 = st * i + mate;
        float e0 = to_f(p[v][u]), e1 = to_f(q[v][u]);
        if (w[v]) {
          e0 *= sc * w[v][d0];
          e1 *= sc * w[v][d1];
        }
        yr[v][d0] = from_f<Y>(fmaf(e0, cs[u], -e1 * sn[u]));
        yr[v][d1] = from_f<Y>(fmaf(e1, cs[u], e0 * sn[u]));
      }
#pragma unroll
      for (int u = 0; u < 2 * NS; ++u) {
        const int d = a.rd + lane + 32 * u;
        const float e = to_f(z[v][u]);
        if (d < D) yr[v][d] = from_f<Y>(w[v] ? e * (sc * w[v][d]) : e);
      }
    }
  }
}

template <class X, class Y, bool NORM>
cudaError_t launch_vec(const RopeArgs& a, bool half, unsigned grid, cudaStream_t st) {
  switch (a.D) {
#define CONFKV_ROPE_D(DD)                                                                      \
  case DD:                                                                                     \
    return half ? launch_chained(rope_kernel<X, Y, true, NORM, DD / 16>, grid, 128, 0, st, a)  \
                : launch_chained(rope_kernel<X, Y, false, NORM, DD / 16>, grid, 128, 0, st, a)
    CONFKV_ROPE_D(32);
    CONFKV_ROPE_D(64);
    CONFKV_ROPE_D(128);
    CONFKV_ROPE_D(256);
#undef CONFKV_ROPE_D
  }
  return cudaErrorInvalidValue;
}

template <class X, class Y>
cudaError_t launch_types(const RopeArgs& a0, bool half, bool vec, cudaStream_t st) {
  RopeArgs a = a0;
  const long long tokens = (long long)a.batch * a.tokens;
  // Share a token's heads among warps until about eight warps an SM are busy
  // (a decode step has few tokens: each round of heads is a trip to HBM), no
  // further than one head a slot.
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int slots = vec ? 32 / (a.D / 16) : 1;
  const int most = (a.heads + slots - 1) / slots;
  a.hsplit = (int)std::min<long long>(most, std::max<long long>(1, 8ll * sms / tokens));
  const long long grid = (tokens * a.hsplit + 3) / 4;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  if (!vec) {
    const auto kernel = a.D <= 64 ? rope_any_kernel<X, Y, 1> : a.D <= 128 ? rope_any_kernel<X, Y, 2> : rope_any_kernel<X, Y, 4>;
    return launch_chained(kernel, (unsigned)grid, 128, 0, st, a, half ? 1 : 0);
  }
  return a.side[0].w || a.side[1].w ? launch_vec<X, Y, true>(a, half, (unsigned)grid, st)
                                    : launch_vec<X, Y, false>(a, half, (unsigned)grid, st);
}

template <class X>
cudaError_t launch_x(const RopeArgs& a, int y_type, bool half, bool vec, cudaStream_t st) {
  switch (y_type) {
    case CONFKV_F32: return launch_types<X, float>(a, half, vec, st);
    case CONFKV_F16: return launch_types<X, __half>(a, half, vec, st);
    default: return launch_types<X, __nv_bfloat16>(a, half, vec, st);
  }
}

// Whether the rows of an output (their strides in elements) lie apart: in the
// order of the strides, each dimension steps over all that those before it span.
bool rows_apart(int D, int batch, long long yb, int tokens, long long yt, int heads, long long yh) {
  struct { int n; long long step; } d[3] = {{batch, yb}, {tokens, yt}, {heads, yh}};
  std::sort(d, d + 3, [](const auto& a, const auto& b) { return a.step < b.step; });
  __int128 span = D;
  for (const auto& x : d) {
    if (x.n <= 1) continue;
    if (x.step < span) return false;
    span += (__int128)(x.n - 1) * x.step;
  }
  return true;
}

bool finite_pos(double v) { return std::isfinite(v) && v > 0.0; }

}  // namespace

}  // namespace confkv

extern "C" {

confkv_status confkv_default_rope_params(confkv_rope_params* p) {
  if (!p) return CONFKV_ERR_ARG;
  std::memset(p, 0, sizeof(*p));
  p->head_dim = 128;
  p->rotary_dim = 128;
  p->layout = CONFKV_ROPE_HALF;
  p->scaling = CONFKV_ROPE_PLAIN;
  p->theta = 10000.0;
  p->factor = 1.0;
  p->low_band = 1.0;
  p->high_band = 4.0;
  p->beta_fast = 32.0;
  p->beta_slow = 1.0;
  p->magnitude = 0.0;
  p->original_length = 8192;
  return CONFKV_OK;
}

confkv_status confkv_rope_prepare(const confkv_rope_params* p, confkv_rope_table* out) {
  using namespace confkv;
  if (!p || !out) return CONFKV_ERR_ARG;
  const int D = p->head_dim, rd = p->rotary_dim;
  if (D < 2 || D > 2 * kMaxPairs || (D & 1) || rd < 0 || rd > D || (rd & 1)) return CONFKV_ERR_ARG;
  if (p->layout != CONFKV_ROPE_HALF && p->layout != CONFKV_ROPE_INTERLEAVED) return CONFKV_ERR_ARG;
  if (p->scaling < CONFKV_ROPE_PLAIN || p->scaling > CONFKV_ROPE_YARN) return CONFKV_ERR_ARG;
  if (!std::isfinite(p->theta) || p->theta <= 1.0) return CONFKV_ERR_ARG;
  if (!std::isfinite(p->magnitude) || p->magnitude < 0.0) return CONFKV_ERR_ARG;
  if (p->scaling != CONFKV_ROPE_PLAIN && !(finite_pos(p->factor) && p->factor >= 1.0)) return CONFKV_ERR_ARG;
  if (p->scaling >= CONFKV_ROPE_BANDED && p->original_length < 1) return CONFKV_ERR_ARG;
  if (p->scaling == CONFKV_ROPE_BANDED &&
      !(finite_pos(p->low_band) && finite_pos(p->high_band) && p->high_band > p->low_band))
    return CONFKV_ERR_ARG;
  if (p->scaling == CONFKV_ROPE_YARN &&
      !(finite_pos(p->beta_fast) && finite_pos(p->beta_slow) && p->beta_fast >= p->beta_slow))
    return CONFKV_ERR_ARG;
  double theta = p->theta, mag = 1.0;
  if (p->scaling == CONFKV_ROPE_NTK && rd > 2) theta *= std::pow(p->factor, (double)rd / (rd - 2));
  if (!std::isfinite(theta)) return CONFKV_ERR_ARG;
  double first = 0.0, last = 0.0;
  if (p->scaling == CONFKV_ROPE_YARN) {
    // the pair that makes `turns` turns within the original length
    auto pair_of = [&](double turns) {
      return rd * std::log(p->original_length / (turns * 2.0 * kPi)) / (2.0 * std::log(theta));
    };
    first = std::max(0.0, std::floor(pair_of(p->beta_fast)));
    last = std::min((double)rd - 1.0, std::ceil(pair_of(p->beta_slow)));
    mag = 0.1 * std::log(p->factor) + 1.0;
  }
  if (p->magnitude > 0.0) mag = p->magnitude;
  if (!finite_pos((float)mag)) return CONFKV_ERR_ARG;   // as the table holds it
  std::memset(out, 0, sizeof(*out));
  out->head_dim = D;
  out->rotary_dim = rd;
  out->layout = p->layout;
  out->magnitude = (float)mag;
  for (int i = 0; i < rd / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rd);   // radians a position
    if (p->scaling == CONFKV_ROPE_LINEAR) {
      f /= p->factor;
    } else if (p->scaling == CONFKV_ROPE_BANDED) {
      const double turns = p->original_length * f / (2.0 * kPi);
      const double keep = std::min(1.0, std::max(0.0, (turns - p->low_band) / (p->high_band - p->low_band)));
      f = f / p->factor * (1.0 - keep) + f * keep;
    } else if (p->scaling == CONFKV_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - first) / std::max(last - first, 0.001)));
      f = f / p->factor * ramp + f * (1.0 - ramp);
    }
    // f <= 1 radian, so the fraction of a turn is below 1/6 and 2^64 times it fits
    out->turns[i] = (uint64_t)std::llround(f / (2.0 * kPi) * 0x1p62) << 2;
  }
  return CONFKV_OK;
}

confkv_status confkv_rope(const confkv_rope_table* table, int32_t batch, int32_t tokens, const int32_t* positions,
                          int32_t x_type, int32_t y_type, float eps, const confkv_rope_rows* q,
                          const confkv_rope_rows* k, void* stream) {
  using namespace confkv;
  if (!table || !q || batch < 0 || tokens < 0) return CONFKV_ERR_ARG;
  const int D = table->head_dim, rd = table->rotary_dim;
  if (D < 2 || D > 2 * kMaxPairs || (D & 1) || rd < 0 || rd > D || (rd & 1)) return CONFKV_ERR_ARG;
  if (table->layout != CONFKV_ROPE_HALF && table->layout != CONFKV_ROPE_INTERLEAVED) return CONFKV_ERR_ARG;
  if (x_type < CONFKV_F32 || x_type > CONFKV_BF16 || y_type < CONFKV_F32 || y_type > CONFKV_BF16) return CONFKV_ERR_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return CONFKV_ERR_ARG;
  if (batch == 0 || tokens == 0) return CONFKV_OK;
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u)) return CONFKV_ERR_ARG;
  const size_t xs = x_type == CONFKV_F32 ? 4 : 2, ys = y_type == CONFKV_F32 ? 4 : 2;
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  const bool half = table->layout == CONFKV_ROPE_HALF;
  bool vec = (D == 32 || D == 64 || D == 128 || D == 256) && (!half || rd % 16 == 0);
  for (int sd = 0; sd < 2; ++sd) {
    if (sd == 1 && !k) continue;
    confkv_rope_rows own = sd ? *k : *q, *r = &own;
    // a dimension of size 1 has no stride, whatever it says
    if (batch == 1) r->x_batch = r->y_batch = 0;
    if (tokens == 1) r->x_token = r->y_token = 0;
    if (r->heads == 1) r->x_head = r->y_head = 0;
    if (r->heads < 1 || r->heads > (1 << 24) || !r->x || !r->y) return CONFKV_ERR_ARG;
    const uintptr_t px = reinterpret_cast<uintptr_t>(r->x), py = reinterpret_cast<uintptr_t>(r->y);
    const uintptr_t pw = reinterpret_cast<uintptr_t>(r->weight);
    if (px % xs || py % ys || pw % 4) return CONFKV_ERR_ARG;
    if (r->x_batch < 0 || r->x_token < 0 || r->x_head < 0 || r->y_batch < 0 || r->y_token < 0 || r->y_head < 0)
      return CONFKV_ERR_ARG;
    // distinct rows must be written to distinct places, those of q and k among them
    if (!rows_apart(D, batch, r->y_batch, tokens, r->y_token, r->heads, r->y_head)) return CONFKV_ERR_ARG;
    if (sd == 1 && r->y == q->y) return CONFKV_ERR_ARG;
    if (px == py && (x_type != y_type || r->x_batch != r->y_batch || r->x_token != r->y_token || r->x_head != r->y_head))
      return CONFKV_ERR_ARG;
    const long long ex = 16 / (long long)xs, ey = 16 / (long long)ys;
    vec = vec && px % 16 == 0 && py % 16 == 0 && pw % 16 == 0;
    vec = vec && r->x_batch % ex == 0 && r->x_token % ex == 0 && r->x_head % ex == 0;
    vec = vec && r->y_batch % ey == 0 && r->y_token % ey == 0 && r->y_head % ey == 0;
    a.side[sd] = RopeSide{r->x, r->y, r->weight, r->heads, r->x_batch, r->x_token, r->x_head,
                          r->y_batch, r->y_token, r->y_head};
    a.heads += r->heads;
  }
  a.pos = positions;
  a.batch = batch;
  a.tokens = tokens;
  a.D = D;
  a.rd = rd;
  a.eps = eps;
  a.mag = table->magnitude;
  std::memcpy(a.turns, table->turns, sizeof(uint64_t) * (size_t)(rd / 2));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (x_type) {
    case CONFKV_F32: e = launch_x<float>(a, y_type, half, vec, st); break;
    case CONFKV_F16: e = launch_x<__half>(a, y_type, half, vec, st); break;
    default: e = launch_x<__nv_bfloat16>(a, y_type, half, vec, st); break;
  }
  if (e == cudaErrorInvalidValue) {
    (void)cudaGetLastError();
    return CONFKV_ERR_ARG;
  }
  return e == cudaSuccess ? CONFKV_OK : CONFKV_ERR_CUDA;
}

}  // extern "C"
