// Sampling of the next token from given uniform numbers, with temperature,
// top-k, top-p (nucleus) and min-p, per row.
//
// With w_i = exp((x_i - max x) / T) and the tokens of a row in descending order
// of x (equal logits: the lower index first),
//   K1 = the first top_k tokens,
//   K2 = the tokens of K1 before which less than top_p of K1's weight lies,
//   K3 = the tokens with x_i >= max x + T ln(min_p),
// the token drawn is the first i, by index, at which the running sum of the
// weights kept (K2 and K3) exceeds u times their total.
//
// One cluster of CTAs takes a row. Each CTA reads its part of the row once and
// keeps it in shared memory; everything after that works from there, so HBM
// sees each logit once. What is left is latency and the instructions per logit:
//   1. maximum and minimum of the row;
//   2. only with top-k or top-p: a histogram over 1024 bins of the distance from
//      the maximum, 1/32 of a factor of two each (less where the row's range is
//      below 16 factors of two): counts for top-k, weights for top-p. The bin in
//      which the cut falls is found by a scan, and all tokens down to it are
//      gathered in the first CTA. If they fit there (the usual case), that CTA
//      finds the cuts and the token alone, by histograms of its own, and the row
//      is done; the cluster's other CTAs leave.
//   3. Otherwise (a wide nucleus, thousands of equal logits) the cut's own bin is
//      gathered, split further where it is too full (by another histogram over it,
//      then by the bits of the (logit, index) pair), which gives the cut as such a
//      pair; the weights of every warp's stretch of the row are summed, and the
//      stretch that holds u times the total is scanned.
// Weights are summed as integers where the order of the additions is not fixed, in
// fp64 and in a fixed order for the draw over a whole row, so two runs agree bit
// for bit. The integers of the top-p cut are units of 2^-30 of a power of two near
// the bin's own weights (of the largest weight of the row, a tail of 100000 light
// tokens came out wrong by as much as it weighs); a bin's sum then goes into units of
// 2^-42 of the largest, and what is left of the cut inside the bin back into the bin's.
// Sums over a gathered list are units of 2^-40 of the largest. The exponent
// (x - max) / (T ln 2) carries a correction for its rounding, which alone would move
// the weights of far tokens by 1e-6.
// Measured: 16 rows of 128256 fp32 with top-k 1000, top-p and min-p 30 us, 256 rows
// with top-p 0.9 206 us (0.64 TB/s: the dozen barriers between a row's phases bound
// it, with 37% of the issue slots used), 33 bf16 rows of 152064 with min-p
// 14 us, one row of 50257 with top-k and top-p 13 us, all latency.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <climits>
#include <cstddef>

#include "../../include/confkv.h"
#include "common.cuh"
#include "kernels.h"

namespace confkv {

namespace {

namespace cg = cooperative_groups;

constexpr int NT = 512, NW = NT / 32;
constexpr int kBins = 1024;            // (with these sizes two CTAs of a 128K row fit on an SM, three where no cuts are set)
constexpr int kGather = 2048;          // tokens that the first CTA's buffer holds
constexpr int kAll = 2048;             // tokens down to a cut from which one CTA finishes the row
constexpr int kGathers = 24;           // more than a row can need: two cuts, each at once, by parts of its bin and by six digits
constexpr int kFew = 128;              // as many are ranked by comparing all with all
static_assert(kAll <= kGather && kFew <= NT && kBins % NT == 0, "sizes of the first CTA's work");
constexpr size_t kMaxShared = 220 * 1024;   // a wider part of a row stays in global memory
constexpr int kMaxVocab = 1 << 20;     // index bits of the (logit, index) pair
constexpr int kIndexBits = 20;

typedef unsigned long long u64;

struct SampleArgs {
  const void* logits;
  long long stride;
  int vocab, chunk;         // chunk: logits per CTA of the cluster (a multiple of 8)
  int staged;               // 1: the chunk fits in shared memory
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  float* prob;
};

template <int CS>
struct Shared {
  u64 scan[NW];
  double dscan[NW];
  uint32_t scan_c[NW];
  int pick, last;
  u64 part[CS];                         // of every CTA: the sum of its slice,
  double weights[CS];                   // what it keeps,
  float4 extremes[CS];                  // the largest and smallest logit, and whether one is bad
  // read by the other CTAs of the cluster
  float mx, mn;
  int bad, first;
  double kept;
  // ---- only where cuts may be set ----
  u64 slice_sum, key;
  uint32_t n_cand[kGathers];            // one counter a gather
  u64 slice[kBins / CS];                // cluster-wide sums of this CTA's share of the bins
  u64 cut_before, cut_here;
  int cut_bin, n_keep;
  int n_list;
  uint32_t light;                       // of this CTA's tokens that a histogram passes over (2^-42)
  u64 list[kFew];
  uint32_t sel[2][kBins];               // select: the low and high 20 bits of the weights
  union {
    uint32_t hist[2][kBins];            // counts; or the low and high 15 bits of the weights
    u64 cand[kGather];
  };
};
template <int CS, bool CUT>
constexpr size_t kSharedBytes = ((CUT ? sizeof(Shared<CS>) : offsetof(Shared<CS>, slice_sum)) + 15) / 16 * 16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// Weights of one row: 2^((x - m) c), c = 1 / (T ln 2) as two floats.
struct Weigher {
  float m, chi, clo;
  float per;   // bins a factor of two, times -1 (a power of two, at least 32 where weights are summed by bin)
  // the exponent, rounded: descending in x, 0 at the maximum
  __device__ __forceinline__ float lead(float x) const { return __fmul_rn(__fsub_rn(x, m), chi); }
  __device__ __forceinline__ int bin(float d) const { return (int)fminf(__fmul_rn(d, per), (float)(kBins - 1)); }
  // the place within a bin, in kBins steps (products by powers of two and this difference are exact)
  __device__ __forceinline__ int sub_bin(float d, int b) const {
    return (int)fminf(__fmul_rn(__fsub_rn(__fmul_rn(d, per), (float)b), (float)kBins), (float)(kBins - 1));
  }
  // the weight of x with exponent d = lead(x): 2^d with the product's rounding
  // error e put back as a factor 1 + e ln 2; 0 below 2^-100
  __device__ __forceinline__ float weight(float x, float d) const {
    const float hi = __fsub_rn(x, m);
    const float e = __fmaf_rn(hi, clo, __fmaf_rn(hi, chi, -d));
    const float w = __fmul_rn(ex2(d), __fmaf_rn(e, 0.69314718f, 1.0f));
    return d > -100.0f ? w : 0.0f;
  }
  __device__ __forceinline__ float weight(float x) const { return weight(x, lead(x)); }
  // the weights of bin b lie between 2^-(e + 1) and 2^-e, e = fall(b) (the last bin's: anywhere below)
  __device__ __forceinline__ int fall(int b) const { return b >> ((__float_as_int(-per) >> 23) - 127); }
};
// About how many tokens of bin b have `mass` (of 2^-42) together (they weigh the same to 2%, the last bin's aside).
__device__ __forceinline__ float about(const Weigher& wt, u64 mass, int b) {
  return (float)mass * ex2(((float)b + 0.5f) / -wt.per - 42.0f);
}
// A weight in units of 2^-(30 + fall), fall that of its bin (below 2^30 units).
__device__ __forceinline__ uint32_t units(float w, int fall) {
  return min(__float2uint_rn(w * __int_as_float((127 + 30 + fall) << 23)), (1u << 30) - 1u);
}
// A bin's sum in units of 2^-42; and of a part of that, rounded up, in the bin's (not above its sum).
__device__ __forceinline__ u64 to_common(u64 sum, int fall) { return (sum << 12) >> fall; }
__device__ __forceinline__ u64 to_bin(u64 part, int fall) { return ((part << fall) + 0xfffull) >> 12; }
// A weight in units of 2^-40, for sums over a list.
__device__ __forceinline__ u64 fine_units(float w) { return min(__float2ull_rn(w * 0x1p40f), (1ull << 40) - 1ull); }

// (logit, index) as an integer that descends along the order of the tokens.
__device__ __forceinline__ u64 pair_key(float x, int i) {
  return ((u64)ordered_bits(x) << kIndexBits) | (unsigned)(kMaxVocab - 1 - i);
}
__device__ __forceinline__ float key_logit(u64 k) {
  const uint32_t o = (uint32_t)(k >> kIndexBits);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_index(u64 k) { return kMaxVocab - 1 - (int)(k & (kMaxVocab - 1)); }

// A cut of the order: the tokens down to a pair, compared without 64-bit keys.
struct Cut {
  float x;
  int i;
  __device__ __forceinline__ bool keeps(float v, int j) const { return (v > x) | ((v == x) & (j <= i)); }
};

template <class T>
__device__ __forceinline__ T warp_total(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Exclusive prefix sum over the CTA's threads, in a fixed order; *total: of all.
template <class T>
__device__ __forceinline__ T block_prefix(T* scratch, T v, T* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T a = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += a;
  }
  __syncthreads();
  if (lane == 31) scratch[w] = inc;
  __syncthreads();
  T base = 0, all = 0;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    if (k == w) base = all;
    all += scratch[k];
  }
  *total = all;
  // the exclusive value is the left neighbour's inclusive one, the same number
  // whichever side asks for it
  T left = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) left = 0;
  return base + left;
}

template <class X>
struct Row {
  const X* g;         // the CTA's part in global memory
  const float* s;     // and in shared memory, when staged (-inf past the end, up to a multiple of 4)
  int n;
  u64 near;           // the logits of this thread in bins before the last, bit 4 j + k for the k-th of its j-th four
  bool few;           // few are: the loops below go by `near` (the same in a warp)
  __device__ __forceinline__ float at(int i) const { return s ? s[i] : to_f(g[i]); }
};

// f(x, i) for every four logits x, at i in the CTA's part; the ones past its end
// are -inf. Four at a time and without branches between them, the loops below keep
// their latencies overlapped. Where only a few tokens of the warp have weight, f
// sees those alone.
template <class X, class F>
__device__ __forceinline__ void each4(const Row<X>& row, F f) {
  float x[4];
  int at[4];
  if (row.few) {
    u64 h = row.near;
    while (h) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int b = h ? __ffsll((long long)h) - 1 : 0;
        at[k] = 4 * threadIdx.x + (b >> 2) * (4 * NT) + (b & 3);
        x[k] = h ? row.s[at[k]] : -CUDART_INF_F;
        h &= h - 1;
      }
      f(x, at);
    }
  } else if (row.s) {
    for (int i = 4 * threadIdx.x; i < row.n; i += 4 * NT) {
      const float4 v = *reinterpret_cast<const float4*>(row.s + i);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
#pragma unroll
      for (int k = 0; k < 4; ++k) at[k] = i + k;
      f(x, at);
    }
  } else {
    for (int i = threadIdx.x; i < row.n; i += 4 * NT) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        at[k] = i + k * NT;
        x[k] = at[k] < row.n ? to_f(row.g[at[k]]) : -CUDART_INF_F;
      }
      f(x, at);
    }
  }
}

// to[k] = from the k-th CTA of the cluster, one thread a CTA; the others read it
// from here (every thread reading all of them keeps the cluster's network busy for
// a thousand cycles and more).
template <int CS, class T, class From>
__device__ __forceinline__ void collect(cg::cluster_group& cl, Shared<CS>& sh, T* to, From from) {
  if (threadIdx.x < CS) to[threadIdx.x] = from(*cl.map_shared_rank(&sh, (int)threadIdx.x));
  __syncthreads();
}

// Histogram of the tokens that `in` selects, by `digit`, summed over the
// cluster: every CTA ends with its share of the bins and that share's sum.
// Returns the sum of all. KIND: token counts; weights by bin (the digit is the
// bin, the sums in units of 2^-42); weights of one bin's tokens by another digit
// (the sums in that bin's units). rest: count, or weight in 2^-42, of this thread's
// tokens in the last bin that each4 passes over.
enum Kind { COUNT, BINS, WITHIN };
template <Kind KIND, int CS, class X, class In, class Digit>
__device__ __forceinline__ u64 histogram(cg::cluster_group& cl, Shared<CS>& sh, const Row<X>& row, const Weigher& wt,
                                         In in, Digit digit, uint32_t rest = 0, int fall = 0) {
  constexpr bool MASS = KIND != COUNT;
  for (int i = threadIdx.x; i < (MASS ? 2 : 1) * kBins; i += NT) (&sh.hist[0][0])[i] = 0;
  if (KIND == BINS && threadIdx.x == 0) sh.light = 0;
  __syncthreads();
  each4(row, [&](const float (&x)[4], const int (&at)[4]) {
    int b[4];
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float d = wt.lead(x[k]);
      const bool mine = x[k] > -CUDART_INF_F && in(x[k], at[k], d);
      b[k] = digit(x[k], at[k], d);
      w[k] = !mine ? 0u : MASS ? units(wt.weight(x[k], d), KIND == BINS ? wt.fall(b[k]) : fall) : 1u;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (MASS) {   // (at most 2^17 tokens a CTA)
        if (w[k] & 0x7fffu) atomicAdd(&sh.hist[0][b[k]], w[k] & 0x7fffu);
        if (w[k] >> 15) atomicAdd(&sh.hist[1][b[k]], w[k] >> 15);
      } else if (b[k] == kBins - 1) {   // the far tokens, most of a confident row: one address
        rest += w[k];
      } else {
        if (w[k]) atomicAdd(&sh.hist[0][b[k]], 1u);
      }
    }
  });
  if (KIND != WITHIN) {
    rest = __reduce_add_sync(0xffffffffu, rest);
    if (rest && (threadIdx.x & 31) == 0) atomicAdd(KIND == BINS ? &sh.light : &sh.hist[0][kBins - 1], rest);
  }
  cl.sync();
  constexpr int share = kBins / CS;
  const int rank = (int)cl.block_rank();
  u64 sum = 0;
  for (int i = threadIdx.x; i < share; i += NT) {
    const int bin = rank * share + i;
    u64 v = 0, light = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      const Shared<CS>* o = cl.map_shared_rank(&sh, r);
      v += o->hist[0][bin];
      if (MASS) v += (u64)o->hist[1][bin] << 15;
      if (KIND == BINS && bin == kBins - 1) light += o->light;
    }
    if (KIND == BINS) v = to_common(v, wt.fall(bin)) + light;
    sh.slice[i] = v;
    sum += v;
  }
  // (only the warps with bins have anything to add)
  sum = warp_total(sum);
  if ((threadIdx.x & 31) == 0) sh.scan[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0;
    for (int w = 0; w < NW; ++w) sum += sh.scan[w];
    sh.slice_sum = sum;
  }
  cl.sync();
  collect(cl, sh, sh.part, [](const Shared<CS>& o) { return o.slice_sum; });
  u64 all = 0;
#pragma unroll
  for (int r = 0; r < CS; ++r) all += sh.part[r];
  return all;
}

// The bin in which the running sum of the last histogram reaches `target` (1 <=
// target <= the sum); *before: the sum ahead of it, *here: its own. Every CTA finds the same.
template <int CS>
__device__ __forceinline__ int find_bin(cg::cluster_group& cl, Shared<CS>& sh, u64 target, u64* before, u64* here) {
  constexpr int share = kBins / CS, per = (share + NT - 1) / NT;
  // the CTA whose share holds it
  u64 ahead = 0;
  int r = 0;
#pragma unroll
  for (int k = 0; k < CS - 1; ++k)
    if (r == k && ahead + sh.part[k] < target) {
      ahead += sh.part[k];
      r = k + 1;
    }
  const Shared<CS>* o = cl.map_shared_rank(&sh, r);
  const int i0 = threadIdx.x * per;
  u64 v[per], sum = 0, all;
#pragma unroll
  for (int k = 0; k < per; ++k) {
    v[k] = i0 + k < share ? o->slice[i0 + k] : 0;
    sum += v[k];
  }
  u64 run = ahead + block_prefix(sh.scan, sum, &all);
#pragma unroll
  for (int k = 0; k < per; ++k) {
    if (run < target && run + v[k] >= target) {
      sh.cut_bin = r * share + i0 + k;
      sh.cut_before = run;
      sh.cut_here = v[k];
    }
    run += v[k];
  }
  __syncthreads();
  *before = sh.cut_before;
  *here = sh.cut_here;
  const int b = sh.cut_bin;
  __syncthreads();
  return b;
}

// The tokens that `in` selects, as keys in the first CTA's `cand` (as many as
// fit). Returns how many there are. `turn` counts the row's gathers. (The last
// barrier before it was past every read of the histogram that `cand` lies over.)
template <int CS, class X, class In>
__device__ __forceinline__ uint32_t gather(cg::cluster_group& cl, Shared<CS>& sh, const Row<X>& row, int i0,
                                           const Weigher& wt, int* turn, In in) {
  Shared<CS>* lead = cl.map_shared_rank(&sh, 0);
  uint32_t* counter = &lead->n_cand[*turn];
  ++*turn;
  // counted first: one addition to the counter a CTA, not one a token
  uint32_t c = 0, all;
  u64 hits = 0;               // of the first 64 logits of this thread
  int seen = 0;
  each4(row, [&](const float (&x)[4], const int (&i)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m |= (uint32_t)(x[k] > -CUDART_INF_F && in(x[k], i[k], wt.lead(x[k]))) << k;
    c += __popc(m);
    if (seen < 64) hits |= (u64)m << seen;
    seen += 4;
  });
  uint32_t at = block_prefix(sh.scan_c, c, &all);
  if (threadIdx.x == 0) sh.pick = all ? (int)atomicAdd(counter, all) : 0;
  __syncthreads();
  if (c && all <= kGather) {
    at += (uint32_t)sh.pick;
    auto put = [&](float x, int i) {
      if (at < kGather) lead->cand[at] = pair_key(x, i0 + i);
      ++at;
    };
    if (row.s && !row.few && seen <= 64) {
      while (hits) {
        const int k = __ffsll((long long)hits) - 1;
        hits &= hits - 1;
        const int i = 4 * threadIdx.x + (k >> 2) * (4 * NT) + (k & 3);
        put(row.s[i], i);
      }
    } else {
      each4(row, [&](const float (&x)[4], const int (&i)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (x[k] > -CUDART_INF_F && in(x[k], i[k], wt.lead(x[k]))) put(x[k], i[k]);
      });
    }
  }
  cl.sync();
  return *counter;
}

// One CTA: v[0 .. n) in descending order, n up to kFew.
__device__ __forceinline__ void sort_descending(u64* v, int n) {
  const u64 mine = threadIdx.x < n ? v[threadIdx.x] : 0;
  int at = 0;
  for (int j = 0; j < n; ++j) at += v[j] > mine;
  __syncthreads();
  if (threadIdx.x < n) v[at] = mine;   // (the keys are distinct)
  __syncthreads();
}

// One CTA: of the keys in `cand`, the one at which the running weight (below 2^40
// each) reaches `target`, along descending order(key); the digits ascend with it.
// The keys of the digit in which the target falls are listed, and split by their
// order's bits (of `bits`) while the list is too long; so no list is ever sorted: a
// sort of a thousand keys takes 13000 cycles, this about 2000.
template <int CS, class Digit, class Weight, class Order>
__device__ __forceinline__ u64 select(Shared<CS>& sh, int n, u64 target, int bits, Digit digit, Weight weight, Order order) {
  constexpr int per = kBins / NT;
  int shift = bits, first = -1;
  u64 prefix = 0;
  while (true) {
    for (int i = threadIdx.x; i < 2 * kBins; i += NT) (&sh.sel[0][0])[i] = 0;
    if (threadIdx.x == 0) sh.n_list = 0;
    __syncthreads();
    const int step = first < 0 ? 0 : min(10, shift), next = shift - step;
    auto mine = [&](u64 k) { return first < 0 || (digit(k) == first && (order(k) >> shift) == prefix); };
    auto at = [&](u64 k) {
      return first < 0 ? digit(k) : ((1 << step) - 1) - (int)((order(k) >> next) & (u64)((1 << step) - 1));
    };
    for (int i = threadIdx.x; i < n; i += NT) {
      const u64 k = sh.cand[i], w = mine(k) ? weight(k) : 0;
      const uint32_t lo = (uint32_t)w & 0xfffffu, hi = (uint32_t)(w >> 20);
      if (lo) atomicAdd(&sh.sel[0][at(k)], lo);
      if (hi) atomicAdd(&sh.sel[1][at(k)], hi);
    }
    __syncthreads();
    u64 v[per], sum = 0, all;
#pragma unroll
    for (int k = 0; k < per; ++k) {
      const int i = threadIdx.x * per + k;
      v[k] = sh.sel[0][i] + ((u64)sh.sel[1][i] << 20);
      sum += v[k];
    }
    u64 run = block_prefix(sh.scan, sum, &all);
#pragma unroll
    for (int k = 0; k < per; ++k) {
      if (run < target && run + v[k] >= target) {
        sh.cut_bin = threadIdx.x * per + k;
        sh.cut_before = run;
      }
      run += v[k];
    }
    __syncthreads();
    const int b = sh.cut_bin;
    target -= sh.cut_before;
    for (int i = threadIdx.x; i < n; i += NT) {
      const u64 k = sh.cand[i];
      if (mine(k) && at(k) == b && weight(k)) {
        const int to = atomicAdd(&sh.n_list, 1);
        if (to < kFew) sh.list[to] = k;
      }
    }
    __syncthreads();
    const int m = sh.n_list;
    if (m <= kFew) {
      if (threadIdx.x < m) {
        const u64 k = sh.list[threadIdx.x], o = order(k);
        u64 before = 0;
        for (int j = 0; j < m; ++j) before += order(sh.list[j]) > o ? weight(sh.list[j]) : 0;
        if (before < target && before + weight(k) >= target) sh.key = k;
      }
      __syncthreads();
      const u64 key = sh.key;
      __syncthreads();
      return key;
    }
    __syncthreads();   // every warp has read n_list, which the next turn sets to 0
    if (first < 0) {
      first = b;
    } else {
      prefix = (prefix << step) | (unsigned)(((1 << step) - 1) - b);
      shift = next;
    }
  }
}

// The key at which the running count (or weight, in the bin's units) reaches
// `target` (what is left of it ahead of bin `bin`), by gathering the bin, split while it is too full:
// first into parts of its width, then by the keys' bits. here: the bin's count
// or an estimate of it.
template <bool MASS, int CS, class X, class In>
__device__ __noinline__ u64 exact_cut(cg::cluster_group& cl, Shared<CS>& sh, const Row<X>& row, int i0,
                                      const Weigher& wt, int* turn, int bin, u64 target, u64 here, In in) {
  int shift = kIndexBits + 32, sub = -1;
  u64 prefix = 0, before;
  const int fall = MASS ? wt.fall(bin) : 0;
  constexpr Kind KIND = MASS ? WITHIN : COUNT;
  auto mine = [&](float x, int i, float d) {
    return wt.bin(d) == bin && (sub < 0 || wt.sub_bin(d, bin) == sub) && in(x, i, d) &&
           (shift == kIndexBits + 32 || (pair_key(x, i0 + i) >> shift) == prefix);
  };
  uint32_t found = here > kGather ? kGather + 1 : 0;
  while ((found > kGather || (found = gather(cl, sh, row, i0, wt, turn, mine)) > kGather) && shift > 0) {
    if (sub < 0) {
      (void)histogram<KIND>(cl, sh, row, wt, mine, [&](float, int, float d) { return wt.sub_bin(d, bin); }, 0, fall);
      sub = find_bin(cl, sh, target, &before, &here);
    } else {
      const int bits = min(10, shift), next = shift - bits, top = (1 << bits) - 1;
      (void)histogram<KIND>(cl, sh, row, wt, mine, [&](float x, int i, float) {
        return top - (int)((pair_key(x, i0 + i) >> next) & (unsigned)top);
      }, 0, fall);
      const int b = find_bin(cl, sh, target, &before, &here);
      prefix = (prefix << bits) | (unsigned)(top - b);
      shift = next;
    }
    target -= before;
    found = !MASS && here > kGather && shift > 0 ? kGather + 1 : 0;
  }
  if (cl.block_rank() == 0) {
    const u64 k = select(sh, min((int)found, kGather), target, kIndexBits + 32,
                         [&](u64 k) { return wt.sub_bin(wt.lead(key_logit(k)), bin); },
                         [&](u64 k) { return MASS ? (u64)units(wt.weight(key_logit(k)), fall) : 1ull; }, [](u64 k) { return k; });
    if (threadIdx.x == 0) sh.key = k;
  }
  cl.sync();
  return cl.map_shared_rank(&sh, 0)->key;
}

// The first CTA finishes a row from the tokens in `cand`, which are the first n
// of the order: top-k, top-p, min-p and the draw. cut_bin: where the cut of top-p
// falls, cut_target in that bin's units; -1: at top_p of the weight of the list's
// first top_k.
template <int CS>
__device__ __noinline__ void finish(Shared<CS>& sh, int n, const Weigher& wt, int top_k, float top_p, int cut_bin,
                                    u64 cut_target, float least, float u, int vocab, int32_t* token, float* prob) {
  if (n > kFew) {
    auto bin = [&](u64 k) { return wt.bin(wt.lead(key_logit(k))); };
    auto same = [](u64 k) { return k; };
    u64 low = 0, sum = 0, all;   // keys from `low` on are kept
    if (top_k > 0 && top_k < n) low = select(sh, n, (u64)top_k, kIndexBits + 32, bin, [](u64) { return 1ull; }, same);
    if (top_p < 1.0f) {
      if (cut_bin < 0) {
        auto weight = [&](u64 k) { return k >= low ? fine_units(wt.weight(key_logit(k))) : 0ull; };
        for (int i = threadIdx.x; i < n; i += NT) sum += weight(sh.cand[i]);
        (void)block_prefix(sh.scan, sum, &all);
        const u64 target = max(1ull, min(all, (u64)ceil((double)top_p * (double)all)));
        low = max(low, select(sh, n, target, kIndexBits + 32, bin, weight, same));
      } else {   // (every token of the bins before it is above that key)
        const int fall = wt.fall(cut_bin);
        low = select(sh, n, cut_target, kIndexBits + 32, [&](u64 k) { return wt.sub_bin(wt.lead(key_logit(k)), cut_bin); },
                     [&](u64 k) { return bin(k) == cut_bin ? (u64)units(wt.weight(key_logit(k)), fall) : 0ull; }, same);
      }
    }
    // the draw in the same units, exact whatever the order of the additions
    auto weight = [&](u64 k) {
      const float x = key_logit(k);
      return k >= low && x >= least ? fine_units(wt.weight(x)) : 0ull;
    };
    sum = 0;
    for (int i = threadIdx.x; i < n; i += NT) sum += weight(sh.cand[i]);
    (void)block_prefix(sh.scan, sum, &all);
    const int shift = max(0, 32 - __clz(vocab - 1) - 10);
    const u64 k = select(sh, n, min(all, (u64)((double)u * (double)all) + 1ull), kIndexBits,
                         [&](u64 k) { return key_index(k) >> shift; }, weight,
                         [](u64 k) { return k & (kMaxVocab - 1); });
    if (threadIdx.x == 0) {
      *token = key_index(k);
      if (prob) *prob = (float)((double)wt.weight(key_logit(k)) * 0x1p40 / (double)all);
    }
    return;
  }
  sort_descending(sh.cand, n);
  if (top_k > 0) n = min(n, top_k);
  constexpr int per = (kFew + NT - 1) / NT;
  const int j0 = threadIdx.x * per;
  u64 key[per], mass[per];
  float w[per];
  u64 sum = 0, all;
  if (threadIdx.x == 0) sh.n_keep = n;
  const int fall = cut_bin < 0 ? 0 : wt.fall(cut_bin);
#pragma unroll
  for (int k = 0; k < per; ++k) {
    key[k] = j0 + k < n ? sh.cand[j0 + k] : 0;
    const float x = key_logit(key[k]);
    w[k] = j0 + k < n ? wt.weight(x) : 0.0f;
    mass[k] = cut_bin < 0 ? fine_units(w[k]) : wt.bin(wt.lead(x)) == cut_bin ? units(w[k], fall) : 0;
    sum += mass[k];
  }
  u64 run = block_prefix(sh.scan, sum, &all);
  if (cut_bin < 0) cut_target = max(1ull, min(all, (u64)ceil((double)top_p * (double)all)));
#pragma unroll
  for (int k = 0; k < per; ++k) {
    const bool in = j0 + k < n && (top_p >= 1.0f || run < cut_target) && key_logit(key[k]) >= least;
    if (j0 + k < n && !in) atomicMin(&sh.n_keep, j0 + k);
    run += mass[k];
  }
  __syncthreads();
  n = sh.n_keep;   // at least the first token
  // by index: the lowest first (a key of the index's complement and the weight's bits)
#pragma unroll
  for (int k = 0; k < per; ++k)
    if (j0 + k < n) sh.cand[j0 + k] = (key[k] & (kMaxVocab - 1)) << 32 | __float_as_uint(w[k]);
  if (threadIdx.x == 0) {
    sh.pick = INT_MAX;
    sh.last = 0;
  }
  __syncthreads();
  sort_descending(sh.cand, n);
  double dsum = 0.0, total;
#pragma unroll
  for (int k = 0; k < per; ++k) {
    key[k] = j0 + k < n ? sh.cand[j0 + k] : 0;
    dsum += (double)__uint_as_float((uint32_t)key[k]);
  }
  double drun = block_prefix(sh.dscan, dsum, &total);
  const double at = (double)u * total;
#pragma unroll
  for (int k = 0; k < per; ++k) {
    drun += (double)__uint_as_float((uint32_t)key[k]);
    if (j0 + k < n && drun > at) {
      atomicMin(&sh.pick, j0 + k);
      break;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const u64 k = sh.cand[min(sh.pick, n - 1)];
    *token = kMaxVocab - 1 - (int)(k >> 32);
    if (prob) *prob = (float)((double)__uint_as_float((uint32_t)k) / total);
  }
}

// CUT: top-k or top-p may be set. (Three CTAs an SM: a row's phases wait for one
// another, and other rows fill the gaps.)
template <class X, int CS, bool CUT>
__global__ void __launch_bounds__(NT, CUT ? 2 : 3) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared<CS>& sh = *reinterpret_cast<Shared<CS>*>(smem);
  float* stage = reinterpret_cast<float*>(smem + kSharedBytes<CS, CUT>);
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int r = blockIdx.x / CS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  chain_enter();
  const float T = a.temperature ? a.temperature[r] : 1.0f;
  const int top_k = CUT && a.top_k ? a.top_k[r] : 0;
  const float top_p = CUT && a.top_p ? a.top_p[r] : 1.0f;
  const float min_p = a.min_p ? a.min_p[r] : 0.0f;
  const float u = a.u[r];
  const bool valid = T >= 0.0f && T <= 3.402823466e38f && top_p == top_p && min_p == min_p && u >= 0.0f && u < 1.0f;

  // ---- the CTA's part of the row: into shared memory, with its maximum ----
  const int i0 = min(rank * a.chunk, a.vocab);
  Row<X> row;
  row.g = static_cast<const X*>(a.logits) + (long long)r * a.stride + i0;
  row.n = min(a.chunk, a.vocab - i0);
  row.s = a.staged ? stage : nullptr;
  row.near = 0;
  row.few = false;
  float mx = -CUDART_INF_F, mn = CUDART_INF_F;   // (mn: of the logits above -inf)
  bool bad = false;
  auto look = [&](float x) {
    bad |= !(x < CUDART_INF_F);   // NaN or +inf
    mx = fmaxf(mx, x);
    if (CUT && x > -CUDART_INF_F) mn = fminf(mn, x);
  };
  constexpr int VEC = 16 / sizeof(X), U = CUT ? 8 : 4;
  const int nv = (reinterpret_cast<uintptr_t>(row.g) & 15u) == 0 ? row.n / VEC : 0;
  for (int v0 = threadIdx.x; v0 < nv; v0 += NT * U) {
    uint4 w[U];
#pragma unroll
    for (int q = 0; q < U; ++q)
      if (v0 + q * NT < nv) w[q] = __ldcs(reinterpret_cast<const uint4*>(row.g) + v0 + q * NT);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (v0 + q * NT >= nv) break;
      const X* e = reinterpret_cast<const X*>(&w[q]);
      float x[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        x[k] = to_f(e[k]);
        look(x[k]);
      }
      if (a.staged) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4)
          *reinterpret_cast<float4*>(stage + (v0 + q * NT) * VEC + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
      }
    }
  }
  for (int i = nv * VEC + threadIdx.x; i < row.n; i += NT) {
    const float x = to_f(row.g[i]);
    look(x);
    if (a.staged) stage[i] = x;
  }
  if (a.staged && threadIdx.x < 3 && row.n + threadIdx.x < (unsigned)((row.n + 3) & ~3)) stage[row.n + threadIdx.x] = -CUDART_INF_F;
  mx = warp_max(mx);
  if (CUT) mn = -warp_max(-mn);
  const bool wbad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    sh.scan_c[warp] = __float_as_uint(mx);
    sh.scan[warp] = wbad;
    if (CUT) sh.dscan[warp] = mn;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    u64 bd = 0;
    for (int w = 0; w < NW; ++w) {
      mx = fmaxf(mx, __uint_as_float(sh.scan_c[w]));
      bd |= sh.scan[w];
      if (CUT) mn = fminf(mn, (float)sh.dscan[w]);
    }
    sh.mx = mx;
    sh.mn = mn;
    sh.bad = (int)bd;
  }
  if (CUT && threadIdx.x < kGathers) sh.n_cand[threadIdx.x] = 0;
  cl.sync();
  collect(cl, sh, sh.extremes, [](const Shared<CS>& o) { return make_float4(o.mx, o.mn, o.bad ? 1.0f : 0.0f, 0.0f); });
  bool any_bad = false;
  mx = -CUDART_INF_F;
#pragma unroll
  for (int k = 0; k < CS; ++k) {
    const float4 o = sh.extremes[k];
    mx = fmaxf(mx, o.x);
    if (CUT) mn = fminf(mn, o.y);
    any_bad |= o.z != 0.0f;
  }
  // ---- rows without a token to draw, and rows with only one ----
  const bool none = !valid || any_bad || mx == -CUDART_INF_F;
  if (none || T < 0x1p-60f || top_k == 1 || top_p <= 0.0f) {
    int first = INT_MAX;
    if (!none) {
      for (int i = threadIdx.x; i < row.n; i += NT)
        if (row.at(i) == mx) {
          first = i0 + i;
          break;
        }
      first = __reduce_min_sync(0xffffffffu, first);
      __syncthreads();
      if (lane == 0) sh.scan_c[warp] = (uint32_t)first;
      __syncthreads();
      if (threadIdx.x == 0) {
        for (int w = 0; w < NW; ++w) first = min(first, (int)sh.scan_c[w]);
        sh.first = first;
      }
      cl.sync();
      if (rank == 0 && threadIdx.x == 0)
        for (int k = 0; k < CS; ++k) first = min(first, cl.map_shared_rank(&sh, k)->first);
    }
    if (rank == 0 && threadIdx.x == 0) {
      a.token[r] = none ? -1 : first;
      if (a.prob) a.prob[r] = none ? 0.0f : 1.0f;
    }
    cl.sync();   // nobody leaves while its shared memory is read
    return;
  }

  Weigher wt;
  wt.m = mx;
  const double c = 1.4426950408889634074 / (double)T;
  wt.chi = (float)c;
  wt.clo = (float)(c - (double)wt.chi);
  // 32 bins a factor of two; as many more as the row's range leaves room for, so
  // that a flat row's bins are as short as they can be
  wt.per = -32.0f;
  if (CUT)
    while (wt.per > -32.0f * kBins && wt.lead(mn) * wt.per * 2.0f < (float)(kBins - 1)) wt.per *= 2.0f;
  // min-p: the border is a logit, rounded up to the next float
  float least = -3.402823466e38f;
  if (min_p > 0.0f)
    least = fmaxf(least, __double2float_ru((double)mx + (double)T * log((double)fminf(min_p, 1.0f))));

  // ---- the cuts of top-k and top-p ----
  // Where most tokens of a row weigh less than 2^-31 of the largest, as in a
  // confident model's, the passes below go over the others alone, as long as no cut
  // falls past those (256 rows of 128256, top-p 0.9: 283 us without the list, 214 with
  // it; not for fewer than five fours a thread, where making it costs as much as it saves).
  uint32_t rest = 0, light = 0;   // tokens of this thread that are passed over: their count and weight (2^-42)
  const bool cuts = CUT && ((top_k > 0 && top_k < a.vocab) || top_p < 1.0f);
  const int fours = (row.n + 4 * NT - 1) / (4 * NT);
  if (cuts && wt.per == -32.0f && row.s && fours > 4 && fours <= 16) {
    int finite = 0, seen = 0;
    float sum = 0.0f;
    each4(row, [&](const float (&x)[4], const int (&)[4]) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float d = wt.lead(x[k]);
        const bool far = !(d * wt.per < (float)(kBins - 1));
        finite += x[k] > -CUDART_INF_F;
        m |= (uint32_t)!far << k;
        sum += far ? ex2(d) : 0.0f;
      }
      row.near |= (u64)m << seen;
      seen += 4;
    });
    const int mine = __popcll(row.near);
    row.few = 3 * ((__reduce_max_sync(0xffffffffu, mine) + 3) / 4) <= 2 * fours;
    if (row.few) {
      rest = (uint32_t)(finite - mine);
      light = __float2uint_rn(sum * 0x1p42f);
    }
  }
  Cut cut{-CUDART_INF_F, kMaxVocab};
  bool done = false;
  int turn = 0;
  if (top_k > 0 && top_k < a.vocab) {
    auto any = [](float, int, float) { return true; };
    const u64 count = histogram<COUNT>(cl, sh, row, wt, any, [&](float, int, float d) { return wt.bin(d); }, rest);
    if ((u64)top_k < count) {
      u64 before, here;
      int b = find_bin(cl, sh, (u64)top_k, &before, &here);
      const float per = wt.per;
      light = 0;   // past the cut, or (below) no longer passed over
      if (b == kBins - 1 && per == -32.0f) {
        // the cut lies past the bins (a confident row): all tokens again, in wider
        // ones that reach down to the smallest, or for 512 factors of two
        row.few = false;
        while (wt.per < -2.0f && wt.lead(mn) * wt.per >= (float)(kBins - 1)) wt.per *= 0.5f;
        (void)histogram<COUNT>(cl, sh, row, wt, any, [&](float, int, float d) { return wt.bin(d); });
        b = find_bin(cl, sh, (u64)top_k, &before, &here);
      }
      if (before + here <= kAll) {
        const uint32_t n = gather(cl, sh, row, i0, wt, &turn, [&](float, int, float d) { return wt.bin(d) <= b; });
        if (rank == 0) finish(sh, (int)n, wt, top_k, top_p, -1, 0, least, u, a.vocab, a.token + r, a.prob ? a.prob + r : nullptr);
        done = true;
      } else {
        const u64 k = exact_cut<false>(cl, sh, row, i0, wt, &turn, b, (u64)top_k - before, here, any);
        cut = Cut{key_logit(k), key_index(k)};
      }
      wt.per = per;
    }
  }
  if (!done && top_p < 1.0f) {
    auto in_k = [&](float x, int i, float) { return cut.keeps(x, i0 + i); };
    auto by_bin = [&](float, int, float d) { return wt.bin(d); };
    auto cut_of = [&](u64 mass) { return max(1ull, min(mass, (u64)ceil((double)top_p * (double)mass))); };
    u64 target = cut_of(histogram<BINS>(cl, sh, row, wt, in_k, by_bin, light));
    u64 before, here;
    int b = find_bin(cl, sh, target, &before, &here);
    if (b == kBins - 1 && wt.per == -32.0f) {   // among the tokens passed over, if there are any: all of them again
      row.few = false;
      target = cut_of(histogram<BINS>(cl, sh, row, wt, in_k, by_bin));
      b = find_bin(cl, sh, target, &before, &here);
    }
    target = to_bin(target - before, wt.fall(b));
    // the tokens down to the bin are at most as many as weigh what the bin's do; a bin
    // that is itself too full is not gathered to find that out
    const float in_bin = about(wt, here, b);
    uint32_t n = kAll + 1;
    if (in_bin < (float)kAll && (float)before * 0x1p-42f < (float)kAll)
      n = gather(cl, sh, row, i0, wt, &turn, [&](float x, int i, float d) { return wt.bin(d) <= b && cut.keeps(x, i0 + i); });
    if (n <= kAll) {
      if (rank == 0) finish(sh, (int)n, wt, 0, top_p, b, target, least, u, a.vocab, a.token + r, a.prob ? a.prob + r : nullptr);
      done = true;
    } else {
      const u64 k = exact_cut<true>(cl, sh, row, i0, wt, &turn, b, target, (u64)in_bin, in_k);
      cut = Cut{key_logit(k), key_index(k)};
    }
  }
  if (done) {
    // The first CTA, whose counter the others read, leaves last; they make room
    // for the next row while it draws.
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (rank == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    return;
  }

  // ---- the draw over the whole row ----
  auto kept = [&](float x, int i) { return x >= least && (!CUT || cut.keeps(x, i0 + i)) ? wt.weight(x) : 0.0f; };
  const int seg = (row.n + 4 * NT - 1) / (4 * NT) * 128;   // a warp's stretch
  const int s0 = warp * seg, s1 = min(row.n, s0 + seg);
  double sum = 0.0;
  if (row.s) {
    for (int i = s0 + 4 * lane; i < s1; i += 128) {
      const float4 v = *reinterpret_cast<const float4*>(row.s + i);
      sum += (double)((kept(v.x, i) + kept(v.y, i + 1)) + (kept(v.z, i + 2) + kept(v.w, i + 3)));
    }
  } else {
    for (int i = s0 + lane; i < s1; i += 32) sum += (double)kept(to_f(row.g[i]), i);
  }
  sum = warp_total(sum);
  __syncthreads();
  if (lane == 0) sh.dscan[warp] = sum;
  if (threadIdx.x == 0) {
    sh.pick = INT_MAX;
    sh.last = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int w = 0; w < NW; ++w) t += sh.dscan[w];
    sh.kept = t;
  }
  cl.sync();
  collect(cl, sh, sh.weights, [](const Shared<CS>& o) { return o.kept; });
  double part[CS], total = 0.0;
#pragma unroll
  for (int k = 0; k < CS; ++k) {
    part[k] = sh.weights[k];
    total += part[k];
  }
  // The CTA and the warp in whose stretch u * total falls, by the same additions
  // everywhere; u < 1, and the last stretch with weight takes what rounding leaves over.
  const double at = (double)u * total;
  double base = 0.0, run = 0.0;
  int own = -1;
#pragma unroll
  for (int k = 0; k < CS; ++k) {
    if (part[k] > 0.0 && run <= at) {
      own = k;
      base = run;
    }
    run += part[k];
  }
  if (own == rank) {
    int ws = 0;
    double wbase = base, wrun = base;
    for (int w = 0; w < NW; ++w) {
      const double v = sh.dscan[w];
      if (v > 0.0 && wrun <= at) {
        ws = w;
        wbase = wrun;
      }
      wrun += v;
    }
    const int per = (seg + NT - 1) / NT;
    const int j0 = ws * seg + threadIdx.x * per, j1 = min(min(j0 + per, ws * seg + seg), row.n);
    sum = 0.0;
    for (int j = j0; j < j1; ++j) sum += (double)kept(row.at(j), j);
    __syncthreads();   // the warps' sums have been read
    double all;
    double before = wbase + block_prefix(sh.dscan, sum, &all);
    for (int j = j0; j < j1; ++j) {
      const double wj = (double)kept(row.at(j), j);
      if (wj > 0.0) {
        atomicMax(&sh.last, j);
        if (before + wj > at) atomicMin(&sh.pick, j);
      }
      before += wj;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      const int j = min(sh.pick, sh.last);   // (none passes: the last one with weight)
      a.token[r] = i0 + j;
      if (a.prob) a.prob[r] = (float)((double)kept(row.at(j), j) / total);
    }
  }
  cl.sync();
}

template <class X, int CS, bool CUT>
cudaError_t launch_cut(const SampleArgs& a0, int rows, cudaStream_t st) {
  SampleArgs a = a0;
  a.chunk = ((a.vocab + CS - 1) / CS + 7) / 8 * 8;
  size_t smem = kSharedBytes<CS, CUT>;
  const size_t part = (size_t)a.chunk * 4;
  a.staged = smem + part <= kMaxShared ? 1 : 0;
  if (a.staged) smem += part;
  // Few rows spread over the SMs: where two CTAs an SM hold them all, as much
  // shared memory is asked for as keeps a third from joining them (33 rows of
  // 152064: 12.8 us, 15.5 with three; 256 rows: 80 and 71). Clusters do not fill every
  // SM, so a tenth is left over; at one CTA an SM that is too little for 16 rows
  // (42 us, 31 with two).
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (10ll * rows * CS <= 18ll * sms) smem = std::max<size_t>(smem, 78 * 1024);
  // The limit is the kernel's, for every thread that calls it: always the same one, so that no call lowers it
  // between another's setting and launch.
  cudaError_t e =
      cudaFuncSetAttribute(sample_kernel<X, CS, CUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxShared);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * CS);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<X, CS, CUT>, a);
}

template <class X, int CS>
cudaError_t launch_row(const SampleArgs& a, int rows, cudaStream_t st) {
  return a.top_k || a.top_p ? launch_cut<X, CS, true>(a, rows, st) : launch_cut<X, CS, false>(a, rows, st);
}

// CTAs a row: eight for wide vocabularies (the row then fits in their shared
// memory), fewer where a CTA would get less than about two thousand logits and
// the cluster's barriers would outweigh the shared work.
template <class X>
cudaError_t launch_sample(const SampleArgs& a, int rows, cudaStream_t st) {
  if (a.vocab > 8192) return launch_row<X, 8>(a, rows, st);
  if (a.vocab > 2048) return launch_row<X, 4>(a, rows, st);
  return launch_row<X, 1>(a, rows, st);
}

}  // namespace

}  // namespace confkv

extern "C" {

confkv_status confkv_sample(int32_t type, const void* logits, int64_t row_stride, int32_t rows, int32_t vocab,
                            const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                            const float* min_p, int32_t* token_out, float* prob_out, void* stream) {
  using namespace confkv;
  if (type < CONFKV_F32 || type > CONFKV_BF16 || rows < 0 || vocab < 1) return CONFKV_ERR_ARG;
  if (rows == 0) return CONFKV_OK;
  if (!logits || !u || !token_out || (rows > 1 && row_stride < vocab)) return CONFKV_ERR_ARG;
  const uintptr_t es = type == CONFKV_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es) return CONFKV_ERR_ARG;
  for (const void* p : {(const void*)u, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                        (const void*)min_p, (const void*)token_out, (const void*)prob_out})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return CONFKV_ERR_ARG;
  if (vocab > kMaxVocab || rows > (1 << 27)) return CONFKV_ERR_CAPACITY;
  SampleArgs a{};
  a.logits = logits;
  a.stride = row_stride;
  a.vocab = vocab;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.token = token_out;
  a.prob = prob_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (type) {
    case CONFKV_F32: e = launch_sample<float>(a, rows, st); break;
    case CONFKV_F16: e = launch_sample<__half>(a, rows, st); break;
    default: e = launch_sample<__nv_bfloat16>(a, rows, st); break;
  }
  if (e != cudaSuccess) (void)cudaGetLastError();   // not left for a later call
  return e == cudaSuccess ? CONFKV_OK : CONFKV_ERR_CUDA;
}

}  // extern "C"
