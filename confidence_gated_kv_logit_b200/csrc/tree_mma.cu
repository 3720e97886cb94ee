// Tree attention for many rows per KV head (nodes * G above a few dozen): both
// products on the fifth-generation tensor cores, accumulators in tensor memory.
// The definition and the numerics (codes widened exactly, scales in fp32, the
// weights in two fp16 parts) are those of tree_attn.cu.
//
// One CTA per SM takes 128 or 256 rows of a (sequence, KV head) over its part
// of the tokens, 128 INT8 tokens or 64 FP16 ones at a time:
//   warps 0-3, 4-7  two softmax groups, one thread per row. Each has its scores
//                   S (which its weights P then overwrite) and its output O in
//                   tensor memory. With more than 128 rows each group has rows
//                   of its own; otherwise they share the rows and take the tiles
//                   in turn, and their sums are merged at the end.
//   warps 8-11      converters: global memory -> registers -> fp16 operands in
//                   shared memory (128-byte swizzle), one tile ahead in
//                   registers. Codes are widened once for all rows of the CTA.
//                   The cache keeps V codes dimension-major, which is the K-major
//                   operand of the second product as it is; FP16 V rows are
//                   transposed 8 x 8 on the way.
//   warp 13         the tiles' scales and validity, one tile ahead
//   warp 12         issues the products: S = Q K^T (shared x shared), O += P V
//                   (P from tensor memory, its high and low parts against the same V).
// What bounds it, in cycles a tile of 128 tokens at head_dim 128:
//   * 256 rows (64 nodes x 4 heads over 32768 tokens x 4 sequences: 297 us, 463
//     TFLOP/s): the softmax, 1700 for the maximum and 3200 for the weights of either
//     group, then about 2100 until its next scores are there, against 3100 of tensor
//     work for both groups.
//   * 64 rows (16 nodes x 4 heads over 2048 tokens x 16 sequences: 59 us): the
//     converters, about 4300 of their own (a third of it waiting for the tile's V
//     codes), and the alternation of the groups. Two copies of the rows with half of the
//     tokens each, to halve the softmax, gained nothing there.
// Every wait is bounded.
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mma.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace confkv {

namespace {

constexpr int kThreads = 16 * 32;
// Registers a thread of the softmax groups, the converters and the rest, out of 128 at launch.
constexpr int kSoftRegs = 152, kConvRegs = 120, kRestRegs = 88;
static_assert(2 * kSoftRegs + kConvRegs + kRestRegs <= 4 * 128, "the shares fit in what the block was launched with");
constexpr int kAux = 4;            // tiles whose scales are kept

struct TileAux {
  float ksc[128];                  // K scale * log2(e) / sqrt(D)
  float vsr[128];                  // V scale * 2^-et of its 32 tokens
  int et[4];
  uint32_t live[4];                // tokens that are there
};

struct Bars {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], aux_full[kAux], aux_empty[kAux], s_full[2], p_full[2], o_done[2],
      drained;
};

template <int D>
struct MCfg {
  static constexpr int HALF = 128 * 128;              // 64 dimensions of 128 rows (K and Q operands)
  static constexpr int KB = (D / 64) * HALF;          // one K stage, or one Q tile
  static constexpr int VB = 2 * D * 128;              // one V stage: 128 tokens
  static constexpr int Q_OFF = 0, K_OFF = 2 * KB, V_OFF = K_OFF + 2 * KB, AUX_OFF = V_OFF + 2 * VB;
  static constexpr int BAR_OFF = AUX_OFF + kAux * (int)sizeof(TileAux);
  static constexpr int MISC_OFF = BAR_OFF + (int)sizeof(Bars);
  static constexpr int SMEM = MISC_OFF + 32;
  static constexpr int MROW = D + 4;                  // floats of a row of the merge area (over the K and V stages)
  static_assert(128 * MROW * 4 <= 2 * KB + 2 * VB, "the merge area fits in the operand stages");
};

// Wait for a phase; gives up when the CTA is aborting or after about two seconds.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > 4000000000ll) {
      *abort_flag = 1;
      return false;
    }
  }
}

__device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

__device__ __forceinline__ uint32_t transpose8x8(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

template <int D, bool CI8>
__global__ void __launch_bounds__(kThreads, 1) tree_mma_kernel(const Cache c, const TreeLaunch a) {
  using C = MCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Bars& bar = *reinterpret_cast<Bars*>(smem + C::BAR_OFF);
  TileAux* aux = reinterpret_cast<TileAux*>(smem + C::AUX_OFF);
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  int* odd_flag = reinterpret_cast<int*>(smem + C::MISC_OFF + 8);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 256);
    mbar_init(&bar.drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], 4);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], 4);
      mbar_init(&bar.v_empty[i], 1);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 128);
      mbar_init(&bar.o_done[i], 1);
    }
    for (int i = 0; i < kAux; ++i) {
      mbar_init(&bar.aux_full[i], 1);
      mbar_init(&bar.aux_empty[i], 1);
    }
    *abort_flag = (smem_addr(smem) & 1023u) != 0;   // the operand layouts need a 1 KB boundary
    *odd_flag = 0;
    fence_mbar_init();
  }
  chain_enter();

  // unit -> (item, row tile, split)
  const int split = blockIdx.x % a.splits;
  const int mt = (blockIdx.x / a.splits) % a.mtiles;
  const int item = blockIdx.x / (a.splits * a.mtiles);
  int l, b, h;
  const int s = seg_of(c, a.r, item, &l, &b, &h);
  const int seq = (l - a.r.l0) * a.r.B + b;
  int count = a.counts ? a.counts[b] : a.nodes;
  if (count < 0 || count > a.nodes) {
    if (threadIdx.x == 0) record_violation(c.err, kSiteTreeCount, s, count);
    count = 0;
  }
  const int R = count * c.G;
  const int row0 = mt * 256;
  if (row0 >= R) {   // nothing here; a sequence without nodes has no attention mass
    if (R == 0 && mt == 0 && split == 0 && a.track)
      for (int g = threadIdx.x; g < c.G; g += kThreads) a.lse_ws[(size_t)s * c.G + g] = CUDART_INF_F;
    return;
  }
  int n_cold = c.n_cold[s];
  if (n_cold < 0 || n_cold > c.cap) {
    if (threadIdx.x == 0) record_violation(c.err, kSiteTreeSeg, s, n_cold);
    n_cold = 0;
  }
  constexpr int TTC = CI8 ? 128 : 64;
  const int tiles_c = (n_cold + TTC - 1) / TTC;
  const int tiles = tiles_c + (c.W + 63) / 64 + 1;   // the last: the drafted rows
  const int t0 = (int)((long long)tiles * split / a.splits), t1 = (int)((long long)tiles * (split + 1) / a.splits);
  const int n = t1 - t0;
  const bool dual = R - row0 > 128;          // each softmax group has rows of its own
  const int jobs = dual ? 2 * n : n;         // job j: group j & 1, tile dual ? j / 2 : j

  if (warp == 12) tmem_alloc(tmem_ptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  const uint32_t sbase = smem_addr(smem);
  const float qs = rsqrtf((float)D) * kLog2e;

  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ------------------------------ converters ------------------------------
    const int cw = warp - 8;
    constexpr int NR = D / 16;
    uint4 rk[NR], rv[NR];
    // Where this lane's 16-byte pieces lie, in the cache (the permutations of
    // layout.cuh) and in the operands (the 128-byte swizzle). The pieces of one
    // lane differ by constants but for one bit of the permutation, so each needs
    // one of two offsets and an immediate.
    const int l7 = lane & 7, q8 = lane >> 3, d16 = lane & 15, c2 = lane >> 4, g = lane >> 2, t4 = lane & 3;
    const uint32_t x0 = (uint32_t)(q8 ^ l7) << 4, x1 = (uint32_t)((4 + q8) ^ l7) << 4;
    const uint32_t ksrc0 = D == 128 ? l7 * 128 + x0 : (l7 * 64 + q8 * 16) ^ ((l7 >> 1) << 4);
    const uint32_t ksrc1 = D == 128 ? l7 * 128 + x1 : (l7 * 64 + q8 * 16) ^ ((4 + (l7 >> 1)) << 4);
    const uint32_t kdst0 = cw * 4096 + l7 * 128 + (((2 * q8) ^ l7) << 4), kdst1 = kdst0 ^ 16;
    const uint32_t vsrc0 = (d16 * 32 + 16 * c2) ^ ((d16 >> 2) << 4), vsrc1 = vsrc0 ^ 64;
    const uint32_t vdst0 = (cw >> 1) * (D * 128) + d16 * 128 + ((((cw & 1) * 4 + c2 * 2) ^ (d16 & 7)) << 4);
    const uint32_t vdst1 = vdst0 ^ 16;
    // the tile's bytes into registers (K and V separately, so that each half is
    // fetched again as soon as it has been written out)
    auto fetch_k = [&](int t) {
      if (CI8 && t < tiles_c) {
        const int j0 = t * 128, cnt = min(128, n_cold - j0);
        const int8_t* src = c.k8 + ((size_t)s * c.cap + j0) * D + cw * (32 * D);
        if (cnt == 128) {
#pragma unroll
          for (int q = 0; q < NR; ++q)
            rk[q] = __ldcs(reinterpret_cast<const uint4*>(src + ((q & 1) ? ksrc1 : ksrc0) +
                                                          (D == 128 ? (q >> 1) * 1024 : q * 512)));
        } else {
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            const int tok = cw * 32 + (D == 128 ? q >> 1 : q) * 8 + l7;
            rk[q] = make_uint4(0, 0, 0, 0);
            if (tok < cnt)
              rk[q] = __ldcs(reinterpret_cast<const uint4*>(src + ((q & 1) ? ksrc1 : ksrc0) +
                                                            (D == 128 ? (q >> 1) * 1024 : q * 512)));
          }
        }
        return;
      }
      if (t == tiles - 1) {
        const __half* src = a.k + ((size_t)seq * a.nodes * c.Hkv + h) * D + q8 * 8;
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          const int tok = (cw * 2 + q / (D / 32)) * 8 + l7;
          rk[q] = make_uint4(0, 0, 0, 0);
          if (tok < count)
            rk[q] = *reinterpret_cast<const uint4*>(src + (size_t)tok * c.Hkv * D + q % (D / 32) * 32);
        }
        return;
      }
      const unsigned char* src;
      if (t < tiles_c) {
        src = reinterpret_cast<const unsigned char*>(c.kc + ((size_t)s * c.cap + t * 64) * D);
      } else {
        src = reinterpret_cast<const unsigned char*>(c.kr + ((size_t)s * c.Wst + (t - tiles_c) * 64) * D);
      }
      src += (cw * 16 + l7) * (2 * D);
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int qq = q % (D / 32);
        rk[q] = __ldcs(reinterpret_cast<const uint4*>(src + q / (D / 32) * (16 * D) + (qq >> 1) * 128 + ((qq & 1) ? x1 : x0)));
      }
    };
    auto fetch_v = [&](int t) {
      if (CI8 && t < tiles_c) {
        const int j0 = t * 128, cnt = min(128, n_cold - j0);
        const int8_t* src = c.v8 + ((size_t)s * c.cap + j0) * D + cw * (32 * D);
        if (32 * cw < cnt) {
#pragma unroll
          for (int q = 0; q < NR; ++q)
            rv[q] = __ldcs(reinterpret_cast<const uint4*>(src + ((q & 1) ? vsrc1 : vsrc0) + q * 512));
        } else {
#pragma unroll
          for (int q = 0; q < NR; ++q) rv[q] = make_uint4(0, 0, 0, 0);
        }
        return;
      }
      uint32_t* w = reinterpret_cast<uint32_t*>(rv);
      if (t == tiles - 1) {
        const __half* src = a.v + ((size_t)seq * a.nodes * c.Hkv + h) * D + t4 * 2;
#pragma unroll
        for (int q = 0; q < 4 * NR; ++q) {
          const int tok = (cw * 2 + q / (D / 8)) * 8 + g;
          w[q] = 0u;
          if (tok < count)
            w[q] = *reinterpret_cast<const uint32_t*>(src + (size_t)tok * c.Hkv * D + q % (D / 8) * 8);
        }
        return;
      }
      const unsigned char* src =
          t < tiles_c ? reinterpret_cast<const unsigned char*>(c.vc + ((size_t)s * c.cap + t * 64) * D)
                      : reinterpret_cast<const unsigned char*>(c.vr + ((size_t)s * c.Wst + (t - tiles_c) * 64) * D);
      src += (cw * 16 + g) * (2 * D) + 4 * t4;
#pragma unroll
      for (int q = 0; q < 4 * NR; ++q) {
        const int dg = q % (D / 8);
        w[q] = *reinterpret_cast<const uint32_t*>(src + q / (D / 8) * (16 * D) + (dg >> 3) * 128 + ((g ^ (dg & 7)) << 4));
      }
    };
    bool ok = true;
    if (n > 0) {
      fetch_k(t0);
      fetch_v(t0);
    }
    for (int i = 0; i < n && ok; ++i) {
      const int t = t0 + i, st = i & 1, use = i >> 1;
      const bool i8 = CI8 && t < tiles_c;
      // FP16 tiles: which tokens are there
      unsigned long long there = 0;
      if (!i8) {
        ok = __all_sync(0xffffffffu, wait_phase(&bar.aux_full[i % kAux], (i / kAux) & 1, abort_flag));
        if (!ok) break;
        there = aux[i % kAux].live[0] | ((unsigned long long)aux[i % kAux].live[1] << 32);
      }
      // ---- K operand ----
      if (use > 0) ok = __all_sync(0xffffffffu, wait_phase(&bar.k_empty[st], (use - 1) & 1, abort_flag));
      if (!ok) break;
      {
        unsigned char* dst = smem + C::K_OFF + st * C::KB;
        if (i8) {
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            unsigned char* row = dst + (D == 128 ? (q & 1) * C::HALF + (q >> 1) * 1024 : q * 1024);
            uint4 lo, hi;
            cvt_codes(rk[q].x, lo.x, lo.y);
            cvt_codes(rk[q].y, lo.z, lo.w);
            cvt_codes(rk[q].z, hi.x, hi.y);
            cvt_codes(rk[q].w, hi.z, hi.w);
            *reinterpret_cast<uint4*>(row + kdst0) = lo;
            *reinterpret_cast<uint4*>(row + kdst1) = hi;
          }
        } else {
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            const int gg = q / (D / 32), qq = q % (D / 32);
            const int tok = (cw * 2 + gg) * 8 + l7;
            *reinterpret_cast<uint4*>(dst + (qq >> 1) * C::HALF + tok * 128 + ((qq & 1) ? x1 : x0)) =
                ((there >> tok) & 1ull) ? rk[q] : make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.k_full[st]);
      }
      if (i + 1 < n) fetch_k(t + 1);
      // ---- V operand ----
      if (use > 0) ok = __all_sync(0xffffffffu, wait_phase(&bar.v_empty[st], (use - 1) & 1, abort_flag));
      if (!ok) break;
      {
        unsigned char* dst = smem + C::V_OFF + st * C::VB;
        if (i8) {
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            uint4 lo, hi;
            cvt_codes(rv[q].x, lo.x, lo.y);
            cvt_codes(rv[q].y, lo.z, lo.w);
            cvt_codes(rv[q].z, hi.x, hi.y);
            cvt_codes(rv[q].w, hi.z, hi.w);
            *reinterpret_cast<uint4*>(dst + vdst0 + q * 2048) = lo;
            *reinterpret_cast<uint4*>(dst + vdst1 + q * 2048) = hi;
          }
        } else {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(rv);
          bool odd = false;
#pragma unroll
          for (int q = 0; q < 4 * NR; ++q) {
            const int tg = cw * 2 + q / (D / 8), dg = q % (D / 8);
            uint32_t v = ((there >> (tg * 8 + g)) & 1ull) ? w[q] : 0u;
            if (t == tiles - 1) {   // values of a node that are not finite must not reach the rows that do not see it
              const uint32_t f = finite_mask(v);
              odd |= f != 0xffffffffu;
              v &= f;
            }
            *reinterpret_cast<uint32_t*>(dst + dg * 1024 + g * 128 + ((tg ^ g) << 4) + 4 * t4) = transpose8x8(v);
          }
          if (odd) *odd_flag = 1;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_full[st]);
      }
      if (i + 1 < n) fetch_v(t + 1);
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    // ------------------------------ products ------------------------------
    if (warp == 12 && n > 0) {
      const uint32_t leader = elect_lane();
      bool ok = true;
      auto wait = [&](uint64_t* p, uint32_t parity) {
        ok = __all_sync(0xffffffffu, ok && wait_phase(p, parity, abort_flag));
      };
      wait(&bar.q_full, 0);
      // descriptors advance by 16 bytes a unit; the operands lie below 256 KB
      const uint64_t dq = sw128_desc(sbase + C::Q_OFF), dk = sw128_desc(sbase + C::K_OFF), dv = sw128_desc(sbase + C::V_OFF);
      auto i8_tile = [&](int i) { return CI8 && t0 + i < tiles_c; };
      auto scores = [&](int j) {
        const int w = j & 1, i = dual ? j >> 1 : j, st = i & 1;
        if (!dual || w == 0) wait(&bar.k_full[st], (i >> 1) & 1);
        // the previous weights of this group's buffer have been read
        if (j >= 2) wait(&bar.o_done[w], ((j >> 1) - 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t q = dq + (dual ? w : 0) * (C::KB >> 4), k = dk + st * (C::KB >> 4);
        const uint32_t idesc = i8_tile(i) ? f16_idesc(128) : f16_idesc(64);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * C::HALF + (ks & 3) * 32) >> 4;
          tc_mma_ss(tmem + w * 128, q + off, k + off, idesc, ks > 0, leader);
        }
        tc_commit(&bar.s_full[w], leader);
        if (!dual || w == 1) tc_commit(&bar.k_empty[st], leader);
      };
      auto output = [&](int j) {
        const int w = j & 1, i = dual ? j >> 1 : j, st = i & 1;
        if (!dual || w == 0) wait(&bar.v_full[st], (i >> 1) & 1);
        wait(&bar.p_full[w], (j >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t v = dv + st * (C::VB >> 4);
        constexpr uint32_t idesc = f16_idesc(D);
        auto steps = [&](auto lo, auto hi) {
#pragma unroll
          for (int ks = decltype(lo)::value; ks < decltype(hi)::value; ++ks) {
            const uint64_t vd = v + (((ks >> 2) * (D * 128) + (ks & 3) * 32) >> 4);
            const uint32_t p = tmem + w * 128 + (ks >> 1) * 32 + (ks & 1) * 8;   // high parts; the low ones 16 columns on
            tc_mma_ts(tmem + 256 + w * 128, p, vd, idesc, j >= 2 || ks > 0, leader);
            tc_mma_ts(tmem + 256 + w * 128, p + 16, vd, idesc, 1, leader);
          }
        };
        steps(std::integral_constant<int, 0>(), std::integral_constant<int, 4>());
        if (i8_tile(i)) steps(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
        tc_commit(&bar.o_done[w], leader);
        if (!dual || w == 1) {
          tc_commit(&bar.v_empty[st], leader);
          tc_commit(&bar.aux_empty[i % kAux], leader);
        }
      };
      if (ok) scores(0);
      if (ok && jobs > 1) scores(1);
      for (int j = 0; j < jobs && ok; ++j) {
        output(j);
        if (ok && j + 2 < jobs) scores(j + 2);
      }
      // on an abort too, nothing of this lane's may be in flight when the CTA ends
      if (!ok) {
        *abort_flag = 1;
        tc_commit(&bar.drained, leader);
        (void)mbar_wait_bounded(&bar.drained, 0);
      }
    }
    // ------------------------------ scales ------------------------------
    if (warp == 13) {
      bool ok = true;
      // lane l: tokens 4 l .. 4 l + 3 of an INT8 tile; fetched one tile ahead
      float4 ks4 = make_float4(0, 0, 0, 0), vs4 = ks4;
      int pos0 = 0, pos1 = 0;
      auto fetch = [&](int t) {
        if (CI8 && t < tiles_c) {   // cap is a multiple of 64, and scales past n_cold are not used
          const int j = t * 128 + 4 * lane;
          if (j < n_cold) {
            ks4 = *reinterpret_cast<const float4*>(c.ks + (size_t)s * c.cap + j);
            vs4 = *reinterpret_cast<const float4*>(c.vs + (size_t)s * c.cap + j);
          }
        } else if (t >= tiles_c && t < tiles - 1) {
          const int j = (t - tiles_c) * 64 + lane;
          const int32_t* pos = c.pos_r + (size_t)s * c.Wst;
          pos0 = pos[j];
          pos1 = pos[j + 32];
        }
      };
      if (n > 0) fetch(t0);
      for (int i = 0; i < n && ok; ++i) {
        const int t = t0 + i;
        if (i >= kAux) ok = __all_sync(0xffffffffu, wait_phase(&bar.aux_empty[i % kAux], (i / kAux - 1) & 1, abort_flag));
        if (!ok) break;
        TileAux& x = aux[i % kAux];
        if (CI8 && t < tiles_c) {
          const int j = t * 128 + 4 * lane;
          float v[4] = {vs4.x, vs4.y, vs4.z, vs4.w}, u[4] = {ks4.x, ks4.y, ks4.z, ks4.w};
          uint32_t bits = 0, top = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool in = j + k < n_cold;
            v[k] = in ? v[k] : 0.0f;
            u[k] = in ? u[k] * qs : 1.0f;   // (above 0: it meets a score of -inf)
            bits |= (uint32_t)in << k;
            top = max(top, __float_as_uint(v[k]));
          }
          // the 32 tokens of a group are eight lanes
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          bits <<= 4 * (lane & 7);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
          const int et = scale_exp(top);
          const float f = pow2i(-et);
          *reinterpret_cast<float4*>(&x.ksc[4 * lane]) = make_float4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<float4*>(&x.vsr[4 * lane]) = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
          if ((lane & 7) == 0) {
            x.et[lane >> 3] = et;
            x.live[lane >> 3] = bits;
          }
        } else {
          bool in0, in1;
          if (t >= tiles_c && t < tiles - 1) {
            const int j = (t - tiles_c) * 64 + lane;
            in0 = j < c.W && pos0 >= 0;
            in1 = j + 32 < c.W && pos1 >= 0;
          } else {
            const int cnt = t == tiles - 1 ? count : min(64, n_cold - t * 64);
            in0 = lane < cnt;
            in1 = lane + 32 < cnt;
          }
          const uint32_t w0 = __ballot_sync(0xffffffffu, in0), w1 = __ballot_sync(0xffffffffu, in1);
          x.ksc[lane] = x.ksc[lane + 32] = qs;
          x.vsr[lane] = in0 ? 0.5f : 0.0f;      // 1 * 2^-et
          x.vsr[lane + 32] = in1 ? 0.5f : 0.0f;
          if (lane == 0) {
            x.et[0] = x.et[1] = x.et[2] = x.et[3] = 1;
            x.live[0] = w0;
            x.live[1] = w1;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.aux_full[i % kAux]);
        if (i + 1 < n) fetch(t + 1);
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------ softmax ------------------------------
    const int w = warp >> 2;                         // group
    const int rr = threadIdx.x & 127;                // row within its tile of 128
    const int r = row0 + (dual ? w * 128 : 0) + rr;  // row of the KV head
    const bool in = r < R;
    const int node = in ? r / c.G : 0, gg = in ? r % c.G : 0;
    // ---- Q operand: rows of zeros past the last ----
    {
      const int tile = dual ? w : 0, part = dual ? 0 : w;   // sharing groups load half the dimensions each
      const __half* q = a.q + (((size_t)seq * a.nodes + node) * c.Hq + h * c.G + gg) * D;
      unsigned char* dst = smem + C::Q_OFF + tile * C::KB + rr * 128;
      constexpr int CH = D / 8;
      const int c0 = dual ? 0 : part * (CH / 2), c1 = dual ? CH : c0 + CH / 2;
      for (int ch = c0; ch < c1; ++ch) {
        const uint4 v = in ? *reinterpret_cast<const uint4*>(q + ch * 8) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dst + (ch >> 3) * C::HALF + (((ch & 7) ^ (rr & 7)) << 4)) = v;
      }
      fence_proxy_async_shared();
      mbar_arrive(&bar.q_full);
    }
    unsigned long long sees = in ? a.mask[(size_t)b * a.nodes + node] : 0ull;
    if (count < 64) sees &= (1ull << count) - 1ull;
    const bool busy = row0 + (dual ? w * 128 : 0) + (warp & 3) * 32 < R;   // the warp has rows
    const bool track = a.track && r < c.G;
    float* sc = a.scores + ((size_t)s * c.G + (r < c.G ? r : 0)) * a.score_stride;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + w * 128, tO = tmem + lanes + 256 + w * 128;
    float m = -CUDART_INF_F, lsum = 0.0f;
    int E = -100;
    bool ok = true;
    for (int j = w; j < jobs && ok; j += 2) {
      const int i = dual ? j >> 1 : j, t = t0 + i, use = j >> 1;
      ok = __all_sync(0xffffffffu, wait_phase(&bar.aux_full[i % kAux], (i / kAux) & 1, abort_flag) &&
                                       wait_phase(&bar.s_full[w], use & 1, abort_flag));
      if (!ok) break;
      __syncwarp();
      tc_fence_after();
      const TileAux& x = aux[i % kAux];
      const bool i8 = CI8 && t < tiles_c, draft = t == tiles - 1;
      const int chunks = i8 ? 4 : 2;
      if (busy) {
        // ---- maximum ----
        float rm = -CUDART_INF_F, rm2 = -CUDART_INF_F;
        int et = -100;
#pragma unroll 1
        for (int ch = 0; ch < chunks; ch += 2) {
          uint32_t sv[2][32];
          tmem_ld32(tS + ch * 32, sv[0]);
          tmem_ld32(tS + ch * 32 + 32, sv[1]);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c32 = ch + e;
            const uint32_t live = x.live[c32] & (draft ? (uint32_t)(sees >> (32 * c32)) : 0xffffffffu);
            et = max(et, x.et[c32]);
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 ks = *reinterpret_cast<const float4*>(&x.ksc[c32 * 32 + k]);
              const float2 u = __fmul2_rn(pair(sv[e][k], sv[e][k + 1]), make_float2(ks.x, ks.y));
              const float2 v = __fmul2_rn(pair(sv[e][k + 2], sv[e][k + 3]), make_float2(ks.z, ks.w));
              sv[e][k] = __float_as_uint(u.x);
              sv[e][k + 1] = __float_as_uint(u.y);
              sv[e][k + 2] = __float_as_uint(v.x);
              sv[e][k + 3] = __float_as_uint(v.y);
            }
            if (live != 0xffffffffu) {
#pragma unroll
              for (int k = 0; k < 32; ++k) sv[e][k] = (live >> k) & 1u ? sv[e][k] : 0xff800000u;
            }
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              rm = fmaxf(rm, fmaxf(__uint_as_float(sv[e][k]), __uint_as_float(sv[e][k + 1])));
              rm2 = fmaxf(rm2, fmaxf(__uint_as_float(sv[e][k + 2]), __uint_as_float(sv[e][k + 3])));
            }
            if (track && !draft) {
              // the root's scaled scores (log2 units), for the attention-mass EMA
              float* dst = sc + (t < tiles_c ? t * TTC : c.cap + (t - tiles_c) * 64) + c32 * 32;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if ((live >> k) & 1u) dst[k] = __uint_as_float(sv[e][k]);
            }
          }
          __syncwarp();   // the next loads take the whole warp
        }
        rm = fmaxf(rm, rm2);
        // ---- move the reference, and with it this row's sums ----
        if (use == 0) {
          m = rm;
          E = et;
        } else {
          const bool move = rm > m + kSlack;
          if (__any_sync(0xffffffffu, move || et > E)) {
            const int En = max(E, et);
            const float mn = move ? rm : m;
            const float fl = m == -CUDART_INF_F ? 0.0f : ex2(m - mn);
            const float f = fl * pow2i(E - En);
            m = mn;
            E = En;
            lsum *= fl;
            for (int ch = 0; ch < D / 32; ++ch) {
              uint32_t ov[32];
              tmem_ld32(tO + ch * 32, ov);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
              tmem_st32(tO + ch * 32, ov);
            }
          }
        }
        // ---- weights, over the scores ----
        const float m0 = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll 1
        for (int ch = 0; ch < chunks; ++ch) {
          const uint32_t live = x.live[ch] & (draft ? (uint32_t)(sees >> (32 * ch)) : 0xffffffffu);
          // Weights carry 2^dE. Where the V scales are so small against the largest that
          // every weight would vanish in fp16, the sum goes without the factor.
          const bool tiny = x.et[ch] - E + kPBits < -33;
          const int dE = tiny ? 0 : x.et[ch] - E + kPBits;
          const float2 off = make_float2((float)dE - m0, (float)dE - m0);
          uint32_t sv[32], pv[32];
          tmem_ld32(tS + ch * 32, sv);
          tc_wait_ld();
          if (__any_sync(0xffffffffu, live != 0xffffffffu)) {
            // a score of -inf in place of what is not there (its scale is above 0)
#pragma unroll
            for (int k = 0; k < 32; ++k) sv[k] = (live >> k) & 1u ? sv[k] : 0xff800000u;
          }
          float2 ls0 = make_float2(0.0f, 0.0f), ls1 = ls0;
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 ks = *reinterpret_cast<const float4*>(&x.ksc[ch * 32 + k]);
            const float4 vs = *reinterpret_cast<const float4*>(&x.vsr[ch * 32 + k]);
            const float2 u = __ffma2_rn(pair(sv[k], sv[k + 1]), make_float2(ks.x, ks.y), off);
            const float2 v = __ffma2_rn(pair(sv[k + 2], sv[k + 3]), make_float2(ks.z, ks.w), off);
            float2 p = make_float2(ex2(u.x), ex2(u.y)), q = make_float2(ex2(v.x), ex2(v.y));
            ls0 = __fadd2_rn(ls0, p);
            ls1 = __fadd2_rn(ls1, q);
            p = __fmul2_rn(p, make_float2(vs.x, vs.y));
            q = __fmul2_rn(q, make_float2(vs.z, vs.w));
            // high part: the mantissa cut to fp16's ten bits (exact in fp16 from 2^-14 up; below, fp16's smallest
            // step bounds both parts); low part: what that leaves
            const float2 ph = pair(__float_as_uint(p.x) & 0xffffe000u, __float_as_uint(p.y) & 0xffffe000u);
            const float2 qh = pair(__float_as_uint(q.x) & 0xffffe000u, __float_as_uint(q.y) & 0xffffe000u);
            const float2 pl = __fadd2_rn(p, make_float2(-ph.x, -ph.y)), ql = __fadd2_rn(q, make_float2(-qh.x, -qh.y));
            pv[k / 2] = pack_h2(ph.x, ph.y);
            pv[k / 2 + 1] = pack_h2(qh.x, qh.y);
            pv[16 + k / 2] = pack_h2(pl.x, pl.y);
            pv[16 + k / 2 + 1] = pack_h2(ql.x, ql.y);
          }
          lsum = fmaf((ls0.x + ls0.y) + (ls1.x + ls1.y), pow2i(-dE), lsum);
          if (tiny) {
#pragma unroll
            for (int k = 0; k < 32; ++k) pv[k] = 0u;
          }
          __syncwarp();
          tmem_st32(tS + ch * 32, pv);
        }
        tc_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&bar.p_full[w]);
    }

    // ---- this group's sums are complete; merge the groups that share rows ----
    const int mine = jobs > w ? (jobs - w + 1) / 2 : 0;   // jobs of this group
    if (ok && mine > 0) ok = __all_sync(0xffffffffu, wait_phase(&bar.o_done[w], (mine - 1) & 1, abort_flag));
    tc_fence_after();
    const float fo = pow2i(E - kPBits);
    float* area = reinterpret_cast<float*>(smem + C::K_OFF) + rr * C::MROW;
    float f0 = 1.0f, f1 = 0.0f;
    bool fine = ok;
    if (!dual) {
      // both groups are past their last product: the operand stages are free
      fine = !named_barrier_or(2, 256, !ok);
      if (w == 1 && fine && busy) {
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t ov[32];
          if (mine > 0) {
            tmem_ld32(tO + ch * 32, ov);
            tc_wait_ld();
          }
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float4 v = make_float4(0, 0, 0, 0);
            if (mine > 0)
              v = make_float4(__uint_as_float(ov[k]) * fo, __uint_as_float(ov[k + 1]) * fo, __uint_as_float(ov[k + 2]) * fo,
                              __uint_as_float(ov[k + 3]) * fo);
            *reinterpret_cast<float4*>(area + ch * 32 + k) = v;
          }
        }
        area[D] = m;
        area[D + 1] = lsum;
      }
      named_barrier_sync(2, 256);
      if (w == 0 && fine && busy) {
        const float m1 = area[D], mn = fmaxf(m, m1);
        f0 = m == -CUDART_INF_F ? 0.0f : ex2(m - mn);
        f1 = m1 == -CUDART_INF_F ? 0.0f : ex2(m1 - mn);
        lsum = lsum * f0 + area[D + 1] * f1;
        m = mn;
      }
    }
    if (fine && busy && (dual || w == 0)) {
      const size_t orow = ((size_t)seq * a.nodes + node) * c.Hq + h * c.G + gg;
      // a row that sees nothing: zeros, and a log-sum-exp of -inf
      const float inv = a.splits > 1 ? 1.0f : lsum == 0.0f ? 0.0f : 1.0f / lsum;
      float* pp = a.part + ((size_t)(item * a.splits + split) * a.nodes * c.G + (in ? r : 0)) * (D + 2);
      const bool odd = *odd_flag && t1 == tiles;
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t ov[32];
        float o[32];
        if (mine > 0) {
          tmem_ld32(tO + ch * 32, ov);
          tc_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          o[k] = mine > 0 ? __uint_as_float(ov[k]) * (fo * f0) : 0.0f;
          if (!dual) o[k] = fmaf(area[ch * 32 + k], f1, o[k]);
        }
        if (odd) {   // values that are not finite reach only the rows that see their node (rare)
          for (int jn = 0; jn < count; ++jn) {
            if (!((sees >> jn) & 1ull)) continue;
            const __half* vrow = a.v + (((size_t)seq * a.nodes + jn) * c.Hkv + h) * D + ch * 32;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float v = __half2float(vrow[k]);
              if (!(fabsf(v) < CUDART_INF_F)) o[k] += v;
            }
          }
        }
        if (in && a.splits > 1) {
#pragma unroll
          for (int k = 0; k < 32; k += 2) *reinterpret_cast<float2*>(pp + ch * 32 + k) = make_float2(o[k], o[k + 1]);
        } else if (in) {
#pragma unroll
          for (int k = 0; k < 32; k += 8)
            *reinterpret_cast<uint4*>(a.out + orow * D + ch * 32 + k) =
                make_uint4(pack_h2(o[k] * inv, o[k + 1] * inv), pack_h2(o[k + 2] * inv, o[k + 3] * inv),
                           pack_h2(o[k + 4] * inv, o[k + 5] * inv), pack_h2(o[k + 6] * inv, o[k + 7] * inv));
        }
        __syncwarp();
      }
      if (in && a.splits > 1) {
        pp[D] = m;
        pp[D + 1] = lsum;
      } else if (in) {
        const float lse = (m + log2f(lsum)) * kLn2;
        if (a.lse_out) a.lse_out[orow] = lse;
        if (a.track && node == 0) a.lse_ws[(size_t)s * c.G + gg] = lse;
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) set_error(c.err, kErrDevice);
  if (warp == 12) {
    tc_fence_after();
    tmem_free(tmem);
  }
}

template <int D, bool CI8>
cudaError_t run(const Cache& c, const TreeLaunch& a, unsigned grid, cudaStream_t st) {
  using C = MCfg<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(tree_mma_kernel<D, CI8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_chained(tree_mma_kernel<D, CI8>, grid, kThreads, C::SMEM, st, c, a);
}

}  // namespace

cudaError_t launch_tree_mma(const Cache& c, const TreeLaunch& a, unsigned grid, cudaStream_t st) {
  if (c.D == 128) return c.cold_int8 ? run<128, true>(c, a, grid, st) : run<128, false>(c, a, grid, st);
  return c.cold_int8 ? run<64, true>(c, a, grid, st) : run<64, false>(c, a, grid, st);
}

}  // namespace confkv
