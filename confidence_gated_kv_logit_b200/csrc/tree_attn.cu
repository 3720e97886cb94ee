// Attention of several drafted tokens per sequence (the nodes of a tree) over
// the mixed FP16/INT8 cache and over one another, and the append of the nodes
// that were accepted.
//
//   row r = node * G + g of a (sequence, KV head):
//   s_j   = q_r . k_j / sqrt(D)   for every cached token j and every node j of
//           the row's mask; k_j, v_j: the stored rows (INT8 code * scale, or FP16)
//   out_r = sum_j e^(s_j - max s) v_j / sum_j e^(s_j - max s)
//
// Decode attention has G rows per KV head and is bound by HBM; a tree has
// nodes * G, up to 512, and both products become real GEMMs with K and V read
// once for all rows. They run on the f16 tensor cores:
//   * this kernel takes up to 32 rows per KV head: a warp holds the fp32 output
//     of 16, and four warps split each tile's tokens. More rows go to the kernel
//     of tree_mma.cu, whose tiles are 128 rows high.
//   * INT8 codes are widened to fp16 in registers (exact), straight from the
//     shared-memory tile; scores get the K scale in fp32, probabilities the V
//     scale, so the codes themselves are never rounded.
//   * P = p * vs is split into two fp16 parts (22 bits, down to fp16's smallest
//     step), relative to a power of two near the largest V scale and to a running
//     maximum that is moved only when a score passes it by 2^8. One part alone would
//     add an error as large as the output's own rounding to fp16, and more where a
//     few keys dominate.
// The token order within a tile is permuted so that one 32-bit word of V codes
// (four tokens of one dimension) is the B operand of a k-step as it lies: column
// c of the score block 2j + e holds token 16 j + 4 (c / 2) + 2 e + (c % 2).
// A producer warp streams the tiles through a shared-memory ring with 1-D bulk
// copies; every wait is bounded.
#include <math_constants.h>

#include <algorithm>

#include "append.cuh"
#include "common.cuh"
#include "kernels.h"
#include "mma.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace confkv {

namespace {

constexpr int kMaxWarps = 8;       // consumer warps
// Rows per KV head of this kernel; more go to the one of tree_mma.cu. Cold, for 32/8
// heads of 128, this kernel against that one: 8 rows over 16384 tokens x 2 sequences
// 48 and 60 us, over 2048 x 16 56 and 63, over 512 x 16 36 and 33; 32 rows 63 and 65,
// 67 and 65, 39 and 35.
constexpr int kMaxRows = 32;

template <int D, bool CI8>
struct TCfg {
  static constexpr int TTC = CI8 ? 128 : 64;    // tokens per cold tile
  static constexpr int KVB = 128 * D;           // bytes of K (and of V) per stage
  static constexpr int STAGE = 2 * KVB + 1024;  // + scales (K, V), or positions
  static constexpr int NSTAGE = D == 128 ? 3 : 4;
  static constexpr int MROW = D + 4;            // floats of one row of the merge area
  static constexpr int RING = NSTAGE * STAGE;
  static constexpr int MERGE = (kMaxWarps - 1) * 16 * MROW * 4;   // at most, reused from the ring
  static constexpr int BAR_OFF = RING > MERGE ? RING : MERGE;
  static constexpr int Q_OFF = (BAR_OFF + 2 * NSTAGE * 8 + 16 + 15) / 16 * 16;
  static constexpr int QROW = 2 * D + 16;       // bytes of a query row (the pad spreads eight rows over the banks)
  static constexpr int SMEM = Q_OFF + kMaxRows * QROW;
};

template <int D>
struct RowState {
  float m[2], l[2];      // rows g and g + 8; m the same in the four lanes of a row, l this lane's share
  float o[D / 8][4];     // times 2^(kPBits - E)
  int E;
};

// Scores s of 32 tokens of one warp become probabilities. valid(k): whether
// this lane's token k (of 8: 4 of each 16-token group) counts for row i.
// vsr[k]: V scale of token k, 0 for tokens that count for no row; Et: exponent of the largest.
template <int D, class Valid>
__device__ __forceinline__ void softmax32(RowState<D>& st, float (&s)[4][4], const float (&ksc)[8], const float (&vs)[8],
                                          int Et, Valid valid, uint32_t (&pa)[2][4], uint32_t (&pb)[2][4]) {
  float rm[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float& v = s[2 * j + e][2 * i + x];
          const int k = 4 * j + 2 * e + x;
          v = valid(i, k) ? v * ksc[k] : -CUDART_INF_F;
          rm[i] = fmaxf(rm[i], v);
        }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    rm[i] = fmaxf(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], 1));
    rm[i] = fmaxf(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], 2));
  }
  const bool move = rm[0] > st.m[0] + kSlack || rm[1] > st.m[1] + kSlack || Et > st.E;
  if (__any_sync(0xffffffffu, move)) {
    const int E = max(st.E, Et);
    const float fe = pow2i(st.E - E);
    st.E = E;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // a maximum of -inf (nothing seen yet) has l and o zero: any factor will do
      const float mn = fmaxf(st.m[i], rm[i]);
      const float f = st.m[i] == -CUDART_INF_F ? 0.0f : ex2(st.m[i] - mn);
      st.m[i] = mn;
      st.l[i] *= f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        st.o[n][2 * i] *= f * fe;
        st.o[n][2 * i + 1] *= f * fe;
      }
    }
  }
  const float scale = pow2i(kPBits - st.E);
  float vsr[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) vsr[k] = vs[k] * scale;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float m = st.m[i] == -CUDART_INF_F ? 0.0f : st.m[i];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p0 = ex2(s[2 * j + e][2 * i] - m), p1 = ex2(s[2 * j + e][2 * i + 1] - m);
        st.l[i] += p0 + p1;
        const float q0 = p0 * vsr[4 * j + 2 * e], q1 = p1 * vsr[4 * j + 2 * e + 1];
        const uint32_t hi = pack_h2(q0, q1);
        const float2 f = h2_to_f2(hi);
        pa[j][2 * e + i] = hi;
        pb[j][2 * e + i] = pack_h2(q0 - f.x, q1 - f.y);
      }
  }
}

template <int D, bool CI8>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1), 1) tree_kernel(const Cache c, const TreeLaunch a) {
  using C = TCfg<D, CI8>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::NSTAGE;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::NSTAGE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ncw = a.wm * a.wn;     // consumer warps; warp ncw produces
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NSTAGE; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], ncw);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  chain_enter();
  __syncthreads();

  // unit -> (item, split)
  const int split = blockIdx.x % a.splits;
  const int item = blockIdx.x / a.splits;
  int l, b, h;
  const int s = seg_of(c, a.r, item, &l, &b, &h);
  const int seq = (l - a.r.l0) * a.r.B + b;
  int count = a.counts ? a.counts[b] : a.nodes;
  if (count < 0 || count > a.nodes) {
    if (threadIdx.x == 0) record_violation(c.err, kSiteTreeCount, s, count);
    count = 0;
  }
  const int R = count * c.G;                 // rows of this sequence and KV head
  if (R == 0) {                              // a sequence without nodes has no attention mass
    if (split == 0 && a.track)
      for (int g = threadIdx.x; g < c.G; g += blockDim.x) a.lse_ws[(size_t)s * c.G + g] = CUDART_INF_F;
    return;
  }
  int n_cold = c.n_cold[s];
  if (n_cold < 0 || n_cold > c.cap) {
    if (threadIdx.x == 0) record_violation(c.err, kSiteTreeSeg, s, n_cold);
    n_cold = 0;
  }
  const int tiles_c = (n_cold + C::TTC - 1) / C::TTC;
  const int tiles_r = (c.W + 63) / 64;
  const int tiles = tiles_c + tiles_r + 1;   // the last: the drafted rows
  const int t0 = (int)((long long)tiles * split / a.splits), t1 = (int)((long long)tiles * (split + 1) / a.splits);

  if (warp == ncw) {
    // ------------------------------ producer ------------------------------
    int issued = 0;
    for (int t = t0; t < t1; ++t, ++issued) {
      const int sg = issued % C::NSTAGE;
      unsigned char* sb = smem + sg * C::STAGE;
      if (issued >= C::NSTAGE) {
        const bool ok = mbar_wait_bounded(&empty[sg], (issued / C::NSTAGE - 1) & 1);
        if (!__all_sync(0xffffffffu, ok) || *abort_flag) {
          if (lane == 0) {
            set_error(c.err, kErrDevice);
            *abort_flag = 1;
          }
          break;
        }
      }
      if (t == tiles - 1) {
        // drafted rows: FP16, [node][kv head][D], placed as window rows are; rows past the count are zeros
        const size_t base = (size_t)seq * a.nodes * c.Hkv * D;
        constexpr int CH = D / 8;              // 16-byte pieces of a row
        for (int i = lane; i < 64 * CH; i += 32) {
          const int j = i / CH, d8 = i % CH;
          const bool in = j < count;
          const size_t off = base + ((size_t)(in ? j : 0) * c.Hkv + h) * D + d8 * 8;
          const uint32_t dst = smem_addr(sb) + (uint32_t)h_off(j, d8 * 16, D);
          const int n = in ? 16 : 0;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(a.k + off), "r"(n) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + C::KVB), "l"(a.v + off), "r"(n)
                       : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[sg]);
      } else if (lane == 0) {
        if (CI8 && t < tiles_c) {
          const int j0 = t * C::TTC, cnt = min(C::TTC, n_cold - j0);
          const uint32_t rows = (uint32_t)((cnt + 31) & ~31);   // whole 32-token blocks (cap is a multiple of 64)
          mbar_arrive_expect_tx(&full[sg], rows * (2 * D + 8));
          const size_t g0 = (size_t)s * c.cap + j0;
          bulk_g2s(sb, c.k8 + g0 * D, rows * D, &full[sg]);
          bulk_g2s(sb + C::KVB, c.v8 + g0 * D, rows * D, &full[sg]);
          bulk_g2s(sb + 2 * C::KVB, c.ks + g0, rows * 4, &full[sg]);
          bulk_g2s(sb + 2 * C::KVB + 512, c.vs + g0, rows * 4, &full[sg]);
        } else if (!CI8 && t < tiles_c) {
          const size_t g0 = (size_t)s * c.cap + t * C::TTC;
          mbar_arrive_expect_tx(&full[sg], 2 * C::KVB);
          bulk_g2s(sb, c.kc + g0 * D, C::KVB, &full[sg]);
          bulk_g2s(sb + C::KVB, c.vc + g0 * D, C::KVB, &full[sg]);
        } else {
          const size_t g0 = (size_t)s * c.Wst + (t - tiles_c) * 64;
          mbar_arrive_expect_tx(&full[sg], 2 * C::KVB + 256);
          bulk_g2s(sb, c.kr + g0 * D, C::KVB, &full[sg]);
          bulk_g2s(sb + C::KVB, c.vr + g0 * D, C::KVB, &full[sg]);
          bulk_g2s(sb + 2 * C::KVB, c.pos_r + g0, 256, &full[sg]);
        }
      }
      __syncwarp();
    }
    // nothing of this CTA may still be in flight when its last warp leaves
    for (int k = max(0, issued - C::NSTAGE); k < issued; ++k)
      (void)mbar_wait_bounded(&full[k % C::NSTAGE], (k / C::NSTAGE) & 1, 1000000000ll);
    return;
  }

  // -------------------------------- consumers --------------------------------
  const int g = lane >> 2, t4 = lane & 3;
  const int wm = warp % a.wm, wn = warp / a.wm;
  const int r0 = 16 * wm + g;                // this lane's rows: r0 and r0 + 8
  const bool busy = 16 * wm < R;      // the warp has rows (the same in all its lanes)
  unsigned long long sees[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * i;
    sees[i] = r < R ? a.mask[(size_t)b * a.nodes + r / c.G] : 0ull;
    if (count < 64) sees[i] &= (1ull << count) - 1ull;
  }
  // query rows, zeros past the last
  for (int i = threadIdx.x; i < 16 * a.wm * (D / 8); i += 32 * ncw) {
    const int row = i / (D / 8), ch = i % (D / 8);
    const int node = row / c.G, gg = row % c.G;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < R) v = *reinterpret_cast<const uint4*>(a.q + (((size_t)seq * a.nodes + node) * c.Hq + h * c.G + gg) * D + ch * 8);
    *reinterpret_cast<uint4*>(smem + C::Q_OFF + row * C::QROW + ch * 16) = v;
  }
  named_barrier_sync(1, 32 * ncw);
  // this lane's part of a k-step's A operand: four dimensions of rows g and g + 8
  const unsigned char* qrow = smem + C::Q_OFF + (16 * wm + g) * C::QROW + 8 * t4;
  auto load_q = [&](int k, uint32_t (&qa)[4]) {
    const uint2 x = *reinterpret_cast<const uint2*>(qrow + 32 * k);
    const uint2 y = *reinterpret_cast<const uint2*>(qrow + 8 * C::QROW + 32 * k);
    qa[0] = x.x;
    qa[1] = y.x;
    qa[2] = x.y;
    qa[3] = y.y;
  };
  const float qs = rsqrtf((float)D) * kLog2e;
  RowState<D> st;
  st.m[0] = st.m[1] = -CUDART_INF_F;
  st.l[0] = st.l[1] = 0.0f;
  st.E = -100;
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) st.o[n][k] = 0.0f;
  // the root's scores, for the attention-mass EMA
  const bool track = a.track && wm == 0;
  float* sc = a.scores + (size_t)s * c.G * a.score_stride;

  bool aborted = false;
  int taken = 0;
  for (int t = t0; t < t1; ++t, ++taken) {
    const int sg = taken % C::NSTAGE;
    const bool arrived = mbar_wait_bounded(&full[sg], (taken / C::NSTAGE) & 1);
    if (!__all_sync(0xffffffffu, arrived) || *abort_flag) {
      if (lane == 0) {
        set_error(c.err, kErrDevice);
        *abort_flag = 1;
      }
      aborted = true;
      break;
    }
    const unsigned char* sb = smem + sg * C::STAGE;
    const uint32_t kt = smem_addr(sb), vt = kt + C::KVB;
    const bool draft = t == tiles - 1, cold = t < tiles_c;
    const int j0 = cold ? t * C::TTC : (t - tiles_c) * 64;
    const int cnt = cold ? min(C::TTC, n_cold - j0) : draft ? count : min(64, c.W - j0);
    if (busy) {
      for (int c0 = 32 * wn; c0 < cnt; c0 += 32 * a.wn) {
        float sacc[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) sacc[n][k] = 0.0f;
        uint32_t pa[2][4], pb[2][4];
        if (CI8 && cold) {
          // ---- scores: B operands are the widened codes ----
          // (the four score blocks take turns: products into one accumulator wait for one another)
          const int i8 = lane & 7, mtx = lane >> 3;
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf) {
            uint32_t w[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int tok = c0 + 16 * (n >> 1) + 4 * (i8 >> 1) + (i8 & 1) + 2 * (n & 1);
              ldsm_x4(w[n], kt + (uint32_t)k8_off(tok, 64 * hf + 16 * mtx, D));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t qa[4];
              load_q(4 * hf + k, qa);
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                uint32_t b0, b1;
                cvt_codes(w[n][k], b0, b1);
                mma_f16(sacc[n], qa, b0, b1);
              }
            }
          }
          const float* ksp = reinterpret_cast<const float*>(sb + 2 * C::KVB);
          float ksc[8], vs[8];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 k4 = *reinterpret_cast<const float4*>(ksp + c0 + 16 * j + 4 * t4);
            const float4 v4 = *reinterpret_cast<const float4*>(ksp + 128 + c0 + 16 * j + 4 * t4);
            ksc[4 * j] = k4.x * qs, ksc[4 * j + 1] = k4.y * qs, ksc[4 * j + 2] = k4.z * qs, ksc[4 * j + 3] = k4.w * qs;
            vs[4 * j] = v4.x, vs[4 * j + 1] = v4.y, vs[4 * j + 2] = v4.z, vs[4 * j + 3] = v4.w;
          }
          uint32_t vb = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (c0 + 16 * (k >> 2) + 4 * t4 + (k & 3) >= cnt) vs[k] = 0.0f;
            vb = max(vb, __float_as_uint(vs[k]));
          }
          const int Et = scale_exp(__reduce_max_sync(0xffffffffu, vb));
          auto valid = [&](int, int k) { return c0 + 16 * (k >> 2) + 4 * t4 + (k & 3) < cnt; };
          softmax32<D>(st, sacc, ksc, vs, Et, valid, pa, pb);
          // ---- P.V ----
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q4 = 0; q4 < D / 32; ++q4) {
              uint32_t w[4];
              ldsm_x4(w, vt + (uint32_t)v8_off(c0 + 16 * j, 32 * q4 + lane, D));
              uint32_t b[4][2];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                cvt_codes(w[k], b[k][0], b[k][1]);
                mma_f16(st.o[4 * q4 + k], pa[j], b[k][0], b[k][1]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_f16(st.o[4 * q4 + k], pb[j], b[k][0], b[k][1]);
            }
        } else {
          // ---- FP16 rows ----
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t qa[4];
            load_q(k, qa);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const int tok = c0 + 16 * (n >> 1) + 4 * (g >> 1) + (g & 1) + 2 * (n & 1);
              const uint2 w = *reinterpret_cast<const uint2*>(sb + h_off(tok, 32 * k + 8 * t4, D));
              mma_f16(sacc[n], qa, w.x, w.y);
            }
          }
          const int32_t* pos = reinterpret_cast<const int32_t*>(sb + 2 * C::KVB);
          uint32_t live = 0;     // bit k: this lane's token k is there
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int j = c0 + 16 * (k >> 2) + 4 * t4 + (k & 3);
            live |= (uint32_t)(j < cnt && (cold || draft || pos[j] >= 0)) << k;
          }
          float ksc[8], vs[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            ksc[k] = qs;
            vs[k] = 1.0f;
          }
          auto valid = [&](int i, int k) {
            const bool there = (live >> k) & 1u;
            return there && (!draft || ((sees[i] >> (c0 + 16 * (k >> 2) + 4 * t4 + (k & 3))) & 1ull));
          };
          softmax32<D>(st, sacc, ksc, vs, 1, valid, pa, pb);
          const int i8 = lane & 7, mtx = lane >> 3;
          bool odd = false;      // a drafted value that is not finite
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // a token that is not there must not reach a sum through 0 * inf
            const uint32_t lv = live >> (4 * j);
            const uint32_t m0 = ((lv & 1u) ? 0xffffu : 0u) | ((lv & 2u) ? 0xffff0000u : 0u);
            const uint32_t m1 = ((lv & 4u) ? 0xffffu : 0u) | ((lv & 8u) ? 0xffff0000u : 0u);
            const int tok = c0 + 16 * j + 4 * (i8 >> 1) + (i8 & 1) + 2 * (mtx & 1);
#pragma unroll
            for (int q2 = 0; q2 < D / 16; ++q2) {
              uint32_t w[4];
              ldsm_x4_t(w, vt + (uint32_t)h_off(tok, 32 * q2 + 16 * (mtx >> 1), D));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                w[k] &= (k & 1) ? m1 : m0;
                if (draft) {
                  const uint32_t f = finite_mask(w[k]);
                  odd |= f != 0xffffffffu;
                  w[k] &= f;
                }
              }
              mma_f16(st.o[2 * q2], pa[j], w[0], w[1]);
              mma_f16(st.o[2 * q2 + 1], pa[j], w[2], w[3]);
              mma_f16(st.o[2 * q2], pb[j], w[0], w[1]);
              mma_f16(st.o[2 * q2 + 1], pb[j], w[2], w[3]);
            }
          }
          if (draft && __any_sync(0xffffffffu, odd)) {
            // values that are not finite reach only the rows that see their node (rare)
            for (int j = c0; j < min(c0 + 32, cnt); ++j)
#pragma unroll
              for (int n = 0; n < D / 8; ++n) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(sb + C::KVB + h_off(j, 16 * n + 4 * t4, D));
                if (finite_mask(w) == 0xffffffffu) continue;
                const float2 v = h2_to_f2(w);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if ((sees[i] >> j) & 1ull) {
                    if (!(fabsf(v.x) < CUDART_INF_F)) st.o[n][2 * i] += v.x;
                    if (!(fabsf(v.y) < CUDART_INF_F)) st.o[n][2 * i + 1] += v.y;
                  }
              }
          }
        }
        if (track && !draft) {
          // sacc holds the scaled scores (log2 units), -inf for tokens that are not there
          const int col0 = cold ? j0 : c.cap + j0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (r0 + 8 * i >= c.G) continue;
            float* dst = sc + (size_t)(r0 + 8 * i) * a.score_stride + col0;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int j = c0 + 16 * (n >> 1) + 4 * t4 + 2 * (n & 1) + x;
                if (j < cnt) dst[j] = sacc[n][2 * i + x];
              }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[sg]);
  }

  // ---- this warp's sums, then over the warps that split the tokens ----
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], 1);
    st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], 2);
  }
  {
    const float f = pow2i(st.E - kPBits);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) st.o[n][k] *= f;
  }
  if (named_barrier_or(1, 32 * ncw, aborted)) return;   // every tile has been read: the ring is free
  if (a.wn > 1) {
    float* area = reinterpret_cast<float*>(smem);
    if (wn > 0 && busy) {
      float* w = area + (size_t)((wn - 1) * a.wm + wm) * 16 * C::MROW;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* row = w + (g + 8 * i) * C::MROW;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(row + 8 * n + 2 * t4) = make_float2(st.o[n][2 * i], st.o[n][2 * i + 1]);
        if (t4 == 0) {
          row[D] = st.m[i];
          row[D + 1] = st.l[i];
        }
      }
    }
    named_barrier_sync(1, 32 * ncw);
    if (wn > 0 || !busy) return;
    for (int k = 1; k < a.wn; ++k) {
      const float* w = area + (size_t)((k - 1) * a.wm + wm) * 16 * C::MROW;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* row = w + (g + 8 * i) * C::MROW;
        const float m2 = row[D], mn = fmaxf(st.m[i], m2);
        const float f1 = st.m[i] == -CUDART_INF_F ? 0.0f : ex2(st.m[i] - mn);
        const float f2 = m2 == -CUDART_INF_F ? 0.0f : ex2(m2 - mn);
        st.m[i] = mn;
        st.l[i] = st.l[i] * f1 + row[D + 1] * f2;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          const float2 v = *reinterpret_cast<const float2*>(row + 8 * n + 2 * t4);
          st.o[n][2 * i] = st.o[n][2 * i] * f1 + v.x * f2;
          st.o[n][2 * i + 1] = st.o[n][2 * i + 1] * f1 + v.y * f2;
        }
      }
    }
  }
  if (!busy) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + 8 * i;
    if (r >= R) continue;
    if (a.splits > 1) {
      float* pp = a.part + ((size_t)(item * a.splits + split) * a.nodes * c.G + r) * (D + 2);
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(pp + 8 * n + 2 * t4) = make_float2(st.o[n][2 * i], st.o[n][2 * i + 1]);
      if (t4 == 0) {
        pp[D] = st.m[i];
        pp[D + 1] = st.l[i];
      }
      continue;
    }
    const int node = r / c.G, gg = r % c.G;
    const size_t orow = ((size_t)seq * a.nodes + node) * c.Hq + h * c.G + gg;
    // a row that sees nothing: zeros, and a log-sum-exp of -inf
    const float inv = st.l[i] == 0.0f ? 0.0f : 1.0f / st.l[i];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<uint32_t*>(a.out + orow * D + 8 * n + 2 * t4) =
          pack_h2(st.o[n][2 * i] * inv, st.o[n][2 * i + 1] * inv);
    const float lse = (st.m[i] + log2f(st.l[i])) * kLn2;
    if (t4 == 0) {
      if (a.lse_out) a.lse_out[orow] = lse;
      if (a.track && node == 0) a.lse_ws[(size_t)s * c.G + gg] = lse;
    }
  }
}

// Merge the splits: one warp per row.
template <int D>
__global__ void __launch_bounds__(256) tree_combine_kernel(const Cache c, const TreeLaunch a) {
  chain_enter();
  const int lane = threadIdx.x & 31;
  const int rows = a.nodes * c.G;
  const long long w = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int item = (int)(w / rows), r = (int)(w % rows);
  if (item >= a.r.items(c.Hkv)) return;
  int l, b, h;
  const int s = seg_of(c, a.r, item, &l, &b, &h);
  const int seq = (l - a.r.l0) * a.r.B + b;
  const int count = a.counts ? a.counts[b] : a.nodes;
  if (count < 0 || count > a.nodes || r >= count * c.G) return;
  const float* pp = a.part + ((size_t)item * a.splits * rows + r) * (D + 2);
  const size_t step = (size_t)rows * (D + 2);
  // lane k holds the maximum and the sum of split k, k + 32, ...; then the rows
  // are added up, several loads in flight
  float m = -CUDART_INF_F;
  for (int k = lane; k < a.splits; k += 32) m = fmaxf(m, pp[k * step + D]);
  m = warp_max(m);
  const float m0 = m == -CUDART_INF_F ? 0.0f : m;
  float lsum = 0.0f, o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.0f;
  for (int k0 = 0; k0 < a.splits; k0 += 32) {
    const int nk = min(32, a.splits - k0);
    float fk = 0.0f;
    if (lane < nk) {
      const float* q = pp + (k0 + lane) * step;
      fk = ex2(q[D] - m0);
      lsum = fmaf(q[D + 1], fk, lsum);
    }
#pragma unroll 8
    for (int k = 0; k < nk; ++k) {
      const float f = __shfl_sync(0xffffffffu, fk, k);
      const float* q = pp + (k0 + k) * step;
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        const float2 v = *reinterpret_cast<const float2*>(q + 64 * e + 2 * lane);
        o[2 * e] = fmaf(v.x, f, o[2 * e]);
        o[2 * e + 1] = fmaf(v.y, f, o[2 * e + 1]);
      }
    }
  }
  lsum = warp_sum(lsum);
  const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;
  const int node = r / c.G, gg = r % c.G;
  const size_t orow = ((size_t)seq * a.nodes + node) * c.Hq + h * c.G + gg;
#pragma unroll
  for (int e = 0; e < D / 64; ++e)
    *reinterpret_cast<uint32_t*>(a.out + orow * D + 64 * e + 2 * lane) = pack_h2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0) {
    const float lse = (m + log2f(lsum)) * kLn2;
    if (a.lse_out) a.lse_out[orow] = lse;
    if (a.track && node == 0) a.lse_ws[(size_t)s * c.G + gg] = lse;
  }
}

// Append of accepted rows: one warp per segment, its tokens one after the other
// (each may push the oldest window token into the INT8 region).
template <int D>
__global__ void __launch_bounds__(128) append_rows_kernel(const Cache c, const Policy pol, const AppendLaunch a) {
  chain_enter();
  const int item = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (item >= a.r.items(c.Hkv)) return;
  int l, b, h;
  const int s = seg_of(c, a.r, item, &l, &b, &h);
  const int seq = (l - a.r.l0) * a.r.B + b;
  const int n = a.counts ? a.counts[b] : a.tokens;
  if (!guard(n >= 0 && n <= a.tokens, c.err, kSiteAppendCount, s, n)) return;
  int t = c.next_pos[s], n_cold = c.n_cold[s];
  if (!guard(t >= 0 && n_cold >= 0 && n_cold <= c.cap, c.err, kSiteAppendSeg, s, t)) return;
  // no token of a list with a bad row is appended
  for (int i = lane; i < n; i += 32) {
    const int row = a.index ? a.index[(size_t)b * a.tokens + i] : i;
    if (row < 0 || row >= a.rows) record_violation(c.err, kSiteAppendRow, s, row);
  }
  bool ok = true;
  for (int i = lane; i < n; i += 32) {
    const int row = a.index ? a.index[(size_t)b * a.tokens + i] : i;
    ok = ok && row >= 0 && row < a.rows;
  }
  if (!__all_sync(0xffffffffu, ok)) return;
  // nor of one that does not fit (the host's bound does not follow replays of a graph)
  if (n_cold + n > c.cap) {
    int cold = n;            // rows that the list adds outside the window
    if (c.W > 0) {
      // the window's tokens that reach age W on the way, and the list's own
      cold = 0;
      for (int sl = lane; sl < c.W; sl += 32) {
        const int pos = c.pos_r[(size_t)s * c.Wst + sl];
        cold += pos >= 0 && pos < t + n - c.W;
      }
      cold = __reduce_add_sync(0xffffffffu, cold) + max(0, n - c.W);
    }
    if (!guard(n_cold + cold <= c.cap, c.err, kSiteAppendRoom, s, n)) return;
  }
  for (int i = 0; i < n; ++i) {
    const int row = a.index ? a.index[(size_t)b * a.tokens + i] : i;
    const size_t in_row = ((size_t)seq * a.rows + row) * c.Hkv + h;
    uint32_t kw[D / 64], vw[D / 64];
    row_load_plain<D>(a.k + in_row * D, lane, kw);
    row_load_plain<D>(a.v + in_row * D, lane, vw);
    const float sc = pol.mode == 1 ? a.prio[in_row] : initial_score(pol, l, b, h, t);
    n_cold = append_row<D>(c, s, lane, t, n_cold, kw, vw, sc);
    if (n_cold < 0) return;
    ++t;
    __syncwarp();   // lane 0's counters and positions before the next token reads them
  }
}

template <int D, bool CI8>
cudaError_t run_tree(const Cache& c, const TreeLaunch& a0, cudaStream_t st, long long* launches, Prof* prof) {
  using C = TCfg<D, CI8>;
  TreeLaunch a = a0;
  const int items = a.r.items(c.Hkv), rows = a.nodes * c.G;
  const int tiles_ub = (a.max_cold_tokens + C::TTC - 1) / C::TTC + (c.W + 63) / 64 + 1;
  const long long room = a.part_rows / ((long long)items * rows);
  cudaError_t e;
  if (rows > kMaxRows) {
    a.mtiles = (rows + 255) / 256;
    // Splits of the token axis: the number with the shortest run of waves, a
    // tile being about a microsecond and a CTA's start and end about three.
    const long long base = (long long)items * a.mtiles;
    const long long most = std::max(1ll, std::min<long long>({room, tiles_ub, 64}));
    double best = 0.0;
    a.splits = 1;
    for (int k = 1; k <= most; ++k) {
      const long long waves = (base * k + a.num_sms - 1) / a.num_sms;
      const double cost = waves * ((double)tiles_ub / k + 3.0) + (k > 1 ? 3.0 : 0.0);
      if (k == 1 || cost < best) {
        best = cost;
        a.splits = k;
      }
    }
    ProfScope ps(prof, kKAttention, st);
    e = launch_tree_mma(c, a, (unsigned)(base * a.splits), st);
  } else {
    // One or two 16-row blocks; the other warps split the tokens of a tile, 32 at a time.
    a.mtiles = 1;
    a.wm = (rows + 15) / 16;
    a.wn = CI8 ? 4 : 2;
    e = cudaFuncSetAttribute(tree_kernel<D, CI8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int threads = 32 * (a.wm * a.wn + 1);
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, tree_kernel<D, CI8>, threads, C::SMEM);
    if (e != cudaSuccess) return e;
    // Splits of the token axis: as many as fill the SMs once, when the segments
    // and row tiles alone do not, with two tiles a split at least.
    const int resident = a.num_sms * std::max(1, per_sm);
    a.splits = (int)std::max<long long>(1, std::min<long long>({resident / items, (tiles_ub + 1) / 2, room}));
    ProfScope ps(prof, kKAttention, st);
    e = launch_chained(tree_kernel<D, CI8>, (unsigned)(items * a.splits), threads, C::SMEM, st, c, a);
  }
  if (e != cudaSuccess) return e;
  ++*launches;
  if (a.splits > 1) {
    ProfScope ps(prof, kKCombine, st);
    const long long warps = (long long)items * a.nodes * c.G;
    e = launch_chained(tree_combine_kernel<D>, (unsigned)((warps + 7) / 8), 256, 0, st, c, a);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_tree_attn(const Cache& c, const TreeLaunch& a, cudaStream_t st, long long* launches, Prof* prof) {
  if (a.r.items(c.Hkv) == 0) return cudaSuccess;
  if (c.D == 128)
    return c.cold_int8 ? run_tree<128, true>(c, a, st, launches, prof) : run_tree<128, false>(c, a, st, launches, prof);
  return c.cold_int8 ? run_tree<64, true>(c, a, st, launches, prof) : run_tree<64, false>(c, a, st, launches, prof);
}

cudaError_t launch_append_rows(const Cache& c, const Policy& pol, const AppendLaunch& a, cudaStream_t st,
                               long long* launches, Prof* prof) {
  const int items = a.r.items(c.Hkv);
  if (items == 0) return cudaSuccess;
  ProfScope ps(prof, kKAppend, st);
  const unsigned grid = (unsigned)((items + 3) / 4);
  const cudaError_t e = c.D == 128 ? launch_chained(append_rows_kernel<128>, grid, 128, 0, st, c, pol, a)
                                   : launch_chained(append_rows_kernel<64>, grid, 128, 0, st, c, pol, a);
  if (e == cudaSuccess) ++*launches;
  return e;
}

}  // namespace confkv
