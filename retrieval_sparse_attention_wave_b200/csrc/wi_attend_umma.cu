// Causal attention over the paged cache on the tensor cores (bf16).
//
// A CTA takes one item: up to two query tiles of 128 rows and a run of
// 128-key tiles.  For query tile i and key tile j (fp32 accumulators in tensor
// memory):
//   S_i = Q_i K_j^T;   P_i = 2^(c S_i - m_i) as bf16, over S_i's columns;
//   O_i += P_i V_j     (P_i straight from tensor memory).
// The weights are rounded to bf16, the type of the values they multiply (half
// a step, 2^-8 of a weight, averages out over the keys; the output's own
// rounding is as large); their sum is taken before that, in fp32.  Where the
// caller asks for exact_weights, a weight is two bf16 parts (P_i and the rest
// of it, in the other half of S_i's columns) and 16 bits of it count: a third
// more time (8192 tokens 679 us against 526, 32768 10.4 ms
// against 7.9) for an output off by its own rounding alone
// (relative 0.0016 against 0.0022).
// Roles:
//   warps 0..3, 4..7  softmax of query tile 0, 1: a thread owns a row
//                     (a tensor-memory lane), so its maximum, mass and output
//                     scale need no exchange;
//   warp 8            the queries (one 3-D tensor copy a tile and 64
//                     channels), then K_0, V_0, K_1, V_1, ... into a ring of
//                     stages: a tensor copy per page and 64 channels;
//   warp 9            issues the MMAs: while tile 0's softmax runs, tile 1's
//                     products do, and the other way round;
//   warps 10, 11      the value tiles on the diagonal: rows no query sees are
//                     zeroed, and values that are not finite in rows only
//                     some queries see (weight 0 times them is not 0) are
//                     taken out and given back to those that see them at the
//                     end.
// The reference point m only keeps the powers in range, P and the mass being
// relative to the same m whatever it is.  It is set 2^24 above a row's maximum
// and moves when the maximum passes it, so the output is seldom rescaled, and
// weights stay at or below 1: the sums are finite as long as tokens x |v| is.
// (Their last bits are lost for |v| below 2^-100.)
//
// What bounds it: a group's own chain.  A tile's softmax takes about 1650
// clocks (read 170, maximum 250, weights 1220: the special-function unit
// alone is 768), its output and next scores 1024, the hand-overs 200; the two
// groups' chains interleave to 2850 clocks a pair of tiles, of which the
// tensor cores work 2048.  8192 tokens of 32 heads on 8 KV heads of 128: 450
// us, 1.22 PFLOP/s (520 us back to back under the power cap); 32768 tokens
// 7.6 to 7.7 ms, 1.15 PFLOP/s.
#include <cmath>

#include "wi_attend_tiles.cuh"
#include "wi_umma.cuh"

namespace wi {
namespace {

constexpr int kUThreads = 384;
// log2 of the reference's distance above the maximum it was set at.  At 2^8
// rescales are common in a sequence's first tiles: short prompts took 22.5 us
// against 20.5.
constexpr float kHead = 24.f;
// Every kPoly-th pair of weights is taken without the special-function unit.
// 8192 tokens: 2 takes 480 us, 3 444, 4 441, 8 445.
constexpr int kPoly = 4;
constexpr int kSoftmaxRegs = 224, kOtherRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kUThreads * 168, "within the launch's registers");

template <int D>
struct UmmaShape {
  static constexpr uint32_t kTile = kRows * D * 2;      // bytes of a tile
  static constexpr uint32_t kBlock = kRows * 128;       // its blocks of 64 channels
  static constexpr int kBlocks = D / 64;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr size_t kSmem = 1024 + (2 + kStages) * (size_t)kTile;
  // tensor-memory columns
  static constexpr uint32_t kS = 0, kO = 256, kCols = 512;
};

__device__ __forceinline__ void tensor_load_3d(void* smem, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(smem)), "l"(tmap), "r"(x), "r"(y), "r"(z),
      "r"(smem_addr(bar)) : "memory");
}

// 2^x without the special-function unit: x = n + f, |f| <= 1/2 (the sum with
// 1.5 * 2^23 rounds x to the integer n, which is then in its low bits), 2^f
// from a degree-5 polynomial (value 1 at 0, the others fitted for the least
// largest relative error, 2^-22.6 in fp32), n added to the exponent.  From
// -127 down the result is 0 (n = -127, f = 0).
__device__ __forceinline__ float2 ex2_poly(float2 x) {
  const auto two = [](float v) { return make_float2(v, v); };
  x = make_float2(fmaxf(x.x, -127.f), fmaxf(x.y, -127.f));
  const float2 t = __fadd2_rn(x, two(12582912.f));
  const float2 f = __ffma2_rn(__fadd2_rn(t, two(-12582912.f)), two(-1.f), x);
  float2 p = __ffma2_rn(f, two(0x1.5bba14p-10f), two(0x1.3cea88p-7f));
  p = __ffma2_rn(p, f, two(0x1.c6b752p-5f));
  p = __ffma2_rn(p, f, two(0x1.ebf9bcp-3f));
  p = __ffma2_rn(p, f, two(0x1.62e42ap-1f));
  p = __ffma2_rn(p, f, two(1.f));
  return make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + __float_as_uint(p.x)),
                     __uint_as_float((__float_as_uint(t.y) << 23) + __float_as_uint(p.y)));
}
// Lane l of four has chunk c of row l in x[c]; afterwards chunk l of row c: the
// four lanes' stores of one row are 64 consecutive bytes.
__device__ __forceinline__ void transpose4(uint4 (&x)[4], int lane) {
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const bool hi = (lane & o) != 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & o) continue;
      uint4 &a = x[c], &b = x[c | o];
      const uint4 send = hi ? a : b;
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, send.x, o);
      got.y = __shfl_xor_sync(0xffffffffu, send.y, o);
      got.z = __shfl_xor_sync(0xffffffffu, send.z, o);
      got.w = __shfl_xor_sync(0xffffffffu, send.w, o);
      if (hi) a = got; else b = got;
    }
  }
}
// eight bf16 values: some is infinite or NaN
__device__ __forceinline__ bool nonfinite(const uint4& x) {
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  __nv_bfloat162 a = zero;
#pragma unroll
  for (int i = 0; i < 4; ++i) a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), zero, a);
  return __hisnan(a.x) || __hisnan(a.y);
}
// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

template <int D, int N, bool kExact>
__global__ void __launch_bounds__(kUThreads, 1)
attend_umma_kernel(const __grid_constant__ AttendTable<N> tb, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const Pool kp, const Pool vp, const AttendOut ao, float scale, uint32_t* status) {
  using S = UmmaShape<D>;
  using T = __nv_bfloat16;
  extern __shared__ unsigned char sh_raw[];
  unsigned char* sq = align_smem_1024(sh_raw);
  unsigned char* ring = sq + 2 * S::kTile;
  __shared__ __align__(8) uint64_t s_full[S::kStages], s_empty[S::kStages];
  __shared__ __align__(8) uint64_t s_q, s_s[2], s_p[2][2], s_o[2], s_go[2], s_fixed[2], s_done;
  __shared__ uint32_t s_tmem, s_bad;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform for the compiler)
  pdl_launch_dependents();
  const Item it = item_of(tb, blockIdx.x, kRows);
  if (it.t0 == it.t1) return;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 1);
    }
    mbar_init(&s_q, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_s[i], 1);
      mbar_init(&s_p[i][0], 4);
      mbar_init(&s_p[i][1], 4);
      mbar_init(&s_o[i], 1);
      mbar_init(&s_go[i], 1);
      mbar_init(&s_fixed[i], 2);
    }
    mbar_init(&s_done, 1);
    mbar_init_fence();
    s_bad = 0;
  }
  if (warp == 9) tmem_alloc(&s_tmem, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's: they start at 0

  const int G = 1 << tb.g_shift, n = it.t1 - it.t0;
  const int nq = it.rows > kRows ? 2 : 1;
  const int first_pos = it.pos0 + (it.row0 >> tb.g_shift);
  // the first key tile on the diagonal: with a key (first_pos + 1, say) that
  // some row of the block does not see
  const int fix_from = max(0, (first_pos + 1) / kRows - it.t0);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------------------- loads
      if (lane == 0) {
        mbar_arrive_expect(&s_q, (uint32_t)nq * S::kTile);
        for (int i = 0; i < nq; ++i)
          for (int c = 0; c < S::kBlocks; ++c)
            tensor_load_3d(sq + i * S::kTile + c * S::kBlock, &map_q, 64 * c, it.h * G,
                           it.q0 + ((it.row0 + i * kRows) >> tb.g_shift), &s_q);
      }
      load_units<D, S::kStages>(it, tb.hkv, kp, vp, map_k, map_v, ring, s_full, s_empty, status);
    } else if (warp == 9) {
      // ----------------------------------------------------------------- MMAs
      // The whole warp runs the loop, so that addresses and descriptors stay in
      // uniform registers; one elected lane issues each batch.
      constexpr uint32_t kIdescS = umma_idesc_bf16_f32<128, 128>();
      constexpr uint32_t kIdescO = umma_idesc_bf16_f32<128, D>() | kIdescBMn;
      constexpr uint64_t kStep = S::kTile >> 4;   // a stage, in descriptor units
      const uint64_t dq = umma_desc_sw128(smem_addr(sq)), dk = umma_desc_sw128(smem_addr(ring));
      const uint64_t dv = umma_desc_sw128_mn(smem_addr(ring), S::kBlock);
      auto scores = [&](int i, int st, bool last) {   // S_i = Q_i K^T
        if (elect_one()) {
          const uint64_t a = dq + i * kStep, b = dk + st * kStep;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t ko = ((uint32_t)(k >> 2) * S::kBlock + (uint32_t)(k & 3) * 32u) >> 4;
            umma_bf16(tmem + S::kS + i * 128, a + ko, b + ko, kIdescS, k != 0);
          }
          umma_commit(&s_s[i]);
          if (last) umma_commit(&s_empty[st]);
        }
        __syncwarp();
      };
      auto output = [&](int i, int st, int half, bool first) {   // O_i += P_i V, half of the keys
        if (elect_one()) {
          const uint64_t b = dv + st * kStep;
#pragma unroll
          for (int kk = 0; kk < kRows / 32; ++kk) {
            const int k = half * (kRows / 32) + kk;
            umma_bf16_ts(tmem + S::kO + i * D, tmem + S::kS + i * 128 + k * 8, b + k * (2048 >> 4), kIdescO,
                         !first || kk != 0);
            if (kExact)   // the weights' second parts
              umma_bf16_ts(tmem + S::kO + i * D, tmem + S::kS + i * 128 + 64 + k * 8, b + k * (2048 >> 4), kIdescO, true);
          }
          if (half == 1) {
            umma_commit(&s_o[i]);
            if (i == nq - 1) umma_commit(&s_empty[st]);
          }
        }
        __syncwarp();
      };
      // a ring position: unit u in stage st, phase ph
      auto full = [&](int st, uint32_t ph) { return wait_bar(&s_full[st], ph, status); };
      bool ok = wait_bar(&s_q, 0, status) && full(0, 0);
      tc_fence_after();
      if (ok)
        for (int i = 0; i < nq; ++i) scores(i, 0, i == nq - 1);
      if (fix_from == 0 && lane == 0) mbar_arrive(&s_go[0]);
      int st = 1;
      uint32_t ph = 0;
      for (int j = 0; j < n && ok; ++j) {
        // the diagonal's values are looked at a tile ahead of their product
        if (j + 1 >= fix_from && j + 1 < n && lane == 0) mbar_arrive(&s_go[(j + 1) & 1]);
        const bool fix = j >= fix_from;
        if (!(ok = full(st, ph))) break;   // V_j
        const int sv = st;
        if (++st == S::kStages) { st = 0; ph ^= 1; }
        for (int i = 0; i < nq && ok; ++i) {
          ok = wait_bar(&s_p[i][0], (uint32_t)j & 1u, status);
          if (ok && fix && i == 0) ok = wait_bar(&s_fixed[j & 1], (uint32_t)((j - fix_from) >> 1) & 1u, status);
          if (!ok) break;
          tc_fence_after();
          output(i, sv, 0, j == 0);
          if (!(ok = wait_bar(&s_p[i][1], (uint32_t)j & 1u, status))) break;
          tc_fence_after();
          output(i, sv, 1, false);
          if (j + 1 < n) {
            if (i == 0 && !(ok = full(st, ph))) break;   // K_(j + 1)
            tc_fence_after();
            scores(i, st, i == nq - 1);
          }
        }
        if (++st == S::kStages) { st = 0; ph ^= 1; }
      }
      // every MMA issued has completed before the columns are released
      if (elect_one()) umma_commit(&s_done);
      __syncwarp();
      wait_bar(&s_done, 0, status);
    } else if (warp >= 10) {
      // ------------------------------------------- value tiles on the diagonal
      for (int j = fix_from; j < n; ++j) {
        // (the ring's phase of V_j is known only from a permission in the MMA
        // warp's order; two of them alternate, as the next may come before this
        // one is seen)
        const int u = 2 * j + 1, base = (it.t0 + j) * kRows;
        bool ok = wait_bar(&s_go[j & 1], (uint32_t)((j - fix_from) >> 1) & 1u, status);
        ok = ok && wait_bar(&s_full[u % S::kStages], (uint32_t)(u / S::kStages) & 1u, status);
        if (!__all_sync(0xffffffffu, ok)) break;
        unsigned char* tile = ring + (size_t)(u % S::kStages) * S::kTile;
        constexpr int CH = D / 8;
        auto chunk_at = [&](int c) {
          return reinterpret_cast<uint4*>(tile + ((c % CH) >> 3) * S::kBlock + swz128(c / CH, c & 7));
        };
        const int r0 = max(0, first_pos + 1 - base);   // the first row some query does not see
        const int r1 = min(kRows, it.key_end - base);   // the first row none sees
        const int at0 = 32 * (warp - 10) + lane;
#pragma unroll 4
        for (int c = r1 * CH + at0; c < kRows * CH; c += 64) *chunk_at(c) = make_uint4(0u, 0u, 0u, 0u);
        // four chunks in flight; a product with 0 tells whether all eight
        // values of a chunk are finite (0 or NaN)
        bool bad = false;
#pragma unroll 1
        for (int c0 = r0 * CH + at0; c0 < r1 * CH; c0 += 256) {
          uint4 x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = *chunk_at(min(c0 + 64 * e, r1 * CH - 1));
          uint32_t odd = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) odd |= nonfinite(x[e]) ? 1u << e : 0u;
          if (odd == 0) continue;
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            if (!((odd >> e) & 1u) || c0 + 64 * e >= r1 * CH) continue;
            uint32_t* w = reinterpret_cast<uint32_t*>(chunk_at(c0 + 64 * e));
            bad = true;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t v = w[q];
              if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
              if ((v & 0x7f800000u) == 0x7f800000u) v &= 0x0000ffffu;
              w[q] = v;
            }
          }
        }
        if (bad) atomicOr(&s_bad, 1u);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_fixed[j & 1]);
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2, r = i * kRows + 32 * (warp & 3) + lane;
    const int pos = it.pos0 + ((it.row0 + r) >> tb.g_shift);
    const int warp_pos = __shfl_sync(0xffffffffu, pos, 0);
    const bool used = i * kRows + 32 * (warp & 3) < it.rows;   // some row of the warp is real
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + S::kS + i * 128, to = tmem + lanes + S::kO + i * D;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (i < nq) {
      for (int j = 0; j < n && ok; ++j) {
        ok = __all_sync(0xffffffffu, wait_bar(&s_s[i], (uint32_t)j & 1u, status));
        if (!ok) break;
        if (used) {
          tc_fence_after();
          uint32_t x[4][32];
          tmem_ld32_issue(ts, x[0]);
          tmem_ld32_issue(ts + 32, x[1]);
          tmem_ld32_issue(ts + 64, x[2]);
          tmem_ld32_issue(ts + 96, x[3]);
          tmem_wait_ld();
          tie32(x[0]); tie32(x[1]); tie32(x[2]); tie32(x[3]);
          const int base = (it.t0 + j) * kRows;
          if (base + kRows - 1 > warp_pos) {
            const int lim = pos - base;   // columns above it are masked
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c + e > lim) x[c][e] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = __uint_as_float(x[c][0]);
#pragma unroll
            for (int e = 1; e < 31; e += 2)
              mx[c] = max3_nan(mx[c], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
          }
          mx[0] = max3_nan(mx[0], __uint_as_float(x[0][31]), __uint_as_float(x[1][31]));
          mx[1] = max3_nan(mx[1], __uint_as_float(x[2][31]), __uint_as_float(x[3][31]));
          // a score that is NaN or +inf makes its row NaN
          float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * scale;
          top = top < INFINITY ? top : NAN;
          const bool up = !(top <= m);
          if (__any_sync(0xffffffffu, up)) {
            const float mn = up ? top + kHead : m;
            const float c = up ? ex2(m - mn) : 1.f;
            l *= c;
            m = mn;
            if (j > 0) {   // O holds the keys before
              ok = __all_sync(0xffffffffu, wait_bar(&s_o[i], (uint32_t)(j - 1) & 1u, status));
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < D; q += 8) tmem_scale8(to + q, c);
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;
          const float2 sc = make_float2(scale, scale), nm = make_float2(-mu, -mu);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16], p2[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), sc, nm);
              const float2 w = e % kPoly == kPoly - 1 ? ex2_poly(y) : make_float2(ex2(y.x), ex2(y.y));
              sum[e & 1] = __fadd2_rn(sum[e & 1], w);
              if (kExact) split_bf16(w.x, w.y, p[e], p2[e]);
              else p[e] = pack_bf16(w.x, w.y);
            }
            tmem_st16(ts + 16 * c, p);
            if (kExact) tmem_st16(ts + 64 + 16 * c, p2);
            if (c == 1) {   // the product over the first half may start
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_p[i][0]);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_p[i][1]);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        } else if (lane == 0) {
          mbar_arrive(&s_p[i][0]);
          mbar_arrive(&s_p[i][1]);
        }
      }
      if (ok) ok = __all_sync(0xffffffffu, wait_bar(&s_o[i], (uint32_t)(n - 1) & 1u, status));
    }
    if (used) {
      tc_fence_after();
      const int row = it.row0 + r;
      const int64_t tok = it.q0 + (row >> tb.g_shift);
      const int head = it.h * G + (row & (G - 1));
      const bool real = r < it.rows;
      const float inv = 1.f / l;
      auto out_row = [&](int rr) {   // of row rr of the block
        const int x = it.row0 + rr;
        return reinterpret_cast<T*>(ao.out) + (it.q0 + (x >> tb.g_shift)) * ao.stride +
               (int64_t)(it.h * G + (x & (G - 1))) * D;
      };
      if (real && it.part >= 0) ao.ml[it.part + r] = make_float2(m, l);
      else if (real && ao.lse) ao.lse[tok * ao.Hq + head] = kLn2 * (m + log2f(l));
      // 64 bytes of a row at a time (16 columns of a part, 32 of the output);
      // four lanes store a row's together: row 4 (lane / 4) + c of the warp
      const bool part = it.part >= 0;
      const int r4 = r - lane + (lane & ~3);
      uint4 x[4];
      float2 odd = make_float2(0.f, 0.f);   // 0, or NaN where a sum is not finite
#pragma unroll 1
      for (int col = 0; col < D; col += 16) {
        uint32_t y[16];
        tmem_ld16(to + col, y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          odd = __ffma2_rn(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), make_float2(0.f, 0.f), odd);
        if (part) {
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = make_uint4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
        } else {
          x[0] = x[2];
          x[1] = x[3];
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = pack_bf16(__uint_as_float(y[2 * e]) * inv, __uint_as_float(y[2 * e + 1]) * inv);
          x[2] = make_uint4(w[0], w[1], w[2], w[3]);
          x[3] = make_uint4(w[4], w[5], w[6], w[7]);
          if (!(col & 16)) continue;
        }
        uint4 t[4] = {x[0], x[1], x[2], x[3]};
        transpose4(t, lane);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (r4 + c >= it.rows) break;
          unsigned char* o = part ? reinterpret_cast<unsigned char*>(ao.o + (it.part + r4 + c) * D + col)
                                  : reinterpret_cast<unsigned char*>(out_row(r4 + c) + (col & ~16));
          *reinterpret_cast<uint4*>(o + 16 * (lane & 3)) = t[c];
        }
      }
      const bool lost = odd.x + odd.y != 0.f && real && l == l;   // (a row whose mass is NaN is NaN)
      if (__any_sync(0xffffffffu, lost || *(volatile uint32_t*)&s_bad != 0)) {
        // Values that are not finite, added to the rows that see them (a
        // positive weight of them is they themselves).  An infinity that every
        // row sees has made NaN of its column where its weight, or the second
        // part of it, came out as 0 or that part is negative: all of a lost
        // row's keys are looked at, and the first such value takes its
        // column's place.
        __syncwarp();
        const int p1 = real ? min(pos + 1, it.t1 * kRows) : 0;
        uint32_t found[D / 32] = {};
#pragma unroll 1
        for (int p = max(lost ? 0 : first_pos + 1, it.t0 * kRows); p < p1; ++p) {
          const int64_t at = pool_row(vp, tb.hkv, D, it.b, it.h, p, status);
#pragma unroll 1
          for (int c = 0; at >= 0 && c < D; ++c) {
            const T* v = reinterpret_cast<const T*>(vp.base) + at + c;
            if (c % 8 == 0 && !nonfinite(*reinterpret_cast<const uint4*>(v))) {
              c += 7;
              continue;
            }
            const float f = __bfloat162float(*v);
            if (isfinite(f)) continue;
            const bool first = lost && !((found[c / 32] >> (c % 32)) & 1u);
            found[c / 32] |= 1u << (c % 32);
            if (part) {
              float* o = ao.o + (it.part + r) * D + c;
              *o = first ? f : *o + f;
            } else {
              T* o = out_row(r) + c;
              *o = __float2bfloat16_rn(first ? f : __bfloat162float(*o) + f);
            }
          }
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }
}

template <int D, bool kExact, int N>
cudaError_t launch_typed(const AttendTable<N>& tb, const AttendPlan& pl, const AttendArgs& a, const AttendOut& ao,
                         cudaStream_t s) {
  using S = UmmaShape<D>;
  CUtensorMap mq, mk, mv;
  // the queries of a group of heads as rows (token, head): 64 channels x G x 128 / G
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)pl.Hq, (cuuint64_t)pl.q_tokens};
  const cuuint64_t qs[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)pl.G, (cuuint32_t)(kRows / pl.G)};
  if (!encode_map(&mq, 3, a.q, qd, qs, qb) || !encode_pools(&mk, &mv, a, pl.hkv, D))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<attend_umma_kernel<D, N, kExact>>(S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attend_umma_kernel<D, N, kExact>, dim3(tb.n_items), kUThreads, S::kSmem, s, false, tb, mq, mk, mv, a.kp,
                       a.vp, ao, kLog2e / std::sqrt((float)D), reinterpret_cast<uint32_t*>(a.ws));
}

}  // namespace

template <int N>
cudaError_t launch_attend_umma(const AttendTable<N>& tb, const AttendPlan& pl, const AttendArgs& a,
                             const AttendOut& ao, cudaStream_t s) {
  if (pl.exact) return pl.D == 128 ? launch_typed<128, true>(tb, pl, a, ao, s) : launch_typed<64, true>(tb, pl, a, ao, s);
  return pl.D == 128 ? launch_typed<128, false>(tb, pl, a, ao, s) : launch_typed<64, false>(tb, pl, a, ao, s);
}
template cudaError_t launch_attend_umma(const AttendTable<kFewSeqs>&, const AttendPlan&, const AttendArgs&,
                                      const AttendOut&, cudaStream_t);
template cudaError_t launch_attend_umma(const AttendTable<kMaxBatch>&, const AttendPlan&, const AttendArgs&,
                                      const AttendOut&, cudaStream_t);

}  // namespace wi
