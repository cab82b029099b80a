// Causal attention over the paged cache on the tensor cores (bf16).
//
// A CTA takes one item: up to two query tiles of 128 rows and a run of
// 128-key tiles.  For query tile i and key tile j (fp32 accumulators in tensor
// memory):
//   S_i = Q_i K_j^T;   P_i = 2^(c S_i - m_i) as bf16, over S_i's columns;
//   O_i += P_i V_j     (P_i straight from tensor memory).
// Roles:
//   warps 0..3, 4..7  softmax of query tile 0, 1: a thread owns a row
//                     (a tensor-memory lane), so its maximum, mass and output
//                     scale need no exchange; a lone query tile (single
//                     tokens, short prompts) has its key tiles taken in turns
//                     by both;
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
// The output is rescaled only when a row's maximum rises by more than 2^8:
// the reference point m only keeps the powers in range, P and the mass being
// relative to the same m whatever it is.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "wi_attend.cuh"
#include "wi_umma.cuh"

namespace wi {
namespace {

constexpr int kRows = 128;          // rows of a query tile, keys of a key tile
constexpr int kUThreads = 384;
constexpr float kRescale = 8.f;     // log2 of the growth that forces a rescale
constexpr int kPoly = 4;            // every kPoly-th pair of weights without the special-function unit
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
// the largest of three, NaN if one is NaN
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int D>
__global__ void __launch_bounds__(kUThreads, 1)
attend_umma_kernel(const __grid_constant__ AttendTable tb, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const Pool kp, const Pool vp, const AttendOut ao, float scale, uint32_t* status) {
  using S = UmmaShape<D>;
  using T = __nv_bfloat16;
  extern __shared__ unsigned char sh_raw[];
  unsigned char* sq = align_smem_1024(sh_raw);
  unsigned char* ring = sq + 2 * S::kTile;
  __shared__ __align__(8) uint64_t s_full[S::kStages], s_empty[S::kStages];
  __shared__ __align__(8) uint64_t s_q, s_s[2], s_p[2][2], s_o[2], s_go, s_fixed, s_done;
  __shared__ float2 s_ml[kRows];
  __shared__ uint32_t s_tmem, s_bad;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (uniform for the compiler)
  pdl_launch_dependents();
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
    }
    mbar_init(&s_go, 1);
    mbar_init(&s_fixed, 2);
    mbar_init(&s_done, 1);
    mbar_init_fence();
    s_bad = 0;
  }
  if (warp == 9) tmem_alloc(&s_tmem, S::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's: they start at 0

  const Item it = item_of(tb, blockIdx.x, kRows);
  const int G = 1 << tb.g_shift, n = it.t1 - it.t0;
  // Two query tiles take every key tile each; a lone one has its key tiles
  // taken in turns by the two softmax groups, each with its own (m, l, O).
  const bool lone = it.rows <= kRows;
  const int ahead = lone ? 2 : 1;   // key tiles whose scores are under way
  const int first_pos = it.pos0 + (it.row0 >> tb.g_shift);
  // a key tile on the diagonal: some row of the block does not see all of it
  auto diagonal = [&](int t) { return t * kRows + kRows - 1 > first_pos; };

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == 8 && n > 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      const int nq = lone ? 1 : 2;
      mbar_arrive_expect(&s_q, (uint32_t)nq * S::kTile);
      for (int i = 0; i < nq; ++i)
        for (int c = 0; c < S::kBlocks; ++c)
          tensor_load_3d(sq + i * S::kTile + c * S::kBlock, &map_q, 64 * c, it.h * G,
                         it.q0 + ((it.row0 + i * kRows) >> tb.g_shift), &s_q);
    }
    const int32_t* bt = kp.bt + (int64_t)it.b * kp.max_pages;
    const int page_mask = (1 << kp.page_shift) - 1;
    bool ok = true;
    if (kp.page_shift >= 3) {
      // a box of min(P, 128) rows per lane; rows no token has, or on a page
      // outside the pool, are read outside the map, as zeros
      const int r_shift = min(kp.page_shift, 7), per = kRows >> r_shift;
      const int bx = lane & (per - 1), c = lane / per;
      const int none = (int)((kp.n_pages * tb.hkv) << kp.page_shift);
      auto page_at = [&](int j) {   // of this lane's box in key tile j (looked up tiles ahead of its use)
        const int key = (it.t0 + j) * kRows + (bx << r_shift);
        return j < n && key < it.key_end ? __ldg(bt + (key >> kp.page_shift)) : INT32_MAX;
      };
      auto row_at = [&](int j, int page) {
        const int key = (it.t0 + j) * kRows + (bx << r_shift);
        if (page >= 0 && page < kp.n_pages)
          return ((page * tb.hkv + it.h) << kp.page_shift) + (key & page_mask);
        if (j < n && key < it.key_end) flag_error(status, WI_DEV_BAD_PAGE);
        return none;
      };
      // unit u: K_0 .. K_(ahead - 1), then V_j, K_(j + ahead) in turns; a
      // tile's row is kept from its keys to its values
      int issued = 0, st = 0, page = page_at(2);
      int y0 = row_at(0, page_at(0)), y1 = row_at(1, page_at(1));
      uint32_t ph = 1;
      auto load = [&](const CUtensorMap* map, int row) {
        if (issued >= S::kStages) ok = __all_sync(0xffffffffu, mbar_wait(&s_empty[st], ph, status));
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect(&s_full[st], S::kTile);
        __syncwarp();
        if (c < S::kBlocks)
          tensor_load_2d(ring + (size_t)st * S::kTile + c * S::kBlock + (bx << r_shift) * 128, map, 64 * c, row, &s_full[st]);
        ++issued;
        if (++st == S::kStages) { st = 0; ph ^= 1; }
      };
      load(&map_k, y0);
      if (lone && n > 1) load(&map_k, y1);
      for (int j = 0; j < n && ok; ++j) {
        const int y2 = row_at(j + 2, page);
        page = page_at(j + 3);
        load(&map_v, y0);
        if (ok && j + ahead < n) load(&map_k, lone ? y2 : y1);
        y0 = y1;
        y1 = y2;
      }
      if (!ok)   // a wait gave up: no copy is left in flight when the CTA ends
        for (int u = max(0, issued - S::kStages); u < issued; ++u)
          mbar_wait(&s_full[u % S::kStages], (uint32_t)(u / S::kStages) & 1u, status);
    } else {
      // pages of fewer than 8 rows: 16-byte copies into the swizzled layout,
      // two units behind the one being issued
      constexpr int CH = D / 8, kLag = 2;
      auto arrive = [&](int u) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_full[u % S::kStages]);
      };
      int u = 0;
      for (; u < 2 * n && ok; ++u) {
        // the same order: past the first `ahead`, values at every other unit
        // until the keys have run out
        const int x = u - min(ahead, n), keys_left = 2 * (n - min(ahead, n));
        const bool val = x >= 0 && ((x & 1) == 0 || x >= keys_left);
        const int j = x < 0 ? u : x >= keys_left ? x - keys_left / 2 : val ? x / 2 : x / 2 + ahead;
        const int t = it.t0 + j, st = u % S::kStages;
        if (u >= S::kStages) ok = __all_sync(0xffffffffu, mbar_wait(&s_empty[st], (uint32_t)(u / S::kStages - 1) & 1u, status));
        if (!ok) break;
        const Pool& p = val ? vp : kp;
        unsigned char* dst = ring + (size_t)st * S::kTile;
#pragma unroll 4
        for (int i = lane; i < kRows * CH; i += 32) {
          const int r = i / CH, ch = i % CH, key = t * kRows + r;
          const int64_t row = key < it.key_end ? pool_row(p, tb.hkv, D, it.b, it.h, key, status) : -1;
          unsigned char* to = dst + (ch >> 3) * S::kBlock + swz128(r, ch & 7);
          if (row >= 0) cp_async16(to, reinterpret_cast<const T*>(p.base) + row + ch * 8);
          else *reinterpret_cast<uint4*>(to) = make_uint4(0u, 0u, 0u, 0u);
        }
        cp_async_commit();
        if (u >= kLag) {
          cp_async_wait<kLag>();
          arrive(u - kLag);
        }
      }
      cp_async_wait<0>();
      if (ok)
        for (int v = max(0, u - kLag); v < u; ++v) arrive(v);
    }
  } else if (warp == 9 && n > 0) {
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
        const uint64_t a = lone ? dq : dq + i * kStep, b = dk + st * kStep;
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
    auto output = [&](int i, int st, int half, bool first, bool last) {   // O_i += P_i V, half of the keys
      if (elect_one()) {
        const uint64_t b = dv + st * kStep;
#pragma unroll
        for (int kk = 0; kk < kRows / 32; ++kk) {
          const int k = half * (kRows / 32) + kk;
          umma_bf16_ts(tmem + S::kO + i * D, tmem + S::kS + i * 128 + k * 8, b + k * (2048 >> 4), kIdescO,
                       !first || kk != 0);
        }
        if (half == 1) {
          umma_commit(&s_o[i]);
          if (last) umma_commit(&s_empty[st]);
        }
      }
      __syncwarp();
    };
    int st = 0, fixes = 0;
    uint32_t ph = 0;
    auto full = [&]() { return mbar_wait(&s_full[st], ph, status); };   // the ring's next unit
    auto next = [&]() { if (++st == S::kStages) { st = 0; ph ^= 1; } };
    bool ok = mbar_wait(&s_q, 0, status) && full();
    tc_fence_after();
    if (ok) {
      scores(0, st, lone);
      if (!lone) scores(1, st, true);
      next();
      if (lone && n > 1 && (ok = full())) {
        tc_fence_after();
        scores(1, st, true);
        next();
      }
    }
    for (int j = 0; j < n && ok; ++j) {
      const bool fix = diagonal(it.t0 + j);
      if (!(ok = full())) break;   // V_j
      if (fix && lane == 0) mbar_arrive(&s_go);
      const int sv = st;
      next();
      const int i0 = lone ? j & 1 : 0, i1 = lone ? i0 : 1;
      const uint32_t pp = (uint32_t)(lone ? j >> 1 : j) & 1u;
      for (int i = i0; i <= i1; ++i) {
        ok = mbar_wait(&s_p[i][0], pp, status);
        if (ok && fix && i == i0) ok = mbar_wait(&s_fixed, (uint32_t)fixes++ & 1u, status);
        if (!ok) break;
        tc_fence_after();
        output(i, sv, 0, j < ahead, false);
        if (!(ok = mbar_wait(&s_p[i][1], pp, status))) break;
        tc_fence_after();
        output(i, sv, 1, false, i == i1);
        if (j + ahead < n) {
          if (i == i0 && !(ok = full())) break;   // K_(j + ahead)
          tc_fence_after();
          scores(i, st, i == i1);
        }
      }
      if (j + ahead < n) next();
    }
    // every MMA issued has completed before the columns are released
    if (elect_one()) umma_commit(&s_done);
    __syncwarp();
    mbar_wait(&s_done, 0, status);
  } else if (warp >= 10 && n > 0) {
    // ------------------------------------------- value tiles on the diagonal
    int fixes = 0;
    for (int j = max(0, (first_pos + 1) / kRows - it.t0); j < n; ++j) {   // first_pos + 1: the first masked key
      const int t = it.t0 + j;
      if (!__all_sync(0xffffffffu, mbar_wait(&s_go, (uint32_t)fixes++ & 1u, status))) break;
      // V_j's unit: `ahead` keys (all n, if fewer) came first, then one more with every value
      const int u = j + min(n, j + ahead);
      unsigned char* tile = ring + (size_t)(u % S::kStages) * S::kTile;
      constexpr int CH = D / 8;
      const int r0 = max(0, first_pos + 1 - t * kRows);    // the first row some query does not see
      const int r1 = min(kRows, it.key_end - t * kRows);   // the first row none sees
      bool bad = false;
      for (int i = r0 * CH + (tid - 320); i < kRows * CH; i += 64) {
        const int r = i / CH, ch = i % CH;
        uint4* at = reinterpret_cast<uint4*>(tile + (ch >> 3) * S::kBlock + swz128(r, ch & 7));
        if (r >= r1) {
          *at = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        uint4 x = *at;
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        bool found = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((w[e] & 0x7f80u) == 0x7f80u) { w[e] &= 0xffff0000u; found = true; }
          if ((w[e] & 0x7f800000u) == 0x7f800000u) { w[e] &= 0x0000ffffu; found = true; }
        }
        if (found) {
          *at = make_uint4(w[0], w[1], w[2], w[3]);
          bad = true;
        }
      }
      if (bad) atomicOr(&s_bad, 1u);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_fixed);
    }
  }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2, r = (lone ? 0 : i * kRows) + 32 * (warp & 3) + lane;
    const int pos = it.pos0 + ((it.row0 + r) >> tb.g_shift);
    const int warp_pos = __shfl_sync(0xffffffffu, pos, 0);
    const bool used = r - lane < it.rows;   // some row of the warp is real
    const int turns = lone ? (n - i + 1) >> 1 : n;   // its key tiles: all, or every other one from the i-th
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + S::kS + i * 128, to = tmem + lanes + S::kO + i * D;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    {
      for (int j = 0; j < turns && ok; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_s[i], (uint32_t)j & 1u, status));
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
          const int base = (it.t0 + (lone ? 2 * j + i : j)) * kRows;
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
          const bool up = !(top <= m + kRescale);
          if (__any_sync(0xffffffffu, up)) {
            const float mn = up ? top : m;
            const float c = up ? ex2(m - mn) : 1.f;
            l *= c;
            m = mn;
            if (j > 0) {   // O holds the keys before
              ok = __all_sync(0xffffffffu, mbar_wait(&s_o[i], (uint32_t)(j - 1) & 1u, status));
              tc_fence_after();
#pragma unroll
              for (int q = 0; q < D / 32; ++q) {
                uint32_t y[32];
                tmem_ld32_issue(to + 32 * q, y);
                tmem_wait_ld();
                tie32(y);
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * c);
                tmem_st32(to + 32 * q, y);
              }
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;
          const float2 sc = make_float2(scale, scale), nm = make_float2(-mu, -mu);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), sc, nm);
              const float2 w = e % kPoly == kPoly - 1 ? ex2_poly(y) : make_float2(ex2(y.x), ex2(y.y));
              sum[e & 1] = __fadd2_rn(sum[e & 1], w);
              p[e] = pack_bf16(w.x, w.y);
            }
            tmem_st16(ts + 16 * c, p);
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
      if (turns > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_o[i], (uint32_t)(turns - 1) & 1u, status));
    }
    tc_fence_after();
    // a lone query tile: group 1 hands its part over in the queries' memory
    // (every product that read them has completed), 16-byte chunks swizzled
    // by row
    float* row1 = reinterpret_cast<float*>(sq) + (32 * (warp & 3) + lane) * D;
    float c0 = 1.f, c1 = 0.f;
    if (lone) {
      if (i == 1 && used && turns > 0) {
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t y[32];
          tmem_ld32_issue(to + 32 * q, y);
          tmem_wait_ld();
          tie32(y);
          if (r < it.rows)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(row1 + 4 * ((8 * q + e) ^ (lane & 7))) =
                  make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        }
      }
      if (i == 1) s_ml[r] = make_float2(m, l);
      named_sync(1, 256);
      if (i == 0) {
        const float2 ml = s_ml[r];
        const float mn = fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.f : mn;
        c0 = ex2(m - mu);
        c1 = ex2(ml.x - mu);
        l = c0 * l + c1 * ml.y;
        m = mn;
      }
    }
    if (used && !(lone && i == 1)) {
      const int row = it.row0 + r;
      const int64_t tok = it.q0 + (row >> tb.g_shift);
      const int head = it.h * G + (row & (G - 1));
      const bool real = r < it.rows;
      const float inv = 1.f / l;
      if (real && it.part >= 0) ao.ml[it.part + r] = make_float2(m, l);
      else if (real && ao.lse) ao.lse[tok * ao.Hq + head] = kLn2 * (m + log2f(l));
      const bool give_back = *(volatile uint32_t*)&s_bad != 0;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t y[32];
        if (n > 0) {
          tmem_ld32_issue(to + 32 * q, y);
          tmem_wait_ld();
          tie32(y);
          if (lone && n > 1 && real)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 f = *reinterpret_cast<const float4*>(row1 + 4 * ((8 * q + e) ^ (lane & 7)));
              const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                y[4 * e + k] = __float_as_uint(fmaf(c1, v[k], c0 * __uint_as_float(y[4 * e + k])));
            }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = 0u;
        }
        if (give_back && real) {
          // values that are not finite, to the rows that see them (a positive
          // weight of them is they themselves)
          const int p1 = min(pos + 1, it.t1 * kRows);
          for (int p = max(first_pos + 1, it.t0 * kRows); p < p1; ++p) {
            const int64_t at = pool_row(vp, tb.hkv, D, it.b, it.h, p, status);
            if (at < 0) continue;
            const T* v = reinterpret_cast<const T*>(vp.base) + at + 32 * q;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float f = __bfloat162float(v[e]);
              if (!isfinite(f)) y[e] = __float_as_uint(__uint_as_float(y[e]) + f);
            }
          }
        }
        if (real && it.part >= 0) {
          float* o = ao.o + (it.part + r) * D + 32 * q;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(o + e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        } else if (real) {
          T* o = reinterpret_cast<T*>(ao.out) + tok * ao.stride + (int64_t)head * D + 32 * q;
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16(__uint_as_float(y[2 * e]) * inv, __uint_as_float(y[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<uint4*>(o + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
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

// cuTensorMapEncodeTiled through the runtime's driver entry point; null when
// unavailable
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

bool encode(CUtensorMap* tm, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const cuuint32_t one[3] = {1, 1, 1};
  auto fn = encode_fn();
  return fn && fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_typed(const AttendTable& tb, const AttendPlan& pl, const AttendArgs& a, const AttendOut& ao,
                         cudaStream_t s) {
  using S = UmmaShape<D>;
  CUtensorMap mq, mk, mv;
  // the queries of a group of heads as rows (token, head): 64 channels x G x 128 / G
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)pl.Hq, (cuuint64_t)pl.q_tokens};
  const cuuint64_t qs[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)pl.G, (cuuint32_t)(kRows / pl.G)};
  // the pools as rows of D channels; page boxes of at most 128 rows (for
  // pages of fewer than 8 rows the maps are not used)
  const cuuint64_t pd[2] = {(cuuint64_t)D, (cuuint64_t)((a.kp.n_pages * pl.hkv) << a.kp.page_shift)};
  const cuuint64_t ps[1] = {(cuuint64_t)D * 2};
  const cuuint32_t pb[2] = {64, (cuuint32_t)std::min(kRows, 1 << a.kp.page_shift)};
  if (!encode(&mq, 3, a.q, qd, qs, qb) || !encode(&mk, 2, a.kp.base, pd, ps, pb) ||
      !encode(&mv, 2, a.vp.base, pd, ps, pb))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<attend_umma_kernel<D>>(S::kSmem);
  if (e != cudaSuccess) return e;
  attend_umma_kernel<D><<<tb.n_items, kUThreads, S::kSmem, s>>>(
      tb, mq, mk, mv, a.kp, a.vp, ao, kLog2e / std::sqrt((float)D), reinterpret_cast<uint32_t*>(a.ws));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_umma(const AttendTable& tb, const AttendPlan& pl, const AttendArgs& a,
                               const AttendOut& ao, cudaStream_t s) {
  return pl.D == 128 ? launch_typed<128>(tb, pl, a, ao, s) : launch_typed<64>(tb, pl, a, ao, s);
}

}  // namespace wi
