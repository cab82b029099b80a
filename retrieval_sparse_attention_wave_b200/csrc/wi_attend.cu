// Causal attention of packed queries over the paged cache (wi_attend).
//
// Row r of a block holds a query q_r at position pos_r; over the key tiles
// t = 0, 1, ... its running maximum, mass and output
//   m' = max(m, max_k s_rk),  c = 2^(m - m'),
//   l' = c l + sum_k 2^(s_rk - m'),  o' = c o + sum_k 2^(s_rk - m') v_k
// (s in units of log2 e / sqrt(d); s_rk = -inf for k > pos_r) end as
// out = o / l and lse = ln2 (m + log2 l): one pass over the keys, nothing of
// size queries x keys in memory.  Key runs of a split block end as parts
// (m, l, o), which attend_merge_kernel joins by the same rule.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "wi_attend.cuh"

namespace wi {
namespace {

// ------------------------------------------------- fp32, on packed FMAs
// 128 threads, 16 of them (half a warp) share a row group of RT rows: each
// takes every 16th key of a tile and every 16th 16-byte chunk of the output
// columns, so a row's statistics and weights stay inside its half warp.
// Products run on packed fp32 FMAs (two head channels at a time).  Bound by
// issue: a tile of 64 x 64 (D = 64) is 2048 packed FMAs a thread, 4096 clocks
// of the FMA pipe, and takes about 8000 with its shared-memory reads, powers
// and four barriers at 2 to 3 warps a scheduler.  42 TFLOP/s at 8192 tokens,
// 32 heads on 8 KV heads of 128 (13.1 ms); 4096 tokens, one head of 64: 82 us.
// A block of at most 16 rows keeps two rows a thread, for more CTAs an SM.
template <int D, int RT>
struct FmaShape {
  static constexpr int kThreads = 128;
  static constexpr int R = 8 * RT;
  static constexpr int KT = D == 128 ? 32 : 64;
  static constexpr int KPT = KT / 16;      // keys per thread
  static constexpr int CPT = D / 64;       // 16-byte output chunks per thread
  static constexpr int LD = D + 4;         // padded row: 8 rows on 8 different bank groups
  static constexpr int PLD = KT + 4;
  static constexpr size_t kSmem = (size_t)(R * LD + 2 * KT * LD + R * PLD) * 4 + 2 * KT * 8;
};

template <int D, int RT, int N>
__global__ void __launch_bounds__(128)
attend_fma_kernel(const __grid_constant__ AttendTable<N> tb, const float* __restrict__ q_, int64_t q_stride,
                  const Pool kp, const Pool vp, const AttendOut ao, float scale, uint32_t* status) {
  using S = FmaShape<D, RT>;
  extern __shared__ __align__(16) float sh_fma[];
  float* sq = sh_fma;
  float* sk = sq + S::R * S::LD;
  float* sv = sk + S::KT * S::LD;
  float* sp = sv + S::KT * S::LD;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  pdl_launch_dependents();
  const Item it = item_of(tb, blockIdx.x, S::KT);
  if (it.t0 == it.t1) return;
  const int G = 1 << tb.g_shift;
  constexpr int CH = D / 4;   // 16-byte chunks of a row

  // Element offsets of a tile's rows in the pools (-1: no token's row), by a
  // thread each, for two tiles; the page of the next one is looked up while a
  // tile is worked on.
  int64_t* srow = reinterpret_cast<int64_t*>(sp + S::R * S::PLD);
  auto page_of = [&](int t) {
    const int key = t * S::KT + tid;
    return tid < S::KT && t < it.t1 && key < it.key_end
               ? __ldg(kp.bt + (int64_t)it.b * kp.max_pages + (key >> kp.page_shift)) : -1;
  };
  auto set_rows = [&](int t, int page) {
    const int key = t * S::KT + tid;
    if (tid < S::KT && t < it.t1)
      srow[(t & 1) * S::KT + tid] = key < it.key_end ? pool_row_pg(kp, tb.hkv, D, it.h, key, page, status) : -1;
  };
  // the rows of tile t from a pool into shared memory; zeros where there is none
  auto load_tile = [&](const Pool& p, float* dst, int t) {
    constexpr int kPerPass = 128 / CH;
#pragma unroll 4
    for (int r = tid / CH; r < S::KT; r += kPerPass) {
      const int64_t row = srow[(t & 1) * S::KT + r];
      float* to = dst + r * S::LD + (tid % CH) * 4;
      if (row >= 0) cp_async16(to, reinterpret_cast<const float*>(p.base) + row + (tid % CH) * 4);
      else *reinterpret_cast<float4*>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    cp_async_commit();
  };

  int page = page_of(it.t0 + 1);
  set_rows(it.t0, page_of(it.t0));
  __syncthreads();
  if (it.t0 < it.t1) load_tile(kp, sk, it.t0);
  for (int c = tid; c < S::R * CH; c += 128) {
    const int r = c / CH, ch = c % CH;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < it.rows) {
      const int row = it.row0 + r;
      x = *reinterpret_cast<const float4*>(q_ + (int64_t)(it.q0 + (row >> tb.g_shift)) * q_stride +
                                           (int64_t)(it.h * G + (row & (G - 1))) * D + ch * 4);
    }
    *reinterpret_cast<float4*>(sq + r * S::LD + ch * 4) = make_float4(x.x * scale, x.y * scale, x.z * scale, x.w * scale);
  }
  float m[RT], l[RT];
  float4 o[RT][S::CPT];
  int pos[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    pos[i] = it.pos0 + ((it.row0 + ty * RT + i) >> tb.g_shift);
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int first_pos = it.pos0 + (it.row0 >> tb.g_shift);

  for (int t = it.t0; t < it.t1; ++t) {
    const int base = t * S::KT;
    load_tile(vp, sv, t);
    set_rows(t + 1, page);
    page = page_of(t + 2);
    cp_async_wait<1>();
    __syncthreads();
    float s[RT][S::KPT];
    {
      float2 a[RT][S::KPT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < S::KPT; ++j) a[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < D / 4; ++c) {
        float4 kk[S::KPT];
#pragma unroll
        for (int j = 0; j < S::KPT; ++j) kk[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * S::LD + 4 * c);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float4 qq = *reinterpret_cast<const float4*>(sq + (ty * RT + i) * S::LD + 4 * c);
#pragma unroll
          for (int j = 0; j < S::KPT; ++j) {
            a[i][j] = __ffma2_rn(make_float2(qq.x, qq.y), make_float2(kk[j].x, kk[j].y), a[i][j]);
            a[i][j] = __ffma2_rn(make_float2(qq.z, qq.w), make_float2(kk[j].z, kk[j].w), a[i][j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < S::KPT; ++j) s[i][j] = a[i][j].x + a[i][j].y;
    }
    __syncthreads();   // the key tile is free
    if (t + 1 < it.t1) load_tile(kp, sk, t + 1);
    else cp_async_commit();
    const bool diag = base + S::KT - 1 > first_pos;   // some row does not see all of the tile
    if (diag) {
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < S::KPT; ++j)
          if (base + tx + 16 * j > pos[i]) s[i][j] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float mx = s[i][0];
#pragma unroll
      for (int j = 1; j < S::KPT; ++j) mx = fmaxf(mx, s[i][j]);
#pragma unroll
      for (int x = 8; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[i], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: weights 0, not NaN
      const float c = exp2f(m[i] - mu);
      m[i] = mn;
      l[i] *= c;
#pragma unroll
      for (int j = 0; j < S::KPT; ++j) {
        const float p = exp2f(s[i][j] - mu);
        l[i] += p;
        sp[(ty * RT + i) * S::PLD + tx + 16 * j] = p;
      }
#pragma unroll
      for (int cc = 0; cc < S::CPT; ++cc) {
        o[i][cc].x *= c; o[i][cc].y *= c; o[i][cc].z *= c; o[i][cc].w *= c;
      }
    }
    cp_async_wait<1>();
    __syncthreads();   // the value tile and the weights are there
    // a masked weight is 0, but 0 * NaN is not: on the diagonal the masked
    // keys are left out of the sum instead of added with weight 0
    auto accumulate = [&](auto masked) {
#pragma unroll 2
      for (int k = 0; k < S::KT; k += 4) {
        float4 p[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (ty * RT + i) * S::PLD + k);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int cc = 0; cc < S::CPT; ++cc) {
            const float4 v = *reinterpret_cast<const float4*>(sv + (k + u) * S::LD + 4 * (tx + 16 * cc));
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              const float w = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
              if (masked && base + k + u > pos[i]) continue;
              float2 lo = make_float2(o[i][cc].x, o[i][cc].y), hi = make_float2(o[i][cc].z, o[i][cc].w);
              lo = __ffma2_rn(make_float2(w, w), make_float2(v.x, v.y), lo);
              hi = __ffma2_rn(make_float2(w, w), make_float2(v.z, v.w), hi);
              o[i][cc] = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
          }
        }
      }
    };
    if (diag) accumulate(std::true_type{});
    else accumulate(std::false_type{});
    __syncthreads();   // the value tile and the weights are free
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int x = 8; x >= 1; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    const int r = ty * RT + i;
    if (r >= it.rows) continue;
    if (it.part >= 0) {
      if (tx == 0) ao.ml[it.part + r] = make_float2(m[i], l[i]);
#pragma unroll
      for (int cc = 0; cc < S::CPT; ++cc)
        *reinterpret_cast<float4*>(ao.o + (it.part + r) * D + 4 * (tx + 16 * cc)) = o[i][cc];
    } else {
      const int row = it.row0 + r;
      const int64_t tok = it.q0 + (row >> tb.g_shift);
      const int head = it.h * G + (row & (G - 1));
      if (tx == 0 && ao.lse) ao.lse[tok * ao.Hq + head] = kLn2 * (m[i] + log2f(l[i]));
      float* to = reinterpret_cast<float*>(ao.out) + tok * ao.stride + (int64_t)head * D;
      const float inv = 1.f / l[i];
#pragma unroll
      for (int cc = 0; cc < S::CPT; ++cc)
        *reinterpret_cast<float4*>(to + 4 * (tx + 16 * cc)) =
            make_float4(o[i][cc].x * inv, o[i][cc].y * inv, o[i][cc].z * inv, o[i][cc].w * inv);
    }
  }
}

// ------------------------------------------------------------------ merge
// The parts' (m, l) of a query row of a split sequence give the weights
// 2^(m_s - m); the parts' outputs are added in order.
constexpr int kMergeWarps = 4;
constexpr int kMergeLanes = 8;   // of a row, where rows are many
constexpr int kMergeRows = 32 * kMergeWarps / kMergeLanes;

struct MergeRow {
  int64_t part, tok;   // its first part (the next one Rb rows on), its token
  uint32_t Rb;
  int ns, head;
};

template <int N>
__device__ inline MergeRow merge_row(const AttendTable<N>& tb, int x) {
  int lo = 0, hi = tb.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.seq[mid].mrow0 <= x) lo = mid; else hi = mid - 1;
  }
  const AttendSeq& s = tb.seq[lo];
  const uint32_t all = (uint32_t)s.n << tb.g_shift, Rb = min((uint32_t)tb.rows, all);
  const uint32_t in = (uint32_t)(x - s.mrow0), h = in / all, row = in - h * all;
  const uint32_t blk = row / (uint32_t)tb.rows, rr = row - blk * tb.rows;
  // its block's runs
  const uint32_t last = min((blk + 1) * (uint32_t)tb.rows, all) - 1;
  const uint32_t tiles = ((uint32_t)(s.T - s.n) + (last >> tb.g_shift) + tb.keys) / tb.keys;   // (of the keys its last row sees)
  MergeRow r;
  r.part = s.part0 + ((int64_t)blk * tb.hkv + h) * s.ns * Rb + rr;
  r.tok = s.q0 + (row >> tb.g_shift);
  r.Rb = Rb;
  r.ns = (int)((tiles + s.run - 1) / s.run);
  r.head = (int)(h << tb.g_shift) + (int)(row & ((1u << tb.g_shift) - 1));
  return r;
}

__device__ inline void store4(float* to, float4 f) { *reinterpret_cast<float4*>(to) = f; }
__device__ inline void store4(__nv_bfloat16* to, float4 f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f.x, f.y), b = __floats2bfloat162_rn(f.z, f.w);
  *reinterpret_cast<uint2*>(to) = make_uint2(reinterpret_cast<const uint32_t&>(a), reinterpret_cast<const uint32_t&>(b));
}

// Many rows: eight lanes a row, so that a warp has four rows' loads in flight
// and looks up four rows at once.
template <typename T, int D, int N>
__global__ void __launch_bounds__(32 * kMergeWarps)
attend_merge_rows_kernel(const __grid_constant__ AttendTable<N> tb, int n_rows, const AttendOut ao) {
  constexpr int C = D / (4 * kMergeLanes);   // quads of columns per lane
  const int sub = threadIdx.x & (kMergeLanes - 1);
  const int x = (int)blockIdx.x * kMergeRows + (int)threadIdx.x / kMergeLanes;
  MergeRow r = merge_row(tb, min(x, n_rows - 1));
  if (x >= n_rows) r.ns = 0;   // (its lanes stay for the shuffles)
  const int ns_warp = (int)__reduce_max_sync(0xffffffffu, (unsigned)r.ns);
  pdl_wait();   // the parts are there
  const float2* ml = ao.ml + r.part;
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 mine = sub < r.ns ? __ldcg(ml + (int64_t)sub * r.Rb) : none;
  float m = mine.x;
  for (int i = sub + kMergeLanes; i < r.ns; i += kMergeLanes)
    m = fmaxf(m, __ldcg(ml + (int64_t)i * r.Rb).x);
#pragma unroll
  for (int k = 1; k < kMergeLanes; k *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < ns_warp; i0 += kMergeLanes) {
    const int at = i0 + sub;
    const float2 f = i0 == 0 ? mine : at < r.ns ? __ldcg(ml + (int64_t)at * r.Rb) : none;
    const float w = at < r.ns ? exp2f(f.x - mu) : 0.f;
    l = fmaf(w, f.y, l);
    const int n = min(kMergeLanes, ns_warp - i0);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i, kMergeLanes);
      if (i0 + i < r.ns) {
        const float4* from = reinterpret_cast<const float4*>(ao.o + (r.part + (int64_t)(i0 + i) * r.Rb) * D) + sub;
        float4 v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = __ldcg(from + kMergeLanes * c);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          o[c].x = fmaf(wi, v[c].x, o[c].x);
          o[c].y = fmaf(wi, v[c].y, o[c].y);
          o[c].z = fmaf(wi, v[c].z, o[c].z);
          o[c].w = fmaf(wi, v[c].w, o[c].w);
        }
      }
    }
  }
#pragma unroll
  for (int k = 1; k < kMergeLanes; k *= 2) l += __shfl_xor_sync(0xffffffffu, l, k);
  if (x >= n_rows) return;
  if (sub == 0 && ao.lse) ao.lse[r.tok * ao.Hq + r.head] = kLn2 * (m + log2f(l));
  const float inv = 1.f / l;
  T* to = reinterpret_cast<T*>(ao.out) + r.tok * ao.stride + (int64_t)r.head * D + 4 * sub;
#pragma unroll
  for (int c = 0; c < C; ++c)
    store4(to + 4 * kMergeLanes * c, make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv));
}

// Few rows (single tokens): a CTA per row, whose four warps take every fourth
// part and add up in a fixed order.
template <typename T, int D, int N>
__global__ void __launch_bounds__(32 * kMergeWarps)
attend_merge_kernel(const __grid_constant__ AttendTable<N> tb, const AttendOut ao) {
  constexpr int E = D / 32;   // columns per lane
  __shared__ float s_o[kMergeWarps][D], s_l[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  const MergeRow r = merge_row(tb, (int)blockIdx.x);
  pdl_wait();   // the parts are there
  float m = -INFINITY;
  for (int i = lane; i < r.ns; i += 32) m = fmaxf(m, __ldcg(&ao.ml[r.part + (int64_t)i * r.Rb]).x);
  m = warp_max(m);
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  // parts warp, warp + kMergeWarps, ..., 32 of them at a time
  for (int i0 = warp; i0 < r.ns; i0 += 32 * kMergeWarps) {
    float w = 0.f;
    if (i0 + kMergeWarps * lane < r.ns) {
      const float2 ml = __ldcg(&ao.ml[r.part + (int64_t)(i0 + kMergeWarps * lane) * r.Rb]);
      w = exp2f(ml.x - mu);
      l = fmaf(w, ml.y, l);
    }
    const int n = min(32, (r.ns - i0 + kMergeWarps - 1) / kMergeWarps);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* from = ao.o + (r.part + (int64_t)(i0 + kMergeWarps * i) * r.Rb) * D + lane * E;
      float v[E];
      if constexpr (E == 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(from));
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      } else {
        const float2 f = __ldcg(reinterpret_cast<const float2*>(from));
        v[0] = f.x; v[1] = f.y;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(wi, v[e], o[e]);
    }
  }
  l = warp_sum(l);
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (warp != 0) return;
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
#pragma unroll
  for (int e = 0; e < E; ++e)
    o[e] = (s_o[0][lane * E + e] + s_o[1][lane * E + e]) + (s_o[2][lane * E + e] + s_o[3][lane * E + e]);
  if (lane == 0 && ao.lse) ao.lse[r.tok * ao.Hq + r.head] = kLn2 * (m + log2f(l));
  const float inv = 1.f / l;
  T* to = reinterpret_cast<T*>(ao.out) + r.tok * ao.stride + (int64_t)r.head * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) store_elem(to + e, o[e] * inv);
}

inline int log2_of(int x) { int r = 0; while ((1 << r) < x) ++r; return r; }

template <int D, int RT, int N>
cudaError_t launch_fma(const AttendTable<N>& tb, const AttendArgs& a, const AttendOut& ao, cudaStream_t s) {
  using S = FmaShape<D, RT>;
  const cudaError_t e = allow_smem<attend_fma_kernel<D, RT, N>>(S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attend_fma_kernel<D, RT, N>, dim3(tb.n_items), S::kThreads, S::kSmem, s, false, tb,
                       static_cast<const float*>(a.q), a.q_stride, a.kp, a.vp, ao, kLog2e / std::sqrt((float)D),
                       reinterpret_cast<uint32_t*>(a.ws));
}

template <typename T, int D, int N>
cudaError_t launch_merge(const AttendTable<N>& tb, int n_rows, const AttendOut& ao, cudaStream_t s) {
  if (n_rows <= 16 * 148)   // one wave of CTAs
    return launch_kernel(attend_merge_kernel<T, D, N>, dim3((unsigned)n_rows), 32 * kMergeWarps, 0, s, true, tb, ao);
  const dim3 grid((unsigned)((n_rows + kMergeRows - 1) / kMergeRows));
  return launch_kernel(attend_merge_rows_kernel<T, D, N>, grid, 32 * kMergeWarps, 0, s, true, tb, n_rows, ao);
}

}  // namespace

// One shape a call, by its largest sequence: a chunk among single tokens puts
// them in blocks of its size (16 tokens over 32768 keys and a chunk of 512: 745
// us; in two calls 375 and 248).
// bf16: 256 rows a block where some sequence has more than a tile of 128.  A
// tile takes about 2850 clocks; an item's queries, pipeline fill and output
// 3.5 times that, a part of 256 rows (133 KB) and its merge 3 times.
// fp32: 64 rows, or 16 where no block has more to fill.  An item's fixed part
// (about 5 us) is two tiles of 64 rows, or six of 16.
// Split items: over 60000 drawn calls of up to 256 sequences and 300000 tokens
// the rule alone chose up to 3200 of 16 rows, 2020 of 128 or 256, 14848 and
// 12548 (fp32); the bounds are a little above those (bf16, d = 128: a workspace
// of at most 34 and 315 MB).
AttendShape attend_shape(int dtype, int D, int most) {
  if (dtype == WI_BF16) {
    if (most <= 16) return AttendShape{16, 128, 148, 2.0, 0.2, 4096};
    const int rows = most <= 128 ? 128 : 256;
    return AttendShape{rows, 128, 148, 3.5, 3.0 * rows / 256, 2368};
  }
  if (most <= 16) return AttendShape{16, D == 128 ? 32 : 64, 4 * 148, 6.0, 1.0, 16384};
  return AttendShape{64, D == 128 ? 32 : 64, (D == 128 ? 2 : 3) * 148, 2.0, 0.5, 13312};
}

namespace {

template <int N>
cudaError_t launch_with(const AttendPlan& pl, const AttendArgs& a, cudaStream_t s) {
  AttendTable<N> tb;
  tb.n_seq = pl.n_seq; tb.n_items = pl.n_items; tb.hkv = pl.hkv;
  tb.g_shift = log2_of(pl.G); tb.rows = pl.rows; tb.keys = pl.keys;
  std::copy(pl.seq, pl.seq + pl.n_seq, tb.seq);
  const AttendOut ao{a.out, a.lse, reinterpret_cast<float2*>(a.ws + pl.off_ml),
                     reinterpret_cast<float*>(a.ws + pl.off_o), a.out_stride, pl.Hq};
  const bool wide = pl.D == 128;
  cudaError_t e;
  if (pl.dtype == WI_BF16)
    e = pl.rows == 16 ? launch_attend_few(tb, pl, a, ao, s) : launch_attend_umma(tb, pl, a, ao, s);
  else if (pl.rows == 16) e = wide ? launch_fma<128, 2>(tb, a, ao, s) : launch_fma<64, 2>(tb, a, ao, s);
  else e = wide ? launch_fma<128, 8>(tb, a, ao, s) : launch_fma<64, 8>(tb, a, ao, s);
  if (e != cudaSuccess || pl.n_merge_rows == 0) return e;
  if (pl.dtype == WI_BF16)
    return wide ? launch_merge<__nv_bfloat16, 128>(tb, pl.n_merge_rows, ao, s)
                : launch_merge<__nv_bfloat16, 64>(tb, pl.n_merge_rows, ao, s);
  return wide ? launch_merge<float, 128>(tb, pl.n_merge_rows, ao, s)
              : launch_merge<float, 64>(tb, pl.n_merge_rows, ao, s);
}

}  // namespace

cudaError_t launch_attend(const AttendPlan& pl, const AttendArgs& a, cudaStream_t s) {
  return pl.n_seq <= kFewSeqs ? launch_with<kFewSeqs>(pl, a, s) : launch_with<kMaxBatch>(pl, a, s);
}

}  // namespace wi
