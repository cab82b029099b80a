// Causal attention over the paged cache for blocks of at most 16 rows (bf16):
// single tokens and a few more, where every key is read for little work and
// the memory's rate is the bound.
//
// A CTA takes one item.  Warp 8 keeps a ring of 192 KB full of key and value
// tiles; warps 0..7 take 16 keys of each 128-key tile, with a running maximum,
// mass and output of their own (products as m16n8k16: the rows are the MMA's
// M, so the scores' accumulators are the weights' operand), and join them at
// the end.  A weight is the sum of two bf16 parts, each multiplied by the
// values, so 16 bits of it count, as in the decode over an index.  With up to
// eight rows (a token of a group of eight heads) the second parts are the
// operand's rows 8..15, so a tile takes as many products as with weights of
// one part (16 tokens over 32768 keys each: 357 us, as before; with products
// of their own 373, and even masked off 363: the clocks fall).  A tile
// costs a warp about 250 instructions, a third of the time its 64 KB take to
// arrive, and a stage is free as soon as eight warps have read it: the
// tensor-memory kernel holds its stages through a softmax of 128 rows, which
// leaves 96 KB in flight and 4.9 TB/s.  16 tokens over 32768 keys each, 8 KV
// heads of 128: 357 to 363 us a call back to back, 5.9 to 6.0 TB/s; one over
// 131072: 92 us, 6 of them the merge.
#include <cmath>
#include <type_traits>

#include "wi_attend_tiles.cuh"

namespace wi {
namespace {

constexpr int kFewRows = 16, kFewWarps = 8, kFewThreads = 32 * (kFewWarps + 1);
constexpr float kFewHead = 24.f;   // log2 of the reference's distance above the maximum it was set at (weights at most 1)

template <int D>
struct FewShape {
  static constexpr uint32_t kTile = kRows * D * 2, kBlock = kRows * 128;
  static constexpr int kStages = 192 * 1024 / kTile;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kTile;
};

// A value fragment word (keys `key` and `key` + 1 of one channel): keys no row
// sees are 0; what is not finite in keys only some rows see is taken out.
__device__ __forceinline__ uint32_t clean(uint32_t w, int key, int first_pos, int key_end, bool& bad) {
  const bool odd0 = key > first_pos && (w & 0x7f80u) == 0x7f80u;
  const bool odd1 = key + 1 > first_pos && (w & 0x7f800000u) == 0x7f800000u;
  bad |= (odd0 && key < key_end) || (odd1 && key + 1 < key_end);
  if (odd0 || key >= key_end) w &= 0xffff0000u;
  if (odd1 || key + 1 >= key_end) w &= 0x0000ffffu;
  return w;
}

template <int D, int N>
__global__ void __launch_bounds__(kFewThreads, 1)
attend_few_kernel(const __grid_constant__ AttendTable<N> tb, const __nv_bfloat16* __restrict__ q, int64_t q_stride,
                  const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const Pool kp, const Pool vp, const AttendOut ao, float scale, uint32_t* status) {
  using S = FewShape<D>;
  extern __shared__ unsigned char sh_raw[];
  unsigned char* ring = align_smem_1024(sh_raw);
  __shared__ __align__(8) uint64_t s_full[S::kStages], s_empty[S::kStages];
  __shared__ float2 s_ml[kFewWarps][kFewRows];
  __shared__ uint32_t s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  pdl_launch_dependents();
  const Item it = item_of(tb, blockIdx.x, kRows);
  if (it.t0 == it.t1) return;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kFewWarps);
    }
    mbar_init_fence();
    s_bad = 0;
  }
  const int G = 1 << tb.g_shift, n = it.t1 - it.t0;
  const int first_pos = it.pos0 + (it.row0 >> tb.g_shift);
  const bool narrow = it.rows <= kFewRows / 2;   // accumulator rows 8..15: the weights' second parts
  __syncthreads();
  if (warp == kFewWarps) {
    load_units<D, S::kStages>(it, tb.hkv, kp, vp, map_k, map_v, ring, s_full, s_empty, status);
    return;
  }

  // thread (g, t) of the warp's fragments: rows g and g + 8, columns 2 t, 2 t + 1
  const int g = lane >> 2, t2 = 2 * (lane & 3);
  auto q_row = [&](int r) {
    const int x = it.row0 + r;
    return q + (int64_t)(it.q0 + (x >> tb.g_shift)) * q_stride + (int64_t)(it.h * G + (x & (G - 1))) * D;
  };
  uint32_t qa[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = g + 8 * (e & 1), c = 16 * k + t2 + 8 * (e >> 1);
      qa[k][e] = r < it.rows ? __ldg(reinterpret_cast<const uint32_t*>(q_row(r) + c)) : 0u;
    }
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  int pos[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) pos[h] = it.pos0 + ((it.row0 + g + 8 * h) >> tb.g_shift);
#pragma unroll
  for (int c = 0; c < D / 8; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
  bool ok = true, bad = false;
  int st = 0;
  uint32_t ph = 0;
  auto full = [&]() { return __all_sync(0xffffffffu, wait_bar(&s_full[st], ph, status)) != 0; };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&s_empty[st]);
    if (++st == S::kStages) { st = 0; ph ^= 1; }
  };
  for (int j = 0; j < n; ++j) {
    if (!(ok = full())) break;
    const int base = (it.t0 + j) * kRows + 16 * warp;   // the warp's keys
    float s[2][4] = {};
    {
      const unsigned char* tile = ring + (size_t)st * S::kTile;
#pragma unroll
      for (int kb = 0; kb < D / 32; ++kb)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int chunk = 4 * kb + (lane >> 3);
          uint32_t b[4];
          ldsm_x4(b, tile + (chunk >> 3) * S::kBlock + swz128(16 * warp + 8 * nt + (lane & 7), chunk & 7));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t(&a)[4] = qa[2 * kb + e];
            mma_bf16_4(s[nt], a[0], a[1], a[2], a[3], b[2 * e], b[2 * e + 1]);
          }
        }
    }
    release();
    const bool diag = base + 15 > first_pos;
    if (diag) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (base + 8 * nt + t2 + (e & 1) > pos[e >> 1]) s[nt][e] = -INFINITY;
    }
    float top[2] = {-INFINITY, -INFINITY};
    bool up = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && narrow) break;
      float x = max3_nan(s[0][2 * h], s[0][2 * h + 1], max3_nan(s[1][2 * h], s[1][2 * h + 1], s[1][2 * h]));
#pragma unroll
      for (int y = 1; y <= 2; y <<= 1) {
        const float z = __shfl_xor_sync(0xffffffffu, x, y);
        x = max3_nan(x, z, z);
      }
      // a score that is NaN or +inf makes its row NaN
      x *= scale;
      top[h] = x < INFINITY ? x : NAN;
      up |= !(top[h] <= m[h]);
    }
    if (__any_sync(0xffffffffu, up)) {
      float c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mn = !(top[h] <= m[h]) ? top[h] + kFewHead : m[h];
        c[h] = mn == m[h] ? 1.f : ex2(m[h] - mn);
        m[h] = mn;
        l[h] *= c[h];
      }
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][e] *= e < 2 || narrow ? c[0] : c[1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && narrow) break;
      const float mu = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = s[nt][2 * h + e];
          x = ex2(fmaf(x, scale, -mu));
          l[h] += x;
        }
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; e += 2) split_bf16(s[e >> 1][0], s[e >> 1][1], hi[e], lo[e]);
    if (narrow) {
      hi[1] = lo[0];
      hi[3] = lo[2];
    } else {
#pragma unroll
      for (int e = 1; e < 4; e += 2) split_bf16(s[e >> 1][2], s[e >> 1][3], hi[e], lo[e]);
    }
    if (!(ok = full())) break;
    auto output = [&](auto second) {   // (a branch a product would leave the second ones in the pipe, masked)
      const unsigned char* tile = ring + (size_t)st * S::kTile;
      const int row = 16 * warp + (lane & 15);
#pragma unroll
      for (int cb = 0; cb < D / 16; ++cb) {
        const int chunk = 2 * cb + (lane >> 4);
        uint32_t b[4];
        ldsm_x4_t(b, tile + (chunk >> 3) * S::kBlock + swz128(row, chunk & 7));
        if (diag) {
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = clean(b[e], base + t2 + 8 * (e & 1), first_pos, it.key_end, bad);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma_bf16_4(o[2 * cb + e], hi[0], hi[1], hi[2], hi[3], b[2 * e], b[2 * e + 1]);
          if (second) mma_bf16_4(o[2 * cb + e], lo[0], lo[1], lo[2], lo[3], b[2 * e], b[2 * e + 1]);
        }
      }
    };
    if (narrow) output(std::false_type{});
    else output(std::true_type{});
    release();
  }
  if (narrow) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) o[c][e] += o[c][e + 2];
  }
  // join the warps' parts in the ring's memory (every unit has been read)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if ((lane & 3) == 0) s_ml[warp][g + 8 * h] = make_float2(m[h], l[h]);
  }
  if (bad) atomicOr(&s_bad, 1u);
  named_sync(1, 32 * kFewWarps);
  float* so = reinterpret_cast<float*>(ring);   // [warps][rows][D]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    if (r >= it.rows) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) mx = fmaxf(mx, s_ml[w][r].x);
    const float f = ex2(m[h] - (mx == -INFINITY ? 0.f : mx));
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      *reinterpret_cast<float2*>(so + (warp * kFewRows + r) * D + 8 * c + t2) =
          make_float2(o[c][2 * h] * f, o[c][2 * h + 1] * f);
  }
  named_sync(1, 32 * kFewWarps);
  for (int x = tid; x < it.rows * (D / 4); x += 32 * kFewWarps) {
    const int r = x / (D / 4), col = 4 * (x % (D / 4)), row = it.row0 + r;
    float mx = -INFINITY, mass = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) mx = fmaxf(mx, s_ml[w][r].x);
    const float mu = mx == -INFINITY ? 0.f : mx;
    float v[4] = {};
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      mass = fmaf(ex2(s_ml[w][r].x - mu), s_ml[w][r].y, mass);
      const float4 f = *reinterpret_cast<const float4*>(so + (w * kFewRows + r) * D + col);
      v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    }
    // A value that is not finite, under a positive weight, is all there is to
    // its column: those taken out on the diagonal, and where the sum is not
    // finite, the others too (a weight's second part, 0 or negative, makes NaN
    // of an infinity).  A row whose mass is NaN is NaN whatever they are.
    const bool lost = mass == mass && !(isfinite(v[0]) && isfinite(v[1]) && isfinite(v[2]) && isfinite(v[3]));
    if (s_bad || lost) {
      const int p1 = min(it.pos0 + (row >> tb.g_shift) + 1, it.t1 * kRows);
      float odd[4] = {};
      uint32_t found = 0;
#pragma unroll 1
      for (int p = max(lost ? 0 : first_pos + 1, it.t0 * kRows); p < p1; ++p) {
        const int64_t at = pool_row(vp, tb.hkv, D, it.b, it.h, p, status);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = at < 0 ? 0.f : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(vp.base)[at + col + e]);
          if (!isfinite(f)) {
            odd[e] += f;
            found |= 1u << e;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((found >> e) & 1u) v[e] = odd[e];
    }
    if (it.part >= 0) {
      if (col == 0) ao.ml[it.part + r] = make_float2(mx, mass);
      *reinterpret_cast<float4*>(ao.o + (it.part + r) * D + col) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      const int64_t tok = it.q0 + (row >> tb.g_shift);
      const int head = it.h * G + (row & (G - 1));
      if (col == 0 && ao.lse) ao.lse[tok * ao.Hq + head] = kLn2 * (mx + log2f(mass));
      const float inv = 1.f / mass;
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(ao.out) + tok * ao.stride + (int64_t)head * D + col) =
          make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
    }
  }
}

template <int D, int N>
cudaError_t launch_typed(const AttendTable<N>& tb, const AttendPlan& pl, const AttendArgs& a, const AttendOut& ao,
                         cudaStream_t s) {
  using S = FewShape<D>;
  CUtensorMap mk, mv;
  if (!encode_pools(&mk, &mv, a, pl.hkv, D)) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<attend_few_kernel<D, N>>(S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_kernel(attend_few_kernel<D, N>, dim3(tb.n_items), kFewThreads, S::kSmem, s, false, tb,
                       static_cast<const __nv_bfloat16*>(a.q), a.q_stride, mk, mv, a.kp, a.vp, ao,
                       kLog2e / std::sqrt((float)D), reinterpret_cast<uint32_t*>(a.ws));
}

}  // namespace

template <int N>
cudaError_t launch_attend_few(const AttendTable<N>& tb, const AttendPlan& pl, const AttendArgs& a,
                             const AttendOut& ao, cudaStream_t s) {
  return pl.D == 128 ? launch_typed<128>(tb, pl, a, ao, s) : launch_typed<64>(tb, pl, a, ao, s);
}
template cudaError_t launch_attend_few(const AttendTable<kFewSeqs>&, const AttendPlan&, const AttendArgs&,
                                      const AttendOut&, cudaStream_t);
template cudaError_t launch_attend_few(const AttendTable<kMaxBatch>&, const AttendPlan&, const AttendArgs&,
                                      const AttendOut&, cudaStream_t);

}  // namespace wi
