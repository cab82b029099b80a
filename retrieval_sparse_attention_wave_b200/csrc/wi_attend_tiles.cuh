// The bf16 attention kernels' tiles: 128 keys of a KV head brought from the
// paged pools into a ring of shared-memory stages in the 128-byte-swizzled
// layout (blocks of 64 channels: 128 rows of 128 bytes), their bounded waits
// and their tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "wi_attend.cuh"

namespace wi {

constexpr int kRows = 128;   // keys of a tile (and rows of a query tile)

// A bounded wait for a barrier's phase that stays a loop in the code (the
// compiler unrolls the shared one: a kilobyte a wait, and these kernels' many
// roles then miss the instruction cache).
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, uint32_t* status) {
  const uint32_t b = smem_addr(bar);
  if (try_bar(b, parity)) return true;
#pragma unroll 1
  for (uint32_t i = 0; i < kSpinLimit; ++i)
    if (try_bar(b, parity)) return true;
  atomicOr(status, WI_DEV_TIMEOUT);
  return false;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// the largest of three, NaN if one is NaN
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A 16-byte asynchronous copy, or 16 bytes of zeros with nothing read.
__device__ __forceinline__ void cp_async16_or_zero(void* smem, const void* gmem, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(smem)), "l"(gmem), "r"(copy ? 16 : 0)
               : "memory");
}

// One warp loads an item's key and value tiles in the order K_0, V_0, K_1, V_1,
// ... (unit u into stage u % kStages): a tensor copy per page and 64 channels.
template <int D, int kStages>
__device__ __forceinline__ void load_units(const Item& it, int hkv, const Pool& kp, const Pool& vp,
                                           const CUtensorMap& map_k, const CUtensorMap& map_v,
                                           unsigned char* ring, uint64_t* s_full, uint64_t* s_empty,
                                           uint32_t* status) {
  constexpr uint32_t kTile = kRows * D * 2, kBlock = kRows * 128;
  const int lane = threadIdx.x & 31, n = it.t1 - it.t0;
  const int32_t* bt = kp.bt + (int64_t)it.b * kp.max_pages;
  const int page_mask = (1 << kp.page_shift) - 1;
  bool ok = true;
  if (kp.page_shift >= 3) {
    // a box of min(P, 128) rows per lane; rows no token has, or on a page
    // outside the pool, are read outside the map, as zeros
    const int r_shift = min(kp.page_shift, 7), per = kRows >> r_shift;
    const int bx = lane & (per - 1), c = lane / per;
    const int none = (int)((kp.n_pages * hkv) << kp.page_shift);
    auto page_at = [&](int t) {
      const int key = t * kRows + (bx << r_shift);
      return key < it.key_end && t < it.t1 ? __ldg(bt + (key >> kp.page_shift)) : -1;
    };
    int page = page_at(it.t0), issued = 0;
    for (int j = 0; j < n && ok; ++j) {
      const int t = it.t0 + j, key = t * kRows + (bx << r_shift);
      int y = none;
      if (key < it.key_end) {
        if (page >= 0 && page < kp.n_pages)
          y = ((page * hkv + it.h) << kp.page_shift) + (key & page_mask);
        else
          flag_error(status, WI_DEV_BAD_PAGE);
      }
      page = page_at(t + 1);
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int u = 2 * j + kv, st = u % kStages;
        if (u >= kStages) ok = __all_sync(0xffffffffu, wait_bar(&s_empty[st], (uint32_t)(u / kStages - 1) & 1u, status));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect(&s_full[st], kTile);
        __syncwarp();
        if (c < D / 64)
          tensor_load_2d(ring + (size_t)st * kTile + c * kBlock + (bx << r_shift) * 128,
                         kv ? &map_v : &map_k, 64 * c, y, &s_full[st]);
        issued = u + 1;
      }
    }
    if (!ok)   // a wait gave up: no copy is left in flight when the CTA ends
      for (int u = max(0, issued - kStages); u < issued; ++u)
        wait_bar(&s_full[u % kStages], (uint32_t)(u / kStages) & 1u, status);
  } else {
    // pages of fewer than 8 rows: 16-byte copies into the swizzled layout,
    // arriving two units behind the one being issued.  Lane l looks up rows l,
    // l + 32, l + 64 and l + 96 of a tile, a tile ahead; the copies of a row
    // get its place by a shuffle.  One warp's issue bounds it: 8192 tokens on
    // pages of one take 743 us, of 16 (tensor copies) 449.
    constexpr int CH = D / 8, kLag = 2;
    auto arrive = [&](int u) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_full[u % kStages]);
    };
    auto key_of = [&](int j, int i) { return (it.t0 + j) * kRows + 32 * i + lane; };
    auto page_at = [&](int j, int i) {
      return j < n && key_of(j, i) < it.key_end ? __ldg(bt + (key_of(j, i) >> kp.page_shift)) : -1;
    };
    int page[4], u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) page[i] = page_at(0, i);
    for (int j = 0; j < n && ok; ++j) {
      int y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key_of(j, i);
        y[i] = -1;
        if (key < it.key_end) {
          if (page[i] >= 0 && page[i] < kp.n_pages)
            y[i] = ((page[i] * hkv + it.h) << kp.page_shift) + (key & page_mask);
          else
            flag_error(status, WI_DEV_BAD_PAGE);
        }
        page[i] = page_at(j + 1, i);
      }
      for (int kv = 0; kv < 2 && ok; ++kv, ++u) {
        const int st = u % kStages;
        if (u >= kStages)
          ok = __all_sync(0xffffffffu, wait_bar(&s_empty[st], (uint32_t)(u / kStages - 1) & 1u, status));
        if (!ok) break;
        const int ch = lane % CH;
        const __nv_bfloat16* base = reinterpret_cast<const __nv_bfloat16*>(kv ? vp.base : kp.base) + ch * 8;
        unsigned char* dst = ring + (size_t)st * kTile + (ch >> 3) * kBlock;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll 4
          for (int k = 0; k < CH; ++k) {
            const int r = k * (32 / CH) + lane / CH;
            const int row = __shfl_sync(0xffffffffu, y[i], r);
            cp_async16_or_zero(dst + swz128(32 * i + r, ch & 7), base + (int64_t)max(row, 0) * D, row >= 0);
          }
        cp_async_commit();
        if (u >= kLag) {
          cp_async_wait<kLag>();
          arrive(u - kLag);
        }
      }
    }
    cp_async_wait<0>();
    if (ok)
      for (int v = max(0, u - kLag); v < u; ++v) arrive(v);
  }
}

// cuTensorMapEncodeTiled through the runtime's driver entry point; null when
// unavailable
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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

inline bool encode_map(CUtensorMap* tm, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const cuuint32_t one[3] = {1, 1, 1};
  auto fn = encode_fn();
  return fn && fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pools as rows of D channels; boxes of at most 128 rows of a page (pages
// of fewer than 8 rows are copied without the maps).
inline bool encode_pools(CUtensorMap* mk, CUtensorMap* mv, const AttendArgs& a, int hkv, int D) {
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)((a.kp.n_pages * hkv) << a.kp.page_shift)};
  const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)std::min(kRows, 1 << a.kp.page_shift)};
  return encode_map(mk, 2, a.kp.base, dims, strides, box) && encode_map(mv, 2, a.vp.base, dims, strides, box);
}

}  // namespace wi
