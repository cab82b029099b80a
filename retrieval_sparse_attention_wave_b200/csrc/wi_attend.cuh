// What the attention kernels share: the call's items, where results go, and
// the launch helpers.
#pragma once

#include <atomic>
#include <cstdint>

#include "wi_serve.h"

namespace wi {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The sequences of a call, a kernel parameter: 10 KB for the largest batch,
// which takes 5 us more to launch, so the kernels are compiled for few
// sequences as well.
constexpr int kFewSeqs = 16;
template <int N>
struct AttendTable {
  int32_t n_seq, n_items, hkv, g_shift, rows, keys;   // (rows of a block, keys of a tile)
  AttendSeq seq[N];
};

// One item of the plan, as its CTA needs it.
struct Item {
  int b, h, T, n, q0;
  int row0, rows;       // its rows of the unit
  int pos0;             // position of query token 0 of the sequence
  int key_end;          // keys its last row sees
  int t0, t1;           // key tiles
  int64_t part;         // first part row, -1: the whole key range
};

template <int N>
__device__ __forceinline__ Item item_of(const AttendTable<N>& tb, int item, int KT) {
  int lo = 0, hi = tb.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.seq[mid].item0 <= item) lo = mid; else hi = mid - 1;
  }
  const AttendSeq& s = tb.seq[lo];
  Item it;
  const uint32_t ns = s.ns, x = item - s.item0, hkv = tb.hkv, nblk = s.nblk;
  const int all = s.n << tb.g_shift;
  uint32_t back, split = 0;   // blocks from the last
  if (ns == 1) {
    back = x / hkv;
    it.h = (int)(x - back * hkv);
  } else {   // the blocks that read a run of keys next to one another
    const uint32_t y = x / nblk;
    back = x - y * nblk;
    split = y / hkv;
    it.h = (int)(y - split * hkv);
  }
  const int blk = (int)(nblk - 1 - back);
  it.b = s.b; it.T = s.T; it.n = s.n; it.q0 = s.q0;
  it.row0 = blk * tb.rows;
  it.rows = min(tb.rows, all - it.row0);
  it.pos0 = s.T - s.n;
  it.key_end = it.pos0 + ((it.row0 + it.rows - 1) >> tb.g_shift) + 1;
  const uint32_t nt = (uint32_t)(it.key_end + KT - 1) / KT;   // at most 2^31 / 32
  it.t0 = 0;
  it.t1 = (int)nt;
  it.part = -1;
  if (ns > 1) {
    it.t0 = (int)min(nt, split * (uint32_t)s.run);
    it.t1 = (int)min(nt, (split + 1) * (uint32_t)s.run);
    it.part = s.part0 + (((int64_t)blk * tb.hkv + it.h) * s.ns + split) * min(tb.rows, all);
  }
  return it;
}

struct AttendOut {
  void* out;
  float* lse;
  float2* ml;
  float* o;
  int64_t stride;
  int Hq;
};

// Dynamic shared memory limit of a kernel, raised once per device.
template <auto kern>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};   // one bit per device (the first 64)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// bf16: blocks of 128 or 256 rows (wi_attend_umma.cu), and of 16
// (wi_attend_few.cu)
template <int N>
cudaError_t launch_attend_umma(const AttendTable<N>& tb, const AttendPlan& pl, const AttendArgs& a,
                               const AttendOut& ao, cudaStream_t s);
template <int N>
cudaError_t launch_attend_few(const AttendTable<N>& tb, const AttendPlan& pl, const AttendArgs& a,
                              const AttendOut& ao, cudaStream_t s);

}  // namespace wi
