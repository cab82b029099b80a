// Serving calls of libwi.so: argument checks and plans of wi_plan_pages,
// wi_append_kv and wi_attend, and the page-plan and append kernels.
// Every argument error is detected here, on the host, before any CUDA call.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <utility>

#include "wi.h"
#include "wi_common.cuh"
#include "wi_serve.h"

namespace wi {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool good_page(int p) { return p >= 1 && p <= 1024 && (p & (p - 1)) == 0; }
int ilog2(int x) { int r = 0; while ((1 << r) < x) ++r; return r; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ------------------------------------------------------------- page plans
// One thread per request holds its lengths; a block scan gives every request
// its first packed token and its first page on the stack, in every CTA (256
// requests at most: one round of loads), so no CTA waits for another.  Then a
// thread takes four packed tokens at a time: a search of the starts in shared
// memory, the slot from the table (a page in use) or straight from the stack
// (a page this call hands out, whose table entry another CTA may be writing),
// and 16-byte stores.  The first CTA writes the lengths and the stack's size
// too; where they are updated in place and other CTAs may still be reading
// them, a kernel of one CTA behind this one does.  Nothing is kept between
// calls.  Latency bounds it (lengths, scan, page, store): 6.5 to 8.3 us for a
// step of 64 requests, cold; 335445 tokens 4.9 us, and 2.8 for the lengths in
// place behind it.
constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 4 * kPlanThreads;   // per CTA and round

struct PlanArgs {
  int32_t batch, page_shift, n_pages, max_pages, max_free, capacity, vec;
  const int32_t *seq_lens, *new_lens, *free_pages, *n_free;
  int32_t *block_table, *seq_lens_out, *n_free_out, *starts, *slot_map, *positions;
  uint32_t* status;
  bool write_lens;   // plan_pages_kernel writes seq_lens_out and n_free_out
};

// the last i < n with tab[i] <= x (tab ascending, tab[0] <= x)
__device__ __forceinline__ int last_at_or_below(const int32_t* tab, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The pages of `have` tokens (which may be all an int holds).
__device__ __forceinline__ int pages_of(int have, int page_shift) {
  return (have >> page_shift) + ((have & ((1 << page_shift) - 1)) != 0);
}

// The step as each of a CTA's threads needs it: its request's lengths (thread
// tid < batch), the new tokens and pages of the requests before it, and the
// sums.  A step that does not fit has no new tokens and no pages.
struct PlanStep {
  int32_t have, fresh;
  int32_t start, taken;
  int32_t tokens, pages, n_free;
  uint32_t bad;
};

__device__ __forceinline__ PlanStep plan_step(const PlanArgs& a) {
  __shared__ int64_t s_sum[2][kPlanThreads / 32];
  __shared__ uint32_t s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page_mask = (1 << a.page_shift) - 1;
  static_assert(kMaxBatch <= kPlanThreads, "a thread per request");
  if (tid == 0) s_bad = 0;
  __syncthreads();
  // lengths in 64 bits: sums of 256 of them can pass 32
  int64_t have = 0, fresh = 0, need = 0;
  const int n_free = *a.n_free;
  if (tid < a.batch) {
    have = a.seq_lens[tid];
    fresh = a.new_lens[tid];
    uint32_t bad = 0;
    if (have < 0 || fresh < 0 || have + fresh > INT32_MAX) {
      bad = WI_DEV_BAD_SLOT;
      fresh = 0;
    }
    const int64_t pages = (have + fresh + page_mask) >> a.page_shift;
    need = pages - ((have + page_mask) >> a.page_shift);
    if (pages > a.max_pages) bad |= WI_DEV_NO_PAGES;
    if (bad) atomicOr(&s_bad, bad);
  }
  int64_t x = fresh, y = need;   // inclusive scans
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t px = __shfl_up_sync(0xffffffffu, x, o), py = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) { x += px; y += py; }
  }
  if (lane == 31) { s_sum[0][warp] = x; s_sum[1][warp] = y; }
  __syncthreads();   // and every thread of this CTA has read the lengths
  int64_t all_fresh = 0, all_need = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) { x += s_sum[0][w]; y += s_sum[1][w]; }
    all_fresh += s_sum[0][w];
    all_need += s_sum[1][w];
  }
  uint32_t bad = s_bad;
  if (n_free < 0 || n_free > a.max_free) bad |= WI_DEV_BAD_PAGE;
  else if (all_need > n_free || all_fresh > a.capacity) bad |= WI_DEV_NO_PAGES;
  if (bad) { all_fresh = all_need = 0; x = y = fresh = need = 0; }
  return PlanStep{(int32_t)have, (int32_t)fresh, (int32_t)(x - fresh), (int32_t)(y - need),
                  (int32_t)all_fresh, (int32_t)all_need, n_free, bad};
}

__device__ __forceinline__ void write_lens(const PlanArgs& a, const PlanStep& st) {
  if ((int)threadIdx.x < a.batch) a.seq_lens_out[threadIdx.x] = st.have + st.fresh;
  if (threadIdx.x == 0) *a.n_free_out = st.n_free - st.pages;
}

// The lengths and the stack's size in place, behind a plan_pages_kernel of
// several CTAs.
__global__ void __launch_bounds__(kPlanThreads) plan_advance_kernel(const PlanArgs a) {
  pdl_wait();   // every CTA of the plan has ended
  write_lens(a, plan_step(a));
}

__global__ void __launch_bounds__(kPlanThreads) plan_pages_kernel(const PlanArgs a) {
  __shared__ int32_t s_start[kMaxBatch + 1], s_need[kMaxBatch + 1], s_have[kMaxBatch];
  const int tid = threadIdx.x;
  const int page_mask = (1 << a.page_shift) - 1;
  pdl_launch_dependents();
  const PlanStep st = plan_step(a);
  const int total = st.tokens, n_need = st.pages, n_free = st.n_free;
  if (tid < a.batch) {
    s_have[tid] = st.have;
    s_start[tid] = st.start;
    s_need[tid] = st.taken;
  }
  if (tid == 0) { s_start[a.batch] = total; s_need[a.batch] = n_need; }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (a.write_lens) write_lens(a, st);
    if (tid == 0 && st.bad) flag_error(a.status, st.bad);
    for (int i = tid; i <= a.batch; i += kPlanThreads) a.starts[i] = s_start[i];
  }

  uint32_t flags = 0;
  // a page off the stack, or -1
  auto taken = [&](int i) {
    const int pg = __ldg(a.free_pages + (n_free - 1 - i));
    if (pg >= 0 && pg < a.n_pages) return pg;
    flags |= WI_DEV_BAD_PAGE;
    return -1;
  };
  const int stride = gridDim.x * kPlanThreads;
  for (int64_t i = blockIdx.x * kPlanThreads + tid; i < n_need; i += stride) {
    const int e = (int)i, b = last_at_or_below(s_need, a.batch, e);
    const int lp = pages_of(s_have[b], a.page_shift) + (e - s_need[b]);
    a.block_table[(int64_t)b * a.max_pages + lp] = taken(e);
  }
  for (int64_t i0 = (int64_t)blockIdx.x * kPlanTokens + 4 * tid; i0 < a.capacity;
       i0 += (int64_t)gridDim.x * kPlanTokens) {
    int slot[4], pos[4];
    int b = i0 < total ? last_at_or_below(s_start, a.batch, (int)i0) : 0;
    int seen_b = -1, seen_lp = -1, pg = -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + j;
      slot[j] = pos[j] = -1;
      if (i < total) {
        while (s_start[b + 1] <= i) ++b;   // ends: s_start[batch] = total > i
        pos[j] = s_have[b] + ((int)i - s_start[b]);
        const int lp = pos[j] >> a.page_shift;
        if (b != seen_b || lp != seen_lp) {
          const int first = pages_of(s_have[b], a.page_shift);
          if (lp >= first) {
            pg = taken(s_need[b] + lp - first);
          } else {
            pg = a.block_table[(int64_t)b * a.max_pages + lp];
            if (pg < 0 || pg >= a.n_pages) { flags |= WI_DEV_BAD_PAGE; pg = -1; }
          }
          seen_b = b;
          seen_lp = lp;
        }
        if (pg >= 0) slot[j] = (pg << a.page_shift) + (pos[j] & page_mask);
      }
    }
    if (a.vec && i0 + 4 <= a.capacity) {
      *reinterpret_cast<int4*>(a.slot_map + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.positions)
        *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j < a.capacity) {
          a.slot_map[i0 + j] = slot[j];
          if (a.positions) a.positions[i0 + j] = pos[j];
        }
    }
  }
  if (flags) flag_error(a.status, flags);
}

// ---------------------------------------------------------------- appends
// A copy: every thread moves 16-byte chunks, kAppendBatch loads in flight,
// from token rows (contiguous over the heads) to the heads' page rows.  HBM
// bounds it: 131072 tokens of 8 heads of 128 (1.07 GB read and written) in
// 178 us a call back to back, 6.0 TB/s (169 us of it the kernel, alone and
// cold); 16 tokens 5.2 us.
constexpr int kAppendThreads = 256;
constexpr int kAppendBatch = 8;

struct AppendArgs {
  const unsigned char *k, *v;
  unsigned char *k_pool, *v_pool;
  const int32_t* slot_map;
  int64_t k_stride, v_stride;   // bytes between tokens
  int64_t n_chunks;             // n_tokens * hkv * chunks per head row
  int64_t n_slots;              // n_pages * P
  int32_t hkv, row_shift, page_shift;   // chunks per head row = 1 << row_shift
  uint32_t* status;
};

__global__ void __launch_bounds__(kAppendThreads) append_kv_kernel(const AppendArgs a) {
  const bool second = blockIdx.y != 0;
  const unsigned char* src = second ? a.v : a.k;
  unsigned char* dst = second ? a.v_pool : a.k_pool;
  const int64_t src_stride = second ? a.v_stride : a.k_stride;
  const uint32_t per_token = (uint32_t)a.hkv << a.row_shift;
  const int64_t base = (int64_t)blockIdx.x * (kAppendThreads * kAppendBatch) + threadIdx.x;
  uint4 x[kAppendBatch];
  int64_t to[kAppendBatch];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kAppendBatch; ++i) {
    const int64_t c = base + (int64_t)i * kAppendThreads;
    to[i] = -1;
    if (c < a.n_chunks) {
      const int64_t t = c / per_token;
      const uint32_t in = (uint32_t)(c - t * per_token);
      const int64_t slot = __ldg(a.slot_map + t);
      if (slot >= a.n_slots) bad = true;
      if (slot >= 0 && slot < a.n_slots) {
        x[i] = ld_stream(src + t * src_stride + (int64_t)in * 16);
        const int h = (int)(in >> a.row_shift), ch = (int)(in & ((1u << a.row_shift) - 1));
        const int64_t page = slot >> a.page_shift, row = slot & ((1 << a.page_shift) - 1);
        to[i] = ((((page * a.hkv + h) << a.page_shift) + row) << a.row_shift) + ch;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kAppendBatch; ++i)
    if (to[i] >= 0) *reinterpret_cast<uint4*>(dst + to[i] * 16) = x[i];
  if (bad) flag_error(a.status, WI_DEV_BAD_SLOT);
}

// -------------------------------------------------------------- attention
// Key runs per block (ns).  Many blocks: one run each, and the item grid
// fills the SMs.  Few: the key axis is split until the longest item and the
// work per SM balance, in key tiles (attend_shape has the other costs).
constexpr double kMergeCost = 3.0;   // the merge's launch and latency (about 4 us)
constexpr int kMinTiles = 2, kMaxSplit = 148;

int64_t tiles_of(const AttendSeq& s, int G, int R, int KT, int blk) {
  const int64_t rows = std::min<int64_t>((int64_t)(blk + 1) * R, (int64_t)s.n * G);
  return cdiv((int64_t)s.T - s.n + cdiv(rows, G), KT);
}

void choose_splits(AttendPlan& pl, const AttendShape& sh) {
  const int R = sh.rows, KT = sh.keys, slots = sh.slots;
  double total = 0;
  int64_t longest = 0;
  uint32_t most[kMaxBatch], least[kMaxBatch];   // tiles of a sequence's last and first block
  for (int i = 0; i < pl.n_seq; ++i) {
    AttendSeq& s = pl.seq[i];
    most[i] = (uint32_t)tiles_of(s, pl.G, R, KT, s.nblk - 1);
    least[i] = (uint32_t)tiles_of(s, pl.G, R, KT, 0);
    total += 0.5 * ((double)most[i] + least[i]) * s.nblk * pl.hkv;
    longest = std::max<int64_t>(longest, most[i]);
    s.ns = 1;
    s.run = 0;
  }
  if ((double)longest + sh.item_cost <= total / slots) return;   // enough blocks
  auto cost = [&](int64_t C) {
    double items = 0, parts = 0;   // parts in full blocks
    int64_t split = 0;             // items of split sequences
    for (int i = 0; i < pl.n_seq; ++i) {
      const AttendSeq& s = pl.seq[i];
      const uint32_t c = (uint32_t)C;
      const double runs = 0.5 * (double)((most[i] + c - 1) / c + (least[i] + c - 1) / c);
      items += s.nblk * pl.hkv * runs;
      const int64_t ns = (most[i] + c - 1) / c;
      if (ns > 1) split += ns * s.nblk * pl.hkv;
      if (runs > 1) parts += pl.hkv * runs * std::min<double>((double)s.n * pl.G / R, s.nblk);
    }
    if (split > sh.most_split) return HUGE_VAL;
    const double one = (double)std::min(C, longest) + sh.item_cost, spread = sh.part_cost * parts / slots;
    const double t = items <= slots ? one : (total + items * sh.item_cost) / slots + 0.5 * one;
    return t + spread + (C < longest ? kMergeCost : 0);
  };
  int64_t best = longest;
  double cheapest = cost(longest);
  // (a candidate costs two divisions a sequence: all 147 for up to two
  // sequences, 27 or 17 of them for more)
  const int coarse = pl.n_seq <= 2 ? kMaxSplit + 1 : pl.n_seq <= 32 ? 8 : 4;
  for (int k = 2; k <= kMaxSplit; k += 1 + k / coarse) {
    const int64_t C = cdiv(longest, k);
    if (C < kMinTiles) break;
    const double c = cost(C);
    if (c < cheapest) { cheapest = c; best = C; }
  }
  for (int i = 0; i < pl.n_seq; ++i) {
    AttendSeq& s = pl.seq[i];
    s.ns = (int)cdiv(most[i], best);
    s.run = (int)cdiv(most[i], s.ns);
  }
}

// The most part rows of a call of up to `batch` sequences with at most n query
// tokens and T tokens each, in blocks of sh.rows rows: those of make_attend_plan
// with every sequence split as far as choose_splits ever does.
int64_t most_parts(const AttendShape& sh, int batch, int hkv, int G, int64_t T, int64_t n) {
  const int64_t rows = n * G, nblk = cdiv(rows, sh.rows);
  const int64_t ns = std::min<int64_t>(kMaxSplit, cdiv(cdiv(T, sh.keys), kMinTiles));
  if (ns < 2) return 0;
  const int64_t full = std::min<int64_t>(sh.rows, rows);
  return full * (int64_t)std::min((double)sh.most_split, (double)batch * hkv * nblk * ns);
}

size_t attend_bytes(int64_t parts, int D, size_t* off_ml, size_t* off_o) {
  size_t o = 256;
  auto take = [&](size_t bytes) { const size_t r = o; o = align_up(o + bytes, 256); return r; };
  *off_ml = take((size_t)parts * 8);
  *off_o = take((size_t)parts * D * 4);
  return o;
}

wi_status make_attend_plan(const wi_kv_cache* kv, const wi_attend_params* p, AttendPlan& pl) {
  if (!kv || !p) return WI_ERR_INVALID_ARG;
  wi_status st = check_common(kv->dtype, kv->batch, kv->n_kv_heads, kv->head_dim, kv->page_size,
                              kv->n_pages, kv->k_pool, kv->v_pool, kv->block_table, kv->max_pages,
                              kv->seq_lens, 0);
  if (st != WI_OK) return st;
  const int H = kv->n_kv_heads;
  if (p->n_q_heads < 1 || p->n_q_heads % H != 0) return WI_ERR_INVALID_ARG;
  if (kv->n_pages * H * kv->page_size >= INT32_MAX) return WI_ERR_UNSUPPORTED;
  const int G = p->n_q_heads / H;
  if (G != 1 && G != 2 && G != 4 && G != 8) return WI_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)p->n_q_heads * kv->head_dim, vec = kv->dtype == WI_BF16 ? 8 : 4;
  for (int64_t s : {p->q_stride, p->out_stride})
    if (s != 0 && (s < row || s % vec != 0)) return WI_ERR_INVALID_ARG;
  std::memset(&pl, 0, sizeof(pl));
  pl.hkv = H; pl.G = G; pl.Hq = p->n_q_heads; pl.D = kv->head_dim; pl.dtype = kv->dtype;
  pl.exact = p->exact_weights != 0;
  int q0 = 0, most = 0;
  for (int b = 0; b < kv->batch; ++b) {
    const int T = kv->seq_lens[b], n = p->q_lens ? p->q_lens[b] : T;
    if (n < 0 || n > T) return WI_ERR_INVALID_ARG;
    // rows are counted in 32 bits, and so are the positions of whole key tiles
    // (with one behind the last)
    if (n > INT32_MAX / G || T > INT32_MAX - 255) return WI_ERR_UNSUPPORTED;
    if (n > 0) {
      AttendSeq& s = pl.seq[pl.n_seq++];
      s.b = b; s.T = T; s.n = n; s.q0 = q0;
      most = std::max(most, n * G);
    }
    q0 += n;   // at most sum T, which check_common bounds
  }
  std::stable_sort(pl.seq, pl.seq + pl.n_seq,
                   [](const AttendSeq& x, const AttendSeq& y) { return x.T > y.T; });
  const AttendShape sh = attend_shape(pl.dtype, pl.D, most);
  pl.rows = sh.rows;
  pl.keys = sh.keys;
  int64_t items = 0;
  for (int i = 0; i < pl.n_seq; ++i) pl.seq[i].nblk = (int)cdiv((int64_t)pl.seq[i].n * G, sh.rows);
  choose_splits(pl, sh);
  int64_t parts = 0, mrows = 0;
  for (int i = 0; i < pl.n_seq; ++i) {
    AttendSeq& s = pl.seq[i];
    s.item0 = (int32_t)items;
    s.part0 = (int32_t)parts;
    s.mrow0 = (int32_t)mrows;
    items += (int64_t)s.nblk * H * s.ns;
    if (s.ns > 1) {
      parts += (int64_t)s.nblk * H * s.ns * std::min<int64_t>(sh.rows, (int64_t)s.n * G);
      mrows += (int64_t)s.n * p->n_q_heads;
    }
    if (items > INT32_MAX || parts > INT32_MAX || mrows > INT32_MAX) return WI_ERR_UNSUPPORTED;
  }
  pl.n_items = (int)items;
  pl.n_merge_rows = (int)mrows;
  pl.q_tokens = q0;
  pl.total = attend_bytes(parts, pl.D, &pl.off_ml, &pl.off_o);
  return WI_OK;
}

// n rows of `row` bytes, sa apart from a on and sb apart from b on, share a byte.
bool rows_overlap(uintptr_t a, int64_t sa, uintptr_t b, int64_t sb, int64_t n, int64_t row) {
  if (a > b) {
    std::swap(a, b);
    std::swap(sa, sb);
  }
  // row i of b against the last row of a that starts at or before it, and the next
  auto meets = [&](int64_t i) {
    const int64_t d = (int64_t)(b - a) + i * sb, j = d / sa, r = d - j * sa;
    return (j < n && r < row) || (j + 1 < n && sa - r < row);
  };
  if (sa == sb) return meets(0);   // (the others lie alike, with fewer rows of a beside them)
  for (int64_t i = 0; i < n && (int64_t)(b - a) + i * sb < (n - 1) * sa + row; ++i)
    if (meets(i)) return true;
  return false;
}

wi_status check_ws(const void* ws, size_t have, size_t need) {
  return !ws || !aligned(ws, 256) || have < need ? WI_ERR_WORKSPACE : WI_OK;
}

}  // namespace

cudaError_t launch_plan_pages(const wi_page_plan& p, unsigned char* ws, cudaStream_t s) {
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(p.capacity, kPlanTokens), 4 * 148));
  const bool in_place = p.seq_lens_out == p.seq_lens || p.n_free_out == p.n_free;
  PlanArgs a{p.batch, ilog2(p.page_size), (int32_t)p.n_pages, p.max_pages, p.max_free, p.capacity,
             aligned(p.slot_map, 16) && aligned(p.positions, 16), p.seq_lens, p.new_lens, p.free_pages,
             p.n_free, p.block_table, p.seq_lens_out, p.n_free_out, p.starts, p.slot_map, p.positions,
             reinterpret_cast<uint32_t*>(ws), grid == 1 || !in_place};
  const cudaError_t e = launch_kernel(plan_pages_kernel, dim3(grid), kPlanThreads, 0, s, false, a);
  if (e != cudaSuccess || a.write_lens) return e;
  return launch_kernel(plan_advance_kernel, dim3(1), kPlanThreads, 0, s, true, a);
}

cudaError_t launch_append_kv(const wi_kv_append& p, unsigned char* ws, cudaStream_t s) {
  const int64_t es = p.dtype == WI_BF16 ? 2 : 4, row = (int64_t)p.n_kv_heads * p.head_dim;
  const int per_row = (int)(p.head_dim * es / 16);
  AppendArgs a{static_cast<const unsigned char*>(p.k), static_cast<const unsigned char*>(p.v),
               static_cast<unsigned char*>(p.k_pool), static_cast<unsigned char*>(p.v_pool), p.slot_map,
               (p.k_stride ? p.k_stride : row) * es, (p.v_stride ? p.v_stride : row) * es,
               (int64_t)p.n_tokens * p.n_kv_heads * per_row, p.n_pages * p.page_size, p.n_kv_heads,
               ilog2(per_row), ilog2(p.page_size), reinterpret_cast<uint32_t*>(ws)};
  const int64_t grid = cdiv(a.n_chunks, kAppendThreads * kAppendBatch);
  return launch_kernel(append_kv_kernel, dim3((unsigned)grid, 2), kAppendThreads, 0, s, false, a);
}

}  // namespace wi

using namespace wi;

extern "C" {

wi_status wi_plan_pages(const wi_page_plan* p, void* ws, size_t ws_bytes, wi_stream_t stream) {
  if (!p) return WI_ERR_INVALID_ARG;
  if (p->batch < 1 || p->max_pages < 1 || p->n_pages < 1 || p->max_free < 0 || p->capacity < 0 ||
      !good_page(p->page_size))
    return WI_ERR_INVALID_ARG;
  if (p->batch > kMaxBatch || p->n_pages > INT32_MAX / p->page_size) return WI_ERR_UNSUPPORTED;
  if (!p->seq_lens || !p->new_lens || !p->block_table || !p->n_free || !p->seq_lens_out || !p->n_free_out ||
      !p->starts || (!p->free_pages && p->max_free > 0) || (!p->slot_map && p->capacity > 0))
    return WI_ERR_INVALID_ARG;
  for (const void* x : {(const void*)p->seq_lens, (const void*)p->new_lens, (const void*)p->block_table,
                        (const void*)p->free_pages, (const void*)p->n_free, (const void*)p->seq_lens_out,
                        (const void*)p->n_free_out, (const void*)p->starts, (const void*)p->slot_map,
                        (const void*)p->positions})
    if (!aligned(x, 4)) return WI_ERR_INVALID_ARG;
  const wi_status st = check_ws(ws, ws_bytes, WI_SERVE_WORKSPACE);
  if (st != WI_OK) return st;
  const cudaError_t e =
      launch_plan_pages(*p, static_cast<unsigned char*>(ws), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WI_OK : cuda_fail(e);
}

wi_status wi_append_kv(const wi_kv_append* a, void* ws, size_t ws_bytes, wi_stream_t stream) {
  if (!a) return WI_ERR_INVALID_ARG;
  if (a->dtype != WI_F32 && a->dtype != WI_BF16) return WI_ERR_INVALID_ARG;
  if (a->n_tokens < 0 || a->n_kv_heads < 1 || a->head_dim < 1 || a->n_pages < 1 || !good_page(a->page_size))
    return WI_ERR_INVALID_ARG;
  if (a->head_dim != 64 && a->head_dim != 128) return WI_ERR_UNSUPPORTED;
  if (a->n_pages > INT32_MAX / a->page_size || a->n_kv_heads > (1 << 16)) return WI_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)a->n_kv_heads * a->head_dim, vec = a->dtype == WI_BF16 ? 8 : 4;
  for (int64_t s : {a->k_stride, a->v_stride})
    if (s != 0 && (s < row || s % vec != 0)) return WI_ERR_INVALID_ARG;
  if (!a->k_pool || !a->v_pool || a->k_pool == a->v_pool) return WI_ERR_INVALID_ARG;
  if (a->n_tokens > 0 && (!a->k || !a->v || !a->slot_map)) return WI_ERR_INVALID_ARG;
  for (const void* x : {a->k, a->v, (const void*)a->k_pool, (const void*)a->v_pool})
    if (!aligned(x, 16)) return WI_ERR_INVALID_ARG;
  if (!aligned(a->slot_map, 4)) return WI_ERR_INVALID_ARG;
  const wi_status st = check_ws(ws, ws_bytes, WI_SERVE_WORKSPACE);
  if (st != WI_OK) return st;
  const int64_t chunks = (int64_t)a->n_tokens * row / vec;
  if (chunks / (kAppendThreads * kAppendBatch) >= INT32_MAX) return WI_ERR_UNSUPPORTED;
  if (a->n_tokens == 0) return WI_OK;
  const cudaError_t e =
      launch_append_kv(*a, static_cast<unsigned char*>(ws), reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WI_OK : cuda_fail(e);
}

wi_status wi_attend_workspace_size(const wi_kv_cache* kv, const wi_attend_params* p, size_t* bytes) {
  if (!bytes) return WI_ERR_INVALID_ARG;
  AttendPlan pl;
  const wi_status st = make_attend_plan(kv, p, pl);
  if (st != WI_OK) return st;
  *bytes = pl.total;
  return WI_OK;
}

wi_status wi_attend_workspace_bound(wi_dtype dtype, int32_t batch, int32_t n_kv_heads, int32_t head_dim,
                                    int32_t n_q_heads, int32_t max_seq_len, int32_t max_q_len, size_t* bytes) {
  if (!bytes || (dtype != WI_F32 && dtype != WI_BF16) || batch < 1 || n_kv_heads < 1 || head_dim < 1 ||
      n_q_heads < 1 || n_q_heads % n_kv_heads != 0 || max_seq_len < 0 || max_q_len < 0)
    return WI_ERR_INVALID_ARG;
  const int G = n_q_heads / n_kv_heads;
  if (batch > kMaxBatch || (head_dim != 64 && head_dim != 128) || (G != 1 && G != 2 && G != 4 && G != 8))
    return WI_ERR_UNSUPPORTED;
  const int64_t n = std::min(max_q_len, max_seq_len);
  // a call may have fewer rows than these, so every shape of fewer counts
  int64_t parts = 0, below = -1;
  for (int64_t most : {(int64_t)16, (int64_t)128, n * G}) {
    most = std::min(most, n * G);
    if (most <= below) continue;
    below = most;
    const AttendShape sh = attend_shape(dtype, head_dim, (int)std::min<int64_t>(most, INT32_MAX));
    parts = std::max(parts, most_parts(sh, batch, n_kv_heads, G, max_seq_len, most / G));
  }
  size_t ml, o;
  *bytes = attend_bytes(parts, head_dim, &ml, &o);
  return WI_OK;
}

wi_status wi_attend(const void* q, const wi_kv_cache* kv, const wi_attend_params* p, void* out, float* lse,
                    void* ws, size_t ws_bytes, wi_stream_t stream) {
  AttendPlan pl;
  wi_status st = make_attend_plan(kv, p, pl);
  if (st != WI_OK) return st;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)) return WI_ERR_INVALID_ARG;
  if (pl.n_seq > 0 && (!q || !out || q == out)) return WI_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, pl.total)) != WI_OK) return st;
  if (pl.n_seq == 0) return WI_OK;
  const int64_t row = (int64_t)pl.Hq * pl.D, es = pl.dtype == WI_BF16 ? 2 : 4;
  if (rows_overlap(reinterpret_cast<uintptr_t>(q), (p->q_stride ? p->q_stride : row) * es,
                   reinterpret_cast<uintptr_t>(out), (p->out_stride ? p->out_stride : row) * es, pl.q_tokens, row * es))
    return WI_ERR_INVALID_ARG;
  AttendArgs a{};
  a.q = q; a.out = out; a.lse = lse;
  a.q_stride = p->q_stride ? p->q_stride : row;
  a.out_stride = p->out_stride ? p->out_stride : row;
  a.kp = Pool{kv->k_pool, kv->block_table, kv->n_pages, kv->max_pages, ilog2(kv->page_size)};
  a.vp = Pool{kv->v_pool, kv->block_table, kv->n_pages, kv->max_pages, ilog2(kv->page_size)};
  a.ws = static_cast<unsigned char*>(ws);
  const cudaError_t e = launch_attend(pl, a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? WI_OK : cuda_fail(e);
}

}  // extern "C"
