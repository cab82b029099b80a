// Host-side plans of the serving calls (page plans, cache appends, attention
// over the paged cache) and their launchers.
#pragma once

#include <cstddef>
#include <cstdint>

#include "wi_common.cuh"

namespace wi {

// in wi_api.cu
wi_status cuda_fail(cudaError_t e);
wi_status check_common(wi_dtype dtype, int batch, int hkv, int d, int page, int64_t n_pages,
                       const void* kp, const void* vp, const int32_t* bt, int max_pages,
                       const int32_t* seq_lens, int min_len = 1);

// A launch whose error is its own (cudaGetLastError after <<<>>> would also
// hand back what an earlier call of this thread left).
template <typename... Params, typename... Args>
cudaError_t launch_kernel(void (*kern)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                          bool behind_previous, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind_previous ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

// ---------------------------------------------------------------- attention
// The query heads of a KV head share its keys, so the rows of a work item are
// (token, head of the group) pairs of one KV head: row r of sequence b's unit
// (b, h) is head h * G + r % G of the sequence's query token r / G.  An item
// is a block of rows and a run of key tiles; a sequence with few blocks has
// its key axis split into runs, whose parts a second kernel merges (the items
// of runs that a block does not reach are empty and leave no part).
struct AttendSeq {
  int32_t b;        // the sequence
  int32_t T;        // its tokens in the cache
  int32_t n;        // its query tokens
  int32_t q0;       // its first query token in the packed q
  int32_t nblk;     // row blocks per unit
  int32_t ns;       // key runs of the longest block
  int32_t run;      // key tiles of a run (ns > 1; a block's last may be shorter)
  int32_t item0;    // its first item: blocks descending (the longest key range
                    // first), then KV heads; split, runs, KV heads, blocks
  int32_t part0;    // its first part row (ns > 1)
  int32_t mrow0;    // its first row of the merge kernel (ns > 1)
};

struct AttendPlan {
  int n_seq;        // sequences with query tokens, the longest key range first
  int n_items, n_merge_rows;
  int hkv, G, Hq, D, dtype;
  bool exact;       // 16 bits of a softmax weight (bf16)
  int rows, keys;   // rows per block, keys per tile
  int64_t q_tokens; // rows of the packed q
  size_t off_ml, off_o, total;   // workspace: {m, l} and o of the part rows
  AttendSeq seq[kMaxBatch];
};

struct AttendArgs {
  const void* q;
  void* out;
  float* lse;
  int64_t q_stride, out_stride;
  Pool kp, vp;
  unsigned char* ws;
};

// Rows per block, keys per tile and items running at once, for a call whose
// blocks have at most `most` rows to fill (wi_attend.cu); in times of a key
// tile of a full block, what an item costs besides its tiles and what writing
// and merging a full block's part costs; and the most items that the split
// sequences of a call have together, which bounds the workspace.
struct AttendShape {
  int rows, keys, slots;
  double item_cost, part_cost;
  int most_split;
};
AttendShape attend_shape(int dtype, int D, int most);
cudaError_t launch_attend(const AttendPlan& pl, const AttendArgs& a, cudaStream_t s);

// ------------------------------------------------------- pages and appends
cudaError_t launch_plan_pages(const wi_page_plan& p, unsigned char* ws, cudaStream_t s);
cudaError_t launch_append_kv(const wi_kv_append& a, unsigned char* ws, cudaStream_t s);

}  // namespace wi
