// mk_kv4.h -- host-side pieces of the 4-bit KV cache shared by its translation units
// and by the handle's park and resume
// (mk_kv4_slot.cu).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "../../include/mk.h"

namespace mk {

mk_status kv4_check_cache(const mk_kv4_cache* c);
mk_status kv4_check(const mk_kv4_cache* c, int32_t layer, const mk_kv4_batch* b, int32_t dtype);
// `written`: the rows are an output, so they must not overlap
mk_status kv4_check_rows(const mk_kv4_rows* r, int32_t dtype, int64_t rows, int32_t heads, int32_t d, bool written);

// The arguments every attention kernel takes.
struct Kv4Attn {
  mk_kv4_cache c;
  mk_kv4_batch b;
  const char* q;
  char* out;
  long long q_row, q_head, o_row, o_head;  // strides in bytes
  int layer, rep;
  float scale_log2;  // scale * log2(e)
};

// ... and how a call is split.  A row tile's rows of one split go to part as
// [reference, sum of the weights, -, -, D sums], in fp32.
struct Kv4AttnSplit : Kv4Attn {
  int n_split, split_len;  // splits of the positions, and positions of each (a multiple of a page, of 128 for prompts)
  int n_rt;                // row tiles of a sequence
  // prompts of unequal sequences: row tiles of the whole batch, sequence i's from
  // (cu[i] >> row_shift) + i on; 0: n_rt to each
  int n_blocks, row_shift;
  float* part;             // [CTA of the grid: row tile, then split][rows of a tile][D + 4]
};

// An error that some earlier call left pending is not these calls' to report or to clear: they
// refuse and leave it in place.
inline bool kv4_error_pending() { return cudaPeekAtLastError() != cudaSuccess; }
// Status of a launch (or of what comes before it); its own error is not left pending.
inline mk_status kv4_status(cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return MK_ERR_CUDA;
}

// Opt-in to more than 48 KiB of shared memory (and to clusters of more than 8 CTAs), once
// per kernel and device.
bool kv4_allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* ready, bool large_cluster = false);

// Attention of many query rows of 16-bit types (mk_kv4_prompt.cu).
constexpr int kKv4PromptRows = 256;  // rows of its tiles
mk_status kv4_prompt(const Kv4AttnSplit& a, int32_t dtype, cudaStream_t s);

// Quantise (write) or read back positions start .. start + n - 1 of a slot of a handle's
// cache [layer][physical page][kv head][K, V][PL][d], all layers; arguments checked by the caller.
mk_status kv4_slot(bool write, const mk_kv4_cache* c, void* kv, const int* slot_table, int n_phys_pages, int PL,
                   bool fp16, const int32_t* table_row, int start, int n, cudaStream_t s);

}  // namespace mk
