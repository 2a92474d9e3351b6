// mk_kv4_slot.cu -- the handle's side of the 4-bit KV cache: parking a slot's positions in
// it and bringing them back.  The handle's struct is private to mk_api.cu, which is therefore
// compiled as part of this translation unit: that file is among those whose hash ties the
// recorded DRAM traffic of the decode kernel to its sources, and nothing of the decode
// step changes here.
#include "mk_api.cu"
#include "mk_kv4.h"

// Positions of one slot between the handle's 16-bit cache and a 4-bit cache, every layer in one launch.
static mk_status move_slot(bool park, mk_handle h, int32_t slot, int32_t start, int32_t n, const mk_kv4_cache* cache,
                           const int32_t* block_table_row, int32_t max_pages, void* stream) {
  if (!h || !block_table_row) return MK_ERR_INVALID_ARG;
  MK_TRY(kv4_check_cache(cache));
  const Dims& D = h->D;
  if (cache->n_layers != D.L || cache->n_kv_heads != D.Hkv || cache->head_dim != D.d) return MK_ERR_INVALID_ARG;
  if (slot < 0 || slot >= D.max_batch || start < 0 || n < 0 || (long long)start + n > D.max_seq ||
      (long long)start + n > (long long)MK_KV4_PAGE * max_pages)
    return MK_ERR_INVALID_ARG;
  if (n == 0) return MK_OK;
  if (kv4_error_pending()) return MK_ERR_CUDA;
  MK_TRY(kv4_status(cudaSetDevice(h->dev)));
  return kv4_slot(park, cache, h->kv, h->page_table + (size_t)slot * D.pages_per_seq, D.n_phys_pages, D.PL, D.kv_fp16,
                  block_table_row, start, n, static_cast<cudaStream_t>(stream));
}

extern "C" mk_status mk_kv4_park(mk_handle h, int32_t slot, int32_t start, int32_t n, const mk_kv4_cache* cache,
                                 const int32_t* block_table_row, int32_t max_pages, void* stream) {
  return move_slot(true, h, slot, start, n, cache, block_table_row, max_pages, stream);
}

extern "C" mk_status mk_kv4_resume(mk_handle h, int32_t slot, int32_t start, int32_t n, const mk_kv4_cache* cache,
                                   const int32_t* block_table_row, int32_t max_pages, void* stream) {
  return move_slot(false, h, slot, start, n, cache, block_table_row, max_pages, stream);
}
