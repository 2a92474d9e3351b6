// mk_kv4_attn.cu -- causal attention over the 4-bit KV cache.
#include <cuda_runtime.h>

#include <cmath>

#include "mk_kv4.cuh"
#include "mk_kv4.h"

namespace mk {
namespace {

struct AttnArgs {
  mk_kv4_cache c;
  mk_kv4_batch b;
  const char* q;
  char* out;
  long long q_row, q_head, o_row, o_head;  // strides in bytes
  int layer, n_heads, rep;
  float scale;
};

__device__ __forceinline__ int seq_of_row(const mk_kv4_batch& b, int row) {
  int lo = 0, hi = b.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.cu[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The plain form: a warp per query row and head, 32 positions at a time (a lane scores
// one position), softmax with a running maximum and sum, a lane per D / 32 output values.
template <int D, class T>
__global__ void __launch_bounds__(128) attn_simple(AttnArgs a) {
  using L = Kv4<D>;
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x, hq = blockIdx.y * 4 + warp;
  __shared__ float qs[4][D];
  if (hq >= a.n_heads) return;
  const int si = seq_of_row(a.b, row);
  const Kv4Seq s = kv4_seq(a.b, si);
  if (!s.ok) {
    if (lane == 0) atomicOr(a.c.status, KV4_BAD_BATCH);
    return;
  }
  if (row < s.row0 || row >= s.row0 + s.n) return;
  const int head = hq / a.rep, see = s.len - s.n + (row - s.row0) + 1;  // positions seen
  const int32_t* table = a.b.block_table + (size_t)si * a.b.max_pages;
  if (lane < D / 8) {
    float x[8];
    load8<T>(a.q + row * a.q_row + hq * a.q_head + lane * 8 * sizeof(T), x);
    for (int i = 0; i < 8; ++i) qs[warp][lane * 8 + i] = x[i];
  }
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[E];
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int p0 = 0; p0 < see; p0 += 32) {
    const int p = p0 + lane;
    float sc = -INFINITY;
    const uint8_t* tile = p < see ? kv4_tile<D>(a.c, table, a.layer, head, p / kKv4Tile) : nullptr;
    if (p < see && !tile) atomicOr(a.c.status, KV4_BAD_PAGE);
    const int r = p % kKv4Tile;
    if (tile) {
      float acc = 0.f;
      for (int g = 0; g < L::G; ++g) {
        float dot = 0.f, sum = 0.f;
        for (int w = 4 * g; w < 4 * g + 4; ++w) {
          const uint32_t codes = *reinterpret_cast<const uint32_t*>(tile + L::k_word(r, w));
          for (int i = 0; i < 8; ++i) {
            const float q = qs[warp][8 * w + i];
            dot = fmaf(q, (float)((codes >> (4 * i)) & 15u), dot);
            sum += q;
          }
        }
        acc += __half2float(*reinterpret_cast<const __half*>(tile + L::kKs + L::scale(r, g))) * dot +
               __half2float(*reinterpret_cast<const __half*>(tile + L::k_min(r, g))) * sum;
      }
      sc = acc * a.scale;
    }
    float mx = sc;
    for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float corr = expf(m - mn), pr = tile ? expf(sc - mn) : 0.f;
    m = mn;
    l = l * corr + pr;
    for (int e = 0; e < E; ++e) o[e] *= corr;
    for (int j = 0; j < 32 && p0 + j < see; ++j) {
      const float pj = __shfl_sync(0xFFFFFFFFu, pr, j);
      const uint8_t* tj = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)tile, j));
      if (!tj) continue;
      const int rj = (p0 + j) % kKv4Tile;
      for (int e = 0; e < E; ++e) {
        const int d = lane * E + e;
        const uint32_t unit = *reinterpret_cast<const uint16_t*>(tj + L::v_unit(rj, d / 4));
        const float v = fmaf(__half2float(*reinterpret_cast<const __half*>(tj + L::kVs + L::scale(rj, d / 32))),
                             (float)((unit >> (4 * (d % 4))) & 15u),
                             __half2float(*reinterpret_cast<const __half*>(tj + L::v_min(rj, d / 32))));
        o[e] = fmaf(pj, v, o[e]);
      }
    }
  }
  for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
  T* dst = reinterpret_cast<T*>(a.out + row * a.o_row + hq * a.o_head);
  for (int e = 0; e < E; ++e) dst[lane * E + e] = (T)(l > 0.f || l != l ? o[e] / l : 0.f);
}

}  // namespace
}  // namespace mk

using namespace mk;

static mk_status check_attention(const mk_kv4_cache* c, int32_t layer, const mk_kv4_batch* b, int32_t n_heads,
                                 int32_t dtype) {
  const mk_status st = kv4_check(c, layer, b, dtype);
  if (st != MK_OK) return st;
  if (n_heads < 1 || n_heads % c->n_kv_heads) return MK_ERR_INVALID_ARG;
  const int rep = n_heads / c->n_kv_heads;
  if (rep != 1 && rep != 2 && rep != 4 && rep != 8) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

extern "C" mk_status mk_kv4_attention_workspace(const mk_kv4_cache* cache, const mk_kv4_batch* batch, int32_t n_heads,
                                                int32_t dtype, int64_t* bytes) {
  if (!bytes) return MK_ERR_INVALID_ARG;
  const mk_status st = check_attention(cache, 0, batch, n_heads, dtype);
  if (st != MK_OK) return st;
  *bytes = 0;
  return MK_OK;
}

extern "C" mk_status mk_kv4_attention(const mk_kv4_cache* cache, int32_t layer, const mk_kv4_batch* batch,
                                      const mk_kv4_rows* q, const mk_kv4_rows* out, int32_t n_heads, int32_t dtype,
                                      float scale, void* workspace, int64_t workspace_bytes, void* stream) {
  mk_status st = check_attention(cache, layer, batch, n_heads, dtype);
  if (st != MK_OK) return st;
  if (!std::isfinite(scale)) return MK_ERR_INVALID_ARG;
  if (batch->n_rows == 0) return MK_OK;
  st = kv4_check_rows(q, dtype, batch->n_rows, n_heads, cache->head_dim, false);
  if (st == MK_OK) st = kv4_check_rows(out, dtype, batch->n_rows, n_heads, cache->head_dim, true);
  if (st != MK_OK) return st;
  const int size = dtype == 2 ? 4 : 2;
  AttnArgs a{*cache, *batch, static_cast<const char*>(q->p), static_cast<char*>(out->p),
             q->row_stride * size, q->head_stride * size, out->row_stride * size, out->head_stride * size,
             layer, n_heads, n_heads / cache->n_kv_heads, scale};
  const dim3 grid(batch->n_rows, (n_heads + 3) / 4);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
#define MK_KV4_ATTN(D, T) attn_simple<D, T><<<grid, 128, 0, s>>>(a)
  if (cache->head_dim == 64) {
    if (dtype == 0) MK_KV4_ATTN(64, __nv_bfloat16);
    else if (dtype == 1) MK_KV4_ATTN(64, __half);
    else MK_KV4_ATTN(64, float);
  } else {
    if (dtype == 0) MK_KV4_ATTN(128, __nv_bfloat16);
    else if (dtype == 1) MK_KV4_ATTN(128, __half);
    else MK_KV4_ATTN(128, float);
  }
#undef MK_KV4_ATTN
  return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
