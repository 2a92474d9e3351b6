// mk_kv4.cuh -- the 4-bit KV cache: where a tile keeps its codes and parameters, how
// a group is quantised, and the argument blocks of its kernels (mk_kv4.cu).
//
// A row (one position's K or V of one kv head, D values) is quantised in groups of 32
// neighbouring values: z = min rounded down to fp16, s = the smallest fp16 with
// z + 15 s >= max, code c = (x - z) / s rounded to nearest even, value = z + s c.
// Since s covers the range from the rounded z, no code leaves 0..15.
//
// 16 positions make a tile of 20 D bytes, 4 tiles a page.  The tile is stored in the
// order the attention's matrix instructions take their operands (mma m16n8k16: lane
// = 4 gid + tig), so a lane reads its operands of a tile with 16-byte loads:
//   K codes: word w of row r (values 8w .. 8w+7): tig = w % 4, gid = r % 8
//   V codes: 16-bit unit q of row r (values 4q .. 4q+3): gid = q % 8, and the rows
//            2 tig, 2 tig + 1 (+ 8) of one unit share a 32-bit word
// followed by fp16 K scales, K minima, V scales and V minima.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/mk.h"
#include "mk_device.cuh"

namespace mk {

constexpr int kKv4Tile = 16;                       // positions per tile
constexpr int kKv4Tiles = MK_KV4_PAGE / kKv4Tile;  // tiles per page

template <int D>
struct Kv4 {
  static constexpr int G = D / 32;         // groups of a row
  static constexpr int kBytes = 20 * D;    // bytes of a tile
  static constexpr int kV = 8 * D;         // byte offsets inside a tile
  static constexpr int kKs = 16 * D;
  static constexpr int kKz = 17 * D;
  static constexpr int kVs = 18 * D;
  static constexpr int kVz = 19 * D;
  // byte offset of K word w of row r
  __host__ __device__ static constexpr int k_word(int r, int w) {
    const int i = (r / 8) * G + w / 4, lane = (r % 8) * 4 + w % 4;
    return 4 * ((i / 4) * 128 + lane * 4 + i % 4);
  }
  // byte offset of V unit q of row r
  __host__ __device__ static constexpr int v_unit(int r, int q) {
    const int i = (q / 8) * 2 + r / 8, lane = (q % 8) * 4 + (r % 8) / 2;
    return kV + 4 * ((i / 4) * 128 + lane * 4 + i % 4) + 2 * (r % 2);
  }
  // byte offset of group g's scale of row r, from kKs or kVs
  __host__ __device__ static constexpr int scale(int r, int g) {
    const int i = (r / 8) * G + g;
    return 4 * ((i / 4) * 16 + ((r % 8) / 2) * 4 + i % 4) + 2 * (r % 2);
  }
  __host__ __device__ static constexpr int k_min(int r, int g) { return kKz + 2 * (r * G + g); }
  __host__ __device__ static constexpr int v_min(int r, int g) { return kVz + 2 * (g * kKv4Tile + r); }
};

// status bits a kernel sets in mk_kv4_cache::status
enum : uint32_t { KV4_BAD_BATCH = 1u, KV4_BAD_PAGE = 2u, KV4_TIMEOUT = 4u };

// A batch's sequence as the kernels see it; ok = 0 where its device-side numbers
// leave the bounds the call was given.
struct Kv4Seq {
  int row0;   // first of its rows in the batch
  int n;      // its rows
  int len;    // its length in the cache after the call
  bool ok;
};
__device__ __forceinline__ Kv4Seq kv4_seq(const mk_kv4_batch& b, int i) {
  Kv4Seq s;
  s.row0 = b.cu[i];
  const int end = b.cu[i + 1];
  s.n = end - s.row0;
  s.len = b.kv_lens[i];
  s.ok = s.row0 >= 0 && end >= s.row0 && end <= b.n_rows && s.n <= b.max_new && s.len >= 0 && s.len <= b.max_len;
  return s;
}

// Tile `tile` of a sequence's kv head in a layer, or null for a page id out of range.
template <int D>
__device__ __forceinline__ uint8_t* kv4_tile(const mk_kv4_cache& c, const int32_t* table_row, int layer, int head,
                                             int tile) {
  const int page = table_row[tile / kKv4Tiles];
  if ((unsigned)page >= (unsigned)c.n_pages) return nullptr;
  const size_t at = (((size_t)layer * c.n_pages + page) * c.n_kv_heads + head) * kKv4Tiles + tile % kKv4Tiles;
  return static_cast<uint8_t*>(c.pool) + at * Kv4<D>::kBytes;
}

// ---- rows of 16-bit or 32-bit values ----
template <class T>
__device__ __forceinline__ void load8(const void* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const void* p, float (&x)[8]) {
  const float4 a = __ldg(static_cast<const float4*>(p)), b = __ldg(static_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const void* p, float (&x)[8]) {
  const uint4 a = ldnc16(p);
  x[0] = bf_lo(a.x); x[1] = bf_hi(a.x); x[2] = bf_lo(a.y); x[3] = bf_hi(a.y);
  x[4] = bf_lo(a.z); x[5] = bf_hi(a.z); x[6] = bf_lo(a.w); x[7] = bf_hi(a.w);
}
template <>
__device__ __forceinline__ void load8<__half>(const void* p, float (&x)[8]) {
  const uint4 a = ldnc16(p);
  x[0] = h_lo(a.x); x[1] = h_hi(a.x); x[2] = h_lo(a.y); x[3] = h_hi(a.y);
  x[4] = h_lo(a.z); x[5] = h_hi(a.z); x[6] = h_lo(a.w); x[7] = h_hi(a.w);
}
__device__ __forceinline__ uint32_t pack_bf(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_h(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <class T>
__device__ __forceinline__ void store8(void* p, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<float>(void* p, const float (&x)[8]) {
  static_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  static_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(void* p, const float (&x)[8]) {
  *static_cast<uint4*>(p) =
      make_uint4(pack_bf(x[0], x[1]), pack_bf(x[2], x[3]), pack_bf(x[4], x[5]), pack_bf(x[6], x[7]));
}
template <>
__device__ __forceinline__ void store8<__half>(void* p, const float (&x)[8]) {
  *static_cast<uint4*>(p) = make_uint4(pack_h(x[0], x[1]), pack_h(x[2], x[3]), pack_h(x[4], x[5]), pack_h(x[6], x[7]));
}

// ---- quantisation ----

// sign of a + b - x, exactly (two-sum: s + e == a + b)
__device__ __forceinline__ int cmp_sum(float a, float b, float x) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  const float e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
  return s > x ? 1 : s < x ? -1 : e > 0.f ? 1 : e < 0.f ? -1 : 0;
}

// Codes of this thread's 8 values (4 bits each, value i at bits 4 i) and the group's
// scale and minimum; the 4 threads of a group are neighbouring lanes of one aligned
// quad, and every lane of the warp calls.  A group that holds anything beyond
// +-2^15, an infinity or a NaN gets NaN parameters, so it reads back as NaN.
// Everything is decided exactly as in real arithmetic: where the fast quotient is
// within its error of a border between two codes, the border z + (k + 1/2) s is
// compared with x through an exact sum.
__device__ __forceinline__ uint32_t kv4_quantise(const float (&x)[8], __half& s_out, __half& z_out) {
  float lo = x[0], hi = x[0];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    bad |= !(fabsf(x[i]) <= 32768.f);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    bad |= __shfl_xor_sync(0xFFFFFFFFu, (int)bad, o) != 0;
  }
  if (bad) {
    s_out = z_out = __ushort_as_half((unsigned short)0x7FFF);
    return 0u;
  }
  const __half zh = __float2half_rd(lo);
  const float z = __half2float(zh);
  // smallest fp16 s with z + 15 s >= max: a guess within one step, then the exact test
  unsigned short sb = __half_as_ushort(__float2half_ru((hi - z) * (1.0f / 15.0f)));
  auto covers = [&](unsigned short b) {
    return cmp_sum(15.0f * __half2float(__ushort_as_half(b)), z, hi) >= 0;
  };
  if (!covers(sb)) ++sb;
  else if (sb != 0 && covers((unsigned short)(sb - 1))) --sb;
  const float s = __half2float(__ushort_as_half(sb));
  const float inv = s > 0.f ? 1.0f / s : 0.f;
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (x[i] - z) * inv;  // within 2^-18 of the quotient (t < 16)
    float n = rintf(t);
    if (fabsf(t - n) > 0.5f - 7.6e-6f) {
      const float k = t > n ? n : n - 1.0f;
      const int c = cmp_sum((k + 0.5f) * s, z, x[i]);  // border - x
      n = c < 0 ? k + 1.0f : c > 0 ? k : (((int)k & 1) ? k + 1.0f : k);
    }
    codes |= (uint32_t)(int)n << (4 * i);
  }
  s_out = __ushort_as_half(sb);
  z_out = zh;
  return codes;
}

}  // namespace mk
