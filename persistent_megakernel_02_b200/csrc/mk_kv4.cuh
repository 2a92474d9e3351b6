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
#include "mk_kv4.h"

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

// The sequence that owns slot `slot`, where sequence i owns the slots from (cu[i] >> shift) + extra i up to
// the next one's first (the caller sees whether the slot is before the first sequence's or behind the
// last one's).  A warp looks at 32 sequences at a time, every lane calls.  -1 where cu does not ascend in
// such a way that some slot of that sequence would lead elsewhere: all of the `cu` looked at are on the
// right side of the sequence's own, so every slot of it takes the same way, and of two sequences that
// are found none has rows of the other.  (kv4_report_order tells of every cu that does not ascend.)
__device__ __forceinline__ int kv4_owner(const mk_kv4_batch& b, int slot, int shift, int extra) {
  if (b.n_seqs == 1) return 0;
  const int lane = threadIdx.x & 31;
  int lo = 0, n = b.n_seqs, below = -0x7FFFFFFF - 1, above = 0x7FFFFFFF;
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lane * step;
    const int c = at < n ? b.cu[lo + at] : 0x7FFFFFFF;
    const bool left = lane == 0 || (at < n && (c >> shift) + extra * (lo + at) <= slot);
    const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, left));
    if (lane <= k) below = max(below, c);
    else above = min(above, c);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return __all_sync(0xFFFFFFFFu, below <= b.cu[lo] && above >= b.cu[lo + 1]) ? lo : -1;
}
// Thread `i` of a call with at least n_seqs of them looks at one pair.  (A sequence alone is looked at in any case.)
__device__ __forceinline__ void kv4_report_order(const mk_kv4_cache& c, const mk_kv4_batch& b, long long i) {
  if (b.n_seqs > 1 && i < b.n_seqs && b.cu[i + 1] < b.cu[i]) atomicOr(c.status, KV4_BAD_BATCH);
}

// The row tile of a prompt's CTA, `idx` counting them without the splits; those that see most of
// their sequence come first.  Every lane calls.
struct Kv4Block {
  int seq, head, tile;  // seq -1: a cu that does not ascend; tile: may be none of the sequence's
};
__device__ __forceinline__ Kv4Block kv4_block(const Kv4AttnSplit& a, int idx) {
  Kv4Block r;
  if (a.n_blocks == 0) {
    r.tile = a.n_rt - 1 - idx / (a.c.n_kv_heads * a.b.n_seqs);
    idx %= a.c.n_kv_heads * a.b.n_seqs;
    r.seq = idx / a.c.n_kv_heads;
  } else {
    const int slot = a.n_blocks - 1 - idx / a.c.n_kv_heads;
    r.seq = kv4_owner(a.b, slot, a.row_shift, 1);
    r.tile = r.seq < 0 ? -1 : slot - (a.b.cu[r.seq] >> a.row_shift) - r.seq;
  }
  r.head = idx % a.c.n_kv_heads;
  return r;
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

// Waits for a phase of an mbarrier, a bounded number of tries; on expiry the cache's
// status word says so.  A look first (27 cycles where the phase is over, the suspending
// try takes 100), then tries that suspend the thread for a while, 4 us measured, so about a second
// in all (spinning instead takes
// issue slots from the other warps: a 2048-token prompt 79 -> 82 us).
constexpr int kKv4Tries = 1 << 18;
__device__ __forceinline__ bool kv4_wait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  uint32_t over;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(over)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (over) return true;
  for (int i = 0; i < kKv4Tries; ++i)
    if (mbar_try_wait_hint(bar, parity, 10000)) return true;
  atomicOr(status, KV4_TIMEOUT);
  return false;
}

// ---- arithmetic of the attention kernels ----
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // at the rate of a maximum of two
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// What accumulated scores are multiplied by to be in powers of two, kept finite: where it is not
// (queries beyond 2^100, a scale beyond 1e34) scores that differ at all do so by 2^-72 of the
// accumulated ones, so that the largest has all the weight with 2^127 too.  Never zero: it
// multiplies the -inf of masked positions.
__device__ __forceinline__ float kv4_score_scale(float k) { return fminf(fmaxf(k, 1e-37f), 1.7e38f); }

// ---- rows of 16-bit or 32-bit values ----
template <class T>
struct Raw8 {  // 8 values as they are in memory
  uint4 v[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ Raw8<T> load_raw8(const void* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = ldnc16(static_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint4 a = r.v[0];
  x[0] = bf_lo(a.x); x[1] = bf_hi(a.x); x[2] = bf_lo(a.y); x[3] = bf_hi(a.y);
  x[4] = bf_lo(a.z); x[5] = bf_hi(a.z); x[6] = bf_lo(a.w); x[7] = bf_hi(a.w);
}
__device__ __forceinline__ void unpack8(const Raw8<__half>& r, float (&x)[8]) {
  const uint4 a = r.v[0];
  x[0] = h_lo(a.x); x[1] = h_hi(a.x); x[2] = h_lo(a.y); x[3] = h_hi(a.y);
  x[4] = h_lo(a.z); x[5] = h_hi(a.z); x[6] = h_lo(a.w); x[7] = h_hi(a.w);
}
template <class T>
__device__ __forceinline__ void load8(const void* p, float (&x)[8]) {
  unpack8(load_raw8<T>(p), x);
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

// minimum and maximum that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// {minimum, -maximum} of 8 values, NaN where one is; 16-bit types in packed pairs
__device__ __forceinline__ float2 extent8(const Raw8<float>& r) {
  float x[8];
  unpack8(r, x);
  return make_float2(
      min_nan(min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), min_nan(min_nan(x[4], x[5]), min_nan(x[6], x[7]))),
      -max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7]))));
}
template <class H2, class T>
__device__ __forceinline__ float2 extent8_packed(const Raw8<T>& r) {
  const H2* h = reinterpret_cast<const H2*>(&r.v[0]);
  const H2 lo = __hmin2_nan(__hmin2_nan(h[0], h[1]), __hmin2_nan(h[2], h[3]));
  const H2 hi = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
  return make_float2(min_nan((float)lo.x, (float)lo.y), -max_nan((float)hi.x, (float)hi.y));
}
__device__ __forceinline__ float2 extent8(const Raw8<__nv_bfloat16>& r) { return extent8_packed<__nv_bfloat162>(r); }
__device__ __forceinline__ float2 extent8(const Raw8<__half>& r) { return extent8_packed<__half2>(r); }

// Scale and minimum of a group with these extremes (low 16 bits the scale).  A group
// that holds anything beyond +-2^15, an infinity or a NaN gets NaN for both, so it
// reads back as NaN.
__device__ __forceinline__ uint32_t kv4_params(float lo, float hi) {
  if (!(lo >= -32768.f && hi <= 32768.f)) return 0x7FFF7FFFu;
  const __half zh = __float2half_rd(lo);
  const float z = __half2float(zh);
  // smallest fp16 s with z + 15 s >= max: rounded up from just below the quotient it is
  // that one or the one before, which the exact sum tells
  uint32_t sb = __half_as_ushort(__float2half_ru((hi - z) * (0.9999995f / 15.0f)));
  if (cmp_sum(15.0f * __half2float(__ushort_as_half((unsigned short)sb)), z, hi) < 0) ++sb;
  return sb | (uint32_t)__half_as_ushort(zh) << 16;
}

constexpr float kRound = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer, kept in the low bits

// The code of x next to a border between two codes, as in real arithmetic: the border
// z + (k + 1/2) s is compared with x through an exact sum; ties go to the even code.
__device__ __forceinline__ uint32_t kv4_code_exact(float x, float s, float z, float inv) {
  const float t = (x - z) * inv;  // within 2^-18 of the quotient
  float n = (t + kRound) - kRound;
  if (fabsf(t - n) > 0.5f - 7.6e-6f) {
    const float k = t > n ? n : n - 1.0f;
    const int c = cmp_sum((k + 0.5f) * s, z, x);  // border - x
    n = c < 0 ? k + 1.0f : c > 0 ? k : (((int)k & 1) ? k + 1.0f : k);
  }
  return (uint32_t)(int)n;
}
// (a call of its own: inlined for every 8 values it made the kernel miss the instruction
// cache, a third of its stalls)
static __device__ __noinline__ uint32_t kv4_codes_exact(float x0, float x1, float x2, float x3, float x4, float x5,
                                                        float x6, float x7, float s, float z, float inv) {
  return kv4_code_exact(x0, s, z, inv) | kv4_code_exact(x1, s, z, inv) << 4 | kv4_code_exact(x2, s, z, inv) << 8 |
         kv4_code_exact(x3, s, z, inv) << 12 | kv4_code_exact(x4, s, z, inv) << 16 |
         kv4_code_exact(x5, s, z, inv) << 20 | kv4_code_exact(x6, s, z, inv) << 24 | kv4_code_exact(x7, s, z, inv) << 28;
}

// Codes of 8 values of a group (4 bits each, value i at bits 4 i); inv is 1 / s to 2^-23,
// 0 where s is 0 or NaN.  Integers come through the low bits of a float: the
// conversion instructions run at an eighth of the rate.
__device__ __forceinline__ uint32_t kv4_codes(const float (&x)[8], uint32_t params, float inv) {
  const float z = h_hi(params), zi = -z * inv;
  if (inv == 0.f) return 0u;  // all equal, or NaN
  // (the shifted bits of kRound are taken off together: one instruction per code)
  constexpr uint32_t kBias = 0x4B400000u * 0x11111111u;
  uint32_t codes = 0u - kBias;
  float off = 0.f;  // largest distance from an integer
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fmaf(x[i], inv, zi), n = t + kRound;
    off = fmaxf(off, fabsf(t - (n - kRound)));
    codes += __float_as_uint(n) << (4 * i);
  }
  // t is off by 2^-24 of z / s (rounded once) and, t being below 16, by 16 (2^-23 + 2^-24)
  if (off > 0.5f - fmaf(fabsf(zi), 1.2e-7f, 3.9e-6f))  // some value is next to a border
    codes = kv4_codes_exact(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], h_lo(params), z, inv);
  return codes;
}

// What a lane sends and keeps when four items, one quarter of each in every lane of a
// quad, are reduced so that lane k of the quad ends up with item k.
__device__ __forceinline__ float quad_scatter_min(float e0, float e1, float e2, float e3, int lane) {
  const bool odd = lane & 1, high = lane & 2;
  const float a = min_nan(odd ? e1 : e0, __shfl_xor_sync(0xFFFFFFFFu, odd ? e0 : e1, 1));
  const float b = min_nan(odd ? e3 : e2, __shfl_xor_sync(0xFFFFFFFFu, odd ? e2 : e3, 1));
  return min_nan(high ? b : a, __shfl_xor_sync(0xFFFFFFFFu, high ? a : b, 2));
}

// the 8 values of a K word (or of two V units) of a group with scale s and minimum z
__device__ __forceinline__ void kv4_values(uint32_t codes, float s, float z, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = __uint_as_float((codes >> (4 * i) & 15u) | __float_as_uint(8388608.0f)) - 8388608.0f;
    x[i] = fmaf(s, c, z);
  }
}

}  // namespace mk
