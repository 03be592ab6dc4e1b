// cache.cuh -- the paged 4-bit key/value cache: layout, writing, reading back,
// and the selection of its blocks for a step's queries. (The attention over it
// is in cache_attn.cuh.)
//
// One page holds one block of bs tokens of every key/value head, per head as
// bs / 64 tiles of 64 tokens. A tile is 72 D bytes:
//   K codes   [64 tokens][D / 2]          token r, channel c: see k_word
//   V codes   [32 token pairs][D]         see v_chunk
//   K scales  [64 tokens][D / 64] (scale, zero) bf16 pairs
//   V scales  [64 tokens][D / 64] (scale, zero) bf16 pairs
// The order of the codes is the one in which the attention kernel's matrix
// instructions want them: each of its threads reads a tile with 16-byte (D =
// 128; 8-byte for D = 64) shared-memory loads free of bank conflicts, and a
// 32-bit word holds eight codes that two masks per byte of shift turn into
// float16 pairs.
//   K: word wi (of D / 32) of quarter t (0..3) of a token's row holds the
//      channels 32 wi + 8 t + 0..7, the lowest four bits the first; words lie
//      in the order [t][wi].
//   V: word wi of chunk g (0..7) of token pair p holds the channels 32 wi + 4 g
//      + 0..3 of token 2 p in its low half and of token 2 p + 1 in its high
//      half; chunks lie in the order g ^ (2 (p % 4)), words in [chunk][wi].
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "bsa_ptx.cuh"

namespace bsa {

constexpr int kCacheTile = 64;  // tokens of a tile

__host__ __device__ constexpr int cache_tile_bytes(int D) { return 72 * D; }
__host__ __device__ constexpr int cache_v_offset(int D) { return 32 * D; }
__host__ __device__ constexpr int cache_ks_offset(int D) { return 64 * D; }
__host__ __device__ constexpr int cache_vs_offset(int D) { return 68 * D; }

// Byte of the 32-bit word with octet `oct` (channels 8 oct .. 8 oct + 7) in a
// token's K row.
__host__ __device__ constexpr int k_word(int oct, int D) { return (oct % 4) * (D / 8) + (oct / 4) * 4; }
// Byte of the word with channels 8 oct + 4 hi .. + 3 in the V row of pair p.
__host__ __device__ constexpr int v_word(int p, int oct, int hi, int D) {
  return ((((oct % 4) * 2 + hi) ^ (2 * (p % 4))) * (D / 8)) + (oct / 4) * 4;
}

// What the cache operators know of one call's sequences.
struct CacheSeqs {
  const int32_t* table;  // [B, max_blocks]: page of each block; outside [0, num_pages): absent
  const int32_t* start;  // [B]: tokens in the cache before this step's
  const int32_t* count;  // [B]: this step's new tokens (null: T)
  int T, num_pages, max_blocks, bs;
};

// Start and count of a sequence, brought into range: a negative start makes the
// sequence empty, count lies in [0, T], start in [0, capacity].
__device__ __forceinline__ void seq_step(const CacheSeqs& s, int b, int& start, int& count) {
  start = s.start[b];
  count = s.count ? s.count[b] : s.T;
  count = start < 0 ? 0 : max(0, min(count, s.T));
  start = max(0, min(start, s.max_blocks * s.bs));
}

// Page of a block, or -1 where the table has none.
__device__ __forceinline__ int seq_page(const CacheSeqs& s, int b, int block) {
  if (block < 0 || block >= s.max_blocks) return -1;
  const int page = s.table[static_cast<long>(b) * s.max_blocks + block];
  return page >= 0 && page < s.num_pages ? page : -1;
}

__device__ __forceinline__ uint8_t* tile_ptr(uint8_t* cache, int page, int h, int tile, int Hkv, int bs, int D) {
  return cache + ((static_cast<long>(page) * Hkv + h) * (bs / kCacheTile) + tile) * cache_tile_bytes(D);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight consecutive channels as they lie in memory.
template <typename T>
struct Octet;
template <>
struct Octet<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* x) { u = __ldg(reinterpret_cast<const uint4*>(x)); }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  // The largest and smallest value, NaN if one is: on bfloat16 pairs, the smallest negated beside the largest, so that
  // one exchange and one maximum serve both.
  using Range = uint32_t;
  __device__ __forceinline__ Range range() const {
    const uint32_t hi = pair_max(pair_max(u.x, u.y), pair_max(u.z, u.w));
    const uint32_t lo = pair_min(pair_min(u.x, u.y), pair_min(u.z, u.w));
    return pair_max(__byte_perm(hi, lo, 0x5410) ^ 0x80000000u, __byte_perm(hi, lo, 0x7632) ^ 0x80000000u);
  }
  static __device__ __forceinline__ Range join(Range a, Range b) { return pair_max(a, b); }
  static __device__ __forceinline__ Range other(Range a, int d) { return __shfl_xor_sync(0xffffffffu, a, d); }
  static __device__ __forceinline__ void limits(Range m, float& mx, float& mn) {
    mx = __uint_as_float(m << 16);
    mn = -__uint_as_float(m & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
};
template <>
struct Octet<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* x) {
    a = __ldg(reinterpret_cast<const float4*>(x)), b = __ldg(reinterpret_cast<const float4*>(x) + 1);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  using Range = float2;  // largest, smallest
  __device__ __forceinline__ Range range() const {
    return make_float2(
        max_nan(max_nan(max_nan(a.x, a.y), max_nan(a.z, a.w)), max_nan(max_nan(b.x, b.y), max_nan(b.z, b.w))),
        min_nan(min_nan(min_nan(a.x, a.y), min_nan(a.z, a.w)), min_nan(min_nan(b.x, b.y), min_nan(b.z, b.w))));
  }
  static __device__ __forceinline__ Range join(Range a, Range b) {
    return make_float2(max_nan(a.x, b.x), min_nan(a.y, b.y));
  }
  static __device__ __forceinline__ Range other(Range a, int d) {
    return make_float2(__shfl_xor_sync(0xffffffffu, a.x, d), __shfl_xor_sync(0xffffffffu, a.y, d));
  }
  static __device__ __forceinline__ void limits(Range m, float& mx, float& mn) { mx = m.x, mn = m.y; }
};
__device__ __forceinline__ void store_octet(__nv_bfloat16* x, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(x) =
      make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store_octet(float* x, const float (&f)[8]) {
  reinterpret_cast<float4*>(x)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(x)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ void unpack_sz(uint32_t sz, float& scale, float& zero) {
  scale = __uint_as_float(sz << 16);
  zero = __uint_as_float(sz & 0xffff0000u);
}

// Scale and zero of a group of 64 channels with these limits, and what the
// quantising multiplies by.
//   z = bf16(min), s = bf16((max - z) * fl(1/15)), code = rint((x - z) * fl(1/s))
// in float32. A scale below the smallest normal float32 becomes 0 (all codes
// 0: the group reads back as its zero). A group with a NaN or infinity, or
// with a range beyond float32, gets NaN for both and reads back as NaN.
__device__ __forceinline__ void group_scale(float mx, float mn, uint32_t& sz, float& inv) {
  const float z = __bfloat162float(__float2bfloat16_rn(mn));
  const float range = __fsub_rn(mx, z);
  float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(range, 1.0f / 15.0f)));
  if (s < 1.17549435e-38f) s = 0.0f;  // a NaN stays
  const bool finite = fabsf(range) < CUDART_INF_F;
  inv = s > 0.0f && finite ? __frcp_rn(s) : 0.0f;
  sz = finite ? (__float_as_uint(s) >> 16) | __float_as_uint(z) : 0x7fff7fffu;
}

// The codes of the eight channels of this lane, packed in channel order (lowest
// bits first), and as whole floats in `code` (pairs).
template <typename T>
__device__ __forceinline__ uint32_t octet_codes(const Octet<T>& x, uint32_t sz, float inv, uint64_t (&code)[4]) {
  const float z = __uint_as_float(sz & 0xffff0000u);
  float f[8];
  x.floats(f);
  // 12582912 = 1.5 * 2^23: adding it rounds to a whole number, half to even, and leaves that number in the low bits
  constexpr float kRound = 12582912.0f;
  const uint64_t zz = f2(z, z), rr = f2(kRound, kRound);
  uint32_t w = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    // the products are single instructions: a packed product and the packed sum after it become one fused
    // multiply-add, whose codes differ at halves
    float lo, hi;
    f2_split(f2_sub(f2(f[2 * i], f[2 * i + 1]), zz), lo, hi);
    lo = __fmul_rn(lo, inv), hi = __fmul_rn(hi, inv);
    if constexpr (sizeof(T) == 4) {
      // a float32 minimum may lie below its bfloat16 zero; of bfloat16 values no quotient leaves [0, 15.04], since
      // the zero is one of them and the scale is off by at most 2^-8
      lo = fminf(fmaxf(lo, 0.0f), 15.0f), hi = fminf(fmaxf(hi, 0.0f), 15.0f);
    }
    const uint64_t t = f2_add(f2(lo, hi), rr);
    f2_split(t, lo, hi);
    // the constant's bits above the number fall out at the top, or are taken off below
    w = (w << 8) + (__float_as_uint(hi) << 4) + __float_as_uint(lo);
    code[i] = f2_sub(t, rr);
  }
  // w = sum of (bits(kRound) + code) << 4 i: the lowest three of those constants reach into 32 bits
  constexpr uint32_t kBits = 0x4b400000u;
  return w - (kBits + (kBits << 4) + (kBits << 8));
}

// Range, scale and codes of one octet; the eight lanes of an aligned group hold
// the 64 channels that share a scale.
template <typename T>
__device__ __forceinline__ uint32_t quantise_octet(const Octet<T>& x, uint32_t& sz, uint64_t (&code)[4]) {
  typename Octet<T>::Range m = x.range();
#pragma unroll
  for (int d = 1; d < 8; d *= 2) m = Octet<T>::join(m, Octet<T>::other(m, d));
  float mx, mn, inv;
  Octet<T>::limits(m, mx, mn);
  group_scale(mx, mn, sz, inv);
  return octet_codes(x, sz, inv, code);
}

// ------------------------------------------------------------------ write
//
// One CTA per (sequence, block that the new tokens touch, key/value head). It
// quantises the block's new rows and sums the keys of all its rows up to the
// last new one, as the cache holds them, so that k_sum depends on the cache's
// contents alone: not on how the tokens were cut into calls, nor on rows that a
// later write with a smaller start has replaced. Row r of a tile belongs to a
// fixed warp and lane group, which adds up scale code and zero of its rows
// apart, in their order, and the partial sums are joined in a fixed order.
// Bound for a prompt: the bytes (2 to 4 in, 9/16 out an element), as long as the
// quantising stays below about 10 instructions an element: the arithmetic runs
// on float32 pairs, minima and maxima on bfloat16 pairs, and the eight lanes of a
// group compute eight octets' scales apart (325 us without that). 131072 tokens of
// 16 heads, D = 128, bf16: 270 us for 1.37 GB, 5.1 TB/s; 87 instructions an octet
// keep the SMs busier than the memory (profiled: issue 62%, the memory's bus 62%). One token of 64 sequences: about 4 us of
// latencies (length, page, older keys, new ones); with the reading back 6.6 us in a captured run, 18.8 issued from Python.
template <typename T, int D>
__global__ void __launch_bounds__(128) cache_write_kernel(const T* __restrict__ k, const T* __restrict__ v,
                                                          uint8_t* cache, float* k_sum, CacheSeqs s, int Hkv,
                                                          int nslot) {
  constexpr int kOct = D / 8, kRows = 32 / kOct, kStep = 4 * kRows, kSteps = kCacheTile / kStep;
  __shared__ float part[4][D];
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x % Hkv, slot = blockIdx.x / Hkv % nslot, b = blockIdx.x / Hkv / nslot;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, oct = lane % kOct, sub = lane / kOct;
  int start, count;
  seq_step(s, b, start, count);
  const int block = start / s.bs + slot;
  const int first = block * s.bs;                       // the block's first token
  const int r0 = max(start - first, 0), r1 = min(start + count - first, s.bs);  // new rows
  const int page = seq_page(s, b, block);
  if (page < 0 || r1 <= r0) return;
  // row r of the block (r0 <= r < r1) of k and v
  const long row_of = static_cast<long>(Hkv) * D, at0 = ((static_cast<long>(b) * s.T + first - start) * Hkv + h) * D + oct * 8;
  uint64_t acc[4] = {};  // sums of scale code, in channel pairs
  float acc_zero = 0.0f;

  auto add_keys = [&](uint32_t sz, const uint64_t (&code)[4]) {
    float sc, ze;
    unpack_sz(sz, sc, ze);
    const uint64_t ss = f2(sc, sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f2_fma(ss, code[i], acc[i]);
    acc_zero += ze;
  };

  for (int tile = 0; tile * kCacheTile < r1; ++tile) {
    uint8_t* base = tile_ptr(cache, page, h, tile, Hkv, s.bs, D);
    const int t0 = tile * kCacheTile, mine = warp * kRows + sub;  // this lane group's rows: mine + step kStep
    if (r0 <= t0 && r1 >= t0 + kCacheTile) {
      // a tile of new rows only: the keys and values of four (float32: two, for registers) rows at a time, so many
      // octets a lane. Each of a group's lanes ends up with one octet's range (four, two and one exchanges instead of
      // three for each), computes its scale for all and stores it.
      using X = Octet<T>;
      constexpr int kAhead = sizeof(T) == 2 ? 4 : 2, kN = 2 * kAhead;
#pragma unroll 1
      for (int i0 = 0; i0 < kSteps; i0 += kAhead) {
        X x[kN];
        typename X::Range m[kN];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const long at = at0 + (t0 + mine + (i0 + i) * kStep) * row_of;
          x[i].load(k + at);
          x[kAhead + i].load(v + at);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) m[i] = x[i].range();
#pragma unroll
        for (int d = kAhead; d; d /= 2) {
          const bool up = lane & d;
#pragma unroll
          for (int i = 0; i < d; ++i)
            m[i] = X::join(up ? m[i + d] : m[i], X::other(up ? m[i] : m[i + d], d));
        }
#pragma unroll
        for (int d = kN; d < 8; d *= 2) m[0] = X::join(m[0], X::other(m[0], d));
        float mx, mn, my_inv;
        uint32_t my_sz;
        X::limits(m[0], mx, mn);
        group_scale(mx, mn, my_sz, my_inv);
        const int my_row = mine + (i0 + lane % kAhead) * kStep;
        if (lane % 8 < kN)
          *reinterpret_cast<uint32_t*>(base + (lane & kAhead ? cache_vs_offset(D) : cache_ks_offset(D)) +
                                       (my_row * (D / 64) + oct / 8) * 4) = my_sz;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int r = mine + (i0 + i % kAhead) * kStep, from = (lane & 24) + i;
          const uint32_t sz = __shfl_sync(0xffffffffu, my_sz, from);
          const float inv = __shfl_sync(0xffffffffu, my_inv, from);
          uint64_t code[4];
          const uint32_t w = octet_codes(x[i], sz, inv, code);
          if (i < kAhead) {
            *reinterpret_cast<uint32_t*>(base + r * (D / 2) + k_word(oct, D)) = w;
            add_keys(sz, code);
          } else {
            // a pair's two rows are neighbouring lane groups: each makes one word of both rows' halves
            const bool odd = sub % 2;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w : w >> 16, kOct);
            const uint32_t both = odd ? __byte_perm(other, w, 0x7610) : __byte_perm(w, other, 0x5410);
            *reinterpret_cast<uint32_t*>(base + cache_v_offset(D) + (r / 2) * D + v_word(r / 2, oct, odd, D)) = both;
          }
        }
      }
      continue;
    }
    // older rows: their keys' codes and scales, all in flight together
    uint32_t w[kSteps], sz[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = mine + i * kStep;
      w[i] = sz[i] = 0;
      if (t0 + r < r0) {
        w[i] = *reinterpret_cast<const uint32_t*>(base + r * (D / 2) + k_word(oct, D));
        sz[i] = *reinterpret_cast<const uint32_t*>(base + cache_ks_offset(D) + (r * (D / 64) + oct / 8) * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      if (t0 + mine + i * kStep < r0) {
        uint64_t code[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          code[c] = f2(static_cast<float>(w[i] >> (8 * c) & 15u), static_cast<float>(w[i] >> (8 * c + 4) & 15u));
        add_keys(sz[i], code);
      }
#pragma unroll 1
    for (int i = 0; i < kSteps; ++i) {
      const int low = t0 + warp * kRows + i * kStep, row = low + sub;  // the warp's rows here begin at `low`
      if (low + kRows <= r0 || low >= r1) continue;
      const bool fresh = row >= r0 && row < r1;
      Octet<T> xk, xv;
      const long at = at0 + (fresh ? row : max(r0, low)) * row_of;  // (of a row that is there)
      xk.load(k + at);
      xv.load(v + at);
      const int r = row - t0, sc_at = (r * (D / 64) + oct / 8) * 4;
      uint32_t z;
      uint64_t code[4];
      uint32_t c = quantise_octet(xk, z, code);
      if (fresh) {
        *reinterpret_cast<uint32_t*>(base + r * (D / 2) + k_word(oct, D)) = c;
        if (oct % 8 == 0) *reinterpret_cast<uint32_t*>(base + cache_ks_offset(D) + sc_at) = z;
        add_keys(z, code);
      }
      c = quantise_octet(xv, z, code);
      if (fresh) {
        uint8_t* to = base + cache_v_offset(D) + (r / 2) * D + (r % 2) * 2;
        *reinterpret_cast<uint16_t*>(to + v_word(r / 2, oct, 0, D)) = static_cast<uint16_t>(c);
        *reinterpret_cast<uint16_t*>(to + v_word(r / 2, oct, 1, D)) = static_cast<uint16_t>(c >> 16);
        if (oct % 8 == 0) *reinterpret_cast<uint32_t*>(base + cache_vs_offset(D) + sc_at) = z;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[2];
    f2_split(acc[i], f[0], f[1]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      f[c] += acc_zero;
#pragma unroll
      for (int d = kOct; d < 32; d *= 2) f[c] += __shfl_xor_sync(0xffffffffu, f[c], d);
      if (lane < kOct) part[warp][oct * 8 + 2 * i + c] = f[c];
    }
  }
  __syncthreads();
  if (threadIdx.x < D)
    k_sum[(static_cast<long>(page) * Hkv + h) * D + threadIdx.x] =
        (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}

// ------------------------------------------------------------------ read
//
// One CTA per (sequence, up to 64 rows of one tile, key/value head): a row's
// eight channels a lane, as the writing lays them. Bound by the bytes (9/16 in, 2
// to 4 out an element): 131072 tokens of 16 heads, D = 128, bf16, in 217 us, 6.3 TB/s.
__device__ __forceinline__ void octet_values(uint32_t w, uint32_t sz, float (&f)[8]) {
  float sc, ze;
  unpack_sz(sz, sc, ze);
  // 2^23 + code is the float with the code in its low bits
  constexpr float kWhole = 8388608.0f;
  const uint64_t ss = f2(sc, sc), zz = f2(ze, ze), ww = f2(kWhole, kWhole);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t = f2(__uint_as_float((w >> (8 * i) & 15u) | 0x4b000000u),
                          __uint_as_float((w >> (8 * i + 4) & 15u) | 0x4b000000u));
    f2_split(f2_fma(ss, f2_sub(t, ww), zz), f[2 * i], f[2 * i + 1]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(128) cache_read_kernel(const uint8_t* __restrict__ cache, T* k, T* v, CacheSeqs s,
                                                         int Hkv, int nslot) {
  constexpr int kOct = D / 8, kRows = 32 / kOct, kStep = 4 * kRows, kSteps = kCacheTile / kStep;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x % Hkv, slot = blockIdx.x / Hkv % nslot, b = blockIdx.x / Hkv / nslot;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, oct = lane % kOct, sub = lane / kOct;
  int start, count;
  seq_step(s, b, start, count);
  const int first = (start / kCacheTile + slot) * kCacheTile;  // the tile's first token
  const int r0 = max(start - first, 0), r1 = min(start + count - first, kCacheTile);
  if (r1 <= r0) return;
  const int page = seq_page(s, b, first / s.bs);
  const uint8_t* base = page >= 0 ? tile_ptr(const_cast<uint8_t*>(cache), page, h, first % s.bs / kCacheTile, Hkv, s.bs, D)
                                  : nullptr;
  const long at0 = ((static_cast<long>(b) * s.T + first - start) * Hkv + h) * D + oct * 8;
  uint32_t kw[kSteps], vw[kSteps], ks[kSteps], vs[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    // whole pairs are read, also where only one row of them is wanted
    const int r = warp * kRows + sub + i * kStep, at = (r * (D / 64) + oct / 8) * 4;
    kw[i] = vw[i] = ks[i] = vs[i] = 0;
    if (base) {
      kw[i] = __ldg(reinterpret_cast<const uint32_t*>(base + r * (D / 2) + k_word(oct, D)));
      vw[i] = __ldg(reinterpret_cast<const uint32_t*>(base + cache_v_offset(D) + (r / 2) * D + v_word(r / 2, oct, r % 2, D)));
      ks[i] = __ldg(reinterpret_cast<const uint32_t*>(base + cache_ks_offset(D) + at));
      vs[i] = __ldg(reinterpret_cast<const uint32_t*>(base + cache_vs_offset(D) + at));
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = warp * kRows + sub + i * kStep;
    const bool odd = r % 2;
    // this lane read the first (even rows) or second four channels of both rows of its pair
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? vw[i] : vw[i] >> 16, kOct);
    const uint32_t w = odd ? __byte_perm(other, vw[i], 0x7610) : __byte_perm(vw[i], other, 0x5410);
    if (r < r0 || r >= r1) continue;
    float f[8];
    octet_values(kw[i], ks[i], f);
    store_octet(k + at0 + r * static_cast<long>(Hkv) * D, f);
    octet_values(w, vs[i], f);
    store_octet(v + at0 + r * static_cast<long>(Hkv) * D, f);
  }
}

// ------------------------------------------------------------------ block selection
//
// One cluster of 1 to 16 CTAs per (sequence, key/value head). Its CTAs score a
// slice of the row's blocks each (eight lanes a block, so that a block's sums are
// one read of D float32 by neighbouring lanes) and store order-preserving keys in
// the first CTA's shared memory; that CTA finds the topk-th largest key by three
// histograms (short rows: by comparing all with all) and writes the ids in
// ascending order.
// The bytes of the sums bound it (B H_kv blocks D 4 bytes) where there are many;
// a short row is a chain of latencies: lengths, pages, sums, three histograms.
// 32 rows x 4 heads of up to 1024 blocks, D = 128: 17 us (lengths, pages and queries 3.4,
// scoring 10.3, selecting 3); 4096 blocks of 8 heads: 15 us (3.4, 4.3, 7.1); 128 blocks: 4.9 us
// in a captured run, 13 issued from Python (the host's time).
// The dot products run in float64 and are rounded to float32 once, so that which
// blocks are kept does not depend on an order of summation.
constexpr int kCacheSelThreads = 256, kCacheSelWarps = kCacheSelThreads / 32;

constexpr uint32_t kForcedKey = 0xffffffffu;  // a forced block ranks above every score, a NaN among the scores first
__device__ __forceinline__ uint32_t cache_score_key(float x) {
  if (x != x) return kForcedKey - 1;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The address of this CTA's shared-memory address `a` in the cluster's first CTA.
__device__ __forceinline__ uint32_t first_cta_addr(uint32_t a) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(kCacheSelThreads) cache_topk_kernel(const T* __restrict__ q,
                                                                      const float* __restrict__ k_sum, int32_t* idx,
                                                                      CacheSeqs s, int H, int Hkv, int topk,
                                                                      int force) {
  constexpr int kVec = D / 32;     // float4s of a lane
  constexpr int kSplit = kCacheSelThreads / D;
  extern __shared__ uint32_t keys[];  // [max_blocks]: pages of this CTA's slice, then (in the first CTA) all keys
  __shared__ double q_part[kSplit][D];
  __shared__ uint2 warp_n[kCacheSelWarps];
  __shared__ __align__(16) uint32_t hist[2048];
  __shared__ uint3 found;
  pdl_launch_dependents();
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  cluster_sync();  // the first CTA's shared memory is there before anyone stores to it
  pdl_wait();
  const int row = blockIdx.x / ctas, h = row % Hkv, b = row / Hkv, G = H / Hkv;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int start, count;
  seq_step(s, b, start, count);
  const int total = min(start + count, s.max_blocks * s.bs);
  const int n = (total + s.bs - 1) / s.bs;
  const int lo = static_cast<int>(static_cast<long>(n) * rank / ctas),
            hi = static_cast<int>(static_cast<long>(n) * (rank + 1) / ctas);
  // this slice's first pages are on their way while the queries are summed
  const int p0 = lo + tid, p1 = p0 + kCacheSelThreads;
  const int page0 = p0 < hi ? seq_page(s, b, p0) : -1, page1 = p1 < hi ? seq_page(s, b, p1) : -1;
  {
    const int d = tid % D, part = tid / D;
    const T* at = q + (static_cast<long>(b) * s.T * H + h * G) * D + d;
    double sum = 0;
#pragma unroll 8
    for (int r = part; r < count * G; r += kSplit) sum += to_float(at[(static_cast<long>(r / G) * H + r % G) * D]);
    q_part[part][d] = sum;
  }
  if (p0 < hi) keys[p0] = static_cast<uint32_t>(page0);
  if (p1 < hi) keys[p1] = static_cast<uint32_t>(page1);
  for (int j = p1 + kCacheSelThreads; j < hi; j += kCacheSelThreads)
    keys[j] = static_cast<uint32_t>(seq_page(s, b, j));
  __syncthreads();
  const int sub = lane % 8, grp = lane / 8;
  double qd[kVec][4];
#pragma unroll
  for (int i = 0; i < kVec; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      double x = 0;
#pragma unroll
      for (int p = 0; p < kSplit; ++p) x += q_part[p][i * 32 + sub * 4 + c];
      qd[i][c] = x;
    }
  const double inv_bs = 1.0 / s.bs;
  const uint32_t to = first_cta_addr(smem_u32(keys));
  // scores of kN runs of 32 blocks from j0 on, their sums' loads all in flight together
  auto score = [&](int j0, auto runs) {
    constexpr int kN = decltype(runs)::value;
    int page[kN];
    float4 x[kN][kVec];
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const int j = j0 + (u * kCacheSelWarps + warp) * 4 + grp;
      page[u] = j < hi ? static_cast<int>(keys[j]) : -1;
      const float4* ks =
          reinterpret_cast<const float4*>(k_sum + (static_cast<long>(max(page[u], 0)) * Hkv + h) * D) + sub;
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[u][i] = __ldg(ks + i * 8);
    }
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const int j = j0 + (u * kCacheSelWarps + warp) * 4 + grp;
      double dot = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        dot = fma(qd[i][0], static_cast<double>(x[u][i].x), dot);
        dot = fma(qd[i][1], static_cast<double>(x[u][i].y), dot);
        dot = fma(qd[i][2], static_cast<double>(x[u][i].z), dot);
        dot = fma(qd[i][3], static_cast<double>(x[u][i].w), dot);
      }
#pragma unroll
      for (int o = 4; o; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (sub == 0 && j < hi) {  // the block's lanes have all read its page
        uint32_t key = 0;        // an absent block: below every score
        if (page[u] >= 0) {
          const int tokens = total - j * s.bs;
          // a full block's size is a power of two: the product with its inverse is exact
          key = cache_score_key(static_cast<float>(tokens >= s.bs ? dot * inv_bs : dot / tokens));
          if (force && count > 0 && (j + 1) * s.bs > start) key = kForcedKey;
        }
        store_cluster(to + 4u * j, key);
      }
    }
  };
  constexpr int kRunBlocks = 4 * kCacheSelWarps;
  int j0 = lo;
  for (; hi - j0 > 2 * kRunBlocks; j0 += 4 * kRunBlocks) score(j0, std::integral_constant<int, 4>{});
  if (hi - j0 > kRunBlocks)
    score(j0, std::integral_constant<int, 2>{});
  else if (hi > j0)
    score(j0, std::integral_constant<int, 1>{});
  cluster_sync();
  if (rank) return;

  int32_t* out = idx + static_cast<long>(row) * topk;
  const uint32_t below = (1u << lane) - 1u;
  int want;
  if (n <= kCacheSelThreads) {
    // a short row: each key's rank by comparison with all others (absent blocks rank nowhere)
    const uint32_t key = tid < n ? keys[tid] : 0u;
    int before = 0;
    if (warp * 32 < n) {
      for (int j = 0; j < warp * 32; ++j) before += keys[j] >= key;
      for (int j = warp * 32; j < min(n, warp * 32 + 32); ++j) before += keys[j] > key || (keys[j] == key && j < tid);
      for (int j = warp * 32 + 32; j < n; ++j) before += keys[j] > key;
    }
    want = min(topk, __syncthreads_count(key != 0));
    const bool up = key && before < want;
    const uint32_t mu = __ballot_sync(0xffffffffu, up);
    if (lane == 0) warp_n[warp] = make_uint2(__popc(mu), 0);
    __syncthreads();
    int at = __popc(mu & below);
    for (int w = 0; w < warp; ++w) at += warp_n[w].x;
    if (up) out[at] = tid;
  } else {
    // the want-th largest key by three histograms of 11, 11 and 10 bits: keys above its interval are in, and `need`
    // of those in it
    uint32_t thr = 0, width = 0;  // the interval: thr and its `width` lower bits
    int need = 0, present = 0;
#pragma unroll 8
    for (int j = tid; j < n; j += kCacheSelThreads) present += keys[j] != 0;
    present = __reduce_add_sync(0xffffffffu, present);
    if (lane == 0) warp_n[warp].x = present;
    __syncthreads();
    present = 0;
    for (int w = 0; w < kCacheSelWarps; ++w) present += warp_n[w].x;
    want = need = min(topk, present);
    if (want) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t bins = pass == 2 ? 1024 : 2048;
        __syncthreads();
        reinterpret_cast<uint4*>(hist)[tid] = reinterpret_cast<uint4*>(hist)[tid + kCacheSelThreads] = uint4{};
        __syncthreads();
#pragma unroll 8
        for (int j = tid; j < n; j += kCacheSelThreads) {
          const uint32_t key = keys[j];
          if (key && (pass == 0 || key >> width == thr >> width)) atomicAdd(&hist[key >> shift & (bins - 1)], 1u);
        }
        __syncthreads();
        // from the top: thread t looks after bins 8 (255 - t) .. + 7
        const int b0 = 8 * (kCacheSelThreads - 1 - tid);
        const uint4 o0 = *reinterpret_cast<const uint4*>(hist + b0), o1 = *reinterpret_cast<const uint4*>(hist + b0 + 4);
        const uint32_t own[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
        const uint32_t sum = o0.x + o0.y + o0.z + o0.w + o1.x + o1.y + o1.z + o1.w;
        uint32_t upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += x;
        }
        if (lane == 31) warp_n[warp].y = upto;
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += warp_n[w].y;
        if (upto >= static_cast<uint32_t>(need) && upto - sum < static_cast<uint32_t>(need)) {  // one thread
          uint32_t over = upto - sum;
#pragma unroll
          for (int i = 7; i >= 0; --i) {
            if (over < static_cast<uint32_t>(need) && over + own[i] >= static_cast<uint32_t>(need))
              found = make_uint3(b0 + i, need - over, own[i]);
            over += own[i];
          }
        }
        __syncthreads();
        thr |= found.x << shift;
        need = found.y;
        width = shift;
        if (need == static_cast<int>(found.z)) break;  // the whole interval is in
      }
    }
    // ids in ascending order, 1024 keys at a time: those above the interval, and in it the first ones
    const bool some = want && need < static_cast<int>(found.z);  // (equal keys then: all 32 bits are known)
    const uint32_t top = thr >> width;
    int above = 0, equal = 0;
    constexpr int kRun = 4;
    for (int base = 0; base < n && want; base += kRun * kCacheSelThreads) {
      uint32_t mu[kRun], ms[kRun];
      int a = 0, e = 0;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int j = base + (warp * kRun + i) * 32 + lane;
        const uint32_t key = j < n ? keys[j] : 0u, digit = key >> width;
        mu[i] = __ballot_sync(0xffffffffu, key && (some ? digit > top : digit >= top));
        ms[i] = __ballot_sync(0xffffffffu, key && some && digit == top);
        a += __popc(mu[i]);
        e += __popc(ms[i]);
      }
      __syncthreads();
      if (lane == 0) warp_n[warp] = make_uint2(a, e);
      __syncthreads();
      a = above, e = equal;
      for (int w = 0; w < kCacheSelWarps; ++w) {
        const uint2 x = warp_n[w];
        if (w < warp) a += x.x, e += x.y;
        above += x.x, equal += x.y;
      }
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const bool up = mu[i] >> lane & 1, same = ms[i] >> lane & 1;
        const int es = e + __popc(ms[i] & below);
        if (up || (same && es < need))
          out[a + __popc(mu[i] & below) + min(es, need)] = base + (warp * kRun + i) * 32 + lane;
        a += __popc(mu[i]);
        e += __popc(ms[i]);
      }
    }
  }
  for (int j = want + tid; j < topk; j += kCacheSelThreads) out[j] = -1;
}

}  // namespace bsa
