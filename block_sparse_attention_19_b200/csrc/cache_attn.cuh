// cache_attn.cuh -- attention of a step's queries over the 4-bit cache.
#pragma once

#include "cache.cuh"

namespace bsa {

// One CTA per (sequence, key/value head, query row); a tile of 64 tokens at a
// time: a thread per token for the scores, a thread per channel for the sums.
template <typename T, int D>
__global__ void __launch_bounds__(128) cache_attn_kernel(const T* __restrict__ q, const uint8_t* cache,
                                                         const int32_t* __restrict__ idx, T* o, CacheSeqs s, int H,
                                                         int Hkv, int topk, float scale_log2) {
  __shared__ float qs[D], p[kCacheTile], red[4];
  pdl_launch_dependents();
  pdl_wait();
  const int G = H / Hkv, tid = threadIdx.x;
  const int row = blockIdx.x % (s.T * G), h = blockIdx.x / (s.T * G) % Hkv, b = blockIdx.x / (s.T * G) / Hkv;
  const int t = row / G, head = h * G + row % G;
  int start, count;
  seq_step(s, b, start, count);
  if (t >= count) return;
  const int limit = min(start + t + 1, s.max_blocks * s.bs);  // tokens that the row sees
  const long at = ((static_cast<long>(b) * s.T + t) * H + head) * D;
  if (tid < D) qs[tid] = to_float(q[at + tid]) * scale_log2;
  float m = -CUDART_INF_F, l = 0.0f, acc = 0.0f;
  const int nblocks = idx ? topk : (limit + s.bs - 1) / s.bs;
  for (int n = 0; n < nblocks; ++n) {
    const int block = idx ? idx[(static_cast<long>(b) * Hkv + h) * topk + n] : n;
    const int page = seq_page(s, b, block);
    if (page < 0) continue;
    for (int tile = 0; tile < s.bs / kCacheTile; ++tile) {
      const int pos = block * s.bs + tile * kCacheTile;
      if (pos >= limit) break;
      const uint8_t* base = tile_ptr(const_cast<uint8_t*>(cache), page, h, tile, Hkv, s.bs, D);
      __syncthreads();
      float x = -CUDART_INF_F;
      if (tid < kCacheTile && pos + tid < limit) {
        x = 0.0f;
        for (int oct = 0; oct < D / 8; ++oct) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(base + tid * (D / 2) + k_word(oct, D));
          float sc, ze;
          unpack_sz(*reinterpret_cast<const uint32_t*>(base + cache_ks_offset(D) + (tid * (D / 64) + oct / 8) * 4), sc,
                    ze);
          for (int i = 0; i < 8; ++i)
            x += qs[oct * 8 + i] * cache_value(sc, ze, static_cast<float>((w >> (4 * i)) & 15u));
        }
      }
      float mx = x;
      for (int d = 16; d; d /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      if (tid % 32 == 0) red[tid / 32] = mx;
      __syncthreads();
      mx = fmaxf(m, fmaxf(red[0], red[1]));
      const float ref = mx == -CUDART_INF_F ? 0.0f : mx;
      if (tid < kCacheTile) p[tid] = exp2f(x - ref);
      const float f = exp2f(m - ref);
      m = mx;
      __syncthreads();
      l *= f, acc *= f;
      for (int r = 0; r < kCacheTile && pos + r < limit; ++r) {
        l += p[r];
        if (tid < D) {
          const int c = tid;
          const uint16_t w = *reinterpret_cast<const uint16_t*>(base + cache_v_offset(D) + (r / 2) * D + (r % 2) * 2 +
                                                                v_word(r / 2, c / 8, c / 4 % 2, D));
          float sc, ze;
          unpack_sz(*reinterpret_cast<const uint32_t*>(base + cache_vs_offset(D) + (r * (D / 64) + c / 64) * 4), sc,
                    ze);
          acc += p[r] * cache_value(sc, ze, static_cast<float>((w >> (4 * (c % 4))) & 15));
        }
      }
    }
  }
  if (tid < D) {
    const float r = l > 0.0f || l != l ? acc / l : 0.0f;
    if constexpr (sizeof(T) == 2)
      o[at + tid] = __float2bfloat16_rn(r);
    else
      o[at + tid] = r;
  }
}

}  // namespace bsa
