// cache_attn.cuh -- attention of a step's queries over the 4-bit cache.
//
// For the R = T G query rows of a (sequence, key/value head) and its tokens i,
//   x = scale log2(e) q.k_i,  o = sum 2^(x - M) v_i / sum 2^(x - M).
// With k = zero + scale code the score splits per group of 64 channels into
//   q.k = k_scale (q . code) + k_zero (sum of q's channels),
// and the output into sum p v_scale code + sum p v_zero, so the codes go to the
// matrix instructions as they are and scales and zeros meet sums only. The
// products run as S^T = K q^T and O^T = V^T P^T (m16n8k16, float16 in, float32
// sums): 16 tokens or 16 channels fill the tall side, and as few as 8 query rows
// the short one.
//
// The bound is the cache's bytes (4.5 bits an element, read once) as long as a
// tile of 64 tokens costs fewer issue slots than its 72 D bytes cost time at the
// memory rate, so the unpacking is kept short. Codes are operands as they are:
//   keys: a code in the low bits of a float16 is the subnormal code 2^-24, in bits
//     4..7 it is 16 code 2^-24, and that factor is taken out of the query. (As e4m3
//     numbers a byte of shift would do for eight codes instead of four, but those
//     matrix instructions made the kernel slower: 110 against 89 us at two CTAs an SM.)
//   values: float16 subnormals, of the byte lo + 16 hi and of lo alone; hi is the
//     difference of the two sums.
// float32 queries take the operands code - 8 instead (with zero + 8 scale): sums
// of both signs stay near the result's own size, and the matrix unit's truncating
// sums cost them nothing (with code, 1e-4 of the result at 6000 tokens).
// All of these operands are exact. For float16's range each query row is
// scaled by a power of two, and so are a row's weights of each group of 64 value
// channels: 2^(x - M) v_scale 2^e is kept below 2^15, with M near the row's largest
// score and e near 8 - log2 of the group's largest 2^(x - M) v_scale.
//
// All units' tiles lie in one line, cut into equal pieces for CTAs that are all
// resident at once; a unit that several CTAs share leaves one part for each, which a
// second launch joins. Measured on one B200 (6.55 TB/s copied), device time of a call in a captured run: 16
// sequences of 32768 tokens, 4 heads, four query rows each: 60 us for 302 MB, 5.0 TB/s; 15% of
// the blocks of up to 131072 tokens: 35 us; one sequence of 397 tokens: 8 us, of
// which 2 are the joining launch. (Issued one by one from Python: 63, 37 and 17 us; the last is the host's time
// for a call.) In the long run a tile costs its bytes' time, 0.214 us of an SM;
// the rest is a chain that every call has: lengths, plan, page, first tile (4 us),
// the last tiles' sums (1.3 us), the joining (2 to 4.5 us).
#pragma once

#include <cuda_fp16.h>

#include "cache.cuh"

namespace bsa {

constexpr int kCaWarps = 4;  // in two pairs: a tile goes to a pair, 32 tokens to a warp
constexpr int kCaThreads = kCaWarps * 32;
constexpr int kCaMaxExtra = 6;  // (see CaPlan)
constexpr int kCaMaxSeqs = 4096;  // sequences whose plan fits in shared memory
// A row's reference M is at least its largest score of the time when it was last raised, and a group's factor 2^e
// puts the largest weight times scale of that time between 2^kCaRaise and 2^(kCaRaise + 1). Later ones may reach 2^15
// before the next raise, and a raise weighs a tile twice: from 8 on at least 2^6 times the largest so far is left, with
// scores of deviation 2 most rows' last raise (40 rows, padded batch: 28.2 us, 34.5 from 12 on; dense: 60.2, 61.8). A weight times scale is off by
// half of float16's smallest number at most, 2^-33 of the group's largest; for float32 queries 2^-37.
// Each group has a factor of its own, so that small scales beside large ones keep their accuracy, and M leaves the
// scales out, so that the sums of weights, and of weights times zeros, stay near one however small the scales are.
template <typename T>
constexpr float kCaRaise = sizeof(T) == 4 ? 12.0f : 8.0f;
constexpr float kCaMaxSum = 0x1p40f;      // a thread's sum of weights beyond it raises M
constexpr float kCaFirstFactor = 0x1p126f;  // 2^e of a group without a scale: the first one overflows and lowers it

// A raise of the reference from `old` to `now` at which the group's largest log2(weight times scale) + `now` is `most`:
// changes the factor, and returns what the group's sums are to be multiplied by (f = 2^(old - now)).
template <typename T>
__device__ __forceinline__ float lower_factor(float& factor, float old, float now, float f, float most) {
  const float e = static_cast<float>(static_cast<int>(__float_as_uint(factor) >> 23) - 127);
  // never above what the sums so far had (fminf and fmaxf drop a NaN, which comes of infinite scores)
  const float to = fmaxf(fminf(ceilf(fminf(kCaRaise<T> - (most - now), e + (now - old))), 126.0f), -126.0f);
  factor = __uint_as_float(static_cast<uint32_t>(static_cast<int>(to) + 127) << 23);
  const float by = fmaxf(fminf(to - e, 126.0f), -126.0f);
  return f * __uint_as_float(static_cast<uint32_t>(static_cast<int>(by) + 127) << 23);
}
// 1 / factor of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float factor_inverse(float factor) {
  return __uint_as_float((254u << 23) - __float_as_uint(factor));
}
constexpr float kCaNone = -0x1.fffffep127f;  // reference of a row that has seen nothing: no finite score is below it

// How many query rows a unit has and how they fill the products' eight columns: each once, or (FOLD = 2, up to four
// rows) twice, the two halves for different tokens.
template <int D, int FOLD>
struct CaShape {
  static constexpr int kCols = 8;
  static constexpr int kRows = kCols / FOLD;  // query rows of a unit
  static constexpr int kCtas = 4;  // CTAs of an SM: four warps to each of its quarters
  static constexpr int kExtra = 6;  // (see CaPlan)
  static constexpr int kOStride = D + 4;  // floats of a row in the join buffer: 16-byte stores free of conflicts
  static constexpr int kJoinBytes = kCaWarps * kCols * kOStride * 4;
  static constexpr int kStages = 2 * 128 / D;  // tiles of a pair's ring
  static size_t smem(int nseq) {
    return 2 * static_cast<size_t>(kStages) * cache_tile_bytes(D) + kJoinBytes + nseq * sizeof(int4);
  }
};

__device__ __forceinline__ void bulk_load(void* smem, const void* gmem, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem)),
               "l"(__cvta_generic_to_global(gmem)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same without a sum to add to, and of bfloat16 operands.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// (16 x 8) (8 x 8) of bfloat16.
__device__ __forceinline__ void mma_bf16_k8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ void mma_bf16_k8_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f));
}
// N consecutive 32-bit words of shared memory, in one load.
template <int N>
__device__ __forceinline__ void load_words(uint32_t p, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(p));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p));
}

// Two codes in the low bits of 16-bit halves as the float16 numbers code - 8.
__device__ __forceinline__ uint32_t centred(uint32_t codes) {
  const uint32_t x = codes | 0x64006400u;  // 1024 + code
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__float2half_rn(1032.0f)));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What packing to float16 left of lo and hi.
__device__ __forceinline__ uint32_t pack_f16_rest(float lo, float hi, uint32_t packed) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&packed));
  return pack_f16(lo - f.x, hi - f.y);
}

// 2^e scale_log2, what a row's products with codes are multiplied by. A row with an element of 2^117 or more, an
// infinity too, has NaN instead: 2^e does not hold its scale any more, and its scores would be wrong, not infinite. So
// has one for which that factor, or the sum of its channels times scale_log2 (up to 2^7 amax scale_log2), leaves
// float32 with a large scale: products below zero would all be -inf, and a row that sees tokens would read as zeros.
__device__ __forceinline__ float score_factor(float amax, int e, float scale_log2) {
  const float f = __uint_as_float(static_cast<uint32_t>(min(e, 127) + 127) << 23) * scale_log2;
  return amax < 0x1p117f && f < CUDART_INF_F && amax * scale_log2 < 0x1p120f ? f : CUDART_NAN_F;
}

// How the tiles of all units are laid in one line and cut into equal pieces, one
// for each CTA. A unit is (sequence, key/value head, run of kRows query rows).
//
// Beginning a unit (its queries, its first tile's references, the sums of the one
// before) takes a CTA as long as `extra` tiles, so the pieces are equal in tiles
// and beginnings together: a unit weighs its tiles and `extra` more, which come
// before them. (Ragged batch of 48: 17.1 us with six, 18.2 with two, 19.1 with none;
// 40 rows: 28.2 with four, 29.0 with two, 33.1 with none.)
struct CaPlan {
  const int4* seqs;  // [B]: tiles before the sequence, weight before it, start, count
  int per_seq;       // units of a sequence
  int row_tiles;     // units of a (sequence, head)
  // x: tiles of a unit where blocks are selected (otherwise 0), y: tokens of a full table. In shared memory, since
  // registers are short in the loop over tiles (dense 32768-token batch: 64.5 us, 59.8 without them).
  const volatile int2* limits;
  int total, weight;  // tiles and weight of all units
  int chunk;          // weight of a CTA
  int extra, B;

  // tiles of each unit of a sequence with these values
  static __device__ __forceinline__ int tiles(int start, int count, int fixed, int most) {
    return count == 0 ? 0 : fixed ? fixed : (min(start + count, most) + kCacheTile - 1) / kCacheTile;
  }

  // The first tile of CTA i.
  __device__ __forceinline__ int cut(int i) const {
    const int at = i * chunk;
    if (at >= weight) return total;
    int lo = 0, hi = B - 1;  // as in locate
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (seqs[mid].y <= at)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int4 q = seqs[lo];
    const int n = tiles(q.z, q.w, limits->x, limits->y), unit = (at - q.y) / (n + extra), in = (at - q.y) % (n + extra);
    return q.x + unit * n + max(in - extra, 0);
  }

  // The unit of tile x: its sequence and number there, first tile and tiles; the sequence's start and count.
  struct Unit {
    int b, unit, first, n, start, count;
  };
  __device__ __forceinline__ Unit locate(int x) const {
    int lo = 0, hi = B - 1;  // the last sequence whose tiles begin at or before x (one without tiles is never last)
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (seqs[mid].x <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int4 q = seqs[lo];
    const int n = tiles(q.z, q.w, limits->x, limits->y), unit = (x - q.x) / n;
    return Unit{lo, unit, q.x + unit * n, n, q.z, q.w};
  }
  __device__ __forceinline__ int head(int unit) const { return row_tiles == 1 ? unit : unit / row_tiles; }
  __device__ __forceinline__ int row0(int unit, int rows) const { return row_tiles == 1 ? 0 : unit % row_tiles * rows; }
};

// Fills the plan and finds the CTA's piece [begin, end); `table` is shared memory for B int4. All threads of the block
// call it; it ends with a barrier. The first CTA leaves what the joining launch needs in `out`.
__device__ __forceinline__ CaPlan make_plan(const CacheSeqs& s, int B, int Hkv, int row_tiles, int topk, int extra,
                                            int4* table, int4* out, int& begin, int& end) {
  __shared__ int total, weight;
  __shared__ int2 limits;
  CaPlan p;
  p.seqs = table, p.row_tiles = row_tiles, p.per_seq = Hkv * row_tiles, p.extra = extra, p.B = B;
  const int fixed = topk * (s.bs / kCacheTile), most = s.max_blocks * s.bs;
  if (threadIdx.x == 0) limits = make_int2(fixed, most);
  p.limits = &limits;
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    int start, count;
    seq_step(s, b, start, count);
    table[b] = make_int4(0, 0, start, count);
  }
  if (B > 32) __syncthreads();
  if (threadIdx.x < 32) {  // warp 0 sums up the sequences' tiles, 32 at a time
    __syncwarp();
    int sum = 0, begun = 0;  // tiles, and sequences with some
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + threadIdx.x;
      const int4 q = b < B ? table[b] : make_int4(0, 0, 0, 0);
      const int n = CaPlan::tiles(q.z, q.w, fixed, most) * p.per_seq;
      int before = n;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int other = __shfl_up_sync(0xffffffffu, before, d);
        if (threadIdx.x >= d) before += other;
      }
      const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
      const int x = sum + before - n;
      if (b < B)
        table[b] = make_int4(x, x + (begun + __popc(some & ((1u << threadIdx.x) - 1))) * p.per_seq * extra, q.z, q.w);
      sum += __shfl_sync(0xffffffffu, before, 31);
      begun += __popc(some);
    }
    if (threadIdx.x == 0) total = sum, weight = sum + begun * p.per_seq * extra;
  }
  __syncthreads();
  p.total = total, p.weight = weight;
  p.chunk = max(1, (p.weight + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  const int x = p.cut(blockIdx.x + threadIdx.x % 2);  // even threads the first tile, odd ones the next CTA's
  begin = __shfl_sync(0xffffffffu, x, 0), end = __shfl_sync(0xffffffffu, x, 1);
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < B; b += blockDim.x) out[1 + b] = table[b];
    if (threadIdx.x == 0) out[0] = make_int4(p.chunk, extra, fixed, most);
  }
  return p;
}

// Position of tile x's first token and where it lies; -1 where its block is absent or past the sequence's tokens.
__device__ __forceinline__ int find_tile(const CacheSeqs& s, const CaPlan& plan, const uint8_t* cache,
                                         const int32_t* idx, int x, int Hkv, int topk, int D, const uint8_t*& src) {
  const CaPlan::Unit u = plan.locate(x);
  const int h = plan.head(u.unit), tile = x - u.first, per = s.bs / kCacheTile, shift = per >> 1;  // (per: 1, 2, 4)
  const int j = tile >> shift;
  const int block = idx ? idx[(static_cast<long>(u.b) * Hkv + h) * topk + j] : j;
  const int page = seq_page(s, u.b, block);
  src = nullptr;
  if (page < 0) return -1;
  const int in = tile & (per - 1), pos = block * s.bs + in * kCacheTile;
  src = tile_ptr(const_cast<uint8_t*>(cache), page, h, in, Hkv, s.bs, D);
  return pos < u.start + u.count ? pos : -1;
}

// Where a CTA leaves its part of a unit that other CTAs share: slot 0 for the
// unit that began before the CTA's tiles, slot 1 for the one that begins among
// them. Floats: references [kRows], weight sums [kRows], sums [kRows][D].
template <int kRows, int D>
__device__ __forceinline__ float* part_of(float* ws, int cta, int slot) {
  return ws + (static_cast<long>(cta) * 2 + slot) * (kRows * (D + 2));
}

template <typename T>
__device__ __forceinline__ void store_out(T* o, float x) {
  if constexpr (sizeof(T) == 2)
    *o = __float2bfloat16_rn(x);
  else
    *o = x;
}

template <typename T, int D, int FOLD>
__global__ void __launch_bounds__(kCaThreads, (CaShape<D, FOLD>::kCtas))
    cache_attn_kernel(const T* __restrict__ q, const uint8_t* __restrict__ cache, const int32_t* __restrict__ idx, T* o,
                      float* ws, CacheSeqs s, int B, int H, int Hkv, int topk, float scale_log2, int4* plan_out) {
  using Shape = CaShape<D, FOLD>;
  constexpr int kStages = Shape::kStages, kRows = Shape::kRows, kCols = Shape::kCols, kTile = cache_tile_bytes(D);
  constexpr int kWords = D / 32, kGroups = D / 64;
  constexpr int kSplit = sizeof(T) == 4 ? 2 : 1;  // float16 parts of a query element and of a weight
  // runs of 16 tokens computed together; folded, two runs share the columns and everything between the products is
  // computed once for both, each thread looking after the tokens of its half
  constexpr int kRuns = kSplit == 1 || FOLD == 2 ? 2 : 1, kSoft = kRuns / FOLD;
  constexpr bool kCentre = kSplit == 2;           // operands code - 8 instead of code
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + 2 * kStages * kTile);
  int4* table = reinterpret_cast<int4*>(smem + 2 * kStages * kTile + Shape::kJoinBytes);
  __shared__ uint64_t bars[2][2][kStages];
  __shared__ int tile_pos[2][kStages];  // position of the stage's first token; -1: the tile's block is absent
  __shared__ int next_pos[2][32];       // the same of the pair's next 32 tiles, and where they lie
  __shared__ const uint8_t* next_src[2][32];
  __shared__ float join_m[2][kCaWarps][kCols], join_l[2][kCaWarps][kCols];
  __shared__ int abort_flag;
  pdl_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, G = H / Hkv, pair = warp / 2;
  const bool leader = warp % 2 == 0;  // the pair's first warp loads its tiles
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kStages; ++i)
      for (int j = 0; j < 2; ++j) {
        mbar_init(&bars[j][0][i], 1);  // filled
        mbar_init(&bars[j][1][i], 1);  // the other warp is done with it
      }
    fence_mbarrier_init();
  }
  pdl_wait();
  int begin, end;
  const CaPlan plan = make_plan(s, B, Hkv, (s.T * G + kRows - 1) / kRows, idx ? topk : 0, Shape::kExtra, table, plan_out,
                                begin, end);
  volatile int* abort = &abort_flag;
  uint8_t* stages = smem + pair * kStages * kTile;
  uint64_t *full = bars[pair][0], *empty = bars[pair][1];

  // The leader: copies tile x (the pair's next to load) into its stage. Where the 32 tiles from x on lie is looked up
  // at once, one lane each.
  int load = begin + pair, load_stage = 0, loads = 0;
  auto fetch = [&]() {
    if (loads % 32 == 0) {
      const int x = load + 2 * lane;
      int pos = -1;
      const uint8_t* src = nullptr;
      if (x < end) pos = find_tile(s, plan, cache, idx, x, Hkv, topk, D, src);
      next_pos[pair][lane] = pos;
      next_src[pair][lane] = src;
      __syncwarp();
    }
    if (lane == 0) {
      const int pos = next_pos[pair][loads % 32];
      tile_pos[pair][load_stage] = pos;
      if (pos >= 0) {
        mbar_arrive_expect_tx(&full[load_stage], kTile);
        bulk_load(stages + load_stage * kTile, next_src[pair][loads % 32], kTile, &full[load_stage]);
      } else {
        mbar_arrive(&full[load_stage]);
      }
    }
    __syncwarp();
    ++loads;
    load += 2;
    if (++load_stage == kStages) load_stage = 0;
  };
  const int g = lane / 4, t4 = lane % 4;
  int flushes = 0, phase = 0, stage = 0, mine = begin + pair;  // this pair's next tile and its place
  for (int x = begin; x < end;) {
    const CaPlan::Unit u = plan.locate(x);
    const int b = u.b, first = u.first, n = u.n, start = u.start;
    const int stop = min(first + n, end);
    const int h = plan.head(u.unit), row0 = plan.row0(u.unit, kRows);
    const int rows = min(kRows, u.count * G - row0);  // rows with a query (may be <= 0)
    Octet<T> raw[kWords];  // this thread's queries: row g, channels 32 w + 8 t4 + 0..7
    const int r = g % kRows, row = row0 + r;
    if (r < rows) {
      const T* at = q + ((static_cast<long>(b) * s.T + row / G) * H + h * G + row % G) * D + t4 * 8;
#pragma unroll
      for (int w = 0; w < kWords; ++w) raw[w].load(at + w * 32);
    } else {
#pragma unroll
      for (int w = 0; w < kWords; ++w) raw[w] = Octet<T>{};
    }
    if (x == begin && leader)  // the first tiles' addresses and copies, while the queries come
      while (loads < kStages && load < end) fetch();

    // the queries as the products' second operand, and per row what a score is multiplied by
    uint32_t qb[kSplit][kWords][2][2];
    uint32_t zb[2];
    float mul[2], qsum[2][kGroups];  // qsum: folded only, in the place of zb
    int limit[2];
    int low_limit = 0x7fffffff;  // positions below it are seen by all rows
    float f[kWords][8], amax = 0.0f, sum[kGroups] = {};
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      raw[w].floats(f[w]);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[w][i])), sum[w / 2] += f[w][i];
    }
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
#pragma unroll
      for (int j = 0; j < kGroups; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
    }
    // the largest element goes to [2^13, 2^14): float16 holds the eight bits of a bfloat16 element down to 2^-27
    // (odd channels 2^-23) of it
    const int up = min(13 - static_cast<int>((__float_as_uint(amax) >> 23) & 255u) + 127, 126);
    const float qscale = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
    const float back = score_factor(amax, (kCentre ? 0 : 24) - up, scale_log2);
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[w][i] *= i % 2 && !kCentre ? qscale * 0.0625f : qscale;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qb[0][w][k][0] = pack_f16(f[w][2 * k], f[w][2 * k + 4]);
        qb[0][w][k][1] = pack_f16(f[w][2 * k + 1], f[w][2 * k + 5]);
        if constexpr (kSplit == 2) {
          qb[1][w][k][0] = pack_f16_rest(f[w][2 * k], f[w][2 * k + 4], qb[0][w][k][0]);
          qb[1][w][k][1] = pack_f16_rest(f[w][2 * k + 1], f[w][2 * k + 5], qb[0][w][k][1]);
        }
      }
    }
    // second operand of zero . (sum of q's channels): a token's (scale, zero) words are the first, group t4 % 2's
    // in this thread's columns, and the sum meets the zero half in up to four bfloat16 parts
    {
      float rest = (kGroups == 2 && t4 % 2 ? sum[kGroups - 1] : sum[0]) * scale_log2;
      uint32_t parts[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat16 h = __float2bfloat16_rn(rest);
        parts[i] = static_cast<uint32_t>(__bfloat16_as_ushort(h)) << 16;  // the zero half, and 8 of it for the scale
        if constexpr (kCentre) parts[i] |= __bfloat16_as_ushort(__float2bfloat16_rn(8.0f * __bfloat162float(h)));
        rest -= __bfloat162float(h);
      }
      if (kGroups == 2) {
        zb[0] = t4 < 2 ? parts[0] : parts[1], zb[1] = t4 < 2 ? parts[2] : parts[3];
      } else {
        zb[0] = t4 < 2 ? (t4 ? parts[1] : parts[0]) : (t4 == 2 ? parts[2] : parts[3]);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {  // this thread's scores belong to rows 2 t4 and 2 t4 + 1
      const int from = (2 * t4 + c) * 4;
      mul[c] = __shfl_sync(0xffffffffu, back, from);
      if constexpr (FOLD == 2) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) qsum[c][j] = __shfl_sync(0xffffffffu, sum[j] * scale_log2, from);
      }
      const int rr = (2 * t4 + c) % kRows;
      limit[c] = rr < rows ? start + (row0 + rr) / G + 1 : 0;
    }
    low_limit = start + row0 / G + 1;

    float m[2], l[2], z[2][kGroups], factor[2][kGroups], acc[kWords][2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[c] = kCaNone, l[c] = 0.0f;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) z[c][j] = 0.0f, factor[c][j] = kCaFirstFactor;
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[w][k][i] = 0.0f;

    // kRuns runs of 16 tokens of a tile, from row r0: their scores, weights and sums. kEdge: some row does not see
    // some token.
    auto tokens = [&](uint32_t base, int pos, int r0, auto edge) {
      constexpr bool kEdge = decltype(edge)::value;
      const int half = FOLD == 2 ? t4 / 2 : 0;  // the run that this thread looks after
      float xs[kSoft][4], dot[kRuns][kGroups][4], zero[kRuns][4];
      uint32_t ksz[kSoft][2][kGroups], vsz[kSoft][2][kGroups];
#pragma unroll
      for (int u = 0; u < kSoft; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          load_words(base + cache_ks_offset(D) + (r0 + 16 * (u + half) + i * 8 + g) * (D / 16), ksz[u][i]);
#pragma unroll
      for (int e = 0; e < kRuns; ++e) {
        const int r = r0 + 16 * e;
        uint32_t kw[2][kWords];
#pragma unroll
        for (int i = 0; i < 2; ++i) load_words(base + (r + i * 8) * (D / 2) + lane * (D / 8), kw[i]);
        if constexpr (FOLD == 1) {
          uint32_t zw[2][1];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            load_words(base + cache_ks_offset(D) + (r + i * 8 + g) * (D / 16) + (t4 % kGroups) * 4, zw[i]);
          mma_bf16_k8_first(zero[e], zw[0][0], zw[1][0], zb[0]);
          if constexpr (kGroups == 2) mma_bf16_k8(zero[e], zw[0][0], zw[1][0], zb[1]);
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t u = kw[0][w] >> (8 * k), v = kw[1][w] >> (8 * k);
            uint32_t a0 = u & kLow, a1 = v & kLow, a2 = u & kHigh, a3 = v & kHigh;
            if constexpr (kCentre) a0 = centred(a0), a1 = centred(a1), a2 = centred(a2 >> 4), a3 = centred(a3 >> 4);
#pragma unroll
            for (int sp = 0; sp < kSplit; ++sp)
              if (w % 2 == 0 && k == 0 && sp == 0)
                mma_f16_first(dot[e][w / 2], a0, a1, a2, a3, qb[sp][w][k][0], qb[sp][w][k][1]);
              else
                mma_f16(dot[e][w / 2], a0, a1, a2, a3, qb[sp][w][k][0], qb[sp][w][k][1]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kSoft; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_words(base + cache_vs_offset(D) + (r0 + 16 * (u + half) + i * 8 + g) * (D / 16), vsz[u][i]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int at = 2 * i + c;
            float d = 0.0f, a = 0.0f;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
              const float one = FOLD == 2 && half ? dot[kRuns - 1][j][at] : dot[u][j][at];
              float sc, ze;
              unpack_sz(ksz[u][i][j], sc, ze);
              if constexpr (kCentre) ze = fmaf(8.0f, sc, ze);
              d = j ? fmaf(sc, one, d) : sc * one;
              if constexpr (FOLD == 2) a = j ? fmaf(ze, qsum[c][j], a) : ze * qsum[c][j];
            }
            if constexpr (FOLD == 1) a = zero[u][at];
            float v = fmaf(d, mul[c], a);
            if (kEdge && pos + r0 + 16 * (u + half) + 8 * i + g >= limit[c]) v = -CUDART_INF_F;
            xs[u][at] = v;
          }
        }
      // weights against the references as they stand, times the groups' factors and the values' scales, in float16;
      // what a row does not see must not count, not even as 0 * NaN
      float p[kSoft][4], sum[2];
      uint32_t w16[kSoft][kGroups][2], high = 0;
      auto weigh = [&]() {
#pragma unroll
        for (int c = 0; c < 2; ++c) sum[c] = l[c];
#pragma unroll
        for (int e = 0; e < kSoft; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              p[e][2 * i + c] = fast_exp2(xs[e][2 * i + c] - m[c]);
              sum[c] += p[e][2 * i + c];
            }
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
              const float vs = __uint_as_float(vsz[e][i][j] << 16);
              float w[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                w[c] = p[e][2 * i + c] * factor[c][j] * vs;
                if (kEdge && pos + r0 + 16 * (e + half) + 8 * i + g >= limit[c]) w[c] = 0.0f;
              }
              w16[e][j][i] = pack_f16(w[0], w[1]);
              high = max_u16x2(high, w16[e][j][i]);
            }
          }
      };
      weigh();
      const float most = fmaxf(sum[0], sum[1]);
      // Is one at 2^15 or above (0x7800; an infinite weight times 0 is a NaN and above it too), or a sum of weights
      // beyond kCaMaxSum? Scales are not negative, so the codes of the float16 halves rank as they do.
      if (__any_sync(0xffffffffu, max_u16x2(high, 0x78007800u) != 0x78007800u || most > kCaMaxSum)) {
        // raise the references to the largest scores, so that no weight is above 1, and lower the factors
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float u[1 + kGroups];  // the largest score, and with log2 of the value's scale
#pragma unroll
          for (int j = 0; j < 1 + kGroups; ++j) {
            u[j] = -CUDART_INF_F;
#pragma unroll
            for (int e = 0; e < kSoft; ++e)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                u[j] = fmaxf(u[j], xs[e][2 * i + c] + (j ? __log2f(__uint_as_float(vsz[e][i][j - 1 + !j] << 16)) : 0.0f));
#pragma unroll
            for (int d = 4; d < 32; d *= 2) u[j] = fmaxf(u[j], __shfl_xor_sync(0xffffffffu, u[j], d));
          }
          const float old = m[c], now = fmaxf(old, u[0]), f = fast_exp2(old - now);
          m[c] = now;
          l[c] *= f;
#pragma unroll
          for (int j = 0; j < kGroups; ++j) {
            z[c][j] *= f;
            const float by = lower_factor<T>(factor[c][j], old, now, f, u[1 + j]);
#pragma unroll
            for (int w = 2 * j; w < 2 * j + 2; ++w)
#pragma unroll
              for (int k = 0; k < 2; ++k) acc[w][k][c] *= by, acc[w][k][2 + c] *= by;
          }
        }
        weigh();
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) l[c] = sum[c];
      uint32_t pb[kSoft][kSplit][kGroups][2];
#pragma unroll
      for (int e = 0; e < kSoft; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < kGroups; ++j) {
            pb[e][0][j][i] = transpose8x8(w16[e][j][i]);
            float vs, vz, w[2];
            unpack_sz(vsz[e][i][j], vs, vz);
            if constexpr (kCentre) vz = fmaf(8.0f, vs, vz);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const bool seen = !kEdge || pos + r0 + 16 * (e + half) + 8 * i + g < limit[c];
              w[c] = seen ? p[e][2 * i + c] * factor[c][j] * vs : 0.0f;
              if (seen) z[c][j] = fmaf(p[e][2 * i + c], vz, z[c][j]);
            }
            if constexpr (kSplit == 2)
              pb[e][1][j][i] = transpose8x8(pack_f16_rest(w[0], w[1], w16[e][j][i]));
          }
#pragma unroll
      for (int e = 0; e < kRuns; ++e) {
        // folded: this run's weights are in columns 4 e .. 4 e + 3, the others' must not meet its values
        const uint32_t mine = FOLD == 1 || g / 4 == e ? 0xffffffffu : 0u;
        uint32_t wb[kSplit][kGroups][2], vw[2][kWords];
#pragma unroll
        for (int i = 0; i < 2 * kSplit * kGroups; ++i)
          (&wb[0][0][0])[i] = (&pb[FOLD == 2 ? 0 : e][0][0][0])[i] & mine;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          load_words(base + cache_v_offset(D) + ((r0 + 16 * e) / 2 + t4 + 4 * i) * D + (g ^ (2 * t4)) * (D / 8), vw[i]);
#pragma unroll
        for (int w = 0; w < kWords; ++w)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if constexpr (kCentre) {
              // float32: from zero, and added in float32 (see put_aside)
              const uint32_t u = vw[0][w] >> (8 * k), v = vw[1][w] >> (8 * k);
              const uint32_t a0 = centred(u & kLow), a1 = centred(u >> 4 & kLow), a2 = centred(v & kLow),
                             a3 = centred(v >> 4 & kLow);
              float part[4];
              mma_f16_first(part, a0, a1, a2, a3, wb[0][w / 2][0], wb[0][w / 2][1]);
              mma_f16(part, a0, a1, a2, a3, wb[kSplit - 1][w / 2][0], wb[kSplit - 1][w / 2][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[w][k][i] += part[i];
            } else {
              // the byte with channels 2 k and 2 k + 1, and the first one alone
              const uint32_t a1 = k ? __byte_perm(vw[0][w], 0, 0x4341) : vw[0][w] & 0x00ff00ffu, a0 = a1 & kLow;
              const uint32_t a3 = k ? __byte_perm(vw[1][w], 0, 0x4341) : vw[1][w] & 0x00ff00ffu, a2 = a3 & kLow;
              mma_f16(acc[w][k], a0, a1, a2, a3, wb[0][w / 2][0], wb[0][w / 2][1]);
            }
          }
      }
    };

    // Sums kept in the matrix unit lose up to a unit of their last place at every step, always downwards: after 2 kAside
    // steps about 2^-24 kAside of the sums of codes, which is 500 times as much of a result in which values of both signs
    // nearly cancel (131072 tokens). So every kAside tiles they go to this thread's places of the join buffer, in
    // float32, at the references of that time. Eight rows of D = 64 over 131072 tokens on one CTA: error 1.87e-3 with 16,
    // 2.3e-3 with 32, 3.8e-3 with 64 (rounding the output alone: 1.68e-3); the dense 32768-token batch takes 1% longer with 16 than with 64.
    constexpr int kAside = 16;
    float aside_m[2];
    bool aside = false;
    auto sums_of = [&](int c, int w, float f, float zero) {
      constexpr float kLo = kCentre ? 1.0f : 0x1p24f, kHi = kCentre ? 1.0f : 0x1p20f;
      const float back = factor_inverse(factor[c][w / 2]);
      float hi[2] = {acc[w][0][2 + c], acc[w][1][2 + c]};
      if constexpr (!kCentre) hi[0] -= acc[w][0][c], hi[1] -= acc[w][1][c];
      return make_float4(fmaf(acc[w][0][c] * kLo * back, f, zero), fmaf(hi[0] * kHi * back, f, zero),
                         fmaf(acc[w][1][c] * kLo * back, f, zero), fmaf(hi[1] * kHi * back, f, zero));
    };
    // the sums so far at reference m + log2(1 / f), with `zero` for each channel
    auto put_aside = [&](int c, float f, float old, const float (&zero)[kGroups]) {
      float4* to = reinterpret_cast<float4*>(join + (warp * kCols + 2 * t4 + c) * Shape::kOStride + 4 * g);
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        float4 v = sums_of(c, w, f, zero[w / 2]);
        if (aside) {
          const float4 u = to[w * 8];
          v = make_float4(fmaf(u.x, old, v.x), fmaf(u.y, old, v.y), fmaf(u.z, old, v.z), fmaf(u.w, old, v.w));
        }
        to[w * 8] = v;
      }
    };

    // a tile goes to one pair of warps, 32 tokens each; the pairs take the CTA's tiles in turn
    while (mine < stop) {
      const int until = kCentre ? stop : min(stop, mine + 2 * kAside);
      for (; mine < until; mine += 2) {
        const int pos = mbar_wait(&full[stage], phase, abort, 802) ? tile_pos[pair][stage] : -1;
        if (pos >= 0) {
          const uint32_t base = smem_u32(stages) + stage * kTile;
          const bool edge = pos + kCacheTile > low_limit;
          for (int run = 0; run < 2; run += kRuns) {
            const int r0 = (warp % 2) * 32 + run * 16;
            if (edge)
              tokens(base, pos, r0, std::true_type{});
            else
              tokens(base, pos, r0, std::false_type{});
          }
        }
        __syncwarp();
        if (!leader) {
          if (lane == 0) mbar_arrive(&empty[stage]);
        } else if (load < end && mbar_wait(&empty[stage], phase, abort, 801)) {
          fetch();
        }
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
      if (mine >= stop) break;
      constexpr float kNone[kGroups] = {};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        put_aside(c, 1.0f, aside ? fast_exp2(aside_m[c] - m[c]) : 0.0f, kNone);
        aside_m[c] = m[c];
      }
      aside = true;
#pragma unroll
      for (int w = 0; w < kWords; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[w][k][i] = 0.0f;
    }
    x = stop;

    // ---------------- the unit's part of this CTA: the warps' (and halves') sums joined in a fixed order
    auto join_top = [](const float (&m)[kCaWarps][kCols], int r) {
      float top = m[0][r];
#pragma unroll
      for (int w = 0; w < kCaWarps; ++w)
#pragma unroll
        for (int e = 0; e < FOLD; ++e) top = fmaxf(top, m[w][r + e * kRows]);
      return top;
    };
    const int fb = flushes++ & 1;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) {
        l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
#pragma unroll
        for (int j = 0; j < kGroups; ++j) z[c][j] += __shfl_xor_sync(0xffffffffu, z[c][j], d);
      }
      if (g == 0) {
        join_m[fb][warp][2 * t4 + c] = m[c];
        join_l[fb][warp][2 * t4 + c] = l[c];
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float top = join_top(join_m[fb], (2 * t4 + c) % kRows), f = fast_exp2(m[c] - top);
      float zero[kGroups];
#pragma unroll
      for (int j = 0; j < kGroups; ++j) zero[j] = z[c][j] * f;
      put_aside(c, f, aside ? fast_exp2(aside_m[c] - top) : 0.0f, zero);
    }
    __syncthreads();
    const bool whole = first >= begin && first + n <= end;
    float* part = part_of<kRows, D>(ws, blockIdx.x, first < begin ? 0 : 1);
    for (int i = threadIdx.x; i < rows * D; i += kCaWarps * 32) {
      const int r = i / D, c = i % D;
      const float top = join_top(join_m[fb], r);
      float sum = 0.0f, val = 0.0f;
#pragma unroll
      for (int w = 0; w < kCaWarps; ++w)
#pragma unroll
        for (int e = 0; e < FOLD; ++e) {
          sum += join_l[fb][w][r + e * kRows] * fast_exp2(join_m[fb][w][r + e * kRows] - top);
          val += join[(w * kCols + r + e * kRows) * Shape::kOStride + c];
        }
      if (whole) {
        const int row = row0 + r;
        store_out(o + ((static_cast<long>(b) * s.T + row / G) * H + h * G + row % G) * D + c,
                  sum == 0.0f ? 0.0f : val / sum);
      } else {
        if (c == 0) part[r] = top, part[kRows + r] = sum;
        part[2 * kRows + r * D + c] = val;
      }
    }
    __syncthreads();  // the join buffer is free for the next unit's sums
  }
  // after a wait that ran out: copies in flight end before the block's shared memory does
  if (*abort && leader && lane == 0)
    for (int i = max(0, loads - kStages); i < loads; ++i) mbar_wait_teardown(&full[i % kStages], i / kStages & 1);
}

// ------------------------------------------------------------------ many query rows
//
// From nine query rows on (bfloat16, D = 128) the work between the products and the
// products themselves outweigh the unpacking, and a warp cannot hold the sums of
// all channels for all rows. (At D = 64 it can, and the kernel above in units of
// eight rows is the faster one: see the measurements where it is chosen.) So the four warps of a CTA share a tile: each scores
// 16 of its 64 tokens against all rows, leaves the weights times the values'
// scales in shared memory in the order of the products' second operand, and after
// one barrier sums 32 of the channels over all 64 tokens. The rows'
// references are the CTA's, in shared memory; a tile whose weights would leave
// float16 raises them and is weighed again. Bound: the matrix instructions, 16 NT
// for 16 tokens at 2.2 cycles of an SM each, 700 cycles a tile at 40 rows
// against 400 for its bytes; measured, 1900 (0.98 us): eight warps an SM do not hide the
// chain of products, exponentials, barrier and products (profiled at 40 rows, 758 instructions of a warp a tile:
// issue 35%, matrix unit 30%, shared memory's data path 48% busy; 2.0 of 5.6 cycles between a warp's instructions are
// fixed latencies, 0.8 shared memory, 0.5 the barrier;
// three CTAs an SM, with spills, 86 -> 110 us for 32768 tokens). Two teams of four warps with half the rows each
// took 1.4 times as long, since both unpack every tile.
constexpr int kCaWideD = 128;
template <int NT>
struct CaWide {
  static constexpr int D = kCaWideD;
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = NT <= 4 ? 3 : 2;
  static constexpr int kExtra = 4;  // (see CaPlan)
  static constexpr int kStages = 4;
  static constexpr int kGroups = D / 64, kSteps = D / 16;
  static constexpr int kQWords = kSteps * NT * 64;            // query operands: [step][nt][lane][2]
  static constexpr int kPWords = 2 * kGroups * 4 * NT * 64;   // weights: [buffer][group][16 tokens][nt][lane][2]
  static size_t smem(int nseq) {
    return static_cast<size_t>(kStages) * cache_tile_bytes(D) + (kQWords + kPWords + 4 * nseq) * 4;
  }
};

// N consecutive 32-bit words, in one load (which the compiler may move between barriers).
template <int N>
__device__ __forceinline__ void get_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ uint64_t load_f2(const float* p) {
  const float2 f = *reinterpret_cast<const float2*>(p);
  return f2(f.x, f.y);
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {  // (may become part of a fused multiply-add)
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int NT>
__global__ void __launch_bounds__(kCaThreads, CaWide<NT>::kCtas)
    cache_attn_wide_kernel(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ cache,
                           const int32_t* __restrict__ idx, __nv_bfloat16* o, float* ws, CacheSeqs s, int B, int H,
                           int Hkv, int topk, float scale_log2, int4* plan_out) {
  using W = CaWide<NT>;
  constexpr int D = W::D, kStages = W::kStages, kRows = W::kRows, kTile = cache_tile_bytes(D), kGroups = W::kGroups;
  constexpr int kWords = D / 32, kMt = 2;  // 32-channel words (one a warp); 16-channel products of a warp
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  extern __shared__ __align__(128) uint8_t smem[];
  uint32_t* sq = reinterpret_cast<uint32_t*>(smem + kStages * kTile);
  uint32_t* sp = sq + W::kQWords;
  int4* table = reinterpret_cast<int4*>(sp + W::kPWords);
  __shared__ uint64_t full[kStages];
  __shared__ int tile_pos[kStages], next_pos[32];
  __shared__ const uint8_t* next_src[32];
  __shared__ __align__(16) float s_mul[kRows], s_qsum[kGroups][kRows], s_ref[kRows], s_factor[kGroups][kRows];
  __shared__ __align__(16) int s_limit[kRows];
  __shared__ float s_top[1 + kGroups][kRows], s_l[kCaWarps][kRows], s_z[kCaWarps][kGroups][kRows];
  __shared__ int abort_flag;
  pdl_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, G = H / Hkv, g = lane / 4, t4 = lane % 4;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    fence_mbarrier_init();
  }
  pdl_wait();
  int begin, end;
  const CaPlan plan = make_plan(s, B, Hkv, (s.T * G + kRows - 1) / kRows, idx ? topk : 0, W::kExtra, table, plan_out,
                                begin, end);
  volatile int* abort = &abort_flag;

  // the last warp: copies the next tile into its stage; where the next 32 lie is looked up at once, one lane each
  int load = begin;
  auto fetch = [&]() {
    const int n0 = load - begin;
    if (n0 % 32 == 0) {
      const int x = load + lane;
      int pos = -1;
      const uint8_t* src = nullptr;
      if (x < end) pos = find_tile(s, plan, cache, idx, x, Hkv, topk, D, src);
      next_pos[lane] = pos;
      next_src[lane] = src;
      __syncwarp();
    }
    if (lane == 0) {
      const int st = n0 % kStages, pos = next_pos[n0 % 32];
      tile_pos[st] = pos;
      if (pos >= 0) {
        mbar_arrive_expect_tx(&full[st], kTile);
        bulk_load(smem + st * kTile, next_src[n0 % 32], kTile, &full[st]);
      } else {
        mbar_arrive(&full[st]);
      }
    }
    __syncwarp();
    ++load;
  };
  const bool loader = warp == kCaWarps - 1;
  if (loader)
    while (load < end && load - begin < kStages - 1) fetch();

  int stage = 0, phase = 0, buf = 0;
  for (int x = begin; x < end;) {
    const CaPlan::Unit u = plan.locate(x);
    const int b = u.b, first = u.first, n = u.n, start = u.start;
    const int stop = min(first + n, end);
    const int h = plan.head(u.unit), row0 = plan.row0(u.unit, kRows);
    const int rows = min(kRows, u.count * G - row0);  // rows with a query (may be <= 0)

    const int group = warp / 2;  // of this warp's value channels

    // ---------------- the queries as the score products' second operand (float16, odd channels / 16: see above)
    constexpr int kPer = (NT + kCaWarps - 1) / kCaWarps;
    Octet<__nv_bfloat16> raw[kPer][kWords];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int r = (warp + e * kCaWarps) * 8 + g, row = row0 + r;
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        if (r < rows)
          raw[e][w].load(q + ((static_cast<long>(b) * s.T + row / G) * H + h * G + row % G) * D + w * 32 + t4 * 8);
        else
          raw[e][w] = Octet<__nv_bfloat16>{};
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int nt = warp + e * kCaWarps;
      if (nt >= NT) break;
      const int r = nt * 8 + g, row = row0 + r;
      float f[kWords][8], amax = 0.0f, sum[kGroups] = {};
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        raw[e][w].floats(f[w]);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[w][i])), sum[w / 2] += f[w][i];
      }
#pragma unroll
      for (int d = 1; d < 4; d *= 2) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
#pragma unroll
        for (int j = 0; j < kGroups; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
      }
      const int up = min(13 - static_cast<int>((__float_as_uint(amax) >> 23) & 255u) + 127, 126);
      const float qscale = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[w][i] *= i % 2 ? qscale * 0.0625f : qscale;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          reinterpret_cast<uint2*>(sq)[((w * 2 + k) * NT + nt) * 32 + lane] =
              make_uint2(pack_f16(f[w][2 * k], f[w][2 * k + 4]), pack_f16(f[w][2 * k + 1], f[w][2 * k + 5]));
      }
      if (t4 == 0) {
        s_mul[r] = score_factor(amax, 24 - up, scale_log2);
#pragma unroll
        for (int j = 0; j < kGroups; ++j) s_qsum[j][r] = sum[j] * scale_log2, s_factor[j][r] = kCaFirstFactor;
        s_limit[r] = r < rows ? start + row / G + 1 : 0;
        s_ref[r] = kCaNone;
      }
    }
    const int low_limit = start + row0 / G + 1;  // positions below it are seen by all rows
    __syncthreads();

    uint64_t l[NT], z[kGroups][NT];
    float acc[kMt][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] = 0;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) z[j][nt] = 0;
#pragma unroll
      for (int k = 0; k < kMt; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][nt][i] = 0.0f;
    }

    bool fresh = true;
    for (; x < stop; ++x) {
      const int pos = mbar_wait(&full[stage], phase, abort, 803) ? tile_pos[stage] : -1;
      const uint8_t* base = smem + stage * kTile;
      const int r0 = warp * 16, p0 = pos + r0 + g;  // this thread's tokens: positions p0 and p0 + 8
      const bool edge = pos + kCacheTile > low_limit;
      uint64_t xs[NT][2], p[NT][2], vs[kGroups][2];
      uint32_t vsz[2][kGroups];
      // the scores of this thread's tokens and columns, and its tokens' value scales
      auto score = [&](auto masked) {
        uint32_t a[kWords][2][4];
        uint64_t sc[kGroups][2], ze[kGroups][2];
        {
          uint32_t kw[2][kWords], sz[2][kGroups];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            get_words(base + (r0 + i * 8) * (D / 2) + lane * (D / 8), kw[i]);
            get_words(base + cache_ks_offset(D) + (r0 + i * 8 + g) * (D / 16), sz[i]);
            get_words(base + cache_vs_offset(D) + (r0 + i * 8 + g) * (D / 16), vsz[i]);
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
              float e, f;
              unpack_sz(sz[i][j], e, f);
              sc[j][i] = f2(e, e), ze[j][i] = f2(f, f);
              e = __uint_as_float(vsz[i][j] << 16);
              vs[j][i] = f2(e, e);
            }
          }
#pragma unroll
          for (int w = 0; w < kWords; ++w)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u = kw[0][w] >> (8 * k), v = kw[1][w] >> (8 * k);
              a[w][k][0] = u & kLow, a[w][k][1] = v & kLow, a[w][k][2] = u & kHigh, a[w][k][3] = v & kHigh;
            }
        }
        float dot[kGroups][NT][4];
#pragma unroll
        for (int w = 0; w < kWords; ++w)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              {
                const uint2 bq = reinterpret_cast<const uint2*>(sq)[((w * 2 + k) * NT + nt) * 32 + lane];
                if (w % 2 == 0 && k == 0)
                  mma_f16_first(dot[w / 2][nt], a[w][k][0], a[w][k][1], a[w][k][2], a[w][k][3], bq.x, bq.y);
                else
                  mma_f16(dot[w / 2][nt], a[w][k][0], a[w][k][1], a[w][k][2], a[w][k][3], bq.x, bq.y);
              }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          {
            const int col = nt * 8 + 2 * t4;
            const uint64_t mul = load_f2(s_mul + col);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint64_t d = f2_mul(sc[0][i], f2(dot[0][nt][2 * i], dot[0][nt][2 * i + 1]));
              uint64_t e = f2_mul(ze[0][i], load_f2(s_qsum[0] + col));
              if constexpr (kGroups == 2) {
                d = f2_fma(sc[1][i], f2(dot[1][nt][2 * i], dot[1][nt][2 * i + 1]), d);
                e = f2_fma(ze[1][i], load_f2(s_qsum[1] + col), e);
              }
              xs[nt][i] = f2_fma(d, mul, e);
              if constexpr (decltype(masked)::value) {
                const int2 lim = *reinterpret_cast<const int2*>(s_limit + col);
                float lo, hi;
                f2_split(xs[nt][i], lo, hi);
                xs[nt][i] = f2(p0 + 8 * i < lim.x ? lo : -CUDART_INF_F, p0 + 8 * i < lim.y ? hi : -CUDART_INF_F);
              }
            }
          }
      };
      // weights against the references as they stand, times the groups' factors and the values' scales, in float16, to
      // shared memory. True where one is at 2^15 or above (or a NaN, see the other kernel), or a weight beyond
      // kCaMaxSum.
      auto weigh = [&](auto masked) -> bool {
        float most = 0.0f;
        uint32_t high = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          {
            const int col = nt * 8 + 2 * t4;
            const uint64_t ref = load_f2(s_ref + col);
            uint32_t w16[kGroups][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float lo, hi;
              f2_split(f2_sub(xs[nt][i], ref), lo, hi);
              lo = fast_exp2(lo), hi = fast_exp2(hi);
              most = fmax3(most, lo, hi);
              p[nt][i] = f2(lo, hi);
#pragma unroll
              for (int j = 0; j < kGroups; ++j) {
                float wl, wh;
                f2_split(f2_mul(f2_mul(p[nt][i], load_f2(s_factor[j] + col)), vs[j][i]), wl, wh);
                if constexpr (decltype(masked)::value) {
                  const int2 lim = *reinterpret_cast<const int2*>(s_limit + col);
                  if (p0 + 8 * i >= lim.x) wl = 0.0f;
                  if (p0 + 8 * i >= lim.y) wh = 0.0f;
                }
                w16[j][i] = pack_f16(wl, wh);
                high = max_u16x2(high, w16[j][i]);
              }
            }
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
              reinterpret_cast<uint2*>(sp)[(((buf * kGroups + j) * 4 + warp) * NT + nt) * 32 + lane] =
                  make_uint2(transpose8x8(w16[j][0]), transpose8x8(w16[j][1]));
          }
        return __any_sync(0xffffffffu, max_u16x2(high, 0x78007800u) != 0x78007800u || most > kCaMaxSum);
      };
      if (pos >= 0) {
        if (edge)
          score(std::true_type{});
        else
          score(std::false_type{});
      }
      // (every warp takes every barrier here, whatever it saw of the tile; a unit's first tile sets the references
      // before it is weighed)
      const bool flag = pos >= 0 && (fresh || (edge ? weigh(std::true_type{}) : weigh(std::false_type{})));
      if (__syncthreads_or(flag)) {
        fresh = false;
        // Raise the references to the largest scores of the tile, lower the factors, and weigh again (a NaN stays one).
        // What each thread has of a column, the largest score and with log2 of the value's scale in each group, meets
        // in the weights' place: they are to be written anew, and every warp is past the tile before this one.
        constexpr int kStride = kCaThreads + 4;  // floats of a list (reading it is free of conflicts)
        static_assert((1 + kGroups) * NT * 2 * kStride <= W::kPWords && (1 + kGroups) * kRows <= kCaThreads);
        float* cand = reinterpret_cast<float*>(sp);
        if (pos >= 0) {
#pragma unroll
          for (int j = 0; j < 1 + kGroups; ++j) {
            const float lv0 = j ? __log2f(__uint_as_float(vsz[0][j - 1 + !j] << 16)) : 0.0f;
            const float lv1 = j ? __log2f(__uint_as_float(vsz[1][j - 1 + !j] << 16)) : 0.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float e[2], f[2];
              f2_split(xs[nt][0], e[0], e[1]);
              f2_split(xs[nt][1], f[0], f[1]);
#pragma unroll
              for (int c = 0; c < 2; ++c)
                cand[((j * NT + nt) * 2 + c) * kStride + threadIdx.x] = fmaxf(e[c] + lv0, f[c] + lv1);
            }
          }
        }
        __syncthreads();
        if (threadIdx.x < (1 + kGroups) * kRows) {
          const int list = threadIdx.x / 4, col = list / 2 % NT * 8 + 2 * t4 + list % 2;
          float top = -CUDART_INF_F;
#pragma unroll 8
          for (int i = 0; i < kCaThreads / 4; ++i) top = fmaxf(top, cand[list * kStride + i * 4 + t4]);
          s_top[list / (2 * NT)][col] = top;
        }
        __syncthreads();
        // each warp's sums follow the factor of the group that its channels are in
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = nt * 8 + 2 * t4 + c;
            const float old = s_ref[col], now = fmaxf(old, s_top[0][col]), f = fast_exp2(old - now);
            float factor = s_factor[group][col];
            const float a = lower_factor<__nv_bfloat16>(factor, old, now, f, s_top[1 + group][col]);
            const uint64_t by = c ? f2(1.0f, f) : f2(f, 1.0f);
            l[nt] = f2_mul(l[nt], by);
#pragma unroll
            for (int i = 0; i < kGroups; ++i) z[i][nt] = f2_mul(z[i][nt], by);
#pragma unroll
            for (int k = 0; k < kMt; ++k) acc[k][nt][c] *= a, acc[k][nt][2 + c] *= a;
          }
        __syncthreads();
        if (threadIdx.x < kRows) {
          const float old = s_ref[threadIdx.x], now = fmaxf(old, s_top[0][threadIdx.x]);
#pragma unroll
          for (int j = 0; j < kGroups; ++j)
            lower_factor<__nv_bfloat16>(s_factor[j][threadIdx.x], old, now, 1.0f, s_top[1 + j][threadIdx.x]);
          s_ref[threadIdx.x] = now;
        }
        __syncthreads();
        if (pos >= 0) weigh(std::true_type{});
        __syncthreads();
      }
      // every warp is past the tile before this one: its stage can be filled again
      if (loader && load < end) fetch();
      if (pos >= 0) {
        auto add_up = [&](auto masked) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
              const float v = __uint_as_float(vsz[i][j] & 0xffff0000u);
              const uint64_t vv = f2(v, v);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (j == 0) l[nt] = f2_add(l[nt], p[nt][i]);
                if constexpr (decltype(masked)::value) {
                  // a weight of 0 that stands for "not seen" must not meet a NaN
                  const int2 lim = *reinterpret_cast<const int2*>(s_limit + nt * 8 + 2 * t4);
                  float lo, hi, zl, zh;
                  f2_split(p[nt][i], lo, hi);
                  f2_split(z[j][nt], zl, zh);
                  z[j][nt] = f2(p0 + 8 * i < lim.x ? fmaf(lo, v, zl) : zl, p0 + 8 * i < lim.y ? fmaf(hi, v, zh) : zh);
                } else {
                  z[j][nt] = f2_fma(p[nt][i], vv, z[j][nt]);
                }
              }
            }
        };
        if (edge)
          add_up(std::true_type{});
        else
          add_up(std::false_type{});
        // a tile's products start from zero and are added in float32 (see the other kernel)
        float sum[kMt][NT][4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          uint32_t vw[2][1], av[kMt][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
            get_words(base + cache_v_offset(D) + (kt * 8 + t4 + 4 * i) * D + (g ^ (2 * t4)) * (D / 8) + warp * 4, vw[i]);
#pragma unroll
          for (int k = 0; k < kMt; ++k) {
            const uint32_t pick = k ? 0x4341u : 0x4240u;
            av[k][1] = __byte_perm(vw[0][0], 0, pick), av[k][0] = av[k][1] & kLow;
            av[k][3] = __byte_perm(vw[1][0], 0, pick), av[k][2] = av[k][3] & kLow;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 bp = reinterpret_cast<const uint2*>(sp)[(((buf * kGroups + group) * 4 + kt) * NT + nt) * 32 + lane];
#pragma unroll
            for (int k = 0; k < kMt; ++k)
              if (kt == 0)
                mma_f16_first(sum[k][nt], av[k][0], av[k][1], av[k][2], av[k][3], bp.x, bp.y);
              else
                mma_f16(sum[k][nt], av[k][0], av[k][1], av[k][2], av[k][3], bp.x, bp.y);
          }
        }
#pragma unroll
        for (int k = 0; k < kMt; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              f2_split(f2_add(f2(acc[k][nt][2 * i], acc[k][nt][2 * i + 1]),
                              f2(sum[k][nt][2 * i], sum[k][nt][2 * i + 1])),
                       acc[k][nt][2 * i], acc[k][nt][2 * i + 1]);
      }
      buf ^= 1;
      if (++stage == kStages) stage = 0, phase ^= 1;
    }

    // ---------------- the unit's part of this CTA: the warps' weight sums joined in a fixed order
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float v[1 + kGroups][2];
      f2_split(l[nt], v[0][0], v[0][1]);
#pragma unroll
      for (int j = 0; j < kGroups; ++j) f2_split(z[j][nt], v[1 + j][0], v[1 + j][1]);
#pragma unroll
      for (int e = 0; e < 1 + kGroups; ++e)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) v[e][c] += __shfl_xor_sync(0xffffffffu, v[e][c], d);
          if (g == 0) (e ? s_z[warp][e - 1] : s_l[warp])[nt * 8 + 2 * t4 + c] = v[e][c];
        }
    }
    __syncthreads();
    const bool whole = first >= begin && first + n <= end;
    float* part = part_of<kRows, D>(ws, blockIdx.x, first < begin ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t4 + c;
        if (r >= rows) continue;
        float sum = 0.0f, zero = 0.0f;
#pragma unroll
        for (int w = 0; w < kCaWarps; ++w) sum += s_l[w][r], zero += s_z[w][group][r];
        const float by = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
        const float back = factor_inverse(s_factor[group][r]);
        const int row = row0 + r;
        __nv_bfloat16* to = o + ((static_cast<long>(b) * s.T + row / G) * H + h * G + row % G) * D;
#pragma unroll
        for (int k = 0; k < kMt; ++k) {
          const int ch = warp * 32 + 4 * g + 2 * k;
          const float v0 = fmaf(acc[k][nt][c] * 0x1p24f, back, zero) * by,
                      v1 = fmaf((acc[k][nt][2 + c] - acc[k][nt][c]) * 0x1p20f, back, zero) * by;
          if (whole)
            *reinterpret_cast<uint32_t*>(to + ch) = pack_bf16x2(v0, v1);
          else
            *reinterpret_cast<float2*>(part + 2 * kRows + r * D + ch) = make_float2(v0, v1);
        }
        if (!whole && warp == 0 && g == 0) part[r] = s_ref[r], part[kRows + r] = sum;
      }
    __syncthreads();
  }
  // after a wait that ran out: copies in flight end before the block's shared memory does
  if (*abort && loader && lane == 0)
    for (int i = max(begin, load - kStages); i < load; ++i)
      mbar_wait_teardown(&full[(i - begin) % kStages], (i - begin) / kStages & 1);
}

// Joins the parts of the units that several CTAs share: one CTA per query row,
// its 8 warps taking the parts in turn and meeting in a fixed order.
constexpr int kCaJoinWarps = 8;

template <typename T, int D, int kRows>
__global__ void __launch_bounds__(kCaJoinWarps * 32)
    cache_attn_join_kernel(T* o, const float* ws, const int4* plan, int tokens, int H, int Hkv) {
  constexpr int kPer = D / 32;  // channels of a lane
  __shared__ float sums[kCaJoinWarps][D], weights[kCaJoinWarps], tops[kCaJoinWarps];
  const int G = H / Hkv, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row_tiles = (tokens * G + kRows - 1) / kRows;
  const int row = blockIdx.x % (tokens * G), h = blockIdx.x / (tokens * G) % Hkv, b = blockIdx.x / (tokens * G) / Hkv;
  const int4 head = plan[0], seq = plan[1 + b];  // (see make_plan)
  if (row / G >= seq.w) return;
  const int chunk = head.x, extra = head.y, n = CaPlan::tiles(seq.z, seq.w, head.z, head.w);
  const int r = row % kRows, first = seq.y + (h * row_tiles + row / kRows) * (n + extra) + extra;  // the first tile's place
  const int c0 = first / chunk, c1 = (first + n - 1) / chunk;
  if (c0 == c1) return;
  // four parts at a time in flight, each against the largest reference so far
  constexpr int kAhead = 4;
  float top = kCaNone, weight = 0.0f, val[kPer] = {};
  for (int c = c0 + warp; c <= c1; c += kAhead * kCaJoinWarps) {
    float m[kAhead], l[kAhead], v[kAhead][kPer], now = top;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int ci = c + i * kCaJoinWarps;
      const float* part = part_of<kRows, D>(const_cast<float*>(ws), min(ci, c1), min(ci, c1) == c0);
      m[i] = ci <= c1 ? part[r] : -CUDART_INF_F;
      l[i] = part[kRows + r];
#pragma unroll
      for (int k = 0; k < kPer; ++k) v[i][k] = part[2 * kRows + r * D + lane * kPer + k];
      now = fmaxf(now, m[i]);
    }
    const float f = fast_exp2(top - now);
    top = now;
    weight *= f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) val[k] *= f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (c + i * kCaJoinWarps > c1) break;  // (a part read twice for nothing may hold a NaN)
      const float e = fast_exp2(m[i] - top);
      weight = fmaf(l[i], e, weight);
#pragma unroll
      for (int k = 0; k < kPer; ++k) val[k] = fmaf(v[i][k], e, val[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) sums[warp][lane * kPer + k] = val[k];
  if (lane == 0) weights[warp] = weight, tops[warp] = top;
  __syncthreads();
  if (threadIdx.x < D) {
    float most = tops[0], v = 0.0f, w = 0.0f;
#pragma unroll
    for (int i = 1; i < kCaJoinWarps; ++i) most = fmaxf(most, tops[i]);
#pragma unroll
    for (int i = 0; i < kCaJoinWarps; ++i) {
      const float e = fast_exp2(tops[i] - most);
      v = fmaf(sums[i][threadIdx.x], e, v), w = fmaf(weights[i], e, w);
    }
    store_out(o + ((static_cast<long>(b) * tokens + row / G) * H + h * G + row % G) * D + threadIdx.x,
              w == 0.0f ? 0.0f : v / w);
  }
}

}  // namespace bsa
