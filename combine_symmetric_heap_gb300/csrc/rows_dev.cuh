// rows_dev.cuh -- device helpers of the row-wise kernels (SwiGLU of expert
// rows, dropout, norms around a block): element types, 16-byte vectors, the
// counter-based random words, sums over a block.
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "symmoe_dev.cuh"

namespace symmoe {
namespace rows {

// VEC elements of T make one 16-byte vector
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float2 get2(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }
  static __device__ __forceinline__ uint32_t put2(float a, float b) { return pack_bf16x2(a, b); }
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float2 get2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  }
  static __device__ __forceinline__ uint32_t put2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// A 16-byte vector of T as floats and back, pairs converted together
template <typename T, int V>
__device__ __forceinline__ void unpack(const uint4 &q, float (&f)[V]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = Elem<T>::get2(w[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ uint4 pack(const float (&f)[V]) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = Elem<T>::put2(f[2 * i], f[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// V consecutive elements as floats: one 16-byte access when V is the vector
// length, one element when V is 1
template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float (&f)[V]) {
  if constexpr (V == 1) f[0] = Elem<T>::get(*p);
  else unpack<T, V>(*reinterpret_cast<const uint4 *>(p), f);
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&f)[V]) {
  if constexpr (V == 1) *p = Elem<T>::put(f[0]);
  else *reinterpret_cast<uint4 *>(p) = pack<T, V>(f);
}

// Four elements: 8 or 16 bytes
template <typename T>
struct Quad {
  using Word = typename std::conditional<sizeof(T) == 4, uint4, uint2>::type;
  static __device__ __forceinline__ void get(const void *p, float (&f)[4]) {
    const Word w = *reinterpret_cast<const Word *>(p);
    if constexpr (sizeof(T) == 4) {
      f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
    } else {
      const float2 a = Elem<T>::get2(w.x), b = Elem<T>::get2(w.y);
      f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    }
  }
  static __device__ __forceinline__ Word put(const float (&f)[4]) {
    if constexpr (sizeof(T) == 4)
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
      return make_uint2(Elem<T>::put2(f[0], f[1]), Elem<T>::put2(f[2], f[3]));
  }
};

// Columns [c, c + V) of a row, of which those outside [0, cols) do not exist
// (zeros on a load, skipped on a store); whole vectors are 16-byte accesses,
// so c places p + c on a 16-byte boundary.
template <typename T, int V>
__device__ __forceinline__ void load_part(const T *p, int c, int cols, float (&f)[V]) {
  if (c >= 0 && c + V <= cols) {
    load<T, V>(p + c, f);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = c + i >= 0 && c + i < cols ? Elem<T>::get(p[c + i]) : 0.f;
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T *p, int c, int cols, const float (&f)[V]) {
  if (c >= 0 && c + V <= cols) {
    store<T, V>(p + c, f);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + i >= 0 && c + i < cols) p[c + i] = Elem<T>::put(f[i]);
}

// ---------------------------------------------------------------------------
// Counter-based random words: Philox 4x32 with 10 rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  Block
// b of the stream (seed, offset) is the cipher of the counter
// (b mod 2^32, b >> 32, offset mod 2^32, offset >> 32) under the key
// (seed mod 2^32, seed >> 32); word j of it belongs to element 4b + j.
// ---------------------------------------------------------------------------
struct Random {
  uint64_t offset;
  uint32_t key[10][2];  // the rounds' keys
  // The first two rounds multiply two words that are the same for all blocks
  // below 2^32: what they leave behind (see random_block).
  uint32_t first[4];
  uint32_t threshold;  // an element is kept where its word >= threshold
  float keep_scale;    // 1 / (1 - p)
};
constexpr uint32_t PHILOX_A = 0xD2511F53u, PHILOX_B = 0xCD9E8D57u;
inline Random make_random(uint64_t seed, uint64_t offset, double p) {
  Random r;
  r.offset = offset;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int i = 0; i < 10; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
    r.key[i][0] = k0;
    r.key[i][1] = k1;
  }
  const uint64_t b = (uint64_t)(uint32_t)offset * PHILOX_B;  // round 1, of the counter's third word
  const uint64_t a = (uint64_t)((uint32_t)(b >> 32) ^ r.key[0][0]) * PHILOX_A;  // round 2, of the first
  r.first[0] = (uint32_t)(offset >> 32) ^ r.key[0][1];  // round 1: third word = high(a) ^ this
  r.first[1] = (uint32_t)b ^ r.key[1][0];               // round 2: first word = high(b) ^ this
  r.first[2] = (uint32_t)(a >> 32) ^ r.key[1][1];       // round 2: third word = low(a of round 1) ^ this
  r.first[3] = (uint32_t)a;                             // round 2: fourth word
  r.threshold = (uint32_t)(p * 4294967296.0);
  r.keep_scale = (float)(1.0 / (1.0 - p));
  return r;
}
__device__ __forceinline__ uint4 random_block(const Random &r, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2, c3;
  auto round = [&](int i) {
    const uint64_t a = (uint64_t)c0 * PHILOX_A, b = (uint64_t)c2 * PHILOX_B;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ r.key[i][0];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ r.key[i][1];
    c3 = (uint32_t)a;
  };
  if (c1 == 0) {
    const uint64_t a = (uint64_t)c0 * PHILOX_A;
    const uint64_t b = (uint64_t)((uint32_t)(a >> 32) ^ r.first[0]) * PHILOX_B;
    c0 = (uint32_t)(b >> 32) ^ r.first[1];
    c1 = (uint32_t)b;
    c2 = (uint32_t)a ^ r.first[2];
    c3 = r.first[3];
  } else {
    c2 = (uint32_t)r.offset, c3 = (uint32_t)(r.offset >> 32);
    round(0);
    round(1);
  }
#pragma unroll
  for (int i = 2; i < 10; ++i) round(i);
  return make_uint4(c0, c1, c2, c3);
}
__device__ __forceinline__ void random_words(const Random &r, uint64_t block, uint32_t (&u)[4]) {
  const uint4 w = random_block(r, block);
  u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
}
// Bit 4b + j: is element j of block first[b] kept?  The blocks' rounds run side
// by side: a round is a chain of two dependent instructions, and one block at a
// time would leave the pipes waiting on it.
template <int NB>
__device__ __forceinline__ uint32_t kept_bits(const Random &r, const uint64_t (&block)[NB]) {
  uint32_t c0[NB], c1[NB], c2[NB], c3[NB];
  bool small = true;
#pragma unroll
  for (int b = 0; b < NB; ++b) small = small && (block[b] >> 32) == 0;
  if (small) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint64_t x = (uint64_t)(uint32_t)block[b] * PHILOX_A;
      const uint64_t y = (uint64_t)((uint32_t)(x >> 32) ^ r.first[0]) * PHILOX_B;
      c0[b] = (uint32_t)(y >> 32) ^ r.first[1];
      c1[b] = (uint32_t)y;
      c2[b] = (uint32_t)x ^ r.first[2];
      c3[b] = r.first[3];
    }
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      c0[b] = (uint32_t)block[b], c1[b] = (uint32_t)(block[b] >> 32);
      c2[b] = (uint32_t)r.offset, c3[b] = (uint32_t)(r.offset >> 32);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t x = (uint64_t)c0[b] * PHILOX_A, y = (uint64_t)c2[b] * PHILOX_B;
        c0[b] = (uint32_t)(y >> 32) ^ c1[b] ^ r.key[i][0];
        c1[b] = (uint32_t)y;
        c2[b] = (uint32_t)(x >> 32) ^ c3[b] ^ r.key[i][1];
        c3[b] = (uint32_t)x;
      }
    }
  }
#pragma unroll
  for (int i = 2; i < 10; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint64_t x = (uint64_t)c0[b] * PHILOX_A, y = (uint64_t)c2[b] * PHILOX_B;
      c0[b] = (uint32_t)(y >> 32) ^ c1[b] ^ r.key[i][0];
      c1[b] = (uint32_t)y;
      c2[b] = (uint32_t)(x >> 32) ^ c3[b] ^ r.key[i][1];
      c3[b] = (uint32_t)x;
    }
  uint32_t kept = 0u;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (c0[b] >= r.threshold) kept |= 1u << (4 * b);
    if (c1[b] >= r.threshold) kept |= 2u << (4 * b);
    if (c2[b] >= r.threshold) kept |= 4u << (4 * b);
    if (c3[b] >= r.threshold) kept |= 8u << (4 * b);
  }
  return kept;
}

// keep factors (0 or 1 / (1 - p)) of the V elements from element `at` on
template <int V>
__device__ __forceinline__ void keep_factors(const Random &r, uint64_t at, float (&k)[V]) {
  if (V >= 4 && (at & 3u) == 0) {  // whole blocks
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const uint4 w = random_block(r, (at + i) >> 2);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4 && i + j < V; ++j) k[i + j] = u[j] >= r.threshold ? r.keep_scale : 0.f;
    }
    return;
  }
  uint64_t have = ~0ull;
  uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint64_t b = (at + i) >> 2;
    if (b != have) {
      w = random_block(r, b);
      have = b;
    }
    const uint32_t j = (uint32_t)(at + i) & 3u;
    const uint32_t u = j == 0 ? w.x : j == 1 ? w.y : j == 2 ? w.z : w.w;
    k[i] = u >= r.threshold ? r.keep_scale : 0.f;
  }
}

// Which of the n elements from element `first` on are kept, one byte each: for
// rows walked element by element, where every block of words would otherwise be
// made four times
__device__ __forceinline__ void fill_mask(const Random &r, uint64_t first, int n, uint8_t *mask, int thread,
                                          int threads) {
  for (uint64_t b = (first >> 2) + thread; 4 * b < first + n; b += threads) {
    uint32_t word[4];
    random_words(r, b, word);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = (int64_t)(4 * b + j - first);
      if (i >= 0 && i < n) mask[i] = word[j] >= r.threshold;
    }
  }
}

// ---------------------------------------------------------------------------
// Sums of K values over the `warps` warps of a row group; every thread gets
// the totals, added in a fixed order.  buf holds 2 * 32 * K floats per group;
// `turn` alternates its halves, so one block barrier per call is enough.
// ---------------------------------------------------------------------------
template <int K>
__device__ __forceinline__ void warp_sums(float (&v)[K]) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], s);
}
template <int K>
__device__ __forceinline__ void group_sums(float (&v)[K], float *buf, int warp, int warps, int &turn) {
  warp_sums<K>(v);
  if (warps == 1) return;
  float *b = buf + turn * 32 * K;
  turn ^= 1;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[warp * K + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? b[lane * K + k] : 0.f;
  warp_sums<K>(v);
}

// Four sums at once for a block of one row.  Inside a warp the lanes trade
// values for halves of the lanes first (6 shuffles instead of 20), so that lane
// 8k ends with sum k; then every warp adds the warps' sums.  buf: 2 * 128
// floats, its halves used in turn.
__device__ __forceinline__ void block_sums4(float (&v)[4], float *buf, int warp, int warps, int &turn) {
  const int lane = threadIdx.x & 31;
  const bool h16 = lane & 16, h8 = lane & 8;
  float a = h16 ? v[2] : v[0], b = h16 ? v[3] : v[1];
  a += __shfl_xor_sync(0xffffffffu, h16 ? v[0] : v[2], 16);
  b += __shfl_xor_sync(0xffffffffu, h16 ? v[1] : v[3], 16);
  float s = h8 ? b : a;
  s += __shfl_xor_sync(0xffffffffu, h8 ? a : b, 8);
#pragma unroll
  for (int i = 4; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
  if (warps == 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(0xffffffffu, s, 8 * k);
    return;
  }
  float *p = buf + turn * 128;
  turn ^= 1;
  if ((lane & 7) == 0) p[warp * 4 + (lane >> 3)] = s;
  __syncthreads();
  // lane l: sum l mod 4 of warps l / 4, l / 4 + 8, ...
  s = 0.f;
  for (int w = lane >> 2; w < warps; w += 8) s += p[w * 4 + (lane & 3)];
#pragma unroll
  for (int i = 16; i > 2; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(0xffffffffu, s, k);
}

// Let launches of `kern` take up to `most` bytes of dynamic shared memory.  The
// limit is one per kernel for the whole process, so every call gives the kernel's
// largest size, whatever its own: with that, a call in another host thread cannot
// lower it between this call and its launch.
template <typename Kern>
inline cudaError_t allow_smem(Kern kern, int most) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

}  // namespace rows
}  // namespace symmoe
