// pair_ops.cuh -- what the products on CTA pairs with operands in either layout
// share (grouped.cu, orthogonalize.cu): bounded waits with the CTA's give-up flag,
// matrix and instruction descriptors, the ring, tensor copies out of shared
// memory, tensor maps and the launch of one CTA pair for each pair of SMs.
#pragma once

#include "gemm2sm.cuh"

namespace symmoe {
namespace pair {

using namespace gemm2;

constexpr int CHUNK_BYTES = BK * 64 * 2;  // 64 contraction rows x 64 features (MN-major tiles)

// Role-local view of the CTA's give-up flag and the wait limit
struct Ctl {
  volatile int *abort;
  int32_t *status;
  uint32_t tmo;
};

__device__ __forceinline__ void raise(int32_t *status, int bits) {
  if (status) atomicOr(status, bits);
}

// Bounded wait (cluster-scope acquire: some arrivals come from the pair's
// other CTA after generic stores); a timeout sets the CTA's abort flag.  A wait
// that may outlast several of the pair's tiles has the limit for each of them.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, const Ctl &c, uint32_t tiles = 1) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait_cluster(a, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  const uint64_t limit = (uint64_t)c.tmo * tiles * 1000ull;
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait_cluster(a, parity)) return true;
    if (*c.abort) return false;
    if ((it & 15u) == 15u && globaltimer_ns() - t0 > limit) {
      *c.abort = 1;
      raise(c.status, SYM_STATUS_TIMEOUT);
      return false;
    }
  }
}

// A wait of this CTA has run out and all its threads have stopped: before its
// shared memory and TMEM are given up, wait (10 ms at most) for the MMAs in
// flight, and 10 ms for the copies.  No barrier this CTA may wait on counts all of
// those (the peer's are counted by the leader, a stage that one CTA did not load
// never completes); a copy takes some microseconds.
__device__ __forceinline__ void settle(uint64_t *drained, bool issuer) {
  constexpr uint32_t LIMIT_US = 10000;
  const uint64_t t0 = globaltimer_ns();
  if (issuer) {
    commit2_both(drained);
    mbar_wait(drained, 0, LIMIT_US, nullptr);
  }
  while (globaltimer_ns() - t0 < LIMIT_US * 1000ull) __nanosleep(1000);
}

// Matrix descriptor of an MN-major tile with the 128-byte swizzle: chunks of
// 64 features, each [64 contraction rows][128 bytes]; the leading offset steps
// over chunks, the stride offset over groups of 8 contraction rows.
__device__ __forceinline__ uint64_t smem_desc_mn(const void *tile, int chunk = CHUNK_BYTES) {
  uint64_t d = 0;
  d |= (smem_u32(tile) >> 4) & 0x3FFFull;
  d |= (uint64_t)(chunk >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= 1ull << 46;
  d |= 2ull << 61;
  return d;
}
constexpr uint64_t MN_STEP = UK * 128 / 16;  // 16 contraction rows, in 16-byte units
constexpr uint64_t K_STEP = UK * 2 / 16;     // 16 contraction columns of a K-major row

// kind::f16 instruction descriptor (idesc_bf16_f32 with the operand type and
// majors as arguments): bits 7-9 / 10-12 operand formats (0 fp16, 1 bf16),
// bits 15 / 16 A / B major (1 = MN).
__device__ __forceinline__ uint32_t idesc(bool fp16, bool a_mn, bool b_mn, int n) {
  const uint32_t fmt = fp16 ? 0u : (1u << 7) | (1u << 10);
  return (1u << 4) | fmt | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
         ((256u >> 4) << 24);
}

__device__ __forceinline__ uint16_t to_half(float v) {
  uint16_t r;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}
template <bool FP16>
__device__ __forceinline__ uint16_t narrow(float v) {
  return FP16 ? to_half(v) : to_bf16(v);
}
template <bool FP16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if (!FP16) return pack_bf16x2(lo, hi);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float widen(bool fp16, uint16_t v) {
  if (!fp16) return __uint_as_float((uint32_t)v << 16);
  float r;
  asm("cvt.f32.f16 %0, %1;" : "=f"(r) : "h"(v));
  return r;
}

template <int N>
struct RingOf {
  uint8_t *base;
  uint64_t *full, *empty;
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == N) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Hand an accumulator (or its head) back to the leader's MMA.  What the arrival
// orders is the warp's finished TMEM reads, nothing in memory, so the peer's
// remote arrival releases at CTA scope: a release at cluster scope waits for
// the warp's stores (a third of the weight gradient's epilogue, 1900 cycles a tile).
__device__ __forceinline__ void give_back(uint64_t *bar, uint32_t rank, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    if (rank == 0) mbar_arrive(bar);
    else asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(map_to(bar, 0)) : "memory");
  }
}

// shared -> global tensor copies of the calling thread's bulk group: a box as
// it is, or added to what is there (fp32); elements past the extents are cut
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, const void *src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap *m, const void *src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
// all but the newest N groups of this thread have read their shared memory
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Order this thread's stores to shared memory before later tensor copies out
// of it.  The unrestricted proxy fence also waits for global accesses: with it
// the weight gradient of the prefill shape took 3.49 ms, with this one 2.99.
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// 16-bit (or fp32) elements [d2][d1][d0], strides in elements, box [1][b1][b0]; elements outside the extents read as zeros
inline bool encode(CUtensorMap *m, uint64_t ptr, uint64_t d0, uint64_t d1, uint64_t d2, int64_t s1, int64_t s2,
                   uint32_t b0, uint32_t b1, bool fp32 = false,
                   CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  typedef CUresult (*Fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                         const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                         CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Fn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<Fn>(p) : nullptr;
  }();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {(cuuint64_t)s1 * (fp32 ? 4 : 2), (cuuint64_t)s2 * (fp32 ? 4 : 2)};
  const cuuint32_t box[3] = {b0, b1, 1}, step[3] = {1, 1, 1};
  return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, reinterpret_cast<void *>(ptr), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Kern, typename... Args>
inline cudaError_t launch_pairs(Kern kern, int threads, size_t smem, int num_sms, cudaStream_t st, Args... args) {
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const int grid = 2 * max_resident_pairs((const void *)kern, threads, smem, num_sms);
  if (grid <= 0) return cudaErrorInvalidConfiguration;
  kern<<<grid, threads, smem, st>>>(args...);
  return cudaGetLastError();
}

}  // namespace pair
}  // namespace symmoe
