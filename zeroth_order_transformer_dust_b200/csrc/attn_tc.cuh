// What the tensor-core kernels of the exact attention share: tile sizes, bounded
// waits, small conversions and the tensor maps.
#pragma once
#include <cudaTypedefs.h>

#include "internal.cuh"
#include "tc_ptx.cuh"

namespace dust {
namespace {

constexpr int BM = 128;  // resident rows: TMEM lanes
constexpr int BN = 128;  // rows of a streamed tile
constexpr int BOX_BYTES = 128 * 64 * 2;  // a TMA box: 128 rows x 64 columns
constexpr int SOFT_WARPS = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

// Wait for phase `parity` of an mbarrier, for at most kWaitLimitNs. On expiry the
// CTA's abort flag and the timeout bit are set and false returns; a raised
// abort flag also ends the wait. The hand-overs between the warps are short, so
// the clock is first read after some polls.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort,
                                       uint32_t* status) {
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort,
                                             uint32_t* status) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_long(bar, parity, abort, status);
}
// The same by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort, status));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float inf_f() { return __int_as_float(0x7f800000); }

// Columns [0, 32 n) of a thread's TMEM lane times `scale` as bf16 to dst.
template <int N32>
__device__ __forceinline__ void store_row(uint32_t taddr, float scale, __nv_bfloat16* dst,
                                          bool in) {
#pragma unroll
  for (int c = 0; c < N32; ++c) {
    float v[32];
    ptx::tmem_ld32(taddr + 32 * c, v);
    if (!in) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 u;
      u.x = pack_bf16(v[8 * i] * scale, v[8 * i + 1] * scale);
      u.y = pack_bf16(v[8 * i + 2] * scale, v[8 * i + 3] * scale);
      u.z = pack_bf16(v[8 * i + 4] * scale, v[8 * i + 5] * scale);
      u.w = pack_bf16(v[8 * i + 6] * scale, v[8 * i + 7] * scale);
      reinterpret_cast<uint4*>(dst + 32 * c)[i] = u;
    }
  }
}

// Zero the last `rows` rows of a landed tile (D / 64 boxes of 128 lines of 128
// bytes; a swizzled row stays inside its line), by a warp, for the MMAs to see.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int rows, int lane) {
  uint4* t = reinterpret_cast<uint4*>(tile);
  for (int i = lane; i < D / 64 * rows * 8; i += 32) {
    const int box = i / (rows * 8), w = i % (rows * 8);
    t[box * (BOX_BYTES / 16) + (BN - rows) * 8 + w] = make_uint4(0, 0, 0, 0);
  }
  ptx::fence_proxy_async();
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return (PFN_cuTensorMapEncodeTiled_v12000)ptr;
    return nullptr;
  }();
  return fn;
}

// T x cols bf16 rows (stride ld) as boxes of 64 columns x 128 rows, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* p, int64_t T, int64_t cols, int64_t ld) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)T};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, BN}, estr[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 16-byte rows: what TMA and the vector loads and stores need.
bool rows16(const void* p, int64_t ld, int64_t T) {
  return ((uintptr_t)p & 15) == 0 && (T <= 1 || (ld & 7) == 0);
}

}  // namespace
}  // namespace dust
