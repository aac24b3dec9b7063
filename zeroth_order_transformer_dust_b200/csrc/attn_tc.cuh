// What the tensor-core kernels of the exact attention share: tile sizes, bounded
// waits, small conversions and the tensor maps.
#pragma once
#include <cudaTypedefs.h>

#include <type_traits>

#include "internal.cuh"
#include "tc_ptx.cuh"

namespace dust {
namespace {

constexpr int BM = 128;  // resident rows: TMEM lanes
constexpr int BN = 128;  // rows of a streamed tile
constexpr int BOX_BYTES = 128 * 64 * 2;  // a TMA box: 128 rows x 64 columns
constexpr int SOFT_WARPS = 8;

// fp32 tensors run on the tensor cores as NP = 3 bf16 planes, x = x0 + x1 + x2
// exactly (each plane takes the next 8 significant bits; bf16 has fp32's range),
// and a product as the six of their nine that are not below 2^-22 of it. The
// tensor cores add to an accumulator by truncation, so the small terms go first:
// only the last one's additions then lose anything of the sum's own size.
// bf16 tensors are one plane, NP = 1.
template <int NP>
constexpr int kTerms = NP == 1 ? 1 : 6;
template <int NP>
__device__ constexpr int term_a(int t) {
  constexpr int a[6] = {2, 0, 1, 0, 1, 0};
  return NP == 1 ? 0 : a[t];
}
template <int NP>
__device__ constexpr int term_b(int t) {
  constexpr int b[6] = {0, 2, 1, 1, 0, 0};
  return NP == 1 ? 0 : b[t];
}
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

// Columns [0, 32 n) of a thread's TMEM lane times `scale` to dst.
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
template <int N32>
__device__ __forceinline__ void store_row(uint32_t taddr, float scale, float* dst, bool in) {
#pragma unroll
  for (int c = 0; c < N32; ++c) {
    float v[32];
    ptx::tmem_ld32(taddr + 32 * c, v);
    if (!in) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      reinterpret_cast<float4*>(dst + 32 * c)[i] =
          make_float4(v[4 * i] * scale, v[4 * i + 1] * scale, v[4 * i + 2] * scale,
                      v[4 * i + 3] * scale);
  }
}
template <int NP>
using Elem = typename std::conditional<NP == 1, __nv_bfloat16, float>::type;

// 32 values of a row as NP bf16 planes of 16 TMEM columns: planes 0 and 1 at t and
// t + 32 (32-column blocks of a 64-column half), plane 2 at t2. v is used up.
template <int NP>
__device__ __forceinline__ void store_planes(uint32_t t, uint32_t t2, float2 (&v)[16]) {
  uint32_t pk[16];
  if (NP == 3) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t x = __float_as_uint(v[i].x), y = __float_as_uint(v[i].y);
        pk[i] = __byte_perm(x, y, 0x7632);  // the upper halves: truncated, so exact to take off
        v[i].x -= __uint_as_float(x & 0xffff0000u);
        v[i].y -= __uint_as_float(y & 0xffff0000u);
      }
      ptx::tmem_st16(t + 32 * q, pk);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) pk[i] = pack_bf16(v[i].x, v[i].y);
  ptx::tmem_st16(NP == 3 ? t2 : t, pk);
}

// The MMAs of S or dP: d = sum over the planes' terms of r s^T, both K-major in
// 64-column boxes, 32 bytes per 16-deep step.
template <int D, int NP>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t r, uint32_t s) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(BM, BN);
  constexpr uint32_t plane = BM * D * 2;
#pragma unroll
  for (int t = 0; t < kTerms<NP>; ++t)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ptx::mma_f16(d, ptx::sdesc_kmajor_sw128(r + term_a<NP>(t) * plane + c * BOX_BYTES + 32 * k),
                     ptx::sdesc_kmajor_sw128(s + term_b<NP>(t) * plane + c * BOX_BYTES + 32 * k), id,
                     (t | c | k) != 0);
}
// The MMAs of a sum: acc += sum over the terms of (planes in TMEM as store_planes
// left them, two halves of 64 rows of the contraction) x (tile read MN-major: 16
// rows, 2048 bytes, per step).
template <int D, int NP>
__device__ __forceinline__ void mma_sum(uint32_t acc, uint32_t p, uint32_t p2, uint32_t s,
                                        bool first) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(BM, D) | ptx::kIdescBMn;
  constexpr uint32_t plane = BM * D * 2;
#pragma unroll
  for (int t = 0; t < kTerms<NP>; ++t)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t a = term_a<NP>(t) < 2 ? p + 64 * (k >> 2) + 32 * term_a<NP>(t) + 8 * (k & 3)
                                       : p2 + 32 * (k >> 2) + 8 * (k & 3);
      ptx::mma_f16_ts(acc, a, ptx::sdesc_mnmajor_sw128(s + term_b<NP>(t) * plane + 2048 * k, BOX_BYTES),
                      id, !first || (t | k) != 0);
    }
}

// Zero the last `rows` rows of a landed tile (D / 64 boxes a plane of 128 lines of
// 128 bytes; a swizzled row stays inside its line), by a warp, for the MMAs to see.
template <int D, int NP>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int rows, int lane) {
  uint4* t = reinterpret_cast<uint4*>(tile);
  for (int i = lane; i < NP * (D / 64) * rows * 8; i += 32) {
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
bool rows16(const AttnArgs& a, const void* p, int64_t ld) {
  return ((uintptr_t)p & 15) == 0 && (ld & (a.dtype == DUST_BF16 ? 7 : 3)) == 0;
}

// The tensor maps of n tensors: of the tensors themselves (NP 1), or of their
// planes in a.planes, which a kernel on `st` fills first (NP 3: T rows of three
// planes side by side, tensor after tensor).
template <int NP>
cudaError_t make_maps(cudaStream_t st, const AttnArgs& a, const SplitSrc* src, CUtensorMap** maps,
                      int n) {
  __nv_bfloat16* at = (__nv_bfloat16*)a.planes;
  for (int i = 0; i < n; ++i) {
    const SplitSrc& x = src[i];
    if (!(NP == 1 ? make_map(maps[i], x.p, a.T, x.width, x.ld)
                  : make_map(maps[i], at, a.T, 3 * x.width, 3 * x.width)))
      return cudaErrorInvalidValue;
    at += a.T * 3 * x.width;
  }
  return NP == 1 ? cudaSuccess : launch_split_planes(st, src, n, a.T, a.planes);
}

}  // namespace
}  // namespace dust
