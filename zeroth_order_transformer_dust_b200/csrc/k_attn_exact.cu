// Causal attention and its exact gradient on CUDA cores, fp32 arithmetic: the
// form for head widths, strides and alignments that the tensor-core forms do not
// take (32-wide heads, 128-wide ones in fp32, rows off 16-byte boundaries).
//
// Mathematics, per sequence and head (key/value head h / (H / H_kv)), for
// pairs j <= i:  s_ij = scale <q_i, k_j>,  p_ij = exp(s_ij - lse_i),
//   o_i = sum_j p_ij v_j,  lse_i = log sum_j exp(s_ij),
//   delta_i = <o_i, e_i>,  dp_ij = <e_i, v_j>,  ds_ij = p_ij (dp_ij - delta_i),
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij e_i,
// the last two also summed over the heads that share the key/value head. The
// backward pass recomputes p from lse, so nothing of size L x L is stored.
//
// Two backward kernels, one per side: a CTA that owns query rows sums dq over
// the keys, a CTA that owns key rows sums dk and dv over the queries and over
// the heads of its group. Scores are formed twice (14 instead of 10 d_h flops a
// pair) and in exchange no sum is shared between CTAs: no atomics, and results
// that do not depend on timing. Bound by the FFMA and shared-memory rates:
// every product reads two 16-byte operands per 16 FFMAs (8 x 1024 tokens, 12 heads
// of 64: forward 637 us, 20 TFLOP/s; backward 2110 us, 15 TFLOP/s of the exact
// flops; 12 heads of 32: 370 and 1056 us in bf16, 370 and 1087 in fp32; of 128 in
// fp32: 1204 and 3640).
//
// Everything is fp32 until the one rounding of the outputs, p and ds too, where
// the tensor-core form of bf16 tensors rounds those to bf16. A sum over a
// sequence is one fp32 chain (about sqrt(n) 2^-24 off for n terms), which is less
// exact than the planes of the fp32 tensor-core form with their sum per tile.
#include <cfloat>

#include "internal.cuh"

namespace dust {
namespace {

constexpr int BT = 64;        // rows of a query or key tile
constexpr int THREADS = 256;  // 16 x 16, each with 4 x 4 of a 64 x 64 tile
constexpr int PP = BT + 4;    // row pitch of the probability tiles

__device__ __forceinline__ float4 load4(const float* p) {
  return make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  return make_float4(__bfloat162float(p[0]), __bfloat162float(p[1]), __bfloat162float(p[2]),
                     __bfloat162float(p[3]));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Rows [r0, r0 + 64) of a head as fp32 into dst (64 x (DH + 4)); rows at or
// past `end` are zero, so that what lies behind a sequence never enters a sum.
template <typename E, int DH>
__device__ __forceinline__ void load_tile(float* dst, const E* src, int64_t ld, int64_t col,
                                          int64_t r0, int64_t end) {
  constexpr int G = DH / 4;
  for (int i = threadIdx.x; i < BT * G; i += THREADS) {
    const int r = i / G, c = (i % G) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r0 + r < end) v = load4(src + (r0 + r) * ld + col + c);
    *reinterpret_cast<float4*>(dst + r * (DH + 4) + c) = v;
  }
}

// acc[a][b] = <A row (4 ty + a), B row (tx + 16 b)>
template <int DH>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx,
                                         float (&acc)[4][4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = 0.0f;
#pragma unroll 2
  for (int d = 0; d < DH; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
      x[a] = *reinterpret_cast<const float4*>(A + (4 * ty + a) * (DH + 4) + d);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      y[b] = *reinterpret_cast<const float4*>(B + (tx + 16 * b) * (DH + 4) + d);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        acc[a][b] = fmaf(x[a].x, y[b].x, acc[a][b]);
        acc[a][b] = fmaf(x[a].y, y[b].y, acc[a][b]);
        acc[a][b] = fmaf(x[a].z, y[b].z, acc[a][b]);
        acc[a][b] = fmaf(x[a].w, y[b].w, acc[a][b]);
      }
  }
}

// acc[a][c] += sum_r P[r][4 ty + a] B[r][column c of the thread]: rows of the
// result are columns of P. Columns: 4 tx + 64 g + {0..3}.
template <int DH>
__device__ __forceinline__ void sum_rows(const float* P, const float* B, int ty, int tx,
                                         float (&acc)[4][DH / 16]) {
  constexpr int NG = DH >= 64 ? DH / 64 : 1;
  constexpr int W = DH >= 64 ? 4 : DH / 16;
#pragma unroll 2
  for (int r = 0; r < BT; ++r) {
    const float4 p = *reinterpret_cast<const float4*>(P + r * PP + 4 * ty);
    const float pa[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float b[W];
#pragma unroll
      for (int w = 0; w < W; ++w) b[w] = B[r * (DH + 4) + g * 64 + W * tx + w];
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int w = 0; w < W; ++w) acc[a][g * W + w] = fmaf(pa[a], b[w], acc[a][g * W + w]);
    }
  }
}
template <int DH>
__device__ __forceinline__ int col_of(int tx, int c) {
  constexpr int W = DH >= 64 ? 4 : DH / 16;
  return (c / W) * 64 + W * tx + c % W;
}

// The tile's sequence: rows [beg, end) of the batch; false where the tile is
// past the sequence's end or the offsets are not usable (then flagged).
__device__ __forceinline__ bool sequence_of(const AttnArgs& a, int seq, int tile, int64_t* beg,
                                            int64_t* end) {
  if (!attn_sequence(a, seq, beg, end)) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadSeq);
    return false;
  }
  return (int64_t)tile * BT < *end - *beg;
}

template <typename E, int DH>
__global__ __launch_bounds__(THREADS, DH == 128 ? 1 : 2) void k_attn_exact_fwd(AttnArgs a) {
  extern __shared__ float sm[];
  float* sq = sm;
  float* sk = sq + BT * (DH + 4);
  float* sv = sk + BT * (DH + 4);
  float* sp = sv + BT * (DH + 4);  // [key][query]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  // the longest rows of tiles first: they take the most key tiles
  const int tile = (int)gridDim.x - 1 - (int)blockIdx.x;
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv);
  int64_t beg, end;
  if (!sequence_of(a, blockIdx.z, tile, &beg, &end)) return;
  const int64_t q0 = beg + (int64_t)tile * BT;
  load_tile<E, DH>(sq, (const E*)a.Q, a.ldq, (int64_t)h * DH, q0, end);
  float o[4][DH / 16] = {};
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -FLT_MAX, l[i] = 0.0f;
  for (int j = 0; j <= tile; ++j) {
    const int64_t k0 = beg + (int64_t)j * BT;
    __syncthreads();
    load_tile<E, DH>(sk, (const E*)a.K, a.ldk, (int64_t)hk * DH, k0, end);
    load_tile<E, DH>(sv, (const E*)a.V, a.ldv, (int64_t)hk * DH, k0, end);
    __syncthreads();
    float s[4][4];
    dot_tile<DH>(sq, sk, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = m[i];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        s[i][b] *= a.scale;
        if (k0 + tx + 16 * b <= q0 + 4 * ty + i) mx = fmaxf(mx, s[i][b]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float f = expf(m[i] - mx);
      float sum = 0.0f;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const bool in = k0 + tx + 16 * b <= q0 + 4 * ty + i;
        const float p = in ? expf(s[i][b] - mx) : 0.0f;
        sum += p;
        sp[(tx + 16 * b) * PP + 4 * ty + i] = p;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = fmaf(l[i], f, sum);
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < DH / 16; ++c) o[i][c] *= f;
    }
    __syncthreads();
    sum_rows<DH>(sp, sv, ty, tx, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = q0 + 4 * ty + i;
    if (r >= end) continue;
    const float inv = 1.0f / l[i];
#pragma unroll
    for (int c = 0; c < DH / 16; ++c)
      store1((E*)a.O + r * a.ldo + (int64_t)h * DH + col_of<DH>(tx, c), o[i][c] * inv);
    if (tx == 0) a.lse_out[r * a.H + h] = m[i] + logf(l[i]);
  }
}

// p and ds of a 64 x 64 tile from its score and dp products: queries q0 + 4 ty
// + i, keys k0 + tx + 16 b; pairs beyond the causal half or a sequence's end give 0.
__device__ __forceinline__ void probs_tile(const AttnArgs& a, float (&s)[4][4], float (&dp)[4][4],
                                           const float* lse, const float* delta, int64_t q0,
                                           int64_t k0, int64_t end, int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = q0 + 4 * ty + i;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bool in = r < end && k0 + tx + 16 * b <= r;
      const float p = in ? expf(fmaf(s[i][b], a.scale, -lse[4 * ty + i])) : 0.0f;
      s[i][b] = p;
      dp[i][b] = in ? p * (dp[i][b] - delta[4 * ty + i]) : 0.0f;
    }
  }
}

// dq of one query tile; also delta = <o, e> of its rows, which the key side reads.
template <typename E, int DH>
__global__ __launch_bounds__(THREADS, DH == 128 ? 1 : 2) void k_attn_exact_dq(AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int TS = BT * (DH + 4);
  float* sq = sm;
  float* se = sq + TS;
  float* sk = se + TS;
  float* sv = sk + TS;
  float* sp = sv + TS;  // ds as [key][query]
  __shared__ float s_lse[BT], s_delta[BT];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int tile = (int)gridDim.x - 1 - (int)blockIdx.x;
  const int h = blockIdx.y, hk = h / (a.H / a.Hkv);
  int64_t beg, end;
  if (!sequence_of(a, blockIdx.z, tile, &beg, &end)) return;
  const int64_t q0 = beg + (int64_t)tile * BT;
  load_tile<E, DH>(sq, (const E*)a.Q, a.ldq, (int64_t)h * DH, q0, end);
  load_tile<E, DH>(se, (const E*)a.E, a.lde, (int64_t)h * DH, q0, end);
  load_tile<E, DH>(sk, (const E*)a.O_in, a.ldo, (int64_t)h * DH, q0, end);
  __syncthreads();
  {  // four threads a row
    const int r = threadIdx.x >> 2;
    float d = 0.0f;
    for (int c = threadIdx.x & 3; c < DH; c += 4)
      d = fmaf(sk[r * (DH + 4) + c], se[r * (DH + 4) + c], d);
    d += __shfl_xor_sync(0xffffffffu, d, 1);
    d += __shfl_xor_sync(0xffffffffu, d, 2);
    if ((threadIdx.x & 3) == 0) {
      const bool in = q0 + r < end;
      s_delta[r] = d;
      s_lse[r] = in ? a.lse[(q0 + r) * a.H + h] : 0.0f;
      if (in) a.delta[(q0 + r) * a.H + h] = d;
    }
  }
  float dq[4][DH / 16] = {};
  for (int j = 0; j <= tile; ++j) {
    const int64_t k0 = beg + (int64_t)j * BT;
    __syncthreads();
    load_tile<E, DH>(sk, (const E*)a.K, a.ldk, (int64_t)hk * DH, k0, end);
    load_tile<E, DH>(sv, (const E*)a.V, a.ldv, (int64_t)hk * DH, k0, end);
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<DH>(sq, sk, ty, tx, s);
    dot_tile<DH>(se, sv, ty, tx, dp);
    probs_tile(a, s, dp, s_lse, s_delta, q0, k0, end, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) sp[(tx + 16 * b) * PP + 4 * ty + i] = dp[i][b];
    __syncthreads();
    sum_rows<DH>(sp, sk, ty, tx, dq);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = q0 + 4 * ty + i;
    if (r >= end) continue;
#pragma unroll
    for (int c = 0; c < DH / 16; ++c)
      store1((E*)a.dQ + r * a.lddq + (int64_t)h * DH + col_of<DH>(tx, c), dq[i][c] * a.scale);
  }
}

// dk and dv of one key tile of a key/value head, over the heads that share it
// and the query tiles at or after it.
template <typename E, int DH>
__global__ __launch_bounds__(THREADS, DH >= 64 ? 1 : 2) void k_attn_exact_dkv(AttnArgs a) {
  extern __shared__ float sm[];
  constexpr int TS = BT * (DH + 4);
  float* sk = sm;
  float* sv = sk + TS;
  float* sq = sv + TS;
  float* se = sq + TS;
  float* sp = se + TS;        // p as [query][key]
  float* sd = sp + BT * PP;   // ds as [query][key]
  __shared__ float s_lse[BT], s_delta[BT];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int tile = blockIdx.x;  // the first key tiles have the most queries
  const int hk = blockIdx.y, group = a.H / a.Hkv;
  int64_t beg, end;
  if (!sequence_of(a, blockIdx.z, tile, &beg, &end)) return;
  const int64_t k0 = beg + (int64_t)tile * BT;
  const int tiles = (int)((end - beg + BT - 1) / BT);
  load_tile<E, DH>(sk, (const E*)a.K, a.ldk, (int64_t)hk * DH, k0, end);
  load_tile<E, DH>(sv, (const E*)a.V, a.ldv, (int64_t)hk * DH, k0, end);
  float dk[4][DH / 16] = {}, dv[4][DH / 16] = {};
  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    for (int i0 = tile; i0 < tiles; ++i0) {
      const int64_t q0 = beg + (int64_t)i0 * BT;
      __syncthreads();
      load_tile<E, DH>(sq, (const E*)a.Q, a.ldq, (int64_t)h * DH, q0, end);
      load_tile<E, DH>(se, (const E*)a.E, a.lde, (int64_t)h * DH, q0, end);
      if (threadIdx.x < BT) {
        const bool in = q0 + threadIdx.x < end;
        s_lse[threadIdx.x] = in ? a.lse[(q0 + threadIdx.x) * a.H + h] : 0.0f;
        s_delta[threadIdx.x] = in ? a.delta[(q0 + threadIdx.x) * a.H + h] : 0.0f;
      }
      __syncthreads();
      float s[4][4], dp[4][4];
      dot_tile<DH>(sq, sk, ty, tx, s);
      dot_tile<DH>(se, sv, ty, tx, dp);
      probs_tile(a, s, dp, s_lse, s_delta, q0, k0, end, ty, tx);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          sp[(4 * ty + i) * PP + tx + 16 * b] = s[i][b];
          sd[(4 * ty + i) * PP + tx + 16 * b] = dp[i][b];
        }
      __syncthreads();
      sum_rows<DH>(sp, se, ty, tx, dv);
      sum_rows<DH>(sd, sq, ty, tx, dk);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = k0 + 4 * ty + i;
    if (r >= end) continue;
#pragma unroll
    for (int c = 0; c < DH / 16; ++c) {
      const int64_t col = (int64_t)hk * DH + col_of<DH>(tx, c);
      store1((E*)a.dK + r * a.lddk + col, dk[i][c] * a.scale);
      store1((E*)a.dV + r * a.lddv + col, dv[i][c]);
    }
  }
}

template <typename F>
cudaError_t launch_tiles(cudaStream_t st, F fn, const AttnArgs& a, int heads, size_t smem) {
  cudaError_t err =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)((a.max_len + BT - 1) / BT), (unsigned)heads, (unsigned)a.n_seqs);
  fn<<<grid, THREADS, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename E, int DH>
cudaError_t fwd_as(cudaStream_t st, const AttnArgs& a) {
  return launch_tiles(st, k_attn_exact_fwd<E, DH>, a, a.H,
                      (3 * BT * (DH + 4) + BT * PP) * sizeof(float));
}
template <typename E, int DH>
cudaError_t bwd_as(cudaStream_t st, const AttnArgs& a) {
  const cudaError_t err = launch_tiles(st, k_attn_exact_dq<E, DH>, a, a.H,
                                       (4 * BT * (DH + 4) + BT * PP) * sizeof(float));
  if (err != cudaSuccess) return err;
  return launch_tiles(st, k_attn_exact_dkv<E, DH>, a, a.Hkv,
                      (4 * BT * (DH + 4) + 2 * BT * PP) * sizeof(float));
}

template <typename E>
cudaError_t simt_as(cudaStream_t st, const AttnArgs& a, bool backward) {
  switch (a.head_dim) {
    case 32: return backward ? bwd_as<E, 32>(st, a) : fwd_as<E, 32>(st, a);
    case 64: return backward ? bwd_as<E, 64>(st, a) : fwd_as<E, 64>(st, a);
    case 128: return backward ? bwd_as<E, 128>(st, a) : fwd_as<E, 128>(st, a);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attn_exact_simt(cudaStream_t st, const AttnArgs& a, bool backward) {
  return a.dtype == DUST_BF16 ? simt_as<__nv_bfloat16>(st, a, backward)
                              : simt_as<float>(st, a, backward);
}

}  // namespace dust
