// Losses over the vocabulary on logits a model has already produced: log
// probabilities of given tokens with entropy and top alternatives, and
// distillation from a teacher's top logits with its logit gradient.
//
// Mathematics. Per row, with m = max_j z_j and e_j = exp((z_j - m) / tau):
//   s = sum_j e_j,  log p_j = (z_j - m) / tau - log s,
//   entropy (tau = 1) = log s - u / s,  u = sum_j (z_j - m) e_j,
//   distillation over the teacher's kept set J, q = softmax_J(v / tau):
//     loss = tau^2 sum_J q_j (log q_j - log p_j),
//     d loss / d z_j = tau (p_j - q_j)   (q_j = 0 outside J).
// All sums run in fp32 with the running maximum of an online softmax, so a row
// is read from HBM once whatever its scale; a thread keeps (m, s, u) of its own
// elements and the threads' triples are combined in a fixed order, so results
// do not depend on timing. z - m is formed before the scale is applied:
// the type's lowest value then stays an ordinary (if unlikely) logit instead of
// overflowing to -inf, and -inf - m gives exp = 0 without a NaN.
//
// Few rows do not fill the GPU with one CTA each, so a row may be split over a
// cluster of up to 8 CTAs whose triples (and top lists) meet in distributed
// shared memory: still one launch.
#include <atomic>
#include <cfloat>

#include "internal.cuh"
#include "tc_ptx.cuh"

namespace dust {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxCluster = 8;  // portable cluster size

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }
__device__ __forceinline__ float inf_f() { return __int_as_float(0x7f800000); }

__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}
// The same for memory that the kernel itself may overwrite later.
__device__ __forceinline__ float load_rw(const float* p) {
  return *reinterpret_cast<const volatile float*>(p);
}
__device__ __forceinline__ float load_rw(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const volatile unsigned short*>(p) << 16);
}
__device__ __forceinline__ void store_e(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_e(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 16 bytes as 4 fp32 or 8 bf16 values.
template <typename E>
struct Vec {
  static constexpr int N = 16 / sizeof(E);
};
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[4]) {
  v[0] = __uint_as_float(w.x);
  v[1] = __uint_as_float(w.y);
  v[2] = __uint_as_float(w.z);
  v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&v)[4]) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A CTA's part of a row: `head` elements up to the first 16-byte boundary (rank
// 0's), whole vectors [v0, v1) of the aligned body behind them, and the `tail`
// elements [tail0, tail1) after it (the last rank's). (V < 2^31.)
struct Slice {
  int head, v0, v1, tail0, tail1;
};
template <typename E>
__device__ __forceinline__ Slice slice_of(const E* row, int64_t V, int rank, int ranks) {
  constexpr int N = Vec<E>::N;
  Slice s;
  const int head = (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(E);
  s.head = head < V ? head : (int)V;
  const int nv = ((int)V - s.head) / N;
  s.v0 = (int)((int64_t)nv * rank / ranks);
  s.v1 = (int)((int64_t)nv * (rank + 1) / ranks);
  s.tail0 = s.head + nv * N;
  s.tail1 = rank == ranks - 1 ? (int)V : s.tail0;
  return s;
}

// Running softmax statistics: maximum, sum of exponentials relative to it and
// (ENT) the sum of (z - m) exp(z - m). The maximum starts at the type's lowest
// finite value, so a row of -inf alone leaves s = 0; a NaN (or +inf) element
// leaves s = NaN.
struct Stat {
  float m, s, u;
};
__device__ __forceinline__ Stat stat_none() { return Stat{-FLT_MAX, 0.0f, 0.0f}; }

template <bool ENT>
__device__ __forceinline__ void stat_rescale(Stat& a, float m, float k2) {
  const float f = ex2((a.m - m) * k2);
  // f = 0: nothing of the old sums is left (and s (m - m') could be 0 x inf)
  if (ENT) a.u = f > 0.0f ? f * fmaf(a.s, a.m - m, a.u) : 0.0f;
  a.s *= f;
  a.m = m;
}

// N (even) more elements, two per packed operation; returns their maximum.
template <bool ENT, int N>
__device__ __forceinline__ float stat_add(Stat& a, const float (&z)[N], float k2) {
  float cm = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) cm = fmaxf(cm, z[i]);
  if (cm > a.m) stat_rescale<ENT>(a, cm, k2);
  const float2 nm = make_float2(-a.m, -a.m), kk = make_float2(k2, k2);
  float2 s = make_float2(0.0f, 0.0f), u = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 d = __fadd2_rn(make_float2(z[i], z[i + 1]), nm);
    const float2 x = __fmul2_rn(d, kk);
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    s = __fadd2_rn(s, e);
    // exp(-1e4) = 0: the clamp only keeps 0 x (-inf) out
    if (ENT) u = __ffma2_rn(make_float2(fmaxf(d.x, -1e4f), fmaxf(d.y, -1e4f)), e, u);
  }
  a.s += s.x + s.y;
  if (ENT) a.u += u.x + u.y;
  return cm;
}
template <bool ENT>
__device__ __forceinline__ void stat_add1(Stat& a, float z, float k2) {
  const float pair[2] = {z, -inf_f()};
  stat_add<ENT, 2>(a, pair, k2);
}

// A warp's statistics, the same value in every lane: the maximum first, so
// that each lane rescales once; the butterflies add in a fixed order.
template <bool ENT>
__device__ __forceinline__ Stat stat_warp(Stat a, float k2) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  stat_rescale<ENT>(a, m, k2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    if (ENT) a.u += __shfl_xor_sync(0xffffffffu, a.u, o);
  }
  return a;
}

// Barrier of the first `threads` threads of a CTA (all but a producer warp), and
// the same with the or of a flag.
__device__ __forceinline__ void sync_threads(int threads) {
  asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}
__device__ __forceinline__ bool sync_threads_or(bool flag, int threads) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)flag), "r"(threads)
      : "memory");
  return r != 0;
}

// The statistics of the first `threads` threads, the same value in each.
template <bool ENT>
__device__ __forceinline__ Stat stat_block(Stat a, float k2, Stat* sh, int threads) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = stat_warp<ENT>(a, k2);
  if (lane == 0) sh[warp] = a;
  sync_threads(threads);
  return stat_warp<ENT>(lane < threads / 32 ? sh[lane] : stat_none(), k2);
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// The row's statistics from its CTAs', the same in every thread of the cluster.
// `mine` (shared memory) stays readable by the others until the cluster's next
// barrier, which the caller makes before it leaves.
template <bool ENT>
__device__ __forceinline__ Stat stat_cluster(const Stat& a, float k2, Stat* mine, int ranks) {
  if (ranks == 1) return a;
  if (threadIdx.x == 0) *mine = a;
  ptx::cluster_sync();
  const int lane = threadIdx.x & 31;
  Stat t = stat_none();
  if (lane < ranks) {
    const uint32_t p = ptx::mapa_shared(ptx::smem_u32(mine), (uint32_t)lane);
    t.m = ld_cluster_f32(p);
    t.s = ld_cluster_f32(p + 4);
    if (ENT) t.u = ld_cluster_f32(p + 8);
  }
  return stat_warp<ENT>(t, k2);
}

// ---- log probabilities, entropy, top alternatives -----------------------------------
//
// Bound by reading the logits once. Without alternatives a thread streams
// vectors straight into its running statistics. With them, a CTA also keeps the
// elements that may still be among its n best in a shared-memory list: an element
// enters when it is not below the CTA's threshold, and when the list has grown
// past its limit it is sorted, cut to n, and the threshold moves to the n-th.
// The first threshold is the n-th largest of the threads' maxima over the
// first tiles (n elements at least are not below it), so on ordinary rows about
// n (1 + ln(V / tile)) elements ever enter. Cutting at 2 n entries and not at 512
// took 4096 x 128256 fp32 with n = 64 from 790 to 467 us together with the
// cheaper ordering (443 and 470 us on two cards since); without alternatives the
// same logits take 303 us, 6.9 TB/s: reads alone run above the rate of a copy,
// 6.55. 8192 x 50257 bf16: 157 and 167 us on two cards, 5.2 and 4.9 TB/s; with n =
// 20, 360 us. 4 x 128256 fp32 with n = 20, eight CTAs a row: 13 us, 7 of them for
// the statistics alone. Any row is handled: a tile that enters whole fits the
// list. List order depends on timing, the sorted list does not: keys are (value,
// ~index), all different.
constexpr int kLpThreads = 256;
constexpr int kTopTile = 8;                           // elements per thread and tile
constexpr int kTopTileElems = kLpThreads * kTopTile;  // a tile
constexpr int kTopList = 4096;                        // list entries, a power of two
constexpr int kTopCut = 256;                          // the list is cut at 2 n entries, at most here
static_assert(kTopCut + 16 + kTopTileElems <= kTopList, "a tile must fit the list");
static_assert(2 * kTopLimit <= kTopCut && kTopCut <= kLpThreads, "one entry per thread");
static_assert(kMaxCluster <= kLpThreads / 32 && kMaxCluster * kTopLimit <= kTopList, "the CTAs' lists meet in one");

__device__ __forceinline__ uint32_t order_bits(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);  // -0 counts as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t top_key(float z, uint32_t col) {
  return ((uint64_t)order_bits(z) << 32) | (0xffffffffu - col);
}
// The smallest float above z: z' >= next_up(z) exactly when z' > z.
__device__ __forceinline__ float next_up(float z) {
  return order_value(order_bits(z) + 1u);
}

// Sort list[0, count) descending; entries up to the next power of two are
// cleared to 0 (below every key). All threads of the CTA; ends with a barrier.
__device__ void sort_list(uint64_t* list, int count) {
  int P = 32;
  while (P < count) P <<= 1;
  for (int i = count + threadIdx.x; i < P; i += blockDim.x) list[i] = 0;
  __syncthreads();
  for (int k = 2; k <= P; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < P / 2; i += blockDim.x) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const uint64_t x = list[a], y = list[b];
        if ((x < y) == ((a & k) == 0)) {
          list[a] = y;
          list[b] = x;
        }
      }
      __syncthreads();
    }
  }
}

// The same for a list of at most an entry per thread: every entry counts the
// keys above it (all keys differ) and moves to its rank, in three barriers
// instead of the sort's thirty.
__device__ void rank_list(uint64_t* list, int count) {
  const int tid = threadIdx.x;
  if (tid == 0) list[count] = 0;  // (below every key)
  __syncthreads();
  uint64_t key = 0;
  int rank = 0;
  if (tid < count) {
    key = list[tid];
#pragma unroll 4
    for (int i = 0; i < count; i += 2) {
      const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(list + i);
      rank += (k.x > key) + (k.y > key);
    }
  }
  __syncthreads();
  if (tid < count) list[rank] = key;
  __syncthreads();
}
__device__ __forceinline__ void order_list(uint64_t* list, int count) {
  if (count <= kLpThreads)
    rank_list(list, count);
  else
    sort_list(list, count);
}

struct TopState {
  int count;
  float thr;       // elements >= thr enter
  uint32_t first;  // order_bits of the first threshold
};

struct LogprobArgs {
  int64_t ld, V;
  const int32_t* tokens;  // or null
  int n;                  // alternatives
  float* logp;            // or null
  float* entropy;         // or null
  int32_t* top_ids;
  float* top_logp;
  uint32_t* status;
};

template <typename E, bool TOP>
__global__ __launch_bounds__(kLpThreads, TOP || sizeof(E) == 2 ? 4 : 3) void k_token_logprobs(
    const E* __restrict__ Z, LogprobArgs a, int ranks) {
  constexpr int N = Vec<E>::N;
  // vectors per thread and tile, and tiles whose loads are in flight: 64 to 128
  // bytes per thread, about 100 KB an SM, cover the latency of HBM
  constexpr int W = TOP ? kTopTile : 16;  // elements per thread and tile
  constexpr int U = W / N, TILE = U * kLpThreads;
  constexpr int AHEAD = TOP ? (sizeof(E) == 4 ? 3 : 4) : (sizeof(E) == 4 ? 2 : 3);
  extern __shared__ __align__(16) uint64_t list[];  // TOP
  __shared__ Stat sh_warp[kLpThreads / 32], sh_cta;
  __shared__ TopState top;
  __shared__ __align__(16) float sh_max[TOP ? kLpThreads : 4];
  const int tid = threadIdx.x;
  const int rank = ranks > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int64_t t = blockIdx.x / ranks;
  const E* row = Z + t * a.ld;
  const Slice sl = slice_of(row, a.V, rank, ranks);
  const int nv = sl.v1 - sl.v0;
  const uint4* src = reinterpret_cast<const uint4*>(row + sl.head) + sl.v0 + tid;
  uint4 w[AHEAD][U];
  auto fetch = [&](uint4 (&x)[U], int v) {
    if (v + TILE <= nv) {
#pragma unroll
      for (int i = 0; i < U; ++i) x[i] = __ldcs(src + v + i * kLpThreads);
    } else if (v < nv) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (v + i * kLpThreads + tid < nv) x[i] = __ldcs(src + v + i * kLpThreads);
    }
  };
#pragma unroll
  for (int q = 0; q < AHEAD; ++q) fetch(w[q], q * TILE);
  Stat st = stat_none();
  bool grown = false;
  if (TOP) {
    if (tid == 0) {
      top.count = 0;
      top.thr = -FLT_MAX;
    }
    __syncthreads();
  }
  const int cut_at = min(max(2 * a.n, 96), kTopCut);
  auto enter = [&](float z, uint32_t col) {
    const int slot = atomicAdd(&top.count, 1);
    list[slot] = top_key(z, col);
    grown |= slot >= cut_at;
  };
  auto edge = [&](int64_t col) {
    const float z = load_f(row + col);
    stat_add1<true>(st, z, kLog2e);
    if (TOP && z >= top.thr) enter(z, (uint32_t)col);
  };
  if (rank == 0 && tid < sl.head) edge(tid);
  // order, cut to the n best and move the threshold past the n-th: every later
  // element has a higher index, so among equal values it loses
  auto cut = [&]() {
    const int count = top.count;
    order_list(list, count);
    if (tid == 0) {  // (cut_at < count, n <= cut_at / 2 or n = 128)
      top.count = min(count, a.n);
      if (count >= a.n) top.thr = next_up(order_value((uint32_t)(list[a.n - 1] >> 32)));
    }
    grown = false;
    __syncthreads();
  };
  // the first threshold, the n-th largest of the threads' maxima over the tiles
  // in flight: the largest maximum that n maxima are not below
  auto first_threshold = [&](float mx) {
    sh_max[tid] = mx;
    if (tid == 0) top.first = 0;
    __syncthreads();
    int ge = 0;
#pragma unroll 4
    for (int i = 0; i < kLpThreads; i += 4) {
      const float4 o = *reinterpret_cast<const float4*>(sh_max + i);
      ge += (o.x >= mx) + (o.y >= mx) + (o.z >= mx) + (o.w >= mx);
    }
    const uint32_t best = __reduce_max_sync(0xffffffffu, ge >= a.n ? order_bits(mx) : 0u);
    if ((tid & 31) == 0) atomicMax(&top.first, best);
    __syncthreads();
    if (tid == 0) top.thr = fmaxf(order_value(top.first), -FLT_MAX);
    __syncthreads();
  };

  const uint32_t col0 = (uint32_t)(sl.head + (sl.v0 + tid) * N);
  if (TOP) {
    float mx = -inf_f();
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (q * TILE + i * kLpThreads + tid < nv) {
          float x[N];
          unpack(w[q][i], x);
#pragma unroll
          for (int e = 0; e < N; ++e) mx = fmaxf(mx, x[e]);  // (NaN is passed over)
        }
    first_threshold(mx);
  }
  for (int v0 = 0; v0 < nv; v0 += AHEAD * TILE) {
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) {
      const int v = v0 + q * TILE;
      if (v >= nv) break;
      float z[W];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float x[N];
        unpack(w[q][i], x);
#pragma unroll
        for (int e = 0; e < N; ++e) z[i * N + e] = x[e];
      }
      if (v + TILE > nv) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (v + i * kLpThreads + tid >= nv) {
#pragma unroll
            for (int e = 0; e < N; ++e) z[i * N + e] = -inf_f();
          }
      }
      fetch(w[q], v + AHEAD * TILE);
      const float mx = stat_add<true, W>(st, z, kLog2e);
      if (TOP) {
        const float thr = top.thr;
        if (mx >= thr) {
          uint32_t in = 0;
#pragma unroll
          for (int e = 0; e < W; ++e) in |= z[e] >= thr ? 1u << e : 0u;
          do {
            const int e = __ffs((int)in) - 1;
            in &= in - 1;
            float x = z[0];
#pragma unroll
            for (int k = 1; k < W; ++k) x = e == k ? z[k] : x;
            enter(x, col0 + (uint32_t)((v + e / N * kLpThreads) * N + e % N));
          } while (in);
        }
        if (__syncthreads_or(grown)) cut();
      }
    }
  }
  if (sl.tail0 + tid < sl.tail1) edge(sl.tail0 + tid);

  st = stat_block<true>(st, kLog2e, sh_warp, kLpThreads);
  if (TOP) {  // (the barrier inside stat_block ordered the last entries)
    const int count = top.count;
    if (ranks == 1 || count > a.n) order_list(list, count);
    if (tid == 0) top.count = min(count, a.n);
    __syncthreads();
  }
  const Stat all = stat_cluster<true>(st, kLog2e, &sh_cta, ranks);
  if (TOP && ranks > 1 && rank == 0) {
    // the CTAs' best behind one another, a warp for each, then in order
    const int r = tid >> 5, lane = tid & 31;
    int cnt = 0, at = 0, total = 0;
    if (lane < ranks)
      cnt = __float_as_int(
          ld_cluster_f32(ptx::mapa_shared(ptx::smem_u32(&top.count), (uint32_t)lane)));
    for (int q = 0; q < ranks; ++q) {
      const int c = __shfl_sync(0xffffffffu, cnt, q);
      at += q < r ? c : 0;
      total += c;
    }
    const int mine = __shfl_sync(0xffffffffu, cnt, r);
    __syncthreads();
    if (r > 0 && r < ranks) {
      const uint32_t src = ptx::mapa_shared(ptx::smem_u32(list), (uint32_t)r);
      for (int i = lane; i < mine; i += 32) list[at + i] = ld_cluster_u64(src + 8u * i);
    }
    __syncthreads();
    order_list(list, total);
    if (tid == 0) top.count = min(total, a.n);
    __syncthreads();
  }
  if (rank == 0) {
    const float logs = logf(all.s);
    const bool bad = isnan(all.s), empty = all.s == 0.0f;
    if (tid == 0) {
      if (a.logp) {
        const int32_t y = a.tokens[t];
        float lp;
        if (y == -1) {
          lp = 0.0f;
        } else if (y < 0 || (int64_t)y >= a.V) {
          atomicOr(a.status, kStatusBadTarget);
          lp = nan_f();
        } else {
          lp = bad ? nan_f() : (empty ? -inf_f() : (load_f(row + y) - all.m) - logs);
        }
        a.logp[t] = lp;
      }
      if (a.entropy) a.entropy[t] = bad ? nan_f() : (empty ? 0.0f : fmaxf(logs - all.u / all.s, 0.0f));
    }
    if (TOP && tid < a.n) {
      const bool there = tid < top.count && !bad;
      const uint64_t key = there ? list[tid] : 0;
      a.top_ids[t * a.n + tid] = there ? (int32_t)(0xffffffffu - (uint32_t)key) : -1;
      a.top_logp[t * a.n + tid] =
          bad ? nan_f() : (there ? (order_value((uint32_t)(key >> 32)) - all.m) - logs : -inf_f());
    }
  }
  if (ranks > 1) ptx::cluster_sync();  // the others' shared memory is no longer read
}

// ---- distillation from a teacher's top logits ---------------------------------------
//
// The gradient reads and writes every logit once, which is its bound: 2 V
// elements a row. A CTA (or a cluster, for rows longer than a CTA's buffer) works
// through rows of its own: it copies its part of a row into shared memory by
// bulk copies, takes the statistics from the chunks as they land, and forms the
// gradient from shared memory, so HBM is read once whatever L2 holds. As soon as
// a chunk's gradient is written the same chunk of the next row is copied in, so
// reads and writes overlap within the CTA; two CTAs share an SM. Rows past 8
// buffers (kReread) are read from global memory twice. The loss alone is a
// streaming pass.
//
// Measured: 8192 x 50304 bf16 (a tenth of the rows left out) 351 us, 4.5 TB/s;
// 2048 x 128256 fp32 415 us, 4.8 TB/s; the loss of 1000 x 50304 fp32 39 us, 5.1
// TB/s (bf16 27 us, 3.7). The gradient takes two exponentials per logit, and
// without them the same copies and stores take 266 and 375 us: what is left is the
// exponentials' issue slots, not the memory. The copies are a warp's own: refilled
// by one of the computing threads, which then waits for the others chunk by chunk,
// the first case took 583 us. A row per CTA or cluster and nothing kept for the
// next, the form this one replaced, took 357 us there and 517 in the second case.
// The loss costs the gradient time, too: a division by tau less at each kept entry
// (log p is not formed, only its difference times tau) took 366 us to 351.
enum DistillMode { kLossOnly = 0, kResident = 1, kReread = 2 };
constexpr int kDsThreads = 480;             // (loss alone: kLpThreads, for more rows at a time)
constexpr int kMaxTeacher = kTopLimit;
constexpr int kChunk = kDsThreads * 32;     // bytes of one bulk copy: two vectors per thread
constexpr int kBufBytes = 7 * kChunk;       // 105 KB: two CTAs fit an SM's shared memory
constexpr int kMaxChunks = kBufBytes / kChunk;

struct DistillArgs {
  int64_t T, ld, ldg, V;
  const int32_t* ids;    // T x k
  const float* vals;     // T x k
  int k;
  float tau, k2;         // temperature, log2(e) / tau
  const float* weights;  // T or null
  float* loss;           // T or null
  uint32_t* status;
};

struct DistillShared {
  Stat warp[kDsThreads / 32], cta[2];
  int4 id[kMaxTeacher / 4];    // the row's entries, -1: none
  float4 q[kMaxTeacher / 4];   // their weights, up to the sum
  float red[2][4], loss[4], scale;
  uint64_t full[kMaxChunks], empty[kMaxChunks];
};

constexpr uint64_t kCopyWaitNs = 2000000000ull;  // 2 s
__device__ const float kOne = 1.0f;                // the weight where none are given

// Wait for a phase of a barrier, for at most kCopyWaitNs: past that the call
// reports a timeout and its outputs are unspecified. Every copy is waited for,
// so none is in flight when the CTA leaves.
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, uint32_t* status) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer_ns() - t0 > kCopyWaitNs) {
      atomicOr(status, kStatusTimeout);
      return;
    }
  }
}
__device__ __forceinline__ void wait_phase(uint64_t& bar, uint32_t parity, uint32_t* status) {
  const uint32_t b = ptx::smem_u32(&bar);
  if (!ptx::mbar_try_wait(b, parity)) wait_slow(b, parity, status);
}

template <typename E, int MODE>
__global__ __launch_bounds__(MODE == kLossOnly ? kLpThreads
                                               : kDsThreads + (MODE == kResident ? 32 : 0),
                             MODE == kResident ? 2 : (MODE == kLossOnly ? 4 : 1))
    void k_distill(const E* Z, E* dZ, DistillArgs a, int ranks) {
  constexpr int N = Vec<E>::N;
  constexpr int THREADS = MODE == kLossOnly ? kLpThreads : kDsThreads;
  extern __shared__ __align__(128) uint8_t buf[];  // kResident: the slice's vectors
  __shared__ DistillShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = ranks > 1 ? (int)ptx::cluster_ctarank() : 0;
  // the k-th row of this cluster: one of every `step` rows, moved on by 7 from one
  // to the next, so that a periodic mask does not leave some clusters all its rows
  // (T <= 2^27: 32 bits do)
  const int T = (int)a.T, step = (int)gridDim.x / ranks, first = (int)blockIdx.x / ranks;
  auto row_of = [&](int k) { return k * step + (first + 7 * k) % step; };
  // this thread's teacher entry of a row: absent (-1) where its id is -1 or its
  // value -inf
  int32_t id = -1;
  float v = -inf_f(), weight = 1.0f;
  // (loaded without a condition, so that nothing waits for the values here)
  auto entry = [&](int t) {
    if (t >= T) t = T - 1;
    const int64_t e = (int64_t)t * a.k + min(tid, a.k - 1);
    id = a.ids[e];
    v = a.vals[e];
    weight = *(a.weights ? a.weights + t : &kOne);
  };
  // From the k-th row on, whose entry is loaded, the first that is not left out
  // (its row T or past it: none). A row without a teacher entry, or of weight 0,
  // gets zeros and its logits are not read. All CTAs of a cluster see the same rows.
  auto next_live = [&](int& k) {
    for (; k * step < T; entry(row_of(++k))) {
      const int t = row_of(k);
      if (t >= T) continue;  // (in the last, incomplete round)
      if (tid >= a.k) id = -1;
      if (id != -1 && (id < 0 || (int64_t)id >= a.V)) {
        atomicOr(a.status, kStatusBadTarget);
        id = -1;
      }
      if (id == -1 || v == -inf_f()) {
        id = -1;
        v = -inf_f();
      }
      if (sync_threads_or(id >= 0, THREADS) && weight != 0.0f) return t;
      if (MODE != kLossOnly) {
        const Slice sl = slice_of(Z + (int64_t)t * a.ld, a.V, rank, ranks);
        E* out = dZ + (int64_t)t * a.ldg;
        const int c0 = rank == 0 ? 0 : sl.head + sl.v0 * N;
        const int c1 = rank == ranks - 1 ? (int)a.V : sl.head + sl.v1 * N;
        const int lead = (int)((16 - ((uintptr_t)(out + c0) & 15)) & 15) / (int)sizeof(E);
        const int c = min(c0 + lead, c1), n = (c1 - c) / N;
        if (c0 + tid < c) store_e(out + c0 + tid, 0.0f);
        for (int i = tid; i < n; i += THREADS)
          __stcs(reinterpret_cast<uint4*>(out + c) + i, make_uint4(0, 0, 0, 0));
        if (c + n * N + tid < c1) store_e(out + c + n * N + tid, 0.0f);
      }
      if (rank == 0 && tid == 0 && a.loss) a.loss[t] = 0.0f;
    }
    return T;
  };
  // chunks of the longest slice of any row
  const int chunks = MODE == kResident
                         ? (((int)a.V / N + ranks) / ranks * 16 + kChunk - 1) / kChunk
                         : 0;
  if (MODE == kResident) {
    if (tid == 0) {
      for (int c = 0; c < chunks; ++c) {
        ptx::mbar_init(ptx::smem_u32(&sh.full[c]), 1);
        ptx::mbar_init(ptx::smem_u32(&sh.empty[c]), THREADS / 32);
      }
      ptx::fence_barrier_init();
      ptx::fence_proxy_async();
    }
    __syncthreads();
    if (tid >= THREADS) {
      // ---------------- the copies ----------------
      int rows = 0;
      for (int k = 0; k * step < T; ++k) {
        const int t = row_of(k);
        if (t >= T) continue;
        bool any = false;
        for (int j = lane; j < a.k; j += 32) {
          const int32_t e = a.ids[(int64_t)t * a.k + j];
          any |= e >= 0 && (int64_t)e < a.V && a.vals[(int64_t)t * a.k + j] != -inf_f();
        }
        if (!__any_sync(0xffffffffu, any) || (a.weights && a.weights[t] == 0.0f)) continue;
        const E* row = Z + (int64_t)t * a.ld;
        const Slice sl = slice_of(row, a.V, rank, ranks);
        const int bytes = (sl.v1 - sl.v0) * 16;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(row + sl.head) + (int64_t)sl.v0 * 16;
        if (lane == 0) {
          for (int c = 0; c < chunks; ++c) {
            if (rows > 0) wait_phase(sh.empty[c], (uint32_t)(rows - 1) & 1u, a.status);
            const int n = min(kChunk, bytes - c * kChunk);
            const uint32_t bar = ptx::smem_u32(&sh.full[c]);
            if (n <= 0) {  // (the slices of a call's rows differ by a vector)
              ptx::mbar_arrive(bar);
            } else {
              ptx::mbar_expect_tx(bar, (uint32_t)n);
              ptx::bulk_load(ptx::smem_u32(buf) + c * kChunk, src + c * kChunk, (uint32_t)n, bar);
            }
          }
        }
        __syncwarp();
        ++rows;
        if (ranks > 1) ptx::cluster_sync();  // the row's exchange of statistics, below
      }
      if (ranks > 1) ptx::cluster_sync();
      return;
    }
  }
  // the student's logit at the entry: gathered a row ahead, and before any of
  // the row is overwritten (dZ may be Z)
  float z_next = 0.0f;
  auto gather = [&](const E* row) { z_next = load_rw(row + max(id, 0)); };
  int k = 0;
  entry(row_of(k));
  int t = next_live(k);
  if (t < T) gather(Z + (int64_t)t * a.ld);
  for (uint32_t par = 0; t < T; par ^= 1u) {
    const E* row = Z + (int64_t)t * a.ld;
    E* out = MODE == kLossOnly ? nullptr : dZ + (int64_t)t * a.ldg;
    const Slice sl = slice_of(row, a.V, rank, ranks);
    const uint4* body = reinterpret_cast<const uint4*>(row + sl.head);
    const int nv = sl.v1 - sl.v0;
    const int32_t my_id = id;
    const float my_v = v, zj = z_next;
    if (tid == 0) sh.scale = weight * a.tau;
    entry(row_of(k + 1));  // on its way while this row is read

    // q over the kept set, up to its sum, by the first warps
    if (warp < kMaxTeacher / 32) {
      float mx = my_v;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (lane == 0) sh.red[0][warp] = mx;
    }
    sync_threads(THREADS);
    const float vm = fmaxf(fmaxf(sh.red[0][0], sh.red[0][1]), fmaxf(sh.red[0][2], sh.red[0][3]));
    const float dv = (my_v - vm) / a.tau;
    const float eq = my_id >= 0 ? expf(dv) : 0.0f;
    if (warp < kMaxTeacher / 32) {
      float sq = eq;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      if (lane == 0) sh.red[1][warp] = sq;
      reinterpret_cast<int32_t*>(sh.id)[tid] = my_id;
      reinterpret_cast<float*>(sh.q)[tid] = eq;
    }

    // statistics of the row
    Stat st = stat_none();
    if (rank == 0 && tid < sl.head) stat_add1<false>(st, load_rw(row + tid), a.k2);
    if (sl.tail0 + tid < sl.tail1) stat_add1<false>(st, load_rw(row + sl.tail0 + tid), a.k2);
    if (MODE == kResident) {
      for (int c = 0; c < chunks; ++c) {
        wait_phase(sh.full[c], par, a.status);
        const int i = 2 * c * THREADS + tid;
        float x[N], y[N], z[2 * N];
        const uint4* src = reinterpret_cast<const uint4*>(buf) + i;
        // (past the slice's end the buffer may hold anything: not read)
        const bool two = i + THREADS < nv;
        if (i < nv) {
          unpack(src[0], x);
          if (two) unpack(src[THREADS], y);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            z[e] = x[e];
            z[N + e] = two ? y[e] : -inf_f();
          }
          stat_add<false, 2 * N>(st, z, a.k2);
        }
      }
    } else {
      constexpr int U = 16 / N, TILE = U * THREADS;
      constexpr int AHEAD = sizeof(E) == 4 ? 1 : 2;
      const uint4* src = body + sl.v0 + tid;
      uint4 w[AHEAD][U];
      auto fetch = [&](uint4 (&x)[U], int p) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (p + i * THREADS + tid < nv)
            x[i] = MODE == kReread ? src[p + i * THREADS] : __ldcs(src + p + i * THREADS);
      };
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) fetch(w[q], q * TILE);
      for (int p0 = 0; p0 < nv; p0 += AHEAD * TILE) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
          const int p = p0 + q * TILE;
          if (p >= nv) break;
          float z[16];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            float x[N];
            unpack(w[q][i], x);
            const bool there = p + i * THREADS + tid < nv;
#pragma unroll
            for (int e = 0; e < N; ++e) z[i * N + e] = there ? x[e] : -inf_f();
          }
          fetch(w[q], p + AHEAD * TILE);
          stat_add<false, 16>(st, z, a.k2);
        }
      }
    }
    st = stat_block<false>(st, a.k2, sh.warp, THREADS);
    const Stat all = stat_cluster<false>(st, a.k2, &sh.cta[par], ranks);
    const float scale = sh.scale;
    const float r = all.s == 0.0f ? 0.0f : scale / all.s;  // NaN rows stay NaN
    auto grad = [&](float z) { return r * ex2((z - all.m) * a.k2); };
    // an entry's part of the loss and, of this CTA's columns, its gradient: p - q
    // in fp32, rounded once; an id that the teacher lists twice has both weights,
    // in list order
    float fix = 0.0f;
    bool mine = false;
    if (warp < kMaxTeacher / 32) {
      const float qsum = (sh.red[1][0] + sh.red[1][1]) + (sh.red[1][2] + sh.red[1][3]);
      const float q = eq / qsum;
      float part = 0.0f;
      if (my_id >= 0 && q != 0.0f) {
        // tau^2 q (log q - log p) with the temperature kept off the differences: the
        // lowest finite logit stays finite (s = 0: a row of -inf, loss +inf)
        const float d = (my_v - vm) - (zj - all.m);
        part = all.s == 0.0f ? inf_f()
                             : a.tau * q * (d + a.tau * (logf(all.s) - logf(qsum)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane == 0) sh.loss[warp] = part;
      const int c0 = rank == 0 ? 0 : sl.head + sl.v0 * N;
      const int c1 = rank == ranks - 1 ? (int)a.V : sl.head + sl.v1 * N;
      mine = MODE != kLossOnly && my_id >= 0 && my_id >= c0 && my_id < c1;
      if (mine) {
        float qs = 0.0f;
        for (int j = 0; j < (a.k + 3) / 4; ++j) {
          const int4 e = sh.id[j];
          const float4 w = sh.q[j];
          qs += e.x == my_id ? w.x : 0.0f;
          qs += e.y == my_id ? w.y : 0.0f;
          qs += e.z == my_id ? w.z : 0.0f;
          qs += e.w == my_id ? w.w : 0.0f;
        }
        fix = grad(zj) - scale * (qs / qsum);
      }
    }
    // the next row's entries, and zeros for the rows left out before it
    const int tn = next_live(++k);
    if (tn < T) gather(Z + (int64_t)tn * a.ld);  // (else the entry is not checked)
    if (MODE != kLossOnly) {
      auto grads = [&](const uint4& w) {
        float z[N];
        unpack(w, z);
        const float2 nm = make_float2(-all.m, -all.m), kk = make_float2(a.k2, a.k2);
        const float2 rr = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float2 x = __fmul2_rn(__fadd2_rn(make_float2(z[i], z[i + 1]), nm), kk);
          const float2 g = __fmul2_rn(make_float2(ex2(x.x), ex2(x.y)), rr);
          z[i] = g.x;
          z[i + 1] = g.y;
        }
        return pack(z);
      };
      const bool aligned = (((uintptr_t)out ^ (uintptr_t)row) & 15) == 0;
      // the edges first: their logits are in global memory
      if (rank == 0 && tid < sl.head) store_e(out + tid, grad(load_rw(row + tid)));
      if (sl.tail0 + tid < sl.tail1)
        store_e(out + sl.tail0 + tid, grad(load_rw(row + sl.tail0 + tid)));
      if (MODE == kResident) {
        uint4* dst = reinterpret_cast<uint4*>(out + sl.head) + sl.v0;
        for (int c = 0; c < chunks; ++c) {
          const int i = 2 * c * THREADS + tid;
          if (aligned) {  // the gradient's rows are aligned as the logits' are
            const uint4* src = reinterpret_cast<const uint4*>(buf);
            if (i < nv) __stcs(dst + i, grads(src[i]));
            if (i + THREADS < nv) __stcs(dst + i + THREADS, grads(src[i + THREADS]));
          } else {
            const int e1 = min(2 * (c + 1) * THREADS, nv) * N;
            for (int e = 2 * c * THREADS * N + tid; e < e1; e += THREADS)
              store_e(out + sl.head + sl.v0 * N + e,
                      grad(load_rw(reinterpret_cast<const E*>(buf) + e)));
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh.empty[c]));
        }
      } else if (aligned) {
        uint4* dst = reinterpret_cast<uint4*>(out + sl.head) + sl.v0;
        for (int i = tid; i < nv; i += THREADS) __stcs(dst + i, grads(body[sl.v0 + i]));
      } else {
        for (int64_t e = tid; e < (int64_t)nv * N; e += THREADS)
          store_e(out + sl.head + sl.v0 * N + e, grad(load_rw(row + sl.head + sl.v0 * N + e)));
      }
    }
    sync_threads(THREADS);  // the row's shared values and dense stores are done
    if (mine) store_e(out + my_id, fix);
    if (rank == 0 && tid == 0 && a.loss)
      a.loss[t] = (sh.loss[0] + sh.loss[1]) + (sh.loss[2] + sh.loss[3]);
    t = tn;
  }
  if (ranks > 1) ptx::cluster_sync();  // the others' shared memory is no longer read
}

// CTAs per row: at least `need`; more while the rows leave SMs without a CTA and
// every CTA keeps a tile of its own to read.
int cluster_for(int64_t T, int64_t V, int need, int64_t tile, int sm_count) {
  int c = need;
  while (2 * c <= kMaxCluster && T * 2 * c <= sm_count && V >= 2 * c * tile) c *= 2;
  return c;
}

template <typename F, typename... Args>
cudaError_t launch_rows(cudaStream_t st, F fn, int64_t clusters, int ranks, int threads,
                        size_t smem, Args... args) {
  cudaError_t err = cudaSuccess;
  if (smem > 48 * 1024)
    err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(clusters * ranks));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, fn, args..., ranks);
  return err != cudaSuccess ? err : cudaGetLastError();
}

template <typename F>
cudaError_t resident_clusters(F fn, int ranks, int threads, size_t smem, int* n) {
  cudaError_t err =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)ranks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaOccupancyMaxActiveClusters(n, fn, &cfg);
  if (err == cudaSuccess && *n < 1) err = cudaErrorInvalidConfiguration;
  return err;
}

template <typename E>
cudaError_t logprobs_as(cudaStream_t st, const void* Z, int64_t T, const LogprobArgs& a,
                        int sm_count) {
  const E* z = (const E*)Z;
  const int c = cluster_for(T, a.V, 1, kTopTileElems, sm_count);
  if (a.n > 0)
    return launch_rows(st, k_token_logprobs<E, true>, T, c, kLpThreads,
                       (size_t)kTopList * sizeof(uint64_t), z, a);
  return launch_rows(st, k_token_logprobs<E, false>, T, c, kLpThreads, 0, z, a);
}

template <typename E>
cudaError_t distill_as(cudaStream_t st, const void* Z, void* dZ, const DistillArgs& a,
                       int sm_count) {
  const E* z = (const E*)Z;
  E* g = (E*)dZ;
  if (!g)  // a row per CTA: the hardware hands out the next
    return launch_rows(st, k_distill<E, kLossOnly>, a.T,
                       cluster_for(a.T, a.V, 1, kLpThreads * 16, sm_count), kLpThreads, 0, z, g, a);
  // a slice has at most V / N / ranks + 1 vectors
  constexpr int64_t kVecs = kBufBytes / 16;
  int64_t need = 1;
  while (need <= kMaxCluster && (a.V / Vec<E>::N + need) / need > kVecs) ++need;
  if (need > kMaxCluster)
    return launch_rows(st, k_distill<E, kReread>, a.T, kMaxCluster, kDsThreads, 0, z, g, a);
  const int c = cluster_for(a.T, a.V, (int)need, kDsThreads * 16, sm_count);
  int64_t clusters = a.T;
  if (a.T * c > sm_count) {
    // the clusters that are resident at once (a grid larger than that would work
    // through the rest of its rows behind them): asked once per size and device
    static std::atomic<int> known[kMaxCluster + 1][64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    int n = dev < 64 ? known[c][dev].load() : 0;
    if (n == 0) {
      err = resident_clusters(k_distill<E, kResident>, c, kDsThreads + 32, kBufBytes, &n);
      if (err != cudaSuccess) return err;
      if (dev < 64) known[c][dev].store(n);
    }
    if (n < clusters) clusters = n;
  }
  return launch_rows(st, k_distill<E, kResident>, clusters, c, kDsThreads + 32,
                     (size_t)kBufBytes, z, g, a);
}

}  // namespace

cudaError_t launch_token_logprobs(cudaStream_t st, const void* Z, int dtype, int64_t T, int64_t V,
                                  int64_t ld, const int32_t* tokens, int top, float* logp,
                                  float* entropy, int32_t* top_ids, float* top_logp, int sm_count,
                                  uint32_t* status) {
  if (T <= 0) return cudaSuccess;
  const LogprobArgs a{ld, V, tokens, top, logp, entropy, top_ids, top_logp, status};
  return dtype == DUST_BF16 ? logprobs_as<__nv_bfloat16>(st, Z, T, a, sm_count)
                            : logprobs_as<float>(st, Z, T, a, sm_count);
}

cudaError_t launch_distill(cudaStream_t st, const void* Z, int dtype, int64_t T, int64_t V,
                           int64_t ld, const int32_t* ids, const float* vals, int k, float tau,
                           const float* weights, float* loss, void* dZ, int64_t ldg, int sm_count,
                           uint32_t* status) {
  if (T <= 0) return cudaSuccess;
  const DistillArgs a{T, ld, ldg, V, ids, vals, k, tau, kLog2e / tau, weights, loss, status};
  return dtype == DUST_BF16 ? distill_as<__nv_bfloat16>(st, Z, dZ, a, sm_count)
                            : distill_as<float>(st, Z, dZ, a, sm_count);
}

}  // namespace dust
