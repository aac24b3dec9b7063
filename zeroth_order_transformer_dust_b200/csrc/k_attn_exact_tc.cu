// Causal attention and its exact gradient on tensor cores (bf16 tensors, 64- or
// 128-wide heads); formulas as in k_attn_exact.cu.
//
// Backward. One kernel body serves both sides. A CTA keeps 128 rows of its side
// resident (queries with their error signal, or keys with their values) and
// streams tiles of 64 rows of the other side. Per tile, with the resident rows
// as TMEM lanes:
//   query side   S = Q K^T, dP = E V^T (64 columns: keys),
//                dS = P (dP - delta) -> bf16 in TMEM, dQ += dS K;
//   key side     S^T = K Q^T, dP^T = V E^T (64 columns: queries),
//                P^T, dS^T -> bf16 in TMEM, dV += P^T E, dK += dS^T Q.
// The streamed tile is staged once by TMA and read twice: K-major by the score
// products and MN-major by the gradient products. P and dS never leave the SM:
// softmax threads write them over the scores' TMEM columns, from where the
// gradient MMAs take them as their A operand. The sums live in TMEM in fp32 for
// the CTA's whole life. Rounding P and dS to bf16 (half a step, 2^-8 relative,
// per term, against fp32 sums) is what puts their products on the tensor cores.
//
// Warp roles: warp 0 TMA producer, warp 1 MMA issuer, warps 2..9 softmax (two
// warps per TMEM lane quarter, 32 of the tile's 64 columns each). With 64-wide
// heads a CTA needs 256 TMEM columns and two CTAs share an SM: one's softmax
// runs under the other's MMAs. With 128-wide heads the accumulators take half of
// TMEM, so one CTA has the SM and keeps two score buffers: the next tile's
// scores are computed while this tile's softmax runs.
//
// Rows at or past the end of a sequence belong to nobody or to another
// sequence, so their content must not enter a sum, not even times 0: in the
// one streamed tile that can hold such rows the producer overwrites them with
// zeros before the MMAs see the tile.
//
// Every wait is bounded: on expiry the CTA raises the timeout bit, drains its own
// copies and MMAs (bounded again), frees its TMEM and returns.
#include <cudaTypedefs.h>

#include "internal.cuh"
#include "tc_ptx.cuh"

namespace dust {
namespace {

constexpr int BM = 128;  // resident rows: TMEM lanes
constexpr int BN = 64;   // rows of a streamed tile
constexpr int BOX_BYTES = 64 * 64 * 2;  // a TMA box: 64 rows x 64 columns
constexpr int SOFT_WARPS = 8;
constexpr int THREADS = 64 + 32 * SOFT_WARPS;
constexpr int STAGES = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

template <int D>
struct Cfg {
  static constexpr int NBUF = D == 128 ? 2 : 1;       // score buffers
  static constexpr int BOXES = D / 64;                // boxes per 64 rows of a tensor
  static constexpr int RES_BYTES = 2 * BM * D * 2;    // both resident tensors
  static constexpr int HALF_STAGE = BN * D * 2;       // one tensor's streamed tile
  static constexpr int STAGE_BYTES = 2 * HALF_STAGE;
  static constexpr int ACC_COL = NBUF * 2 * BN;       // TMEM: score buffers, then the sums
  static constexpr int TMEM_COLS = D == 128 ? 512 : 256;
  static constexpr size_t SMEM = 1024 + (size_t)RES_BYTES + (size_t)STAGES * STAGE_BYTES + 2048 + 256;
  static_assert(ACC_COL + 2 * D <= TMEM_COLS, "TMEM columns");
  static_assert(SMEM * (D == 64 ? 2 : 1) <= 226 * 1024, "shared memory per SM");
};

struct Bars {
  uint64_t res, land, full[STAGES], empty[STAGES], sfull[2], pfull[2], vdone[2], afull;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// As the GEMM's bounded wait: false (and the abort flag and timeout bit) on expiry.
__device__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort,
                             uint32_t* status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
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

// Resident tensors r0, r1 and streamed tensors s0, s1 of the score products
// S = r0 s0^T and dP = r1 s1^T: (Q, E; K, V) on the query side, (K, V; Q, E) on
// the key side.
template <int D, bool KEY>
__global__ __launch_bounds__(THREADS, D == 64 ? 2 : 1) void k_attn_exact_bwd_tc(
    const __grid_constant__ CUtensorMap tmR0, const __grid_constant__ CUtensorMap tmR1,
    const __grid_constant__ CUtensorMap tmS0, const __grid_constant__ CUtensorMap tmS1,
    AttnArgs a) {
  using C = Cfg<D>;
  constexpr int NBUF = C::NBUF;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  const uint32_t sRes = base, sStage = base + C::RES_BYTES;
  // query side: partial deltas (2 x 128); key side: per stage lse and delta (2 x 64)
  float* s_col = reinterpret_cast<float*>(basep + C::RES_BYTES + STAGES * C::STAGE_BYTES);
  Bars* sh = reinterpret_cast<Bars*>(reinterpret_cast<uint8_t*>(s_col) + 2048);
  volatile int* abort = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // longest work first: query tiles from the end, key tiles from the start
  const int heads = KEY ? a.Hkv : a.H;
  const int head = (int)(blockIdx.x % heads), seq = (int)(blockIdx.x / heads);
  const int tile = KEY ? (int)blockIdx.y : (int)(gridDim.y - 1 - blockIdx.y);
  const int group = a.H / a.Hkv;
  int64_t beg, end;
  if (!attn_sequence(a, seq, &beg, &end)) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadSeq);
    return;
  }
  const int len = (int)(end - beg);
  const int r_first = tile * BM;  // first resident row of the sequence
  if (r_first >= len) return;
  const int tiles64 = (len + BN - 1) / BN;
  // streamed tiles: keys [0, diagonal] of one head, or for every head of the
  // group the queries from the diagonal on
  const int per_head = KEY ? tiles64 - 2 * tile : min(tiles64, 2 * tile + 2);
  const int n = KEY ? group * per_head : per_head;
  const int s_off = KEY ? 2 * tile : 0;

  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&sh->res), 1);
    ptx::mbar_init(ptx::smem_u32(&sh->land), 1);
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(ptx::smem_u32(&sh->full[s]), 2);  // the bytes, and the producer's word
      ptx::mbar_init(ptx::smem_u32(&sh->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&sh->sfull[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&sh->pfull[b]), SOFT_WARPS);
      ptx::mbar_init(ptx::smem_u32(&sh->vdone[b]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&sh->afull), 1);
    sh->abort = 0;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async();
    ptx::prefetch_map(&tmR0);
    ptx::prefetch_map(&tmR1);
    ptx::prefetch_map(&tmS0);
    ptx::prefetch_map(&tmS1);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&sh->tmem_base), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    const int res_col = head * D;
    if (lane == 0) {
      const uint32_t bar = ptx::smem_u32(&sh->res);
      ptx::mbar_expect_tx(bar, C::RES_BYTES);
      for (int t = 0; t < 2; ++t)
        for (int c = 0; c < C::BOXES; ++c)
          for (int h = 0; h < 2; ++h)
            ptx::tma_load_2d(sRes + t * (BM * D * 2) + (2 * c + h) * BOX_BYTES, t ? &tmR1 : &tmR0,
                             res_col + 64 * c, (int)(beg + r_first + 64 * h), bar);
    }
    // key side: lse (log2) and delta of a tile's queries, two rows per lane;
    // +inf past the sequence's end, which makes p = 0 there
    float nl[2], nd[2];
    auto fetch_cols = [&](int j) {
      const int h = head * group + j / per_head;
      const int r = (s_off + j % per_head) * BN;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int q = r + lane + 32 * i;
        const bool in = j < n && q < len;
        nl[i] = in ? a.lse[(beg + q) * a.H + h] * kLog2e : inf_f();
        nd[i] = in ? a.delta[(beg + q) * a.H + h] : 0.0f;
      }
    };
    if (KEY) fetch_cols(0);
    uint32_t land_phase = 0;
    int armed = 0;  // tiles whose copies were issued
    for (int j = 0; j < n; ++j) {
      const int st = j % STAGES;
      const uint32_t ph = (uint32_t)(j / STAGES) & 1u;
      if (!wait_warp(ptx::smem_u32(&sh->empty[st]), ph ^ 1u, abort, a.status)) break;
      const int h = KEY ? head * group + j / per_head : head / group;
      const int r = (s_off + j % per_head) * BN;
      const uint32_t dst = sStage + (uint32_t)(st * C::STAGE_BYTES);
      const uint32_t full = ptx::smem_u32(&sh->full[st]), land = ptx::smem_u32(&sh->land);
      const bool partial = r + BN > len;
      if (lane == 0) {
        const uint32_t bar = partial ? land : full;
        ptx::mbar_expect_tx(bar, C::STAGE_BYTES);
        for (int t = 0; t < 2; ++t)
          for (int c = 0; c < C::BOXES; ++c)
            ptx::tma_load_2d(dst + t * C::HALF_STAGE + c * BOX_BYTES, t ? &tmS1 : &tmS0,
                             h * D + 64 * c, (int)(beg + r), bar);
      }
      armed = j + 1;
      if (KEY) {
        float* col = s_col + st * 2 * BN;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          col[lane + 32 * i] = nl[i];
          col[BN + lane + 32 * i] = nd[i];
        }
        fetch_cols(j + 1);
      }
      if (partial) {
        if (!wait_warp(land, land_phase, abort, a.status)) break;
        land_phase ^= 1u;
        // zero the 128-byte lines of the rows past the end (a swizzled row stays
        // inside its line)
        const int rows = r + BN - len;
        uint4* st0 = reinterpret_cast<uint4*>(basep + C::RES_BYTES + st * C::STAGE_BYTES);
        for (int i = lane; i < 2 * C::BOXES * rows * 8; i += 32) {
          const int box = i / (rows * 8), w = i % (rows * 8);
          st0[box * (BOX_BYTES / 16) + (BN - rows) * 8 + w] = make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) {
        if (partial) ptx::mbar_arrive(full);
        ptx::mbar_arrive(full);
      }
    }
    // every copy has landed before the CTA can exit (after an abort the last
    // stages may not have been waited for by the MMAs)
    if (*abort) {
      int dummy = 0;
      wait_warp(ptx::smem_u32(&sh->res), 0, &dummy, a.status);
      for (int j = max(0, armed - STAGES); j < armed; ++j) {
        const int r = (s_off + j % per_head) * BN;
        const bool partial = r + BN > len;
        if (partial)
          wait_warp(ptx::smem_u32(&sh->land), land_phase, &dummy, a.status);
        else
          wait_warp(ptx::smem_u32(&sh->full[j % STAGES]), (uint32_t)(j / STAGES) & 1u, &dummy,
                    a.status);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0) {
      constexpr uint32_t id_s = ptx::idesc_bf16_f32(BM, BN);
      constexpr uint32_t id_g = ptx::idesc_bf16_f32(BM, D) | ptx::kIdescBMn;
      // S or dP: K-major operands, 64-column boxes, 32 bytes per 16-deep step
      auto product = [&](uint32_t d, uint32_t r, uint32_t s) {
#pragma unroll
        for (int c = 0; c < C::BOXES; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::mma_f16(d, ptx::sdesc_kmajor_sw128(r + c * 2 * BOX_BYTES + 32 * k),
                         ptx::sdesc_kmajor_sw128(s + c * BOX_BYTES + 32 * k), id_s, (c | k) != 0);
      };
      // sum += (bf16 tile in TMEM) x (streamed tile read MN-major: 16 rows, 2048
      // bytes, per step). The softmax warps of column half h left their 32
      // columns at 32 h: two steps each.
      auto gradient = [&](uint32_t acc, uint32_t p, uint32_t s, bool first) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::mma_f16_ts(acc, p + 32 * (k >> 1) + 8 * (k & 1),
                          ptx::sdesc_mnmajor_sw128(s + 2048 * k, BOX_BYTES), id_g,
                          !first || k != 0);
      };
      auto wait = [&](uint64_t& bar, int use) {
        return wait_bounded(ptx::smem_u32(&bar), (uint32_t)use & 1u, abort, a.status);
      };
      const uint32_t acc0 = tmem + C::ACC_COL, acc1 = acc0 + D;
      bool issued = false;
      // The score buffer's columns are free once the gradient MMAs that read
      // them are complete; the second product waits while the first runs.
      auto scores = [&](int j) {
        const int st = j % STAGES, b = j % NBUF, o = j - NBUF;
        const uint32_t s = sStage + (uint32_t)(st * C::STAGE_BYTES);
        if (!wait(sh->full[st], j / STAGES)) return false;
        if (KEY && o >= 0 && !wait(sh->vdone[b], o / NBUF)) return false;
        ptx::tc_fence_after();
        product(tmem + b * 2 * BN, sRes, s);
        issued = true;
        if (o >= 0 && !wait(sh->empty[o % STAGES], o / STAGES)) return false;
        ptx::tc_fence_after();
        product(tmem + b * 2 * BN + BN, sRes + BM * D * 2, s + C::HALF_STAGE);
        ptx::mma_commit(ptx::smem_u32(&sh->sfull[b]));
        return true;
      };
      auto grads = [&](int j) {
        const int st = j % STAGES, b = j % NBUF;
        const uint32_t s = sStage + (uint32_t)(st * C::STAGE_BYTES);
        if (!wait(sh->pfull[b], j / NBUF)) return false;
        ptx::tc_fence_after();
        const uint32_t p = tmem + b * 2 * BN, ds = p + BN;
        if (KEY) {
          gradient(acc0, p, s + C::HALF_STAGE, j == 0);  // dV += P^T E
          ptx::mma_commit(ptx::smem_u32(&sh->vdone[b]));
          gradient(acc1, ds, s, j == 0);                 // dK += dS^T Q
        } else {
          gradient(acc0, ds, s, j == 0);                 // dQ += dS K
        }
        ptx::mma_commit(ptx::smem_u32(&sh->empty[st]));
        return true;
      };
      bool ok = wait(sh->res, 0);
      if (NBUF == 2 && ok) ok = scores(0);
      for (int j = 0; j < n && ok; ++j) {
        if (NBUF == 2) {
          if (j + 1 < n) ok = scores(j + 1);
        } else {
          ok = scores(j);
        }
        ok = ok && grads(j);
      }
      if (issued) {
        // all MMAs complete before the sums are read, or TMEM is released
        ptx::mma_commit(ptx::smem_u32(&sh->afull));
        int dummy = 0;
        wait_bounded(ptx::smem_u32(&sh->afull), 0, &dummy, a.status);
      }
    }
  } else {
    // ---------------- softmax warps 2..9 ----------------
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int row = quad * 32 + lane;       // TMEM lane: resident row
    const int rr = r_first + row;           // its place in the sequence
    const bool in = rr < len;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const float c2 = a.scale * kLog2e;
    float lse2 = inf_f(), delta = 0.0f;
    if (!KEY) {
      // delta = <o, e>: this thread's half of the row's columns
      float d = 0.0f;
      if (in) {
        const int64_t r = beg + rr;
        const uint4* o = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.O_in + r * a.ldo +
                                                        head * D + half * (D / 2));
        const uint4* e = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.E + r * a.lde +
                                                        head * D + half * (D / 2));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 x = __ldg(o + i), y = __ldg(e + i);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            d = fmaf(__uint_as_float(xs[w] << 16), __uint_as_float(ys[w] << 16), d);
            d = fmaf(__uint_as_float(xs[w] & 0xffff0000u), __uint_as_float(ys[w] & 0xffff0000u), d);
          }
        }
        lse2 = a.lse[r * a.H + head] * kLog2e;
      }
      s_col[half * BM + row] = d;
      asm volatile("bar.sync 1, %0;" ::"n"(32 * SOFT_WARPS) : "memory");
      delta = s_col[row] + s_col[BM + row];
      if (in && half == 0) a.delta[(beg + rr) * a.H + head] = delta;
    }
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int b = j % NBUF, st = j % STAGES;
      const int c0 = (s_off + j % per_head) * BN + 32 * half;  // first column's place
      ok = wait_warp(ptx::smem_u32(&sh->sfull[b]), (uint32_t)(j / NBUF) & 1u, abort, a.status);
      // (the producer's lse and delta are ordered by its own barrier)
      if (KEY && ok)
        ok = wait_warp(ptx::smem_u32(&sh->full[st]), (uint32_t)(j / STAGES) & 1u, abort, a.status);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t ts = lane_base + b * 2 * BN + 32 * half, td = ts + BN;
      uint32_t s[32], d[32];
      ptx::tmem_ld32x2(ts, s, td, d);
      // the tiles that cross the diagonal
      const bool diag = KEY ? j % per_head < 2 : j >= 2 * tile;
      uint32_t p16[16], d16[16];
      const float* cl = s_col + st * 2 * BN + 32 * half;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float4 l4 = make_float4(lse2, lse2, lse2, lse2), d4 = make_float4(delta, delta, delta, delta);
        if (KEY) {
          l4 = *reinterpret_cast<const float4*>(cl + i);
          d4 = *reinterpret_cast<const float4*>(cl + BN + i);
        }
        const float ls[4] = {l4.x, l4.y, l4.z, l4.w}, dl[4] = {d4.x, d4.y, d4.z, d4.w};
        float p[4], ds[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x = fmaf(__uint_as_float(s[i + k]), c2, -ls[k]);
          if (diag && (KEY ? c0 + i + k < rr : c0 + i + k > rr)) x = -inf_f();
          p[k] = ex2(x);
          ds[k] = p[k] * (__uint_as_float(d[i + k]) - dl[k]);
        }
        p16[i / 2] = pack_bf16(p[0], p[1]);
        p16[i / 2 + 1] = pack_bf16(p[2], p[3]);
        d16[i / 2] = pack_bf16(ds[0], ds[1]);
        d16[i / 2 + 1] = pack_bf16(ds[2], ds[3]);
      }
      if (KEY) ptx::tmem_st16(ts, p16);
      ptx::tmem_st16(td, d16);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->pfull[b]));
    }
    if (ok) ok = wait_warp(ptx::smem_u32(&sh->afull), 0, abort, a.status);
    if (ok && !*abort) {
      ptx::tc_fence_after();
      const uint32_t acc = lane_base + C::ACC_COL + half * (D / 2);
      const int64_t r = beg + rr;
      const int64_t col = (int64_t)head * D + half * (D / 2);
      if (KEY) {
        store_row<D / 64>(acc, 1.0f, (__nv_bfloat16*)a.dV + r * a.lddv + col, in);
        store_row<D / 64>(acc + D, a.scale, (__nv_bfloat16*)a.dK + r * a.lddk + col, in);
      } else {
        store_row<D / 64>(acc, a.scale, (__nv_bfloat16*)a.dQ + r * a.lddq + col, in);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
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

// T x cols bf16 rows (stride ld) as boxes of 64 columns x 64 rows, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* p, int64_t T, int64_t cols, int64_t ld) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)T};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, 64}, estr[2] = {1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool KEY>
cudaError_t launch_side(cudaStream_t st, const AttnArgs& a, const CUtensorMap& q,
                        const CUtensorMap& e, const CUtensorMap& k, const CUtensorMap& v) {
  auto fn = k_attn_exact_bwd_tc<D, KEY>;
  const cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Cfg<D>::SMEM);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)(KEY ? a.Hkv : a.H) * (unsigned)a.n_seqs,
                  (unsigned)((a.max_len + BM - 1) / BM));
  if (KEY)
    fn<<<grid, THREADS, Cfg<D>::SMEM, st>>>(k, v, q, e, a);
  else
    fn<<<grid, THREADS, Cfg<D>::SMEM, st>>>(q, e, k, v, a);
  return cudaGetLastError();
}

template <int D>
cudaError_t backward_as(cudaStream_t st, const AttnArgs& a) {
  CUtensorMap q, e, k, v;
  const int64_t wq = (int64_t)a.H * D, wk = (int64_t)a.Hkv * D;
  if (!make_map(&q, a.Q, a.T, wq, a.ldq) || !make_map(&e, a.E, a.T, wq, a.lde) ||
      !make_map(&k, a.K, a.T, wk, a.ldk) || !make_map(&v, a.V, a.T, wk, a.ldv))
    return cudaErrorInvalidValue;
  const cudaError_t err = launch_side<D, false>(st, a, q, e, k, v);
  if (err != cudaSuccess) return err;
  return launch_side<D, true>(st, a, q, e, k, v);
}

// 16-byte rows: what TMA and the vector loads and stores need.
bool rows16(const void* p, int64_t ld, int64_t T) {
  return ((uintptr_t)p & 15) == 0 && (T <= 1 || (ld & 7) == 0);
}

}  // namespace

bool attn_exact_tc_supported(const AttnArgs& a, bool backward) {
  if (!backward) return false;
  if (a.dtype != DUST_BF16 || (a.head_dim != 64 && a.head_dim != 128) || !encode_fn()) return false;
  return rows16(a.Q, a.ldq, a.T) && rows16(a.K, a.ldk, a.T) && rows16(a.V, a.ldv, a.T) &&
         rows16(a.O_in, a.ldo, a.T) && rows16(a.E, a.lde, a.T) && rows16(a.dQ, a.lddq, a.T) &&
         rows16(a.dK, a.lddk, a.T) && rows16(a.dV, a.lddv, a.T);
}

cudaError_t launch_attn_exact_tc(cudaStream_t st, const AttnArgs& a, bool backward) {
  (void)backward;
  return a.head_dim == 64 ? backward_as<64>(st, a) : backward_as<128>(st, a);
}

}  // namespace dust
