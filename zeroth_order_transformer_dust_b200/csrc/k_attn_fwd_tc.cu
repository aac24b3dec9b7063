// Causal attention on tensor cores (bf16 tensors with 64- or 128-wide heads, fp32
// tensors with 64-wide ones as three bf16 planes): the forward pass of the exact
// attention; formulas as in k_attn_exact.cu.
//
// A CTA owns 256 query rows of a head as two tiles of 128 and streams key/value
// tiles of 128 rows. Per streamed tile and query tile g, with the query rows as
// TMEM lanes: S_g = Q_g K^T, P_g = exp2(S_g c - m_g) -> bf16 over S_g's TMEM
// columns, O_g += P_g V with P_g taken from TMEM. While one tile's rows are in
// softmax the tensor pipe works for the other. Bound by the exponentials as
// much as by the MMAs: a 128 x 128 tile takes 1024 cycles of either with
// 128-wide heads.
//
// One thread has one row, so no maximum crosses threads. The maximum that P is
// taken against is only moved when a row's has grown by more than 8 (log2): P
// then stays below 2^8, which costs a float nothing, and O, which lives in TMEM,
// is rescaled in the few tiles where that happens instead of in every one. The
// sum l is taken over the unrounded P; rounding P to bf16 for the product (half
// a step, 2^-8 relative, per term) is what puts it on the tensor cores.
//
// fp32 tensors: a CTA owns one query tile with two S buffers instead, which leaves
// TMEM for the third plane of P and a total. The tensor cores truncate as they
// add, so a tile's P V starts from zero and the softmax threads add it to the
// total in fp32, rounded (1.9e-6 off over a sequence of 1024 without that).
//
// Measured: packed sequences of 3000 to 1000, 16 query and 4 key/value heads of
// 128, bf16 117 us (0.67 PFLOP/s of the exact flops); 8 x 1024 tokens, 12 heads of
// 64, bf16 46 us (0.28), fp32 160 us with the 29 for its planes; 12 heads of 128,
// bf16 57 us (0.46).
//
// Warp roles: warp 0 TMA producer, warp 1 issues S products, warp 2 the PV
// products, warps 4..7 and 8..11 are the softmax of either query tile. Rows past
// a sequence's end and bounded waits as in k_attn_bwd_tc.cu.
#include <cfloat>

#include "attn_tc.cuh"

namespace dust {
namespace {

constexpr int THREADS = 128 + 32 * SOFT_WARPS;
constexpr float kGrow = 8.0f;  // log2 growth of a row's maximum that rescales O

template <int D, int NP>
struct Cfg {
  static constexpr int G = NP == 3 ? 1 : 2;  // query tiles
  // key and value stages
  static constexpr int STK = NP == 3 ? 2 : (D == 64 ? 4 : 3), STV = NP == 3 ? 1 : (D == 64 ? 4 : 2);
  static constexpr int BOXES = D / 64;
  static constexpr int TILE_BYTES = NP * BM * D * 2;
  static constexpr int K0 = G * TILE_BYTES, V0 = K0 + STK * TILE_BYTES;
  static constexpr int BARS = V0 + STV * TILE_BYTES;
  static constexpr size_t SMEM = 1024 + (size_t)BARS + 256;
  // TMEM: two S (of two query tiles, or of one in turn), O of each; NP 3: the total
  // and P's third plane
  static constexpr int O = 2 * BN, TOTAL = O + D, P2 = TOTAL + D;
  static_assert(NP == 3 ? P2 + 64 <= 512 : O + 2 * D <= 512, "TMEM columns");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct Bars {
  uint64_t res[2], land, kfull[4], vfull[4], kempty[4], vempty[4], sfull[2], pfull[2], odone[2],
      sdone, pvdone;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

template <int D, int NP>
__global__ __launch_bounds__(THREADS, 1) void k_attn_fwd_tc(
    const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
    const __grid_constant__ CUtensorMap tmV, AttnArgs a) {
  using C = Cfg<D, NP>;
  using E = Elem<NP>;
  constexpr int STK = C::STK, STV = C::STV, G = C::G;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  Bars* sh = reinterpret_cast<Bars*>(basep + C::BARS);
  volatile int* abort = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int head = (int)(blockIdx.x % a.H), seq = (int)(blockIdx.x / a.H);
  const int hk = head / (a.H / a.Hkv);
  const int tile = (int)(gridDim.y - 1 - blockIdx.y);  // the longest rows first
  int64_t beg, end;
  if (!attn_sequence(a, seq, &beg, &end)) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadSeq);
    return;
  }
  const int len = (int)(end - beg);
  const int r_first = G * tile * BM;
  if (r_first >= len) return;
  // key tiles up to the diagonal; the second query tile may lie past the end
  const int n0 = G * tile + 1, n1 = G == 2 && r_first + BM < len ? 2 * tile + 2 : 0;
  const int n = max(n0, n1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      ptx::mbar_init(ptx::smem_u32(&sh->kfull[s]), 2);  // the bytes, and the producer's word
      ptx::mbar_init(ptx::smem_u32(&sh->vfull[s]), 2);
      ptx::mbar_init(ptx::smem_u32(&sh->kempty[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&sh->vempty[s]), 1);
    }
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(ptx::smem_u32(&sh->res[g]), 1);
      ptx::mbar_init(ptx::smem_u32(&sh->sfull[g]), 1);
      ptx::mbar_init(ptx::smem_u32(&sh->pfull[g]), SOFT_WARPS / 2);
      ptx::mbar_init(ptx::smem_u32(&sh->odone[g]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&sh->land), 1);
    ptx::mbar_init(ptx::smem_u32(&sh->sdone), 1);
    ptx::mbar_init(ptx::smem_u32(&sh->pvdone), 1);
    sh->abort = 0;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async();
    // the query rows are on their way while TMEM is allocated
    for (int g = 0; g < (n1 ? 2 : 1); ++g) {
      const uint32_t bar = ptx::smem_u32(&sh->res[g]);
      ptx::mbar_expect_tx(bar, C::TILE_BYTES);
      for (int c = 0; c < NP * C::BOXES; ++c)
        ptx::tma_load_2d(base + g * C::TILE_BYTES + c * BOX_BYTES, &tmQ,
                         c / C::BOXES * a.H * D + head * D + 64 * (c % C::BOXES),
                         (int)(beg + r_first + g * BM), bar);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&sh->tmem_base), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  // by one thread: use `use` of a barrier
  auto wait = [&](uint64_t& bar, int use) {
    return wait_bounded(ptx::smem_u32(&bar), (uint32_t)use & 1u, abort, a.status);
  };

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    uint32_t land_phase = 0;
    int armed_k = 0, armed_v = 0;  // tiles whose copies were issued
    auto load = [&](const CUtensorMap* map, uint32_t off, int stages, uint64_t* full,
                    uint64_t* empty, int j, int* armed) {
      const int st = j % stages;
      if (!wait_warp(ptx::smem_u32(&empty[st]), ((uint32_t)(j / stages) & 1u) ^ 1u, abort,
                     a.status))
        return false;
      const uint32_t fb = ptx::smem_u32(&full[st]), land = ptx::smem_u32(&sh->land);
      const bool partial = (j + 1) * BN > len;
      if (lane == 0) {
        const uint32_t bar = partial ? land : fb;
        ptx::mbar_expect_tx(bar, C::TILE_BYTES);
        for (int c = 0; c < NP * C::BOXES; ++c)
          ptx::tma_load_2d(base + off + st * C::TILE_BYTES + c * BOX_BYTES, map,
                           c / C::BOXES * a.Hkv * D + hk * D + 64 * (c % C::BOXES),
                           (int)(beg + j * BN), bar);
      }
      *armed = j + 1;
      if (partial) {
        if (!wait_warp(land, land_phase, abort, a.status)) return false;
        land_phase ^= 1u;
        zero_rows<D, NP>(basep + off + st * C::TILE_BYTES, (j + 1) * BN - len, lane);
      }
      __syncwarp();
      if (lane == 0) {
        if (partial) ptx::mbar_arrive(fb);
        ptx::mbar_arrive(fb);
      }
      return true;
    };
    for (int j = 0; j < n; ++j)
      if (!load(&tmK, C::K0, STK, sh->kfull, sh->kempty, j, &armed_k) ||
          !load(&tmV, C::V0, STV, sh->vfull, sh->vempty, j, &armed_v))
        break;
    // every copy has landed before the CTA can exit (after an abort the last
    // stages may not have been waited for by the MMAs)
    if (*abort) {
      int dummy = 0;
      for (int g = 0; g < (n1 ? 2 : 1); ++g)
        wait_warp(ptx::smem_u32(&sh->res[g]), 0, &dummy, a.status);
      auto landed = [&](uint64_t* full, int stages, int armed) {
        for (int j = max(0, armed - stages); j < armed; ++j) {
          if ((j + 1) * BN > len)
            wait_warp(ptx::smem_u32(&sh->land), land_phase, &dummy, a.status);
          else
            wait_warp(ptx::smem_u32(&full[j % stages]), (uint32_t)(j / stages) & 1u, &dummy,
                      a.status);
        }
      };
      landed(sh->kfull, STK, armed_k);
      landed(sh->vfull, STV, armed_v);
    }
  } else if (warp == 1) {
    // ---------------- S_g = Q_g K^T ----------------
    if (lane == 0) {
      bool issued = false, ok = true;
      for (int j = 0; j < n && ok; ++j) {
        ok = wait(sh->kfull[j % STK], j / STK);
        for (int g = 0; g < G && ok; ++g) {
          if (j >= (g ? n1 : n0)) continue;
          // P of the buffer's previous tile lies over S: its product is complete
          const int b = G == 2 ? g : j & 1;
          if (j == 0) ok = wait(sh->res[g], 0);
          if (G == 2 && j > 0) ok = wait(sh->odone[g], j - 1);
          if (G == 1 && j > 1) ok = wait(sh->odone[b], (j >> 1) - 1);
          if (!ok) break;
          ptx::tc_fence_after();
          mma_scores<D, NP>(tmem + b * BN, base + g * C::TILE_BYTES,
                            base + C::K0 + (j % STK) * C::TILE_BYTES);
          ptx::mma_commit(ptx::smem_u32(&sh->sfull[b]));
          issued = true;
        }
        if (ok) ptx::mma_commit(ptx::smem_u32(&sh->kempty[j % STK]));
      }
      if (issued) {  // complete before TMEM is released
        int dummy = 0;
        ptx::mma_commit(ptx::smem_u32(&sh->sdone));
        wait_bounded(ptx::smem_u32(&sh->sdone), 0, &dummy, a.status);
      }
    }
  } else if (warp == 2) {
    // ---------------- O_g += P_g V ----------------
    if (lane == 0) {
      bool ok = true;
      for (int j = 0; j < n && ok; ++j) {
        ok = wait(sh->vfull[j % STV], j / STV);
        for (int g = 0; g < G && ok; ++g) {
          if (j >= (g ? n1 : n0)) continue;
          ok = wait(sh->pfull[g], j);
          if (!ok) break;
          ptx::tc_fence_after();
          const int b = G == 2 ? g : j & 1;
          mma_sum<D, NP>(tmem + C::O + g * D, tmem + b * BN, tmem + C::P2,
                         base + C::V0 + (j % STV) * C::TILE_BYTES, NP == 3 || j == 0);
          ptx::mma_commit(ptx::smem_u32(&sh->odone[b]));
        }
        if (ok) ptx::mma_commit(ptx::smem_u32(&sh->vempty[j % STV]));
      }
      int dummy = 0;  // complete before TMEM is released
      ptx::mma_commit(ptx::smem_u32(&sh->pvdone));
      wait_bounded(ptx::smem_u32(&sh->pvdone), 0, &dummy, a.status);
    }
  } else if (warp >= 4 && warp < 4 + 4 * G) {
    // ---------------- softmax ----------------
    const int g = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;                  // TMEM lane
    const int rr = r_first + g * BM + row;             // the row's place in the sequence
    const int ng = g ? n1 : n0;
    const bool in = rr < len;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t to = lane_base + C::O + g * D, total = lane_base + C::TOTAL;
    const float c2 = a.scale * kLog2e;
    float m = 0.0f, l = 0.0f;
    bool ok = true;
    // the product of tile j is complete
    auto done = [&](int j) {
      ok = wait_warp(ptx::smem_u32(&sh->odone[G == 2 ? g : j & 1]),
                     (uint32_t)(G == 2 ? j : j >> 1) & 1u, abort, a.status);
      ptx::tc_fence_after();
      return ok;
    };
    // NP 3: total = (total + the product of tile j) f
    auto flush = [&](int j, float f) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32], y[32], w[16];
        ptx::tmem_ld32x2(to + 32 * c, x, total + 32 * c, y);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float o = __uint_as_float(x[16 * b + i]);
            w[i] = __float_as_uint((j == 0 ? o : o + __uint_as_float(y[16 * b + i])) * f);
          }
          ptx::tmem_st16(total + 32 * c + 16 * b, w);
        }
      }
    };
    for (int j = 0; j < ng; ++j) {
      const int sb = G == 2 ? g : j & 1;
      const uint32_t ts = lane_base + sb * BN;
      ok = wait_warp(ptx::smem_u32(&sh->sfull[sb]), (uint32_t)(G == 2 ? j : j >> 1) & 1u, abort,
                     a.status);
      if (!ok) break;
      ptx::tc_fence_after();
      const bool diag = j == ng - 1;
      uint32_t s[2][32];
      // 64 columns of S; on the diagonal tile keys past the row's are -inf
      auto load = [&](int h) {
        ptx::tmem_ld32x2(ts + 64 * h, s[0], ts + 64 * h + 32, s[1]);
        if (diag) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (64 * h + i > row) s[i >> 5][i & 31] = 0xff800000u;
        }
      };
      float mx[4] = {-inf_f(), -inf_f(), -inf_f(), -inf_f()};
#pragma unroll
      for (int h = 1; h >= 0; --h) {
        load(h);
#pragma unroll
        for (int i = 0; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i >> 5][i & 31]));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
      // (a lane past the end has a neighbour's row, or nobody's: it has no vote)
      const bool grown = __any_sync(0xffffffffu, in && top > m + kGrow);
      if (j == 0) {
        // finite: a tile whose scores are all -inf gives p = 0 and is forgotten by
        // the first maximum behind it
        m = fmaxf(top, -FLT_MAX);
      } else if (NP == 3) {
        // (P's third plane has one buffer, so this tile's waits for the product anyway)
        if (!done(j - 1)) break;
        float f = 1.0f;
        if (grown) {
          const float mn = fmaxf(m, top);
          f = ex2(m - mn);
          m = mn;
          l *= f;
        }
        flush(j - 1, f);
        // (the first half's registers are needed again: the loads below)
        load(0);
      } else if (grown) {
        if (!done(j - 1)) break;  // O holds the tiles before this one
        const float mn = fmaxf(m, top), f = ex2(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          ptx::tmem_ld32(to + 32 * c, v);
          uint32_t w[2][16];
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i >> 4][i & 15] = __float_as_uint(v[i] * f);
          ptx::tmem_st16(to + 32 * c, w[0]);
          ptx::tmem_st16(to + 32 * c + 16, w[1]);
        }
      }
      const float2 cc = make_float2(c2, c2), nm = make_float2(-m, -m);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1) load(1);  // (the first half is still in registers)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float2 v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[b][2 * i]),
                                                    __uint_as_float(s[b][2 * i + 1])),
                                        cc, nm);
            v[i] = make_float2(ex2(x.x), ex2(x.y));
            sum[i & 1] = __fadd2_rn(sum[i & 1], v[i]);
          }
          // P's columns lie over those of S that this thread has read
          store_planes<NP>(ts + 64 * h + 16 * b, lane_base + C::P2 + 32 * h + 16 * b, v);
        }
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->pfull[g]));
    }
    if (ok && ng > 0 && done(ng - 1) && !*abort) {
      if (NP == 3) {
        flush(ng - 1, 1.0f);
        ptx::tmem_wait_st();
      }
      const int64_t r = beg + rr;
      if (in) a.lse_out[r * a.H + head] = 0.6931471805599453f * m + logf(l);
      store_row<D / 32>(NP == 3 ? total : to, 1.0f / l, (E*)a.O + r * a.ldo + (int64_t)head * D, in);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

template <int D, int NP>
cudaError_t forward_as(cudaStream_t st, const AttnArgs& a) {
  CUtensorMap q, k, v;
  const int64_t wq = (int64_t)a.H * D, wk = (int64_t)a.Hkv * D;
  const SplitSrc src[3] = {{a.Q, a.ldq, wq}, {a.K, a.ldk, wk}, {a.V, a.ldv, wk}};
  CUtensorMap* maps[3] = {&q, &k, &v};
  cudaError_t err = make_maps<NP>(st, a, src, maps, 3);
  if (err != cudaSuccess) return err;
  auto fn = k_attn_fwd_tc<D, NP>;
  constexpr size_t smem = Cfg<D, NP>::SMEM;
  err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)a.H * (unsigned)a.n_seqs,
                  (unsigned)((a.max_len + Cfg<D, NP>::G * BM - 1) / (Cfg<D, NP>::G * BM)));
  fn<<<grid, THREADS, smem, st>>>(q, k, v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd_tc(cudaStream_t st, const AttnArgs& a) {
  if (a.dtype == DUST_F32) return forward_as<64, 3>(st, a);
  return a.head_dim == 64 ? forward_as<64, 1>(st, a) : forward_as<128, 1>(st, a);
}

}  // namespace dust
