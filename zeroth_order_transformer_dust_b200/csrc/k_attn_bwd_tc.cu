// The exact gradient of causal attention on tensor cores (bf16 tensors with 64- or
// 128-wide heads, fp32 tensors with 64-wide ones as three bf16 planes); formulas
// as in k_attn_exact.cu.
//
// One kernel body serves both sides. A CTA keeps 128 rows of its side
// resident (queries with their error signal, or keys with their values) and
// streams tiles of 128 rows of the other side. Per tile, with the resident rows
// as TMEM lanes:
//   query side   S = Q K^T, dP = E V^T (columns: keys),
//                dS = P (dP - delta) -> bf16 in TMEM, dQ += dS K;
//   key side     S^T = K Q^T, dP^T = V E^T (columns: queries),
//                P^T, dS^T -> bf16 in TMEM, dV += P^T E, dK += dS^T Q.
// The streamed tile is staged once by TMA and read twice: K-major by the score
// products and MN-major by the gradient products. P and dS never leave the SM:
// softmax threads write them over the scores' TMEM columns, from where the
// gradient MMAs take them as their A operand. The sums live in TMEM in fp32 for
// the CTA's whole life. Rounding P and dS to bf16 (half a step, 2^-8 relative,
// per term, against fp32 sums) is what puts their products on the tensor cores.
//
// Tiles of 128 and not 64 streamed rows: a 128 x 64 x 16 product takes 47 cycles
// where a 128 x 128 x 16 one takes 62 (its A operand is read at the same rate),
// and the hand-overs between the warps, about 150 cycles each, come half as often.
//
// Warp roles: warp 0 TMA producer, warp 1 issues the score products, warp 10 the
// gradient products (one thread for both spends more time between its waits
// than the tensor pipe does on the MMAs), warps 2..9 softmax (two warps per TMEM
// lane quarter, 64 of the tile's 128 columns each). The softmax of a tile has two
// halves, P from S and dS from dP. Where TMEM has room (bf16, all but the key side
// of 128-wide heads) S has two buffers, and P and dS go over the columns of the
// tile's S, which is dead by then: the next tile's P starts at once, from scores
// that are already there, and the gradient products and the next dP run under it.
// Else P goes over S and dS over dP, and the MMAs alternate so that S of the next
// tile runs while dS is formed.
//
// delta = <o, e> is taken from the bf16 output o, whose rounding matters where
// few keys average it out; in a sequence's first 128 rows the kernel sums
// P dP instead, which is the same number without that rounding.
//
// fp32 tensors: the key side runs as two kernels, one for dV and one for dK, since
// TMEM does not hold the third planes of P and dS and both sums. The tensor cores
// truncate as they add, always towards zero: over a sequence of 1024 that took
// 1.4e-5 off dK and dV. So a tile's sum starts from zero, and the softmax
// threads add it to the total (TMEM columns too) in fp32, rounded.
//
// Rows at or past the end of a sequence belong to nobody or to another
// sequence, so their content must not enter a sum, not even times 0: in the
// one streamed tile that can hold such rows the producer overwrites them with
// zeros before the MMAs see the tile.
//
// Measured (query side + key side): 8 x 1024 tokens, 12 heads of 64, bf16 60 + 70 us
// (0.25 PFLOP/s of the exact flops); packed sequences of 3000 to 1000, 16 query and
// 4 key/value heads of 128, bf16 167 + 228 us (0.50 PFLOP/s); the first in fp32
// planes 38 + 170 + 137 + 161 us. By stamps inside one CTA a tile takes about 2100
// cycles with 64-wide heads and 2500 to 4000 with 128-wide ones, against 770 to
// 2050 of MMAs: the chain of hand-overs S -> P -> sum -> S; a CTA's start takes
// 4000. That does not account for the whole: the first case's query side has 23.4
// tiles and 5.2 starts an SM, 36 of its 60 us, and the rest (the sums' way out,
// one CTA's end and the next one's launch, the last wave) has not been stamped.
// The key side of grouped heads also waits for its longest CTA (94 tiles where
// the mean SM has 70).
//
// Every wait is bounded: on expiry the CTA raises the timeout bit, drains its own
// copies and MMAs (bounded again), frees its TMEM and returns.
#include "attn_tc.cuh"

namespace dust {
namespace {

constexpr int THREADS = 96 + 32 * SOFT_WARPS;

// The kernels: the query side, the key side, and the key side's two gradients apart.
enum Side { kQuery = 0, kKey = 1, kKeyV = 2, kKeyK = 3 };

template <int D, int SIDE, int NP>
struct Cfg {
  static constexpr bool KEY = SIDE != kQuery;
  static constexpr bool DV = SIDE == kKey || SIDE == kKeyV;  // sums dV
  static constexpr bool DS = SIDE != kKeyV;                  // forms dS, sums dK or dQ
  static constexpr int NS = (KEY && D == 128) || NP == 3 ? 1 : 2;  // score buffers
  // stages of either streamed tensor
  static constexpr int ST0 = NP == 3 ? 1 : (D == 64 ? 4 : (KEY ? 2 : 3));
  static constexpr int ST1 = NP == 3 ? 1 : (D == 64 ? 4 : 2);
  static constexpr int BOXES = D / 64;                // boxes per 128 rows of a tensor
  static constexpr int TILE_BYTES = NP * BM * D * 2;  // 128 rows of a tensor
  // shared memory: the resident tensors, the stages, then (key side) -lse and
  // -delta per stage of s0 or (query side) partial deltas
  static constexpr int S0 = 2 * TILE_BYTES, S1 = S0 + ST0 * TILE_BYTES;
  static constexpr int COL = S1 + ST1 * TILE_BYTES;
  static constexpr int COL_BYTES = (KEY ? ST0 : 1) * 2 * BN * 4;
  static constexpr size_t SMEM = 1024 + (size_t)COL + COL_BYTES + 256;
  // TMEM columns: score buffers, dP, third planes of P and dS, the sums
  static constexpr int DP = NS * BN, P2 = DP + BN, ACC = P2 + (NP == 3 ? 64 : 0);
  static constexpr int TOTAL = ACC + D;  // NP 3: the sum of the tiles before
  // where a column half's dS goes, from its S columns (NS 2) or its dP columns (NS 1)
  static constexpr int DS_AT = KEY && NS == 2 ? 32 : 0;
  static_assert(ACC + (SIDE == kKey || NP == 3 ? 2 : 1) * D <= 512, "TMEM columns");
  static_assert(NP == 1 || SIDE != kKey, "one sum at a time");
  static_assert(SMEM <= 227 * 1024 && COL_BYTES >= 2 * BM * 4, "shared memory");
};

struct Bars {
  uint64_t res, land, full0[4], full1[4], empty0[4], empty1[4], sfull[2], pfull[2], dsfull[2], dpfull,
      vdone, sdone, afull;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// Resident tensors r0, r1 and streamed tensors s0, s1 of the score products
// S = r0 s0^T and dP = r1 s1^T: (Q, E; K, V) on the query side, (K, V; Q, E) on
// the key side.
template <int D, int SIDE, int NP>
__global__ __launch_bounds__(THREADS, 1) void k_attn_bwd_tc(
    const __grid_constant__ CUtensorMap tmR0, const __grid_constant__ CUtensorMap tmR1,
    const __grid_constant__ CUtensorMap tmS0, const __grid_constant__ CUtensorMap tmS1,
    AttnArgs a) {
  using C = Cfg<D, SIDE, NP>;
  constexpr bool KEY = C::KEY, DV = C::DV, DS = C::DS;
  using E = Elem<NP>;
  constexpr int NS = C::NS, ST0 = C::ST0, ST1 = C::ST1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw);
  // key side: per stage -lse and -delta (2 x 128); query side: partial deltas (2 x 128)
  float* s_col = reinterpret_cast<float*>(basep + C::COL);
  Bars* sh = reinterpret_cast<Bars*>(basep + C::COL + C::COL_BYTES);
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
  // streamed tiles: keys [0, diagonal] of one head, or for every head of the
  // group the queries from the diagonal on
  const int per_head = KEY ? (len + BN - 1) / BN - tile : tile + 1;
  const int n = KEY ? group * per_head : per_head;
  const int s_off = KEY ? tile : 0;
  // columns between the planes of the resident and the streamed tensors
  const int r_plane = heads * D, s_plane = (KEY ? a.H : a.Hkv) * D;

  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&sh->res), 1);
    ptx::mbar_init(ptx::smem_u32(&sh->land), 1);
    for (int s = 0; s < 4; ++s) {
      ptx::mbar_init(ptx::smem_u32(&sh->full0[s]), 2);  // the bytes, and the producer's word
      ptx::mbar_init(ptx::smem_u32(&sh->full1[s]), 2);
      ptx::mbar_init(ptx::smem_u32(&sh->empty0[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&sh->empty1[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_u32(&sh->sfull[b]), 1);
      ptx::mbar_init(ptx::smem_u32(&sh->pfull[b]), SOFT_WARPS);
      ptx::mbar_init(ptx::smem_u32(&sh->dsfull[b]), SOFT_WARPS);
    }
    ptx::mbar_init(ptx::smem_u32(&sh->dpfull), 1);
    ptx::mbar_init(ptx::smem_u32(&sh->vdone), 1);
    ptx::mbar_init(ptx::smem_u32(&sh->sdone), 1);
    ptx::mbar_init(ptx::smem_u32(&sh->afull), 1);
    sh->abort = 0;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async();
    // the resident rows are on their way while TMEM is allocated
    const uint32_t bar = ptx::smem_u32(&sh->res);
    ptx::mbar_expect_tx(bar, (DS ? 2 : 1) * C::TILE_BYTES);
    for (int t = 0; t < (DS ? 2 : 1); ++t)
      for (int c = 0; c < NP * C::BOXES; ++c)
        ptx::tma_load_2d(base + t * C::TILE_BYTES + c * BOX_BYTES, t ? &tmR1 : &tmR0,
                         c / C::BOXES * r_plane + head * D + 64 * (c % C::BOXES),
                         (int)(beg + r_first), bar);
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
    // key side: -lse (log2) and -delta of a tile's queries, four rows per lane;
    // -inf past the sequence's end, which makes p = 0 there
    float nl[4], nd[4];
    auto fetch_cols = [&](int j) {
      const int h = head * group + j / per_head;
      const int r = (s_off + j % per_head) * BN;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = r + lane + 32 * i;
        const bool in = j < n && q < len;
        nl[i] = in ? -a.lse[(beg + q) * a.H + h] * kLog2e : -inf_f();
        nd[i] = DS && in ? -a.delta[(beg + q) * a.H + h] : 0.0f;
      }
    };
    if (KEY) fetch_cols(0);
    uint32_t land_phase = 0;
    int armed0 = 0, armed1 = 0;  // tiles of s0 and s1 whose copies were issued
    // one tile of one streamed tensor into its stage; false after an abort
    auto load = [&](const CUtensorMap* map, uint32_t off, int stages, uint64_t* full,
                    uint64_t* empty, int j, int* armed) {
      const int st = j % stages;
      if (!wait_warp(ptx::smem_u32(&empty[st]), ((uint32_t)(j / stages) & 1u) ^ 1u, abort,
                     a.status))
        return false;
      const int h = KEY ? head * group + j / per_head : head / group;
      const int r = (s_off + j % per_head) * BN;
      const uint32_t fb = ptx::smem_u32(&full[st]), land = ptx::smem_u32(&sh->land);
      const bool partial = r + BN > len;
      if (lane == 0) {
        const uint32_t bar = partial ? land : fb;
        ptx::mbar_expect_tx(bar, C::TILE_BYTES);
        for (int c = 0; c < NP * C::BOXES; ++c)
          ptx::tma_load_2d(base + off + st * C::TILE_BYTES + c * BOX_BYTES, map,
                           c / C::BOXES * s_plane + h * D + 64 * (c % C::BOXES), (int)(beg + r),
                           bar);
      }
      *armed = j + 1;
      if (KEY && off == C::S0) {
        float* col = s_col + st * 2 * BN;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          col[lane + 32 * i] = nl[i];
          col[BN + lane + 32 * i] = nd[i];
        }
        fetch_cols(j + 1);
      }
      if (partial) {
        if (!wait_warp(land, land_phase, abort, a.status)) return false;
        land_phase ^= 1u;
        zero_rows<D, NP>(basep + off + st * C::TILE_BYTES, r + BN - len, lane);
      }
      __syncwarp();
      if (lane == 0) {
        if (partial) ptx::mbar_arrive(fb);
        ptx::mbar_arrive(fb);
      }
      return true;
    };
    for (int j = 0; j < n; ++j)
      if (!load(&tmS0, C::S0, ST0, sh->full0, sh->empty0, j, &armed0) ||
          !load(&tmS1, C::S1, ST1, sh->full1, sh->empty1, j, &armed1))
        break;
    // every copy has landed before the CTA can exit (after an abort the last
    // stages may not have been waited for by the MMAs)
    if (*abort) {
      int dummy = 0;
      wait_warp(ptx::smem_u32(&sh->res), 0, &dummy, a.status);
      auto landed = [&](uint64_t* full, int stages, int armed) {
        for (int j = max(0, armed - stages); j < armed; ++j) {
          if ((s_off + j % per_head) * BN + BN > len)
            wait_warp(ptx::smem_u32(&sh->land), land_phase, &dummy, a.status);
          else
            wait_warp(ptx::smem_u32(&full[j % stages]), (uint32_t)(j / stages) & 1u, &dummy,
                      a.status);
        }
      };
      landed(sh->full0, ST0, armed0);
      landed(sh->full1, ST1, armed1);
    }
  } else if (warp == 1) {
    // ---------------- score products: S and dP ----------------
    if (lane == 0) {
      bool issued = false;
      auto s_product = [&](int j) {
        if (!wait(sh->full0[j % ST0], j / ST0)) return false;
        ptx::tc_fence_after();
        mma_scores<D, NP>(tmem + (j % NS) * BN, base, base + C::S0 + (j % ST0) * C::TILE_BYTES);
        ptx::mma_commit(ptx::smem_u32(&sh->sfull[j % NS]));
        issued = true;
        return true;
      };
      auto dp_product = [&](int j) {
        if (!wait(sh->full1[j % ST1], j / ST1)) return false;
        ptx::tc_fence_after();
        mma_scores<D, NP>(tmem + C::DP, base + C::TILE_BYTES,
                          base + C::S1 + (j % ST1) * C::TILE_BYTES);
        ptx::mma_commit(ptx::smem_u32(&sh->dpfull));
        if (!DV) ptx::mma_commit(ptx::smem_u32(&sh->empty1[j % ST1]));
        return true;
      };
      // the gradient MMAs of tile j are complete
      auto done0 = [&](int j) { return wait(sh->empty0[j % ST0], j / ST0); };
      bool ok = wait(sh->res, 0) && s_product(0) && (!DS || dp_product(0));
      if (NS == 2 && n > 1) ok = ok && s_product(1);
      for (int j = 0; j + 1 < n && ok; ++j) {
        if (NS == 2)  // dP's columns are read once dS is there; S's free after the tile's MMAs
          ok = wait(sh->dsfull[j & 1], j >> 1) && dp_product(j + 1) &&
               (j + 2 >= n || (done0(j) && s_product(j + 2)));
        else  // S's columns are free after dV's MMAs (no dV: once read), dP's after dK's
          ok = (DV ? wait(sh->vdone, j) : wait(sh->dsfull[j & 1], j >> 1)) && s_product(j + 1) &&
               (!DS || (done0(j) && dp_product(j + 1)));
      }
      if (issued) {  // complete before TMEM is released
        int dummy = 0;
        ptx::mma_commit(ptx::smem_u32(&sh->sdone));
        wait_bounded(ptx::smem_u32(&sh->sdone), 0, &dummy, a.status);
      }
    }
  } else if (warp == 2 + SOFT_WARPS) {
    // ---------------- gradient products ----------------
    if (lane == 0) {
      const uint32_t acc0 = tmem + C::ACC, acc1 = acc0 + D;
      bool issued = false;
      for (int j = 0; j < n; ++j) {
        const uint32_t s_at = tmem + (j % NS) * BN;
        // (P needs only s0's tile: s1's is waited for here, too)
        if (DV) {  // dV += P^T E
          if (!wait(sh->full1[j % ST1], j / ST1) || !wait(sh->pfull[j & 1], j >> 1)) break;
          ptx::tc_fence_after();
          mma_sum<D, NP>(acc0, s_at, tmem + C::P2, base + C::S1 + (j % ST1) * C::TILE_BYTES,
                         NP == 3 || j == 0);
          ptx::mma_commit(ptx::smem_u32(&sh->vdone));
          if (!DS) {  // (s0's stage too only here: its lse is read for P)
            ptx::mma_commit(ptx::smem_u32(&sh->empty0[j % ST0]));
            ptx::mma_commit(ptx::smem_u32(&sh->empty1[j % ST1]));
          }
          issued = true;
        }
        if (!DS) continue;
        // dK += dS^T Q, dQ += dS K; dS also means that dP's MMAs are done with s1's tile
        if (!wait(sh->full0[j % ST0], j / ST0) || !wait(sh->dsfull[j & 1], j >> 1)) break;
        ptx::tc_fence_after();
        mma_sum<D, NP>(DV ? acc1 : acc0, (NS == 2 ? s_at : tmem + C::DP) + C::DS_AT, tmem + C::P2,
                       base + C::S0 + (j % ST0) * C::TILE_BYTES, NP == 3 || j == 0);
        ptx::mma_commit(ptx::smem_u32(&sh->empty0[j % ST0]));
        if (DV) ptx::mma_commit(ptx::smem_u32(&sh->empty1[j % ST1]));
        issued = true;
      }
      if (issued) {  // complete before the sums are read, or TMEM is released
        int dummy = 0;
        ptx::mma_commit(ptx::smem_u32(&sh->afull));
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
    // the other column half's thread of this row, through shared memory
    auto row_sum = [&](float v) {
      s_col[half * BM + row] = v;
      asm volatile("bar.sync 1, %0;" ::"n"(32 * SOFT_WARPS) : "memory");
      return s_col[row] + s_col[BM + row];
    };
    float nlse2 = -inf_f(), ndelta = 0.0f;  // -lse (log2; p = 0 past the end), -delta
    if (!KEY) {
      if (in) nlse2 = -a.lse[(beg + rr) * a.H + head] * kLog2e;
      if (tile > 0) {
        // delta = <o, e>: this thread's half of the row's columns
        float d = 0.0f;
        if (in) {
          const int64_t r = beg + rr;
          const uint4* o =
              reinterpret_cast<const uint4*>((const E*)a.O_in + r * a.ldo + head * D + half * (D / 2));
          const uint4* e =
              reinterpret_cast<const uint4*>((const E*)a.E + r * a.lde + head * D + half * (D / 2));
#pragma unroll
          for (int i = 0; i < D / 2 * (int)sizeof(E) / 16; ++i) {
            const uint4 x = __ldg(o + i), y = __ldg(e + i);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (NP == 1) {
                d = fmaf(__uint_as_float(xs[w] << 16), __uint_as_float(ys[w] << 16), d);
                d = fmaf(__uint_as_float(xs[w] & 0xffff0000u),
                         __uint_as_float(ys[w] & 0xffff0000u), d);
              } else {
                d = fmaf(__uint_as_float(xs[w]), __uint_as_float(ys[w]), d);
              }
            }
          }
        }
        ndelta = -row_sum(d);
      }
    }
    // NP 3: total += the sum of tile j, whose MMAs are waited for; this thread's half
    // of the row's columns
    const uint32_t acc = lane_base + C::ACC + half * (D / 2);
    auto flush = [&](int j) {
      uint64_t& bar = DS ? sh->empty0[j % ST0] : sh->vdone;
      if (!wait_warp(ptx::smem_u32(&bar), (uint32_t)(j / (DS ? ST0 : 1)) & 1u, abort, a.status))
        return false;
      ptx::tc_fence_after();
      uint32_t x[32], y[32], w[16];
      ptx::tmem_ld32x2(acc, x, lane_base + C::TOTAL + half * (D / 2), y);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = j == 0 ? x[16 * b + i]
                        : __float_as_uint(__uint_as_float(x[16 * b + i]) +
                                          __uint_as_float(y[16 * b + i]));
        ptx::tmem_st16(lane_base + C::TOTAL + half * (D / 2) + 16 * b, w);
      }
      return true;
    };
    bool ok = true, summed = KEY || tile > 0;
    for (int j = 0; j < n; ++j) {
      const int b = j % NS, st = j % ST0;
      const uint32_t ts = lane_base + b * BN + 64 * half;
      const float* cl = s_col + st * 2 * BN + 64 * half;
      float2 p[32];
      {  // P from S
        // (the producer's lse and delta are ordered by its own barrier)
        if (KEY)
          ok = wait_warp(ptx::smem_u32(&sh->full0[st]), (uint32_t)(j / ST0) & 1u, abort, a.status);
        ok = ok &&
             wait_warp(ptx::smem_u32(&sh->sfull[b]), (uint32_t)(j / NS) & 1u, abort, a.status);
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[2][32];
        ptx::tmem_ld32x2(ts, s[0], ts + 32, s[1]);
        if (j % per_head == (KEY ? 0 : tile)) {  // the tile on the diagonal: column > or < row
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (KEY ? 64 * half + i < row : 64 * half + i > row)
              s[i >> 5][i & 31] = 0xff800000u;  // -inf: p = 0
        }
        const float2 cc = make_float2(c2, c2);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float4 l4 = make_float4(nlse2, nlse2, nlse2, nlse2);
          if (KEY) l4 = *reinterpret_cast<const float4*>(cl + 2 * i);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int e = 2 * (i + k);
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[e >> 5][e & 31]),
                                                    __uint_as_float(s[e >> 5][(e & 31) + 1])),
                                        cc, k ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y));
            p[i + k] = make_float2(ex2(x.x), ex2(x.y));
          }
          if (DV && (i & 15) == 14) {
            float2 v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = p[(i & 16) + k];
            store_planes<NP>(ts + (i & 16), lane_base + C::P2 + 32 * half + (i & 16), v);
          }
        }
        if (DV) {
          if (NP == 3 && j > 0 && !flush(j - 1)) {
            ok = false;
            break;
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->pfull[j & 1]));
        }
      }
      if (DS) {  // dS from P and dP
        ok = wait_warp(ptx::smem_u32(&sh->dpfull), (uint32_t)j & 1u, abort, a.status);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t td = lane_base + C::DP + 64 * half;
        uint32_t d[2][32];
        ptx::tmem_ld32x2(td, d[0], td + 32, d[1]);
        auto dpair = [&](int i) {
          const int e = 2 * i;
          return make_float2(__uint_as_float(d[e >> 5][e & 31]),
                             __uint_as_float(d[e >> 5][(e & 31) + 1]));
        };
        if (!KEY && tile == 0) {  // one tile: delta = sum_j P dP, all at hand
          float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc = __ffma2_rn(p[i], dpair(i), acc);
          ndelta = -row_sum(acc.x + acc.y);
          summed = true;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 v[16];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float4 d4 = make_float4(ndelta, ndelta, ndelta, ndelta);
            if (KEY) d4 = *reinterpret_cast<const float4*>(cl + BN + 32 * h + 2 * i);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              v[i + k] = __fmul2_rn(
                  p[16 * h + i + k],
                  __fadd2_rn(dpair(16 * h + i + k),
                             k ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y)));
          }
          store_planes<NP>((NS == 2 ? ts : td) + C::DS_AT + 16 * h,
                           lane_base + C::P2 + 32 * half + 16 * h, v);
        }
        if (NP == 3 && j > 0 && !flush(j - 1)) {
          ok = false;
          break;
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->dsfull[j & 1]));
      }
    }
    // (after an abort: the other warps do not wait for this one's part of delta)
    if (!summed) asm volatile("bar.arrive 1, %0;" ::"n"(32 * SOFT_WARPS) : "memory");
    if (!KEY && in && half == 0) a.delta[(beg + rr) * a.H + head] = -ndelta;
    if (ok) ok = wait_warp(ptx::smem_u32(&sh->afull), 0, abort, a.status);
    if (NP == 3 && ok) ok = flush(n - 1);
    if (NP == 3) ptx::tmem_wait_st();
    if (ok && !*abort) {
      ptx::tc_fence_after();
      const uint32_t sum = NP == 3 ? acc + D : acc;  // (TOTAL, or the accumulator)
      const int64_t r = beg + rr;
      const int64_t col = (int64_t)head * D + half * (D / 2);
      if (SIDE == kKey) {
        store_row<D / 64>(sum, 1.0f, (E*)a.dV + r * a.lddv + col, in);
        store_row<D / 64>(sum + D, a.scale, (E*)a.dK + r * a.lddk + col, in);
      } else if (SIDE == kKeyV) {
        store_row<D / 64>(sum, 1.0f, (E*)a.dV + r * a.lddv + col, in);
      } else if (SIDE == kKeyK) {
        store_row<D / 64>(sum, a.scale, (E*)a.dK + r * a.lddk + col, in);
      } else {
        store_row<D / 64>(sum, a.scale, (E*)a.dQ + r * a.lddq + col, in);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

template <int D, int SIDE, int NP>
cudaError_t launch_side(cudaStream_t st, const AttnArgs& a, const CUtensorMap& q,
                        const CUtensorMap& e, const CUtensorMap& k, const CUtensorMap& v) {
  auto fn = k_attn_bwd_tc<D, SIDE, NP>;
  constexpr bool KEY = SIDE != kQuery;
  constexpr size_t smem = Cfg<D, SIDE, NP>::SMEM;
  const cudaError_t err =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)(KEY ? a.Hkv : a.H) * (unsigned)a.n_seqs,
                  (unsigned)((a.max_len + BM - 1) / BM));
  if (KEY)
    fn<<<grid, THREADS, smem, st>>>(k, v, q, e, a);
  else
    fn<<<grid, THREADS, smem, st>>>(q, e, k, v, a);
  return cudaGetLastError();
}

template <int D, int NP>
cudaError_t backward_as(cudaStream_t st, const AttnArgs& a) {
  CUtensorMap q, e, k, v;
  const int64_t wq = (int64_t)a.H * D, wk = (int64_t)a.Hkv * D;
  const SplitSrc src[4] = {{a.Q, a.ldq, wq}, {a.E, a.lde, wq}, {a.K, a.ldk, wk}, {a.V, a.ldv, wk}};
  CUtensorMap* maps[4] = {&q, &e, &k, &v};
  cudaError_t err = make_maps<NP>(st, a, src, maps, 4);
  if (err == cudaSuccess) err = launch_side<D, kQuery, NP>(st, a, q, e, k, v);
  if constexpr (NP == 1) {
    if (err == cudaSuccess) err = launch_side<D, kKey, NP>(st, a, q, e, k, v);
  } else {
    if (err == cudaSuccess) err = launch_side<D, kKeyV, NP>(st, a, q, e, k, v);
    if (err == cudaSuccess) err = launch_side<D, kKeyK, NP>(st, a, q, e, k, v);
  }
  return err;
}

}  // namespace

bool attn_exact_tc_supported(const AttnArgs& a, bool backward) {
  const bool heads = a.dtype == DUST_BF16 ? a.head_dim == 64 || a.head_dim == 128
                                          : a.head_dim == 64 && a.planes;
  if (!heads || !encode_fn()) return false;
  if (!rows16(a, a.Q, a.ldq) || !rows16(a, a.K, a.ldk) || !rows16(a, a.V, a.ldv)) return false;
  if (!backward) return rows16(a, a.O, a.ldo);
  return rows16(a, a.O_in, a.ldo) && rows16(a, a.E, a.lde) && rows16(a, a.dQ, a.lddq) &&
         rows16(a, a.dK, a.lddk) && rows16(a, a.dV, a.lddv);
}

cudaError_t launch_attn_bwd_tc(cudaStream_t st, const AttnArgs& a) {
  if (a.dtype == DUST_F32) return backward_as<64, 3>(st, a);
  return a.head_dim == 64 ? backward_as<64, 1>(st, a) : backward_as<128, 1>(st, a);
}

}  // namespace dust
