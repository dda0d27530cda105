// sol_attn_bwd: gradients of sol_attn_fwd for given lists, recomputing the
// probabilities from Q, K and the saved normaliser.
//
// Per query row r with normaliser L_r and delta_r = sum_d dO_rd O_rd, for a key
// row t of a listed block:
//   p = exp(s q.k_t - L_r),  dp = dO.v_t,  ds = p (dp - delta_r)
//   dq_r += s ds k_t,  dk_t += s ds q_r,  dv_t += p dO_r
// and for the centroid (kc_j, vc_j, offset c_j) of an unlisted block the same
// with gradients gk_j, gv_j and, for the offset, gb_j = sum ds, which the pooling
// passes on to the block's rows (the lists are constants, and the rounding of
// the centroids to bf16 is passed straight through):
//   mode 0: dk_t += gk_j / n, dv_t += gv_j / n
//   mode 1: c_j holds the log-mass bias; with w_t the anchor's softmax over the
//           block's rows, beta_t = s gb_j (w_t - 1/n): dk_t also gets beta_t a
//   mode 2: h_t = gk_j.k_t - gb_j s a.k_t + gv_j.v_t, beta_t = s w_t (h_t - sum_u w_u h_u):
//           dk_t += w_t gk_j + beta_t a, dv_t += w_t gv_j
//   anchor (modes 1, 2): da = sum_t beta_t k_t over all rows, spread evenly over
//           the anchor's query rows.
// No gradient is added atomically: the queries' pass and the keys' pass each own
// their outputs (the logits are computed in both), so results are deterministic.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "ptx.cuh"

namespace sol {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// ---- row statistics ------------------------------------------------------------------------------
// -lse (log2 units) and -delta of every query row.  HBM-bound: O and dO are read
// once.  A CTA owns one 64-row block of 8 heads; D/8 lanes hold a row.
constexpr int kStatHeads = 8;

template <int D>
__global__ void __launch_bounds__(256) stat_kernel(const BwdArgs a) {
  constexpr int LPR = D / 8, G = 256 / LPR;   // row groups of the CTA
  __shared__ float sd[kStatHeads][65];
  const int hg = (a.H + kStatHeads - 1) / kStatHeads, blk = blockIdx.x / hg % a.nb;
  const int b = blockIdx.x / hg / a.nb, h0 = (int)(blockIdx.x % hg) * kStatHeads;
  const int c = threadIdx.x % LPR, g = threadIdx.x / LPR;
#pragma unroll 4
  for (int e = g; e < 64 * kStatHeads; e += G) {   // heads fastest: contiguous rows of BTHD
    const int hh = e % kStatHeads, r = e / kStatHeads, n = 64 * blk + r, h = h0 + hh;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (h < a.H && n < a.N) {
      const int64_t at = (int64_t)b * a.ob + (int64_t)n * a.on + (int64_t)h * a.oh + 8 * c;
      x = *reinterpret_cast<const uint4*>(a.o + at);
      y = *reinterpret_cast<const uint4*>(a.d_o + at);
    }
    float f[8], d[8], s = 0.f;
    unpack8(x, f);
    unpack8(y, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(f[i], d[i], s);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (c == 0) sd[hh][r] = s;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 64 * kStatHeads; e += 256) {
    const int hh = e >> 6, r = e & 63, n = 64 * blk + r, h = h0 + hh;
    if (h >= a.H) continue;
    const int64_t bh = (int64_t)b * a.H + h, at = bh * 64 * a.nb + n;
    float nl = -INFINITY, nd = 0.f;
    if (n < a.N) {
      const float l = a.lse[bh * a.N + n];
      if (l > -INFINITY) { nl = -l * kLog2e; nd = -sd[hh][r]; }   // a row without keys: p = 0 everywhere
    }
    a.nlse[at] = nl;
    a.ndelta[at] = nd;
  }
}

// ---- the keys' plan: lists transposed --------------------------------------------------------------
// A CTA turns 32 key blocks' column of the query blocks' bitmaps (word m of every
// query block) into 32 rows of bits over the query blocks (32 x 32 transposes by
// ballot), then each warp lists two of its 16 key tiles.
constexpr int kTWarps = 8;

__global__ void __launch_bounds__(kTWarps * 32) tplan_kernel(const BwdArgs a) {
  __shared__ uint32_t T[32][kMaxKeyBlocks / 32 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = blockIdx.y;
  const int64_t bh = blockIdx.x;
  const int ntq = (a.nb + 1) / 2, qw = (a.nb + 31) / 32, pi = plan_ints(a.mask_words, a.nb);
  for (int w = warp; w < qw; w += kTWarps) {
    const int i = 32 * w + lane;
    uint32_t bits = 0u;
    if (i < a.nb) bits = (uint32_t)a.plan[(bh * ntq + (i >> 1)) * pi + 16 + (i & 1) * a.mask_words + m];
    uint32_t mine = 0u;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint32_t col = __ballot_sync(0xffffffffu, (bits >> e) & 1u);
      if (lane == e) mine = col;
    }
    T[lane][w] = mine;
  }
  __syncthreads();
  for (int t = warp; t < 16; t += kTWarps) {
    const int j0 = 32 * m + 2 * t;
    if (j0 >= a.nb) break;
    const uint32_t wa = lane < qw ? T[2 * t][lane] : 0u, wb = lane < qw ? T[2 * t + 1][lane] : 0u;
    const int cnt = __popc(wa | wb);
    int at = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    int* P = a.tplan + (bh * ntq + (j0 >> 1)) * tplan_ints(a.nb);
    if (lane == 31) P[0] = at;
    at -= cnt;
    for (uint32_t u = wa | wb; u; u &= u - 1) {
      const int e = __ffs(u) - 1;
      P[16 + at++] = (32 * lane + e) | (int)((wa >> e) & 1u) << 16 | (int)((wb >> e) & 1u) << 17;
    }
  }
}

// ---- the passes over block pairs ---------------------------------------------------------------------
// Both passes run on the tensor cores with 64-row blocks of the streamed side.
//
//   dq_kernel    a CTA owns 128 query rows (two consecutive query blocks, M = 128)
//                and walks the union of their lists, one 64-key block a step, then
//                64 centroids a step: S = Q K^T, dP = dO V^T, dQ += dS K.  Q and dO
//                sit in TMEM as A operands, so a step reads only K and V from
//                shared memory.
//   dkv_kernel   a CTA owns 128 key rows (two consecutive key blocks) or 128
//                centroids and walks the query blocks that take either, one a step,
//                transposed: S = K Q^T, dP = V dO^T, dV += P dO, dK += dS Q.  P and
//                dS come out with their rows in TMEM lanes, as an A operand needs.
//
// A half of the tile (64 of its 128 rows) that a step does not concern is left out
// of that step's MMAs by their row mask, and its softmax warps only pass the
// barriers on: the MMA takes the same time, but a masked row costs no power.  On
// lists whose steps mostly concern one half this is what sets the clock of long
// calls (a loop of such MMAs, 148 SMs at the 1 kW limit: 1.58 GHz unmasked, 1.85
// GHz with half the rows masked).  Accumulators start from zeros stored by the
// softmax threads, since a half's first step may not be the tile's.  Roles (12 warps): warp 0 loads the tiles with TMA, warps 1
// and 2 issue the MMAs, warps 4-11 are two softmax warpgroups that take alternate
// steps, one thread per TMEM lane.  A step's S and dP live in one of two 128-column
// TMEM stages; P (bf16) is written over S and dS over dP.  S and dP are handed over
// apart: S(t+2) is issued as soon as S(t) is read (dq) or dV has P(t) queued (dkv),
// so a group starts its next exponentials while dS(t)'s products and dP(t+2) run.
// An MMA that overwrites P or dS is issued by the warp that issued the one that
// reads it, and the pipe keeps their order.  Two issuing warps, because the waits
// between two batches cost the issuer 150 to 400 clocks, which the pipe's short
// queue does not cover: while one warp waits the other's MMAs run.  Every wait is bounded; on expiry the kernel raises
// SOL_ERR_TIMEOUT, drains what it issued and frees TMEM.
constexpr int kThreads = 384;            // 4 control warps + 2 softmax warpgroups
constexpr int kMaxWords = kMaxKeyBlocks / 32;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void cta_sync() {
  __syncwarp();
  __syncthreads();
}

// Shared-memory and TMEM layout.  Streamed tiles are 64 rows in 128-byte column
// chunks (SW128); the owned tiles of dkv_kernel are 128 rows.
template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kSChunk = 64 * 128;            // one column chunk of a streamed tile
  static constexpr int kSTile = 64 * D * 2;           // streamed tile
  static constexpr int kOChunk = 128 * 128;           // one column chunk of an owned tile
  static constexpr int kOTile = 128 * D * 2;
  static constexpr int kDqStages = 5, kKvStages = 4;  // pairs of streamed tiles in flight
  // TMEM columns.  dq: Q | dO | dQ | two stages; dkv: dV | dK | two stages.
  static constexpr uint32_t kStage = 256;             // stage g: S at kStage + 128 g, dP 64 columns on
  static constexpr uint32_t kQ = 0, kDo = 64, kDq = 128;
  static constexpr uint32_t kDv = 0, kDk = 128;
};

struct Bars {
  uint64_t own_full;                // owned tiles have landed (dkv: TMA) / are in TMEM (dq: softmax threads)
  uint64_t full[5], empty[5];       // ring of streamed tile pairs
  uint64_t s_full[2], dp_full[2];   // a step's S / dP are in TMEM
  uint64_t p_full[2], ds_full[2];   // S is read (dq) or P is in its place (dkv) / dS is in dP's place
  uint64_t own_tile;                // dq: Q and dO are in shared memory, on their way to TMEM
  uint64_t cent_ready;              // dq: the centroids' offsets are in shared memory
  uint64_t final_mma;
};

struct DqExtra {
  Bars bar;
  uint32_t tmem_base;
  int abort_flag, n_union, n_cent;
  uint32_t sel[2][kMaxWords];
  int list[kMaxKeyBlocks];                        // union entries: j | needA << 16 | needB << 17
  int clist[16];                                  // 64-centroid units: u | liveA << 16 | liveB << 17
  alignas(16) float cent_add[16][2][64];          // their offsets (log2 units), -inf where masked
  alignas(16) float tail_add[64];                 // 0 for valid rows of the last key block, -inf past N
};

template <int S>
struct KvExtra {
  Bars bar;
  uint32_t tmem_base;
  int abort_flag, n_steps;
  int list[kMaxKeyBlocks];                        // query blocks: i | needA << 16 | needB << 17
  uint32_t cword[128][4];                         // centroids: the step's exact-block bits of this tile
  alignas(16) float nl[S][64], nd[S][64];         // per ring stage: -lse, -delta of the query rows
  alignas(16) float gsum[2][2][128];              // exact: the two blocks' gk, gv
  float gb[128];
};

// TMA loads of one streamed pair (two 64-row tiles).
template <int D>
__device__ __forceinline__ void load_pair4(uint8_t* dst, const CUtensorMap* m1, const CUtensorMap* m2, int row, int h, int b,
                                           uint64_t* bar) {
  for (int c = 0; c < Cfg<D>::kChunks; ++c) {
    tma_load_4d(dst + c * Cfg<D>::kSChunk, m1, c * 64, h, row, b, bar);
    tma_load_4d(dst + Cfg<D>::kSTile + c * Cfg<D>::kSChunk, m2, c * 64, h, row, b, bar);
  }
}

// Rows of half hf that a step with this list entry leaves out of its MMAs.
__device__ __forceinline__ uint32_t off(int entry, int hf) { return (entry >> (16 + hf)) & 1 ? 0u : 0xffffffffu; }

// Position in the ring of streamed tiles: stage and the parity of its current load.
template <int S>
struct RingPos {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == S) { s = 0; ph ^= 1u; }
  }
};

// Streamed-tile descriptors: as B operand with the head dims as K (K-major), and
// with the rows as K (MN-major).
template <int D>
__device__ __forceinline__ uint64_t kmaj(uint64_t base, int kk, int chunk) {
  return base + (uint64_t)(((kk >> 2) * chunk + (kk & 3) * 32) >> 4);
}

// Row r's 32 values of columns 32c .. 32c+31, as bf16, into a SW128 tile of 128 rows
// (64-column chunks), the layout of the tile stores.
template <int D>
__device__ __forceinline__ void put_row(uint8_t* tile, int r, int c, const float* v) {
  uint8_t* row = tile + (c >> 1) * Cfg<D>::kOChunk + r * 128;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int at = 4 * (c & 1) + u;
    *reinterpret_cast<uint4*>(row + ((at ^ (r & 7)) << 4)) =
        make_uint4(pack_bf16(v[8 * u], v[8 * u + 1]), pack_bf16(v[8 * u + 2], v[8 * u + 3]),
                   pack_bf16(v[8 * u + 4], v[8 * u + 5]), pack_bf16(v[8 * u + 6], v[8 * u + 7]));
  }
}
// The same tile's halves to rows row0 .. row0 + 127 of a BTHD tensor (one thread).
template <int D>
__device__ __forceinline__ void store_rows(const CUtensorMap* m, const uint8_t* tile, int row0, int h, int b, int N) {
  for (int hf = 0; hf < 2; ++hf)
    if (row0 + 64 * hf < N)
      for (int c = 0; c < Cfg<D>::kChunks; ++c)
        tma_store_4d(m, c * 64, h, row0 + 64 * hf, b, tile + c * Cfg<D>::kOChunk + hf * (Cfg<D>::kOChunk / 2));
  tma_store_wait();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdo, const __grid_constant__ CUtensorMap mdq,
          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
          const __grid_constant__ CUtensorMap mkb, const __grid_constant__ CUtensorMap mvb, const BwdArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* own = ring + (C::kDqStages - 2) * 2 * C::kSTile;   // Q, dO at the start; the ring's last two stages after
  DqExtra& x = *reinterpret_cast<DqExtra*>(ring + C::kDqStages * 2 * C::kSTile);
  Bars& bar = x.bar;
  volatile int* abort_flag = &x.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ntq = (a.nb + 1) / 2, mw = a.mask_words;
  const int tq = blockIdx.x % ntq;
  const int64_t bh = blockIdx.x / ntq;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H), i0 = 2 * tq;

  if (tid == 0) {
    mbar_init(&bar.own_full, 256);
    mbar_init(&bar.own_tile, 1);
    mbar_init(&bar.cent_ready, 1);
    for (int s = 0; s < C::kDqStages; ++s) { mbar_init(&bar.full[s], 1); mbar_init(&bar.empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.s_full[s], 1); mbar_init(&bar.dp_full[s], 1);
      mbar_init(&bar.p_full[s], 4); mbar_init(&bar.ds_full[s], 4);
    }
    mbar_init(&bar.final_mma, 2);
    x.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // Q and dO rest in the ring's last two stages until the softmax threads have them
    // in TMEM (row-per-thread global loads instead held up the plan's by 3,000 clocks)
    mbar_expect_tx(&bar.own_tile, 2 * C::kOTile);
    for (int c = 0; c < C::kChunks; ++c)
      for (int hf = 0; hf < 2; ++hf) {
        tma_load_4d(own + c * C::kOChunk + hf * (C::kOChunk / 2), &mq, c * 64, h, 64 * (i0 + hf), b, &bar.own_tile);
        tma_load_4d(own + C::kOTile + c * C::kOChunk + hf * (C::kOChunk / 2), &mdo, c * 64, h, 64 * (i0 + hf), b, &bar.own_tile);
      }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(&x.tmem_base)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  const int n_tail = a.N - 64 * (a.nb - 1);
  if (tid < 64) x.tail_add[tid] = tid < n_tail ? 0.f : -INFINITY;
  {
    const int* P = a.plan + (bh * ntq + tq) * plan_ints(mw, a.nb);
    for (int e = tid; e < 2 * mw + a.nb; e += kThreads) {
      const int v = P[16 + e];
      if (e >= 2 * mw) x.list[e - 2 * mw] = v;
      else x.sel[e / mw][e % mw] = (uint32_t)v;
    }
    if (tid < 32) {   // 64-centroid units (two bitmap words) that either query block leaves to its centroids
      const uint32_t w0 = (uint32_t)P[12], w1 = (uint32_t)P[13];
      const bool l0 = tid < 16 && ((w0 >> (2 * tid)) & 3u), l1 = tid < 16 && ((w1 >> (2 * tid)) & 3u);
      const uint32_t any = __ballot_sync(0xffffffffu, l0 || l1);
      if (l0 || l1) x.clist[__popc(any & ((1u << tid) - 1u))] = tid | (int)l0 << 16 | (int)l1 << 17;
      if (tid == 0) { x.n_union = P[0]; x.n_cent = __popc(any); }
    }
  }
  fence_before();
  cta_sync();
  fence_after();
  const uint32_t tmem = x.tmem_base;
  const int n_union = x.n_union, T = n_union + x.n_cent;
  auto entry = [&](int t) { return *(t < n_union ? &x.list[t] : &x.clist[t - n_union]); };
  if (warp == 0) {
    if (lane == 0) {   // K and V (centroid) tiles
      int nl = 0;
      for (int t = 0; t < T; ++t) {
        const int s = t % C::kDqStages, n = t / C::kDqStages;
        if (!wait_bar(&bar.empty[s], (n & 1) ^ 1, abort_flag, a.status)) break;
        if (t == C::kDqStages - 2 && !wait_bar(&bar.own_full, 0, abort_flag, a.status)) break;
        uint8_t* dst = ring + s * 2 * C::kSTile;
        ++nl;
        mbar_expect_tx(&bar.full[s], 2 * C::kSTile);
        if (t < n_union) {
          load_pair4<D>(dst, &mk, &mv, 64 * (x.list[t] & 0xffff), h, b, &bar.full[s]);
        } else {
          const int row = 64 * (x.clist[t - n_union] & 0xffff);
          for (int c = 0; c < C::kChunks; ++c) {
            tma_load_3d(dst + c * C::kSChunk, &mkb, c * 64, row, (int)bh, &bar.full[s]);
            tma_load_3d(dst + C::kSTile + c * C::kSChunk, &mvb, c * 64, row, (int)bh, &bar.full[s]);
          }
        }
      }
      for (int s = 0; s < C::kDqStages; ++s) {   // every armed load has landed before the CTA may exit
        const int cnt = (nl + C::kDqStages - 1 - s) / C::kDqStages;
        if (cnt) drain_bar(&bar.full[s], (cnt - 1) & 1, a.status);
      }
      drain_bar(&bar.own_tile, 0, a.status);
    }
  } else if (warp == 1 || warp == 2) {
    constexpr uint32_t id_s = idesc_bf16(128, 64, 0, 0), id_g = idesc_bf16(128, D, 0, 1);
    constexpr uint64_t kStep = 2 * (C::kSTile >> 4);   // descriptor step per ring stage
    const uint64_t sd0 = sdesc(smem_u32(ring), 16, 1024), gd0 = sdesc(smem_u32(ring), C::kSChunk, 1024);
    RingPos<C::kDqStages> ld, use;   // the next step to start, the step to finish
    auto wait_ld = [&]() { return wait_bar(&bar.full[ld.s], ld.ph, abort_flag, a.status); };
    // A(TMEM) times a streamed tile: S from Q and K, dP from dO and V.  Half-way
    // through, the next step's barriers are looked at: the answer comes back while
    // the second half is issued, and a step whose barriers are already complete
    // (the usual case) starts without a wait.
    auto start = [&](uint32_t col, uint32_t own, uint64_t bd, uint64_t* done, int e, auto&& probe) {
      const uint64_t b0 = bd + ld.s * kStep;
      ld.next();
      bool r = false;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if (kk == D / 32) r = probe();
        mma_ts_m(tmem + col, tmem + own + kk * 8, kmaj<D>(b0, kk, C::kSChunk), id_s, kk > 0 ? 1u : 0u, off(e, 0), off(e, 1));
      }
      mma_commit_w(done);
      return r;
    };
    bool ok = __all_sync(0xffffffffu, wait_bar(&bar.own_full, 0, abort_flag, a.status));
    fence_after();
    if (warp == 1) {   // S(t+2) once S(t) is in the softmax threads' registers
      bool early = false;
      int e0 = T > 0 ? entry(0) : 0;
      for (int t = 0; t < T && ok; ++t) {
        const uint32_t par = ((t >> 1) & 1) ^ 1;
        if (!__all_sync(0xffffffffu, early)) {
          ok = wait_ld() && (t < 2 || wait_bar(&bar.p_full[t & 1], par, abort_flag, a.status));
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        fence_after();
        const int e = e0;
        early = start(C::kStage + 128 * (t & 1), C::kQ, sd0, &bar.s_full[t & 1], e, [&]() {
          const int u = t + 1;
          const bool l = mbar_test(&bar.full[ld.s], ld.ph);
          e0 = entry(min(u, T - 1));
          return (u < 2 || mbar_test(&bar.p_full[u & 1], ((u >> 1) & 1) ^ 1)) && l;
        });
      }
    } else {           // dQ += dS(t) K, then dP(t+2) over dS(t)
      for (int t = 0; t < 2 && t < T && ok; ++t)
        if ((ok = __all_sync(0xffffffffu, wait_ld())))
          start(C::kStage + 128 * t + 64, C::kDo, sd0 + (C::kSTile >> 4), &bar.dp_full[t], entry(t), []() { return false; });
      auto dq_mma = [&](int t, int e) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_m(tmem + C::kDq, tmem + C::kStage + 128 * (t & 1) + 64 + kk * 8, gd0 + use.s * kStep + (uint64_t)(kk * 2048 >> 4),
                   id_g, 1u, off(e, 0), off(e, 1));
        mma_commit_w(&bar.empty[use.s]);   // S(t), on which dS(t) depends, has read its tile too
        use.next();
      };
      bool early = false;
      int t = 0, e0 = T > 0 ? entry(0) : 0, e1 = T > 1 ? entry(1) : 0, e2 = T > 2 ? entry(2) : 0;   // steps t, t+1, t+2
      for (; t < T - 2 && ok; ++t) {   // (no condition around a batch: see the last two steps below)
        if (!__all_sync(0xffffffffu, early)) {
          ok = wait_ld() && wait_bar(&bar.ds_full[t & 1], (t >> 1) & 1, abort_flag, a.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        fence_after();
        dq_mma(t, e0);
        const int e = e2;
        e0 = e1;
        e1 = e2;
        early = start(C::kStage + 128 * (t & 1) + 64, C::kDo, sd0 + (C::kSTile >> 4), &bar.dp_full[t & 1], e, [&]() {
          const bool l = mbar_test(&bar.full[ld.s], ld.ph);
          e2 = entry(min(t + 3, T - 1));
          return mbar_test(&bar.ds_full[(t + 1) & 1], ((t + 1) >> 1) & 1) && l;
        });
      }
      for (; t < T && ok; ++t) {
        if (!(ok = __all_sync(0xffffffffu, wait_bar(&bar.ds_full[t & 1], (t >> 1) & 1, abort_flag, a.status)))) break;
        fence_after();
        dq_mma(t, e0);
        e0 = e1;
      }
    }
    mma_commit_w(&bar.final_mma);
    if (warp == 1) drain_bar(&bar.final_mma, 0, a.status);
  } else if (warp == 3) {   // the centroids' offsets, needed after the last listed block
    for (int e = lane; e < 128 * x.n_cent; e += 32) {
      const int slot = e >> 7, hf = (e >> 6) & 1, j = 64 * (x.clist[slot] & 0xffff) + (e & 63);
      const bool live = j < a.nb && i0 + hf < a.nb && !((x.sel[hf][j >> 5] >> (j & 31)) & 1u);
      x.cent_add[slot][hf][e & 63] = live ? a.cbias[bh * a.nb + j] * kLog2e : -INFINITY;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.cent_ready);
  } else if (warp >= 4) {
    const int g = (warp >> 2) - 1, sub = warp & 3, r = 32 * sub + lane, hf = r >> 6;
    const int row = 64 * i0 + r;
    bool ok = __all_sync(0xffffffffu, wait_bar(&bar.own_tile, 0, abort_flag, a.status));
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * sub) << 16);
    {   // group 0 puts Q, group 1 dO into TMEM
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 v = *reinterpret_cast<const uint4*>(own + g * C::kOTile + c * C::kOChunk + r * 128 + ((u ^ (r & 7)) << 4));
          w[4 * u] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
        }
        tmem_st32(lane_addr + (g == 0 ? C::kQ : C::kDo) + 32 * c, w);
#pragma unroll
        for (int u = 0; u < 32; ++u) w[u] = 0u;
        tmem_st32(lane_addr + C::kDq + g * (D / 2) + 32 * c, w);   // dQ starts from zero (its half)
      }
      tmem_wait_st();
      fence_async();   // the rows are read before the ring's loads overwrite them
      fence_before();
      mbar_arrive(&bar.own_full);
    }
    const bool in_range = i0 + hf < a.nb;
    const float nl = in_range ? a.nlse[bh * 64 * a.nb + row] : -INFINITY;
    const float nd = in_range ? a.ndelta[bh * 64 * a.nb + row] : 0.f;
    const float sl2 = a.scale * kLog2e;
    const uint64_t sl22 = f2pack(sl2, sl2), nl2 = f2pack(nl, nl), nd2 = f2pack(nd, nd);
    for (int t = g; t < T && ok; t += 2) {
      const float* add = nullptr;
      const int e = entry(t);
      const bool need = (e >> (16 + hf)) & 1;
      if (t < n_union) {
        if ((e & 0xffff) == a.nb - 1) add = x.tail_add;
      } else {
        if (t < n_union + 2) ok = __all_sync(0xffffffffu, wait_bar(&bar.cent_ready, 0, abort_flag, a.status));
        if (!ok) break;
        add = x.cent_add[t - n_union][hf];
      }
      ok = __all_sync(0xffffffffu, wait_bar(&bar.s_full[g], (t >> 1) & 1, abort_flag, a.status));
      if (!ok) break;
      fence_after();
      const uint32_t st = lane_addr + C::kStage + 128 * g;
      float p[64];
      if (need) {
        tmem_ld32(st, p);
        tmem_ld32(st + 32, p + 32);
        tmem_wait_ld();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[g]);
      if (need) {
        uint64_t mul2 = sl22;
        if (add) {   // centroids and the last key block: offsets first (log2 units)
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 o = reinterpret_cast<const float2*>(add)[c];
            f2unpack(ffma2(f2pack(p[2 * c], p[2 * c + 1]), sl22, f2pack(o.x, o.y)), p[2 * c], p[2 * c + 1]);
          }
          mul2 = f2pack(1.f, 1.f);
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float e0, e1;
          f2unpack(ffma2(f2pack(p[2 * c], p[2 * c + 1]), mul2, nl2), e0, e1);
          p[2 * c] = ex2(e0);
          p[2 * c + 1] = ex2(e1);
        }
      }
      ok = __all_sync(0xffffffffu, wait_bar(&bar.dp_full[g], (t >> 1) & 1, abort_flag, a.status));
      if (!ok) break;
      fence_after();
      if (need) {
        uint32_t pk[32];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float dp[32];
          tmem_ld32(st + 64 + 32 * hh, dp);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int k = 32 * hh + 2 * c;
            float d0, d1;
            f2unpack(fmul2(f2pack(p[k], p[k + 1]), fadd2(f2pack(dp[2 * c], dp[2 * c + 1]), nd2)), d0, d1);
            pk[16 * hh + c] = pack_bf16(d0, d1);
          }
        }
        tmem_st32(st + 64, pk);
        tmem_wait_st();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ds_full[g]);
    }
    if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bar.final_mma, 0, abort_flag, a.status));
    __syncwarp();
    if (ok) {
      fence_after();
      const bool anch = a.da && (row >= a.prefix || a.prefix == a.N);
      const float4* da = reinterpret_cast<const float4*>(a.da + bh * D);
      for (int c = g; c < D / 32; c += 2) {
        float v[32];
        __syncwarp();
        tmem_ld32(lane_addr + C::kDq + 32 * c, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= a.scale;
        if (anch) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 d = da[8 * c + e];
            v[4 * e] += d.x; v[4 * e + 1] += d.y; v[4 * e + 2] += d.z; v[4 * e + 3] += d.w;
          }
        }
        put_row<D>(ring, r, c, v);   // the ring is idle: every step is complete
      }
      fence_async();
    }
    bar_sync(1, 256);
    if (tid == 128 && ok && !*abort_flag) store_rows<D>(&mdq, ring, 64 * i0, h, b, a.N);
  }
  fence_before();
  cta_sync();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512));
  }
}

template <int D, bool kCent>
__global__ void __launch_bounds__(kThreads, 1)
dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdo,
           const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
           const __grid_constant__ CUtensorMap mgk, const __grid_constant__ CUtensorMap mgv, const BwdArgs a) {
  using C = Cfg<D>;
  constexpr int S = C::kKvStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* own = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = own + 2 * C::kOTile;
  KvExtra<S>& x = *reinterpret_cast<KvExtra<S>*>(ring + S * 2 * C::kSTile);
  Bars& bar = x.bar;
  volatile int* abort_flag = &x.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ntq = (a.nb + 1) / 2, mw = a.mask_words;
  const int tiles = kCent ? (a.nb + 127) / 128 : ntq;
  const int tk = blockIdx.x % tiles;
  const int64_t bh = (blockIdx.x / tiles) % ((int64_t)a.B * a.H), bhs = (int64_t)a.B * a.H;
  const int split = kCent ? (int)(blockIdx.x / tiles / bhs) : 0;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H);

  if (tid == 0) {
    mbar_init(&bar.cent_ready, 1);
    mbar_init(&bar.own_full, 1 + 256);   // the owned tiles' load, and the softmax threads' zeroed accumulators
    for (int s = 0; s < S; ++s) { mbar_init(&bar.full[s], 1); mbar_init(&bar.empty[s], 2); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.s_full[s], 1); mbar_init(&bar.dp_full[s], 1);
      mbar_init(&bar.p_full[s], 4); mbar_init(&bar.ds_full[s], 4);
    }
    mbar_init(&bar.final_mma, 2);
    x.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    mbar_expect_tx(&bar.own_full, 2 * C::kOTile);
    for (int c = 0; c < C::kChunks; ++c) {
      uint8_t* dk = own + c * C::kOChunk;
      uint8_t* dv = dk + C::kOTile;
      if (kCent) {
        for (int hf = 0; hf < 2; ++hf) {
          tma_load_3d(dk + hf * (C::kOChunk / 2), &mk, c * 64, 128 * tk + 64 * hf, (int)bh, &bar.own_full);
          tma_load_3d(dv + hf * (C::kOChunk / 2), &mv, c * 64, 128 * tk + 64 * hf, (int)bh, &bar.own_full);
        }
      } else {
        for (int hf = 0; hf < 2; ++hf) {
          tma_load_4d(dk + hf * (C::kOChunk / 2), &mk, c * 64, h, 128 * tk + 64 * hf, b, &bar.own_full);
          tma_load_4d(dv + hf * (C::kOChunk / 2), &mv, c * 64, h, 128 * tk + 64 * hf, b, &bar.own_full);
        }
      }
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(&x.tmem_base)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (kCent) {
    // the range's query blocks that leave any of the tile's key blocks to its centroid
    const int lo = (int)((int64_t)a.nb * split / a.splits), hi = (int)((int64_t)a.nb * (split + 1) / a.splits);
    if (warp == 2) {
      int n = 0;
      for (int i = lo; i < hi; i += 32) {
        uint32_t w[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (i + lane < hi) {
          const int* P = a.plan + (bh * ntq + ((i + lane) >> 1)) * plan_ints(mw, a.nb) + 16 + ((i + lane) & 1) * mw;
          for (int e = 0; e < 4; ++e) {
            const int base = 128 * tk + 32 * e;
            if (base >= a.nb) continue;
            w[e] = (uint32_t)P[4 * tk + e];
            if (a.nb - base < 32) w[e] |= ~((1u << (a.nb - base)) - 1u);
          }
        }
        const bool live = (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu;
        const uint32_t any = __ballot_sync(0xffffffffu, live);
        if (live) {
          const int at = n + __popc(any & ((1u << lane) - 1u));
          x.list[at] = i + lane;
          for (int e = 0; e < 4; ++e) x.cword[at][e] = w[e];
        }
        n += __popc(any);
      }
      if (lane == 0) x.n_steps = n;
    }
  } else {
    const int* P = a.tplan + (bh * ntq + tk) * tplan_ints(a.nb);
    for (int e = tid; e < a.nb; e += kThreads) x.list[e] = P[16 + e];
    if (tid == 0) x.n_steps = P[0];
  }
  fence_before();
  cta_sync();
  fence_after();
  const uint32_t tmem = x.tmem_base;
  const int T = x.n_steps;

  if (warp == 0) {
    if (lane == 0) {   // Q and dO tiles, -lse and -delta of their rows
      int nl = 0;
      for (int t = 0; t < T; ++t) {
        const int s = t % S, n = t / S, i = x.list[t] & 0xffff;
        if (!wait_bar(&bar.empty[s], (n & 1) ^ 1, abort_flag, a.status)) break;
        ++nl;
        mbar_expect_tx(&bar.full[s], 2 * C::kSTile + 512);
        load_pair4<D>(ring + s * 2 * C::kSTile, &mq, &mdo, 64 * i, h, b, &bar.full[s]);
        bulk_load(x.nl[s], a.nlse + (bh * a.nb + i) * 64, 256, &bar.full[s]);
        bulk_load(x.nd[s], a.ndelta + (bh * a.nb + i) * 64, 256, &bar.full[s]);
      }
      for (int s = 0; s < S; ++s) {
        const int cnt = (nl + S - 1 - s) / S;
        if (cnt) drain_bar(&bar.full[s], (cnt - 1) & 1, a.status);
      }
      drain_bar(&bar.own_full, 0, a.status);
    }
  } else if (warp == 1 || warp == 2) {
    // warp 1: dV += P(t) dO, then S(t+2) over P(t); warp 2: dK += dS(t) Q, then dP(t+2) over dS(t)
    constexpr uint32_t id_s = idesc_bf16(128, 64, 0, 0), id_g = idesc_bf16(128, D, 0, 1);
    constexpr uint64_t kStep = 2 * (C::kSTile >> 4);   // descriptor step per ring stage
    const bool first = warp == 1;
    const uint64_t tile = C::kSTile >> 4;
    const uint64_t od = sdesc(smem_u32(own), 16, 1024) + (first ? 0 : C::kOTile >> 4);            // K / V
    const uint64_t sd = sdesc(smem_u32(ring), 16, 1024) + (first ? 0 : tile);                       // Q / dO, K-major
    const uint64_t gd = sdesc(smem_u32(ring), C::kSChunk, 1024) + (first ? tile : 0);               // dO / Q, MN-major
    const uint32_t col = tmem + C::kStage + (first ? 0 : 64), acc = tmem + (first ? C::kDv : C::kDk);
    uint64_t* done = first ? bar.s_full : bar.dp_full;
    uint64_t* ready = first ? bar.p_full : bar.ds_full;
    RingPos<S> ld, use;
    auto wait_ld = [&]() { return wait_bar(&bar.full[ld.s], ld.ph, abort_flag, a.status); };
    auto start = [&](int g, int e) {
      const uint64_t b0 = sd + ld.s * kStep;
      ld.next();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_m(col + 128 * g, kmaj<D>(od, kk, C::kOChunk), kmaj<D>(b0, kk, C::kSChunk), id_s, kk > 0 ? 1u : 0u, off(e, 0), off(e, 1));
      mma_commit_w(&done[g]);
    };
    auto finish = [&](int t, int e) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ts_m(acc, col + 128 * (t & 1) + kk * 8, gd + use.s * kStep + (uint64_t)(kk * 2048 >> 4), id_g, 1u, off(e, 0), off(e, 1));
      mma_commit_w(&bar.empty[use.s]);
      use.next();
    };
    // a step's list entry (its halves); centroid tiles take every row
    auto entry = [&](int t) { return kCent ? 3 << 16 : x.list[t]; };
    bool ok = __all_sync(0xffffffffu, wait_bar(&bar.own_full, 0, abort_flag, a.status));
    fence_after();
    for (int t = 0; t < 2 && t < T && ok; ++t)
      if ((ok = __all_sync(0xffffffffu, wait_ld()))) start(t, entry(t));
    int t = 0, e0 = T > 0 ? entry(0) : 0, e1 = T > 1 ? entry(1) : 0, e2 = T > 2 ? entry(2) : 0;   // steps t, t+1, t+2
    for (; t < T - 2 && ok; ++t) {   // (no condition around a batch: see the last two steps below)
      ok = wait_ld() && wait_bar(&ready[t & 1], (t >> 1) & 1, abort_flag, a.status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      fence_after();
      finish(t, e0);
      const int e = e2;
      e0 = e1;
      e1 = e2;
      e2 = entry(min(t + 3, T - 1));
      start(t & 1, e);
    }
    for (; t < T && ok; ++t) {
      if (!(ok = __all_sync(0xffffffffu, wait_bar(&ready[t & 1], (t >> 1) & 1, abort_flag, a.status)))) break;
      fence_after();
      finish(t, e0);
      e0 = e1;
    }
    mma_commit_w(&bar.final_mma);
    if (first) drain_bar(&bar.final_mma, 0, a.status);
  } else if (!kCent && warp == 3) {
    // the two blocks' centroid gradients, summed over the query ranges in order (read after the last step)
    if (a.centroids) {
#pragma unroll
      for (int e = lane; e < D; e += 32) {   // float4s of [gk, gv][half][D]
        const int d = e % (D / 4), half = (e / (D / 4)) & 1, which = e / (D / 2), jj = 2 * tk + half;
        const float4* src = reinterpret_cast<const float4*>((which ? a.gv : a.gk) + (bh * a.nb + jj) * D) + d;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (jj < a.nb) {
#pragma unroll 8
          for (int s = 0; s < a.splits; ++s) {
            const float4 u = src[s * bhs * a.nb * (D / 4)];
            v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
          }
        }
        reinterpret_cast<float4*>(x.gsum[which][half])[d] = v;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.cent_ready);
  } else if (warp >= 4) {
    const int g = (warp >> 2) - 1, sub = warp & 3, r = 32 * sub + lane, hf = r >> 6;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * sub) << 16);
    const float sl2 = a.scale * kLog2e;
    const uint64_t sl22 = f2pack(sl2, sl2);
    const int j = kCent ? 128 * tk + r : 2 * tk + hf;   // this row's centroid / key block
    const float cadd = kCent && j < a.nb ? a.cbias[bh * a.nb + j] * kLog2e : -INFINITY;
    {   // accumulators from zero: group 0 dK, group 1 dV
      uint32_t z[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) z[c] = 0u;
      for (int c = 0; c < D / 32; ++c) tmem_st32(lane_addr + (g ? C::kDv : C::kDk) + 32 * c, z);
      tmem_wait_st();
      fence_before();
      mbar_arrive(&bar.own_full);
    }
    uint64_t gb2 = 0ull;   // kCent: the sums of ds of even and odd queries
    bool ok = true;
    for (int t = g; t < T && ok; t += 2) {
      const int rs = t % S;
      bool need = true;
      uint64_t add2 = 0ull;
      if (kCent) {
        const float v = (x.cword[t][sub] >> lane) & 1u ? -INFINITY : cadd;
        add2 = f2pack(v, v);
      } else {
        need = (x.list[t] >> (16 + hf)) & 1;
      }
      ok = __all_sync(0xffffffffu, wait_bar(&bar.full[rs], (t / S) & 1, abort_flag, a.status) &&
                                       wait_bar(&bar.s_full[g], (t >> 1) & 1, abort_flag, a.status));
      if (!ok) break;
      fence_after();
      const uint32_t st = lane_addr + C::kStage + 128 * g;
      float p[64];
      uint32_t pk[32];
      if (need) {
        tmem_ld32(st, p);
        tmem_ld32(st + 32, p + 32);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 l4 = reinterpret_cast<const float4*>(x.nl[rs])[c];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint64_t l2 = u ? f2pack(l4.z, l4.w) : f2pack(l4.x, l4.y);
            if (kCent) l2 = fadd2(l2, add2);
            const int k = 4 * c + 2 * u;
            float e0, e1;
            f2unpack(ffma2(f2pack(p[k], p[k + 1]), sl22, l2), e0, e1);
            p[k] = ex2(e0);
            p[k + 1] = ex2(e1);
            pk[2 * c + u] = pack_bf16(p[k], p[k + 1]);
          }
        }
        tmem_st32(st, pk);
        tmem_wait_st();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[g]);
      ok = __all_sync(0xffffffffu, wait_bar(&bar.dp_full[g], (t >> 1) & 1, abort_flag, a.status));
      if (!ok) break;
      fence_after();
      if (need) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float dp[32];
          tmem_ld32(st + 64 + 32 * hh, dp);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float4 d4 = reinterpret_cast<const float4*>(x.nd[rs])[8 * hh + c];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint64_t n2 = u ? f2pack(d4.z, d4.w) : f2pack(d4.x, d4.y);
              const int k = 4 * c + 2 * u;
              float d0, d1;
              const uint64_t d2 = fmul2(f2pack(p[32 * hh + k], p[32 * hh + k + 1]), fadd2(f2pack(dp[k], dp[k + 1]), n2));
              if (kCent) gb2 = fadd2(gb2, d2);
              f2unpack(d2, d0, d1);
              pk[16 * hh + 2 * c + u] = pack_bf16(d0, d1);
            }
          }
        }
        tmem_st32(st + 64, pk);
        tmem_wait_st();
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ds_full[g]);
    }
    float gbs, gb_odd;
    f2unpack(gb2, gbs, gb_odd);
    gbs += gb_odd;
    if (kCent && g == 0) x.gb[r] = gbs;
    if (ok) ok = __all_sync(0xffffffffu, wait_bar(&bar.final_mma, 0, abort_flag, a.status));
    if (!kCent && ok) ok = __all_sync(0xffffffffu, wait_bar(&bar.cent_ready, 0, abort_flag, a.status));
    __syncwarp();
    if (kCent) bar_sync(1, 256);   // x.gb
    // Group 0 brings out dk (gk), group 1 dv (gv), through the shared memory that the
    // tiles no longer need and tile stores.
    const float sc = g ? 1.f : a.scale;
    if (ok) {
      fence_after();
      if (kCent) {
        if (g == 1 && j < a.nb) a.gb_[(split * bhs + bh) * a.nb + j] = x.gb[r] + gbs;
        uint8_t* tile = own + g * (128 * D * 4);
        for (int c = 0; c < D / 32; ++c) {   // fp32 rows: 32-column chunks of 128 bytes, SW128
          float v[32];
          __syncwarp();
          tmem_ld32(lane_addr + (g ? C::kDv : C::kDk) + 32 * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<float4*>(tile + c * C::kOChunk + r * 128 + ((u ^ (r & 7)) << 4)) =
                make_float4(sc * v[4 * u], sc * v[4 * u + 1], sc * v[4 * u + 2], sc * v[4 * u + 3]);
        }
      } else {
        const int row = 128 * tk + r;
        const int64_t plane = bhs * 64 * a.nb, cr = bh * 64 * a.nb + row;
        float mul = 0.f, beta = 0.f;   // the row's share of its centroid's gradient, and of the anchor's
        if (row < a.N && a.centroids) {
          mul = a.mode ? a.coef[(g ? 2 : 0) * plane + cr] : 1.f / (float)min(64, a.N - 64 * j);
          if (a.mode && g == 0) beta = a.coef[plane + cr];
        }
        const float4* an = reinterpret_cast<const float4*>(a.anchor + bh * D);
        const float4* gs = reinterpret_cast<const float4*>(x.gsum[g][hf]);
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          __syncwarp();
          tmem_ld32(lane_addr + (g ? C::kDv : C::kDk) + 32 * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= sc;
          if (a.centroids) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 u = gs[8 * c + e];
              v[4 * e] = fmaf(mul, u.x, v[4 * e]); v[4 * e + 1] = fmaf(mul, u.y, v[4 * e + 1]);
              v[4 * e + 2] = fmaf(mul, u.z, v[4 * e + 2]); v[4 * e + 3] = fmaf(mul, u.w, v[4 * e + 3]);
            }
            if (a.mode && g == 0) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 u = an[8 * c + e];
                v[4 * e] = fmaf(beta, u.x, v[4 * e]); v[4 * e + 1] = fmaf(beta, u.y, v[4 * e + 1]);
                v[4 * e + 2] = fmaf(beta, u.z, v[4 * e + 2]); v[4 * e + 3] = fmaf(beta, u.w, v[4 * e + 3]);
              }
            }
          }
          put_row<D>(own + g * C::kOTile, r, c, v);
        }
      }
      fence_async();
    }
    bar_sync(2 + g, 128);
    if ((tid & 127) == 0 && ok && !*abort_flag) {
      if (kCent) {
        for (int c = 0; c < D / 32; ++c)
          tma_store_3d(g ? &mgv : &mgk, 32 * c, 128 * tk, (int)(split * bhs + bh), own + g * (128 * D * 4) + c * C::kOChunk);
        tma_store_wait();
      } else {
        store_rows<D>(g ? &mgv : &mgk, own + g * C::kOTile, 128 * tk, h, b, a.N);
      }
    }
  }
  fence_before();
  cta_sync();
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512));
  }
}

// ---- the pooling's gradient (modes 1, 2) -----------------------------------------------------------------
// Per key block: the anchor's weights over its rows again, the rows' coefficients
// (dk_t += alpha_t gk_j + beta_t a, dv_t += gamma_t gv_j) and the block's part of
// the anchor's gradient.  One CTA a block, its K rows held in registers (K read
// once, in mode 2 V too); HBM-bound.
template <int D>
__global__ void __launch_bounds__(256) pool_bwd_kernel(const BwdArgs a) {
  constexpr int LPR = D / 8, G = 256 / LPR, R = 64 / G;   // rows a lane group holds
  __shared__ float sw[64], sh[64], red[G][D], cst[4];
  __shared__ alignas(16) float sg[2][D];
  const int j = blockIdx.y;
  const int64_t bh = blockIdx.x, bhs = (int64_t)a.B * a.H;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H);
  const int c = threadIdx.x % LPR, g = threadIdx.x / LPR, n = min(64, a.N - 64 * j);
  uint4 kr[R], vr[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = g + G * i;
    const int64_t at = (int64_t)b * a.sb + (int64_t)(64 * j + r) * a.sn + (int64_t)h * a.sh + 8 * c;
    kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
    if (r < n) kr[i] = *reinterpret_cast<const uint4*>(a.k + at);
    if (r < n && a.mode == 2) vr[i] = *reinterpret_cast<const uint4*>(a.v + at);
  }
  // the block's gk and gv, summed over the query ranges in order (one dim of one of them a thread)
  for (int e = threadIdx.x; e < 2 * D; e += 256) {
    const float* src = (e < D ? a.gk : a.gv) + (bh * a.nb + j) * D + e % D;
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) v += src[s * bhs * a.nb * D];
    sg[e / D][e % D] = v;
  }
  float an[8], gk[8], gv[8], gb = 0.f;
#pragma unroll 8
  for (int s = 0; s < a.splits; ++s) gb += a.gb_[(s * bhs + bh) * a.nb + j];
#pragma unroll
  for (int i = 0; i < 8; ++i) an[i] = a.anchor[bh * D + 8 * c + i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) { gk[i] = sg[0][8 * c + i]; gv[i] = sg[1][8 * c + i]; }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float f[8], w[8], e = 0.f, hh = 0.f;
    unpack8(kr[i], f);
    unpack8(vr[i], w);
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      e = fmaf(an[d], f[d], e);
      hh = fmaf(gk[d], f[d], fmaf(gv[d], w[d], hh));
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
      e += __shfl_xor_sync(0xffffffffu, e, o);
      hh += __shfl_xor_sync(0xffffffffu, hh, o);
    }
    const int r = g + G * i;
    e *= a.scale;
    if (c == 0) { sw[r] = r < n ? e : -INFINITY; sh[r] = hh - gb * e; }
  }
  __syncthreads();
  if (threadIdx.x < 32) {   // softmax weights of the 64 rows and the weighted mean of h
    const int l = threadIdx.x;
    const float e0 = sw[l], e1 = sw[l + 32];
    float m = fmaxf(e0, e1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float x0 = expf(e0 - m), x1 = expf(e1 - m);
    float z = x0 + x1, hs = x0 * (l < n ? sh[l] : 0.f) + x1 * (l + 32 < n ? sh[l + 32] : 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, o);
      hs += __shfl_xor_sync(0xffffffffu, hs, o);
    }
    const float inv = 1.f / z;
    sw[l] = x0 * inv;
    sw[l + 32] = x1 * inv;
    if (l == 0) cst[0] = hs * inv;
  }
  __syncthreads();
  const float hbar = cst[0], rn = 1.f / n;
  const int64_t plane = bhs * 64 * a.nb, row0 = bh * 64 * a.nb + 64 * j;
  float da[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) da[i] = 0.f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = g + G * i;
    const float w = sw[r];
    const float beta = r >= n ? 0.f : a.mode == 2 ? a.scale * w * (sh[r] - hbar) : a.scale * gb * (w - rn);
    float f[8];
    unpack8(kr[i], f);
#pragma unroll
    for (int d = 0; d < 8; ++d) da[d] = fmaf(beta, f[d], da[d]);
    if (c == 0) {
      a.coef[row0 + r] = a.mode == 2 ? w : rn;
      a.coef[plane + row0 + r] = beta;
      a.coef[2 * plane + row0 + r] = a.mode == 2 ? w : rn;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[g][8 * c + i] = da[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int i = 0; i < G; ++i) s += red[i][threadIdx.x];
    a.da_part[(bh * a.nb + j) * D + threadIdx.x] = s;
  }
}

// The anchor's gradient over its row count: the blocks' parts added in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) anchor_bwd_kernel(const BwdArgs a) {
  constexpr int K = 1024 / D;
  __shared__ float red[K][D];
  const int64_t bh = blockIdx.x;
  const int d = threadIdx.x % D, s = threadIdx.x / D;
  float v = 0.f;
  for (int j = s; j < a.nb; j += K) v += a.da_part[(bh * a.nb + j) * D + d];
  red[s][d] = v;
  __syncthreads();
  if (s == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) v += red[i][d];
    a.da[bh * D + d] = v / (float)(a.prefix < a.N ? a.N - a.prefix : a.N);
  }
}

template <int D>
constexpr size_t dq_smem() { return 1024 + Cfg<D>::kDqStages * 2 * Cfg<D>::kSTile + sizeof(DqExtra); }
template <int D>
constexpr size_t dkv_smem() {
  return 1024 + 2 * Cfg<D>::kOTile + Cfg<D>::kKvStages * 2 * Cfg<D>::kSTile + sizeof(KvExtra<Cfg<D>::kKvStages>);
}
static_assert(2 * 128 * 128 * 4 <= 2 * Cfg<128>::kOTile + Cfg<128>::kKvStages * 2 * Cfg<128>::kSTile, "fp32 tiles");
static_assert(dq_smem<128>() <= 232448 && dkv_smem<128>() <= 232448, "shared memory");

// Once per device (so that launches stay free of attribute calls, e.g. inside a
// stream capture): opt in to the shared memory.
template <int D>
cudaError_t prepare() {
  static std::atomic<int> done[64];   // zero-initialised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire))) return e;
  const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(dq_kernel<D>, at, (int)dq_smem<D>())) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(dkv_kernel<D, false>, at, (int)dkv_smem<D>())) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(dkv_kernel<D, true>, at, (int)dkv_smem<D>())) != cudaSuccess) return e;
  if (dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_release);
  return cudaSuccess;
}

// 64-row boxes of a BTHD tensor (strides in elements) and of the [BH, nb, D] centroids.
bool map_rows(CUtensorMap* m, const __nv_bfloat16* p, const BwdArgs& a, int D, int64_t sb, int64_t sn, int64_t sh) {
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)a.H, (cuuint64_t)a.N, (cuuint64_t)a.B};
  const cuuint64_t str[3] = {(cuuint64_t)(a.H > 1 ? sh : D) * 2, (cuuint64_t)(a.N > 1 ? sn : D) * 2,
                             (cuuint64_t)(a.B > 1 ? sb : D) * 2};
  const cuuint32_t box[4] = {64, 1, 64, 1};
  return make_map(m, p, 4, dims, str, box, kSw128);
}
bool map_cent(CUtensorMap* m, const __nv_bfloat16* p, const BwdArgs& a, int D) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.nb, (cuuint64_t)a.B * a.H};
  const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.nb * D * 2};
  const cuuint32_t box[3] = {64, 64, 1};
  return make_map(m, p, 3, dims, str, box, kSw128);
}
// 128-row boxes of the centroid gradients' partial sums, fp32 [splits * BH, nb, D].
bool map_part(CUtensorMap* m, const float* p, const BwdArgs& a, int D) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.nb, (cuuint64_t)a.splits * a.B * a.H};
  const cuuint64_t str[2] = {(cuuint64_t)D * 4, (cuuint64_t)a.nb * D * 4};
  const cuuint32_t box[3] = {32, 128, 1};
  return make_map(m, p, 3, dims, str, box, kSw128, CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
}

template <int D>
cudaError_t launch(const BwdArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mdo, mkb, mvb, mdq, mdk, mdv, mgk, mgv;
  if (!map_rows(&mq, a.q, a, D, a.sb, a.sn, a.sh) || !map_rows(&mk, a.k, a, D, a.sb, a.sn, a.sh) ||
      !map_rows(&mv, a.v, a, D, a.sb, a.sn, a.sh) || !map_rows(&mdo, a.d_o, a, D, a.ob, a.on, a.oh) ||
      !map_cent(&mkb, a.kbar16, a, D) || !map_cent(&mvb, a.vbar16, a, D) || !map_rows(&mdq, a.dq, a, D, a.gb, a.gn, a.gh) ||
      !map_rows(&mdk, a.dk, a, D, a.gb, a.gn, a.gh) || !map_rows(&mdv, a.dv, a, D, a.gb, a.gn, a.gh) ||
      (a.centroids && (!map_part(&mgk, a.gk, a, D) || !map_part(&mgv, a.gv, a, D))))
    return cudaErrorInvalidValue;
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess) return e;
  stat_kernel<D><<<(unsigned)(a.B * a.nb) * ((a.H + kStatHeads - 1) / kStatHeads), 256, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  AttnArgs pa{};
  pa.row_ptr = a.row_ptr; pa.col_idx = a.col_idx; pa.plan = a.plan; pa.status = a.status;
  pa.B = a.B; pa.H = a.H; pa.N = a.N; pa.nqb = pa.nkb = a.nb; pa.centroids = a.centroids;
  if ((e = launch_plan(pa, st)) != cudaSuccess) return e;
  tplan_kernel<<<dim3(a.B * a.H, a.mask_words), kTWarps * 32, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const unsigned bh = (unsigned)(a.B * a.H), tiles = bh * ((a.nb + 1) / 2);
  if (a.centroids) {
    dkv_kernel<D, true><<<bh * ((a.nb + 127) / 128) * a.splits, kThreads, dkv_smem<D>(), st>>>(mq, mdo, mkb, mvb, mgk, mgv, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.centroids && a.mode) {
    pool_bwd_kernel<D><<<dim3(a.B * a.H, a.nb), 256, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    anchor_bwd_kernel<D><<<a.B * a.H, 1024, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  dq_kernel<D><<<tiles, kThreads, dq_smem<D>(), st>>>(mq, mdo, mdq, mk, mv, mkb, mvb, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  dkv_kernel<D, false><<<tiles, kThreads, dkv_smem<D>(), st>>>(mq, mdo, mk, mv, mdk, mdv, a);
  return cudaGetLastError();
}

}  // namespace

// Query ranges of the centroid pass.  By the length alone, so that a head's
// result does not depend on how many heads a call has; sixteen query blocks a
// range keep short sequences' CTAs many, eight ranges at most bound the partial
// sums' memory.
int attn_bwd_splits(int nb) { return nb <= 16 ? 1 : nb >= 128 ? 8 : (nb + 15) / 16; }

cudaError_t launch_attn_bwd(const BwdArgs& a, int D, cudaStream_t st) {
  return D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace sol
