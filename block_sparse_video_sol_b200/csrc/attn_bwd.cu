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

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "ptx.cuh"

namespace sol {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Fault-test build: the "dS ready" arrive of a tile's step g_drop_ds_arrive is withheld, so
// that the issuing warp's bounded wait for dS expires (sol_debug_drop_arrive).
#ifdef SOL_FAULT_TEST
__device__ int g_drop_ds_arrive = -1;
__device__ __forceinline__ bool withheld(int step) { return step == g_drop_ds_arrive; }
#else
__device__ __forceinline__ bool withheld(int) { return false; }
#endif

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
// once.  A CTA owns 16 rows of 8 heads, all their loads in flight together (64 rows
// in four rounds: 34.6 us against 27.4 at N = 4096, H = 56); D/8 lanes hold a row.
constexpr int kStatHeads = 8, kStatRows = 16;

template <int D>
__global__ void __launch_bounds__(256) stat_kernel(const BwdArgs a) {
  constexpr int LPR = D / 8, G = 256 / LPR;   // row groups of the CTA
  __shared__ float sd[kStatHeads][kStatRows + 1];
  const int hg = (a.H + kStatHeads - 1) / kStatHeads, per = 64 / kStatRows * a.nb;
  const int n0 = (int)(blockIdx.x / hg % per) * kStatRows, b = blockIdx.x / hg / per, h0 = (int)(blockIdx.x % hg) * kStatHeads;
  griddep_launch();   // the plans do not depend on this
  if (blockIdx.x == 0 && threadIdx.x < 4) a.counter[threadIdx.x] = 0;   // the later passes' tile counters
  const int c = threadIdx.x % LPR, g = threadIdx.x / LPR;
  const int heads = min(kStatHeads, a.H - h0);
#pragma unroll 8
  for (int e = g; e < kStatRows * kStatHeads; e += G) {   // heads fastest: contiguous rows of BTHD
    const int hh = e % heads, r = e / heads, n = n0 + r, h = h0 + hh;
    if (kStatRows * heads <= (e & ~(32 / LPR - 1))) break;   // uniform over the warp
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (r < kStatRows && n < a.N) {
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
    if (c == 0 && r < kStatRows) sd[hh][r] = s;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kStatRows * heads; e += 256) {
    const int hh = e / kStatRows, r = e % kStatRows, n = n0 + r, h = h0 + hh;
    const int64_t bh = (int64_t)b * a.H + h, at = (bh * a.nb + (n >> 6)) * 128 + (n & 63);
    float nl = -INFINITY, nd = 0.f;
    if (n < a.N) {
      const float l = a.lse[bh * a.N + n];
      if (l != -INFINITY) { nl = -l * kLog2e; nd = -sd[hh][r]; }   // a row without keys: p = 0 everywhere; NaN stays NaN
    }
    a.stat[at] = nl;
    a.stat[at + 64] = nd;
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
  griddep_launch();
  griddep_wait();
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
// softmax threads, since a half's first step may not be the tile's.
//
// Roles (12 warps): warp 0 loads the tiles with TMA, warps 1 and 2 issue the MMAs,
// warp 3 reads the next tile's plan and stores the results, warps 4-11 are two
// softmax warpgroups that take alternate steps, one thread per TMEM lane.
//
// What bounds a step (D = 128, both halves): dq_kernel's MMAs read A from TMEM and
// take 768 clocks, the step 950 (waits around the softmax); dkv_kernel's S and dP
// read both operands from shared memory, 48 clocks an MMA instead of 32, and a
// step's MMAs take 1,280, the step 1,290.  Around a tile's steps dq_kernel spends
// some 3 us and dkv_kernel 4.5 (first loads, last products, way out).  N = 8192,
// H = 56, 20% of the blocks: tensor pipe active 78% and 73% of the time.  Long calls
// are at the power limit (N = 32768: 1.65 GHz), where the energy of a step counts.
//
// A step's S and dP live in one of two 128-column TMEM stages; P (bf16) is written over S and dS over dP.  S and dP are handed over
// apart: S(t+2) is issued as soon as S(t) is read (dq) or dV has P(t) queued (dkv),
// so a group starts its next exponentials while dS(t)'s products and dP(t+2) run.
// An MMA that overwrites P or dS is issued by the warp that issued the one that
// reads it, and the pipe keeps their order.  Two issuing warps, because the waits
// between two batches cost the issuer 150 to 400 clocks, which the pipe's short
// queue does not cover: while one warp waits the other's MMAs run.  Every wait is
// bounded; on expiry the kernel raises SOL_ERR_TIMEOUT, drains what it issued and
// frees TMEM.
constexpr int kThreads = 384;            // 4 control warps + 2 softmax warpgroups
constexpr unsigned kSms = 148;
// A persistent CTA takes its next tile when this many steps of the present one are
// left to load: early enough for its plan, late enough that a CTA in a long tile
// does not hold a tile that another could run (N = 38247, H = 7, prefix 2407: 5.32 ms
// with 12 or 24, 5.35 with 4 or with a whole tile).
constexpr int kAhead = 12;

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

// Bounded wait in as few instructions as it takes: false on expiry (recorded in the
// abort flag, which the CTA reports at its end) or once another warp gave up.  These
// kernels' code has to stay in the instruction cache: a first pass over straight
// code costs some ten clocks an instruction (dq_kernel at N = 4096, H = 56: 184 us
// with wait_bar's loop in every place and unrolled ways in and out, 146 without).
__device__ __forceinline__ bool wait_for(uint64_t* b, uint32_t parity, volatile int* abort_flag) {
  for (uint32_t i = 0; !mbar_try(b, parity); ++i) {
    if (*abort_flag) return false;
    if (i >= kSpinLimit) { *abort_flag = 1; return false; }
  }
  return true;
}
// The same with its polling out of line.  Smaller still (dq_kernel above: 148 us
// against 161), but a call costs registers: dkv_kernel's softmax threads spill.
__device__ __noinline__ bool wait_poll(uint64_t* b, uint32_t parity, volatile int* abort_flag) {
  return wait_for(b, parity, abort_flag);
}
__device__ __forceinline__ bool wait_call(uint64_t* b, uint32_t parity, volatile int* abort_flag) {
  return mbar_try(b, parity) || wait_poll(b, parity, abort_flag);
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
  static constexpr int kStages = 4;                    // dkv: pairs of streamed tiles in flight
  static constexpr int kDqStages = 6;                  // dq: ring slots of one pair
  // TMEM columns.  dq: Q | dO | dQ | two stages; dkv: dV | dK | two stages.
  static constexpr uint32_t kStage = 256;             // stage g: S at kStage + 128 g, dP 64 columns on
  static constexpr uint32_t kQ = 0, kDo = 64, kDq = 128;
  static constexpr uint32_t kDv = 0, kDk = 128;
};

// What the roles of a persistent CTA read of a tile: its plan, in one of two
// buffers filled by the planning warp while the previous tile runs.
struct DqTile {
  int tile, n_union, n_cent;                      // tile < 0: no more
  int i0, bh, h, b;                               // its first query block and head
  int list[kMaxKeyBlocks];                        // union entries: j | needA << 16 | needB << 17
  int clist[16];                                  // 64-centroid units: u | liveA << 16 | liveB << 17
  alignas(16) float cent_add[16][2][64];          // their offsets (log2 units), -inf where masked
  __device__ __forceinline__ int steps() const { return n_union + n_cent; }
  __device__ __forceinline__ int entry(int t) const { return *(t < n_union ? &list[t] : &clist[t - n_union]); }
};
struct DqBars {
  uint64_t plan_full[2], plan_cent[2], plan_empty[2];   // a buffer's lists / centroid offsets are there; all roles are done
  uint64_t plan_go;                 // time to take the next tile
  uint64_t own_full[2], own_free[2];   // Q / dO are in TMEM; the tile's S / dP products have read them
  uint64_t full[6], empty[6];       // ring slots
  uint64_t s_full[2], dp_full[2];   // a step's S / dP are in TMEM
  uint64_t p_full[2], ds_full[2];   // S is read / dS is in dP's place
  uint64_t dq_full, dq_clear;       // the tile's dQ is complete / read and zeroed for the next tile
  uint64_t out_full;                // dQ is in its ring slot, to be stored
  uint64_t mma_done;                // the issuers' last commits, at the end
};
struct DqExtra {
  DqBars bar;
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float tail_add[64];                 // 0 for valid rows of the last key block, -inf past N
  DqTile info[2];
};

struct KvTile {
  int tile, n;                                    // tile < 0: no more
  int tk, bh, h, b, split;                        // its index in the head, its head, its query range (centroids)
  int list[kMaxKeyBlocks];                        // query blocks: i | needA << 16 | needB << 17
  uint32_t cword[128][4];                         // centroids: each step's exact-block bits of the tile
  alignas(16) float gsum[4 * 128];                // exact: [gk, gv][block][D] of the tile's two blocks
  float coef[3][128];                             // and the rows' alpha, beta, gamma
};
struct KvBars {
  uint64_t plan_full[2], plan_cent[2], plan_empty[2];   // a buffer's list / centroid sums are there; all roles are done
  uint64_t plan_go;                 // time to take the next tile
  uint64_t own_full[2], own_free[2];   // the tile's K / V are in shared memory; its S / dP products have read them
  uint64_t full[4], empty[4];       // ring slots
  uint64_t s_full[2], dp_full[2];   // a step's S / dP are in TMEM
  uint64_t p_full[2], ds_full[2];   // P is in S's place / dS is in dP's place
  uint64_t acc_full[2], acc_clear[2];   // dK / dV are complete; read and zeroed for the next tile
  uint64_t gb_full[2], out_full[2]; // group 0's offset sums of a tile are there; dK / dV are in their ring slots, to be stored
  uint64_t mma_done;                // the issuers' last commits, at the end
};
struct KvExtra {
  KvBars bar;
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float stat[4][128];                 // per ring slot: -lse and -delta of the query rows
  float gb[2][128];
  KvTile info[2];
};

// TMA load of a tile of a BTHD tensor: one instruction, since one takes its thread some
// 150 clocks and steps are short.  The maps have the 64-column chunks as a dimension
// of their own outside the rows, which is the tiles' layout.
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* m, int row, int h, int b, uint64_t* bar) {
  tma_load_5d(dst, m, 0, row, 0, h, b, bar);
}

// A plan's list (up to nb entries) into shared memory by one warp; returns its length.  The
// length and the first 64 entries are read at once: a tile of few steps waits for this.
__device__ __forceinline__ int copy_list(int* dst, const int* src, const int* length, int nb, int lane) {
  const int a = lane < nb ? src[lane] : 0, b = 32 + lane < nb ? src[32 + lane] : 0, n = *length;
  dst[lane] = a;
  dst[32 + lane] = b;
#pragma unroll 4
  for (int e = 64 + lane; e < n; e += 32) dst[e] = src[e];
  return n;
}

// Rows of half hf that a step with this list entry leaves out of its MMAs.
__device__ __forceinline__ uint32_t off(int entry, int hf) { return (entry >> (16 + hf)) & 1 ? 0u : 0xffffffffu; }

// The i-th of all heads' tiles (`per` a head) in the order in which they are run:
// every head's first `lead` tiles, the prefix's, whose lists are the longest, then
// the others, head by head (neighbours share K and V, or Q and dO, in L2).
__device__ __forceinline__ int tile_at(int i, int heads, int per, int lead) {
  if (i < heads * lead) return i / lead * per + i % lead;
  i -= heads * lead;
  return i / (per - lead) * per + lead + i % (per - lead);
}

// Position in the ring of streamed tiles: stage and the parity of its current load.
template <int S>
struct RingPos {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == S) { s = 0; ph ^= 1u; }
  }
  __device__ __forceinline__ void skip(int n) {
    s += n;
    ph ^= (uint32_t)(s / S) & 1u;
    s %= S;
  }
};

// Streamed-tile descriptors: as B operand with the head dims as K (K-major), and
// with the rows as K (MN-major).
template <int D>
__device__ __forceinline__ uint64_t kmaj(uint64_t base, int kk, int chunk) {
  return base + (uint64_t)(((kk >> 2) * chunk + (kk & 3) * 32) >> 4);
}

// Eight values to a 32-byte aligned address.
__device__ __forceinline__ void st_global32(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}
// Row r's 16 values of columns 16c .. 16c+15, as bf16, into a SW128 tile of 128 rows
// (64-column chunks), the layout of the tile stores.
template <int D>
__device__ __forceinline__ void put_row(uint8_t* tile, int r, int c, const float* v) {
  uint8_t* row = tile + (c >> 2) * Cfg<D>::kOChunk + r * 128;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int at = 2 * (c & 3) + u;
    *reinterpret_cast<uint4*>(row + ((at ^ (r & 7)) << 4)) =
        make_uint4(pack_bf16(v[8 * u], v[8 * u + 1]), pack_bf16(v[8 * u + 2], v[8 * u + 3]),
                   pack_bf16(v[8 * u + 4], v[8 * u + 5]), pack_bf16(v[8 * u + 6], v[8 * u + 7]));
  }
}
// The same tile to rows row0 .. row0 + 127 of a BTHD tensor (one thread; rows past N are not written).
__device__ __forceinline__ void store_rows(const CUtensorMap* m, const uint8_t* tile, int row0, int h, int b) {
  tma_store_5d(m, 0, row0, 0, h, b, tile);
  tma_store_commit();
}

// The queries' pass is persistent: a CTA takes tiles off a counter until none is
// left.  While a tile runs, its planning warp fetches the next one's lists; the
// loading warp runs ahead through one ring of 32 KB slots, which carry for each
// tile Q, dO, the steps' K and V and, last, dQ on its way out.  The next tile's
// Q and dO go into TMEM as soon as this one's products have read theirs, so its
// first S and dP are computed while dQ is brought out; only dQ's accumulator is
// waited for.  Steps, slots and barrier phases count on through the tiles.  (A CTA
// per tile spent 12,000 clocks around its steps: launch, plan, loads, the first
// products and the way out; now about 6,000.)
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdo, const __grid_constant__ CUtensorMap mdq,
          const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
          const __grid_constant__ CUtensorMap mkb, const __grid_constant__ CUtensorMap mvb, const BwdArgs a) {
  using C = Cfg<D>;
  constexpr int S = C::kDqStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  static_assert(C::kOTile == 2 * C::kSTile, "a slot holds a streamed pair or one owned tile");
  DqExtra& x = *reinterpret_cast<DqExtra*>(ring + S * 2 * C::kSTile);
  DqBars& bar = x.bar;
  volatile int* abort_flag = &x.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ntq = (a.nb + 1) / 2, mw = a.mask_words;

  griddep_launch();   // the next pass may take up idle SMs
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.plan_full[s], 1); mbar_init(&bar.plan_cent[s], 1); mbar_init(&bar.plan_empty[s], 1 + 2 + 8);
      mbar_init(&bar.s_full[s], 1); mbar_init(&bar.dp_full[s], 1);
      mbar_init(&bar.p_full[s], 4); mbar_init(&bar.ds_full[s], 4);
    }
    for (int s = 0; s < S; ++s) { mbar_init(&bar.full[s], 1); mbar_init(&bar.empty[s], 1); }
    for (int s = 0; s < 2; ++s) { mbar_init(&bar.own_full[s], 128); mbar_init(&bar.own_free[s], 1); }
    mbar_init(&bar.dq_full, 1);
    mbar_init(&bar.dq_clear, 256);
    mbar_init(&bar.out_full, 8);
    mbar_init(&bar.plan_go, 1);
    mbar_init(&bar.mma_done, 2);
    x.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(&x.tmem_base)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid < 64) x.tail_add[tid] = tid < a.N - 64 * (a.nb - 1) ? 0.f : -INFINITY;
  fence_before();
  cta_sync();
  fence_after();
  const uint32_t tmem = x.tmem_base;
  // every wait's outcome is made warp-uniform where a whole warp takes part
  auto wait = [&](uint64_t* b, uint32_t par) { return wait_call(b, par & 1u, abort_flag); };
  auto wait_w = [&](uint64_t* b, uint32_t par) { return __all_sync(0xffffffffu, wait(b, par)) != 0; };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      RingPos<S> pos;
      int slots = 0;
      bool ok = true;
      auto slot = [&]() { return ok = ok && wait(&bar.empty[pos.s], pos.ph ^ 1u); };
      auto next = [&]() { pos.next(); ++slots; };
      for (int k = 0;; ++k) {
        if (!(ok = ok && wait(&bar.plan_full[k & 1], k >> 1))) break;
        const DqTile& in = x.info[k & 1];
        if (in.tile < 0) break;
        const int h = in.h, b = in.b, T = in.steps();
        for (int o = 0; o < 2 && slot(); ++o, next()) {   // Q, dO
          mbar_expect_tx(&bar.full[pos.s], C::kOTile);
          load_rows(ring + pos.s * C::kOTile, o ? &mdo : &mq, 64 * in.i0, h, b, &bar.full[pos.s]);
        }
        const int go = max(0, T - kAhead);
        if (T == 0) mbar_arrive(&bar.plan_go);
        for (int t = 0; t < T && slot(); ++t, next()) {
          if (t == go) mbar_arrive(&bar.plan_go);
          uint8_t* dst = ring + pos.s * C::kOTile;
          uint64_t* full = &bar.full[pos.s];
          mbar_expect_tx(full, 2 * C::kSTile);
          const int row = 64 * (in.entry(t) & 0xffff);
          if (t < in.n_union) {
            load_rows(dst, &mk, row, h, b, full);
            load_rows(dst + C::kSTile, &mv, row, h, b, full);
          } else {
            tma_load_4d(dst, &mkb, 0, row, 0, in.bh, full);
            tma_load_4d(dst + C::kSTile, &mvb, 0, row, 0, in.bh, full);
          }
        }
        if (!slot()) break;   // the slot that carries dQ out: handed over empty
        mbar_arrive(&bar.full[pos.s]);
        next();
        mbar_arrive(&bar.plan_empty[k & 1]);
      }
      // every armed load has landed before the CTA may exit
      for (int i = max(0, slots - S); i < slots; ++i) drain_bar(&bar.full[i % S], (i / S) & 1, a.status);
    }
  } else if (warp == 1 || warp == 2) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t id_s = idesc_bf16(128, 64, 0, 0), id_g = idesc_bf16(128, D, 0, 1);
    constexpr uint64_t kStep = 2 * (C::kSTile >> 4);   // descriptor step per ring stage
    const uint64_t sd0 = sdesc(smem_u32(ring), 16, 1024), gd0 = sdesc(smem_u32(ring), C::kSChunk, 1024);
    RingPos<S> ld, use;   // the next step to start, the step to finish
    auto wait_ld = [&]() { return wait(&bar.full[ld.s], ld.ph); };
    // A(TMEM) times a streamed tile: S from Q and K, dP from dO and V.  Half-way
    // through, the next step's barriers are looked at: the answer comes back while
    // the second half is issued, and a step whose barriers are already complete
    // (the usual case) starts without a wait.
    auto start = [&](uint32_t col, uint32_t own_col, uint64_t bd, uint64_t* done, int e, auto&& probe) {
      const uint64_t b0 = bd + ld.s * kStep;
      ld.next();
      bool r = false;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if (kk == D / 32) r = probe();
        mma_ts_m(tmem + col, tmem + own_col + kk * 8, kmaj<D>(b0, kk, C::kSChunk), id_s, kk > 0 ? 1u : 0u, off(e, 0), off(e, 1));
      }
      mma_commit_w(done);
      return r;
    };
    bool ok = true;
    int base = 0;   // steps of the earlier tiles
    for (int k = 0; ok; ++k) {
      if (!(ok = wait_w(&bar.plan_full[k & 1], k >> 1))) break;
      const DqTile& in = x.info[k & 1];
      if (in.tile < 0) break;
      const int T = in.steps(), o = warp - 1;
      if (!(ok = wait_w(&bar.own_full[o], k))) break;
      fence_after();
      if (o) ld.next();
      if (lane == 0) mbar_arrive(&bar.empty[ld.s]);   // Q's / dO's slot
      ld.skip(2 - o);
      if (warp == 1) {   // S(u+2) once S(u) is in the softmax threads' registers (u counts through the tiles)
        bool early = false;
        int e0 = T > 0 ? in.entry(0) : 0;
        for (int u = base; u < base + T && ok; ++u) {
          const uint32_t par = ((u >> 1) & 1) ^ 1;
          if (!__all_sync(0xffffffffu, early)) {
            ok = wait_ld() && (u < 2 || wait(&bar.p_full[u & 1], par));
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
          }
          fence_after();
          const int e = e0;
          early = start(C::kStage + 128 * (u & 1), C::kQ, sd0, &bar.s_full[u & 1], e, [&]() {
            const bool l = mbar_test(&bar.full[ld.s], ld.ph);
            e0 = in.entry(min(u + 1 - base, T - 1));
            return (u + 1 < 2 || mbar_test(&bar.p_full[(u + 1) & 1], (((u + 1) >> 1) & 1) ^ 1)) && l;
          });
        }
        mma_commit_w(&bar.own_free[0]);
      } else {           // dQ += dS(u) K, then dP(u+2) over dS(u)
        for (int t = 0; t < 2 && t < T && ok; ++t)
          if ((ok = __all_sync(0xffffffffu, wait_ld())))
            start(C::kStage + 128 * ((base + t) & 1) + 64, C::kDo, sd0 + (C::kSTile >> 4), &bar.dp_full[(base + t) & 1], in.entry(t),
                  []() { return false; });
        use.skip(2);
        if (!(ok = ok && wait_w(&bar.dq_clear, k))) break;
        fence_after();
        auto dq_mma = [&](int u, int e) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts_m(tmem + C::kDq, tmem + C::kStage + 128 * (u & 1) + 64 + kk * 8, gd0 + use.s * kStep + (uint64_t)(kk * 2048 >> 4),
                     id_g, 1u, off(e, 0), off(e, 1));
          mma_commit_w(&bar.empty[use.s]);   // S(u), on which dS(u) depends, has read its tile too
          use.next();
        };
        bool early = false;
        int u = base, e0 = T > 0 ? in.entry(0) : 0, e1 = T > 1 ? in.entry(1) : 0, e2 = T > 2 ? in.entry(2) : 0;   // steps u, u+1, u+2
        for (; u < base + T - 2 && ok; ++u) {   // (no condition around a batch: see the last two steps below)
          if (!__all_sync(0xffffffffu, early)) {
            ok = wait_ld() && wait(&bar.ds_full[u & 1], u >> 1);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
          }
          fence_after();
          dq_mma(u, e0);
          const int e = e2;
          e0 = e1;
          e1 = e2;
          early = start(C::kStage + 128 * (u & 1) + 64, C::kDo, sd0 + (C::kSTile >> 4), &bar.dp_full[u & 1], e, [&]() {
            const bool l = mbar_test(&bar.full[ld.s], ld.ph);
            e2 = in.entry(min(u + 3 - base, T - 1));
            return mbar_test(&bar.ds_full[(u + 1) & 1], ((u + 1) >> 1) & 1) && l;
          });
        }
        mma_commit_w(&bar.own_free[1]);
        for (; u < base + T && ok; ++u) {
          if (!(ok = wait_w(&bar.ds_full[u & 1], u >> 1))) break;
          fence_after();
          dq_mma(u, e0);
          e0 = e1;
        }
        mma_commit_w(&bar.dq_full);
        use.next();   // dQ's slot
      }
      ld.next();      // dQ's slot
      base += T;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.plan_empty[k & 1]);
    }
    mma_commit_w(&bar.mma_done);
    if (warp == 1) drain_bar(&bar.mma_done, 0, a.status);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- plans, and dQ's way out
    const int total = a.B * a.H * ntq;
    auto plan = [&](int k) {   // the next tile off the counter into buffer k & 1
      DqTile& in = x.info[k & 1];
      int tile = 0;
      if (lane == 0) tile = atomicAdd(a.counter, 1);
      tile = __shfl_sync(0xffffffffu, tile, 0);
      if (tile >= total) {
        if (lane == 0) { in.tile = -1; mbar_arrive(&bar.plan_full[k & 1]); }
        return;
      }
      tile = tile_at(tile, a.B * a.H, ntq, min(ntq, (a.prefix + 127) / 128));
      const int* P = a.plan + (int64_t)tile * plan_ints(mw, a.nb);
      const int n = copy_list(in.list, P + 16 + 2 * mw, P, a.nb, lane);
      const uint32_t w0 = (uint32_t)P[12], w1 = (uint32_t)P[13];   // bitmap words that leave a block to its centroid
      const bool l0 = lane < 16 && ((w0 >> (2 * lane)) & 3u), l1 = lane < 16 && ((w1 >> (2 * lane)) & 3u);
      const uint32_t any = __ballot_sync(0xffffffffu, l0 || l1);
      if (l0 || l1) in.clist[__popc(any & ((1u << lane) - 1u))] = lane | (int)l0 << 16 | (int)l1 << 17;
      const int bh = tile / ntq, i0 = 2 * (tile % ntq), nc = __popc(any);
      if (lane == 0) {
        in.tile = tile; in.n_union = n; in.n_cent = nc;
        in.i0 = i0; in.bh = bh; in.h = bh % a.H; in.b = bh / a.H;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.plan_full[k & 1]);
      for (int s = 0; s < nc; ++s) {
        const int unit = in.clist[s] & 0xffff;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = lane + 32 * q, hf = e >> 6, j = 64 * unit + (e & 63);
          uint32_t bits = 0xffffffffu;   // (both loads at once)
          float v = 0.f;
          if (j < a.nb && i0 + hf < a.nb) {
            bits = (uint32_t)P[16 + hf * mw + (j >> 5)];
            v = a.cbias[(int64_t)bh * a.nb + j] * kLog2e;
          }
          in.cent_add[s][hf][e & 63] = (bits >> (j & 31)) & 1u ? -INFINITY : v;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.plan_cent[k & 1]);
    };
    RingPos<S> pos;
    plan(0);
    for (int k = 0;; ++k) {
      const DqTile& in = x.info[k & 1];
      if (in.tile < 0) break;
      if (!wait_w(&bar.plan_go, k) || (k >= 1 && !wait_w(&bar.plan_empty[(k + 1) & 1], ((k + 1) >> 1) - 1))) break;
      plan(k + 1);
      pos.skip(2 + in.steps());
      if (!wait_w(&bar.out_full, k)) break;
      if (lane == 0) {
        store_rows(&mdq, ring + pos.s * C::kOTile, 64 * in.i0, in.h, in.b);
        tma_store_wait<0>();
        mbar_arrive(&bar.empty[pos.s]);
      }
      pos.next();
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- softmax warpgroups
    const int g = (warp >> 2) - 1, sub = warp & 3, r = 32 * sub + lane, hf = r >> 6;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * sub) << 16);
    const float sl2 = a.scale * kLog2e;
    const uint64_t sl22 = f2pack(sl2, sl2);
    int base = 0;        // steps of the earlier tiles
    RingPos<S> pos;      // the tile's first slot
    float nl = 0.f, nd = 0.f;
    // A tile's rows: -lse and -delta, and Q (group 0) or dO (group 1) from its slot into TMEM
    auto take_own = [&](const DqTile& in) {
      const int i = in.i0 + hf;
      const float* st = a.stat + ((int64_t)in.bh * a.nb + i) * 128 + (r & 63);
      nl = i < a.nb ? st[0] : -INFINITY;
      nd = i < a.nb ? st[64] : 0.f;
      RingPos<S> p = pos;
      if (g) p.next();
      if (!wait_w(&bar.full[p.s], p.ph)) return false;
      const uint8_t* src = ring + p.s * C::kOTile + r * 128;
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + c * C::kOChunk + ((u ^ (r & 7)) << 4));
          w[4 * u] = v.x; w[4 * u + 1] = v.y; w[4 * u + 2] = v.z; w[4 * u + 3] = v.w;
        }
        tmem_st32(lane_addr + (g == 0 ? C::kQ : C::kDo) + 32 * c, w);
      }
      tmem_wait_st();
      fence_async();   // the rows are read before later loads overwrite the slot
      fence_before();
      mbar_arrive(&bar.own_full[g]);
      return true;
    };
    // dQ starts from zero: each group clears the columns that it brings out (16 at a time)
    auto clear = [&](int c) {
      uint32_t z[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) z[u] = 0u;
      tmem_st16(lane_addr + C::kDq + 16 * c, z);
    };
    bool ok = wait_w(&bar.plan_full[0], 0);
    if (ok && x.info[0].tile >= 0) {
      ok = take_own(x.info[0]);
#pragma unroll 1
      for (int c = g; c < D / 16; c += 2) clear(c);
      tmem_wait_st();
      fence_before();
      mbar_arrive(&bar.dq_clear);
    }
    for (int k = 0; ok; ++k) {
      const DqTile& in = x.info[k & 1];
      if (in.tile < 0) break;
      const int n_union = in.n_union, T = in.steps();
      const uint64_t nl2 = f2pack(nl, nl), nd2 = f2pack(nd, nd);
      for (int u = base + ((base + g) & 1); u < base + T; u += 2) {   // the steps of this group's stage
        const int t = u - base, e = in.entry(t);
        const bool need = (e >> (16 + hf)) & 1;
        const float* add = nullptr;
        if (t < n_union) {
          if ((e & 0xffff) == a.nb - 1) add = x.tail_add;
        } else {
          if (!(ok = wait_w(&bar.plan_cent[k & 1], k >> 1))) break;
          add = in.cent_add[t - n_union][hf];
        }
        if (!(ok = wait_w(&bar.s_full[g], u >> 1))) break;
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
        if (!(ok = wait_w(&bar.dp_full[g], u >> 1))) break;
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
              const int q = 32 * hh + 2 * c;
              float d0, d1;
              f2unpack(fmul2(f2pack(p[q], p[q + 1]), fadd2(f2pack(dp[2 * c], dp[2 * c + 1]), nd2)), d0, d1);
              pk[16 * hh + c] = pack_bf16(d0, d1);
            }
          }
          tmem_st32(st + 64, pk);
          tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0 && !withheld(u - base)) mbar_arrive(&bar.ds_full[g]);
      }
      if (!ok) break;
      base += T;
      RingPos<S> out = pos;
      out.skip(2 + T);
      pos = out;
      pos.next();
      // the next tile's rows, once this tile's products have read its own
      if (!(ok = wait_w(&bar.plan_full[(k + 1) & 1], (k + 1) >> 1))) break;
      const bool more = x.info[(k + 1) & 1].tile >= 0;
      if (more && !(ok = wait_w(&bar.own_free[g], k) && take_own(x.info[(k + 1) & 1]))) break;
      // dQ into its slot, from where the planning warp stores it
      if (!(ok = wait_w(&bar.dq_full, k) && wait_w(&bar.full[out.s], out.ph))) break;
      fence_after();
      const int row = 64 * in.i0 + r;
      const bool anch = a.da && (row >= a.prefix || a.prefix == a.N);
      if (a.da && k == 0) griddep_wait();   // launched early: the anchor's gradient (and the pass in front) has to be complete
      const float4* da = reinterpret_cast<const float4*>(a.da + (int64_t)in.bh * D);
#pragma unroll 1
      for (int c = g; c < D / 16; c += 2) {
        float v[16];
        tmem_ld16(lane_addr + C::kDq + 16 * c, v);
        tmem_wait_ld();
        clear(c);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] *= a.scale;
        if (anch) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 d = da[4 * c + e];
            v[4 * e] += d.x; v[4 * e + 1] += d.y; v[4 * e + 2] += d.z; v[4 * e + 3] += d.w;
          }
        }
        put_row<D>(ring + out.s * C::kOTile, r, c, v);
        __syncwarp();
      }
      tmem_wait_st();
      fence_async();
      fence_before();
      mbar_arrive(&bar.dq_clear);
      __syncwarp();
      if (lane == 0) { mbar_arrive(&bar.out_full); mbar_arrive(&bar.plan_empty[k & 1]); }
    }
  }
  fence_before();
  cta_sync();
  if (tid == 0 && x.abort_flag) raise_status(a.status, SOL_ERR_TIMEOUT);
  griddep_wait();   // not complete before the pass in front of it
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512));
  }
}

// The keys' pass (and, kCent, the centroids'), persistent like the queries': a tile
// is 128 key rows (128 centroids and one range of the query blocks), its K and V
// stay in shared memory, and the ring's slots carry the steps' Q and dO and then
// dV and dK on their way out, each stored as it is ready.  The next tile's K and V are loaded
// as soon as this tile's products have read theirs.
template <int D, bool kCent>
__global__ void __launch_bounds__(kThreads, 1)
dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdo,
           const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
           const __grid_constant__ CUtensorMap mdk, const __grid_constant__ CUtensorMap mdv, const BwdArgs a) {
  using C = Cfg<D>;
  constexpr int S = C::kStages, kOut = kCent ? 0 : 2;   // ring slots; those that carry a tile's results
  extern __shared__ uint8_t smem_raw[];
  uint8_t* own = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = own + 2 * C::kOTile;
  KvExtra& x = *reinterpret_cast<KvExtra*>(ring + S * C::kOTile);
  KvBars& bar = x.bar;
  volatile int* abort_flag = &x.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ntq = (a.nb + 1) / 2, mw = a.mask_words;
  const int tiles = kCent ? (a.nb + 127) / 128 : ntq;   // of one head (and range)
  const int bhs = a.B * a.H;

  if (kCent) griddep_wait();   // the plans and row statistics: the passes after this one rely on them without a wait
  griddep_launch();            // the next pass may take up idle SMs
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.plan_full[s], 1); mbar_init(&bar.plan_cent[s], 1); mbar_init(&bar.plan_empty[s], 1 + 2 + 8);
      mbar_init(&bar.own_full[s], 1); mbar_init(&bar.own_free[s], 1);
      mbar_init(&bar.s_full[s], 1); mbar_init(&bar.dp_full[s], 1);
      mbar_init(&bar.p_full[s], 4); mbar_init(&bar.ds_full[s], 4);
      mbar_init(&bar.acc_full[s], 1); mbar_init(&bar.acc_clear[s], 128);
    }
    for (int s = 0; s < S; ++s) { mbar_init(&bar.full[s], 1); mbar_init(&bar.empty[s], 2); }
    for (int s = 0; s < 2; ++s) { mbar_init(&bar.gb_full[s], 128); mbar_init(&bar.out_full[s], 4); }
    mbar_init(&bar.plan_go, 1);
    mbar_init(&bar.mma_done, 2);
    x.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_u32(&x.tmem_base)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  cta_sync();
  fence_after();
  const uint32_t tmem = x.tmem_base;
  auto wait = [&](uint64_t* b, uint32_t par) { return wait_for(b, par & 1u, abort_flag); };
  auto wait_w = [&](uint64_t* b, uint32_t par) { return __all_sync(0xffffffffu, wait(b, par)) != 0; };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      RingPos<S> pos;
      int slots = 0, owns[2] = {0, 0};   // armed loads: ring slots; K's, V's
      bool ok = true;
      auto slot = [&]() { return ok = ok && wait(&bar.empty[pos.s], pos.ph ^ 1u); };
      auto next = [&]() { pos.next(); ++slots; };
      for (int k = 0;; ++k) {
        if (!(ok = ok && wait(&bar.plan_full[k & 1], k >> 1))) break;
        const KvTile& in = x.info[k & 1];
        if (in.tile < 0) break;
        const int tk = in.tk, h = in.h, b = in.b, T = in.n;
#pragma unroll
        for (int o = 0; o < 2; ++o) {   // K, V, once the previous tile's products have read theirs
          if (k > 0 && !(ok = ok && wait(&bar.own_free[o], k - 1))) break;
          mbar_expect_tx(&bar.own_full[o], C::kOTile);
          if (kCent) tma_load_4d(own + o * C::kOTile, o ? &mv : &mk, 0, 128 * tk, 0, in.bh, &bar.own_full[o]);
          else load_rows(own + o * C::kOTile, o ? &mv : &mk, 128 * tk, h, b, &bar.own_full[o]);
          ++owns[o];   // (counted apart: V's wait may give up with K's load on its way)
        }
        if (!ok) break;
        const int go = max(0, T - kAhead);
        if (T == 0) mbar_arrive(&bar.plan_go);
        for (int t = 0; t < T && slot(); ++t, next()) {   // Q and dO, -lse and -delta of their rows
          if (t == go) mbar_arrive(&bar.plan_go);
          const int i = in.list[t] & 0xffff;
          mbar_expect_tx(&bar.full[pos.s], 2 * C::kSTile + 512);
          load_rows(ring + pos.s * C::kOTile, &mq, 64 * i, h, b, &bar.full[pos.s]);
          load_rows(ring + pos.s * C::kOTile + C::kSTile, &mdo, 64 * i, h, b, &bar.full[pos.s]);
          bulk_load(x.stat[pos.s], a.stat + ((int64_t)in.bh * a.nb + i) * 128, 512, &bar.full[pos.s]);
        }
        for (int o = 0; o < kOut && slot(); ++o, next()) mbar_arrive(&bar.full[pos.s]);   // handed over empty
        if (!ok) break;
        mbar_arrive(&bar.plan_empty[k & 1]);
      }
      // every armed load has landed before the CTA may exit
      for (int i = max(0, slots - S); i < slots; ++i) drain_bar(&bar.full[i % S], (i / S) & 1, a.status);
#pragma unroll
      for (int o = 0; o < 2; ++o)
        if (owns[o]) drain_bar(&bar.own_full[o], (owns[o] - 1) & 1, a.status);
    }
  } else if (warp == 1 || warp == 2) {
    // ---------------------------------------------------------------- products
    // warp 1: dV += P(u) dO, then S(u+2) over P(u); warp 2: dK += dS(u) Q, then dP(u+2) over dS(u)
    constexpr uint32_t id_s = idesc_bf16(128, 64, 0, 0), id_g = idesc_bf16(128, D, 0, 1);
    constexpr uint64_t kStep = 2 * (C::kSTile >> 4);   // descriptor step per ring slot
    const bool first = warp == 1;
    const int o = first ? 0 : 1;
    const uint64_t tile = C::kSTile >> 4;
    const uint64_t od = sdesc(smem_u32(own), 16, 1024) + (first ? 0 : C::kOTile >> 4);            // K / V
    const uint64_t sd = sdesc(smem_u32(ring), 16, 1024) + (first ? 0 : tile);                       // Q / dO, K-major
    const uint64_t gd = sdesc(smem_u32(ring), C::kSChunk, 1024) + (first ? tile : 0);               // dO / Q, MN-major
    const uint32_t col = tmem + C::kStage + (first ? 0 : 64), acc = tmem + (first ? C::kDv : C::kDk);
    uint64_t* done = first ? bar.s_full : bar.dp_full;
    uint64_t* ready = first ? bar.p_full : bar.ds_full;
    RingPos<S> ld, use;
    auto wait_ld = [&]() { return wait(&bar.full[ld.s], ld.ph); };
    auto start = [&](int g, int e) {
      const uint64_t b0 = sd + ld.s * kStep;
      ld.next();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_m(col + 128 * g, kmaj<D>(od, kk, C::kOChunk), kmaj<D>(b0, kk, C::kSChunk), id_s, kk > 0 ? 1u : 0u, off(e, 0), off(e, 1));
      mma_commit_w(&done[g]);
    };
    auto finish = [&](int g, int e) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ts_m(acc, col + 128 * g + kk * 8, gd + use.s * kStep + (uint64_t)(kk * 2048 >> 4), id_g, 1u, off(e, 0), off(e, 1));
      mma_commit_w(&bar.empty[use.s]);
      use.next();
    };
    bool ok = true;
    int base = 0;   // steps of the earlier tiles
    for (int k = 0; ok; ++k) {
      if (!(ok = wait_w(&bar.plan_full[k & 1], k >> 1))) break;
      const KvTile& in = x.info[k & 1];
      if (in.tile < 0) break;
      const int T = in.n;
      // a step's list entry (its halves); centroid tiles take every row
      auto entry = [&](int t) { return kCent ? 3 << 16 : in.list[t]; };
      if (!(ok = wait_w(&bar.own_full[o], k))) break;
      for (int t = 0; t < 2 && t < T && ok; ++t)
        if ((ok = __all_sync(0xffffffffu, wait_ld()))) start((base + t) & 1, entry(t));
      if (!(ok = ok && wait_w(&bar.acc_clear[1 - o], k))) break;
      fence_after();
      int u = base, e0 = T > 0 ? entry(0) : 0, e1 = T > 1 ? entry(1) : 0, e2 = T > 2 ? entry(2) : 0;   // steps u, u+1, u+2
      for (; u < base + T - 2 && ok; ++u) {   // (no condition around a batch: see the last two steps below)
        if (!(ok = wait_w(&ready[u & 1], u >> 1))) break;
        fence_after();
        finish(u & 1, e0);
        const int e = e2;
        e0 = e1;
        e1 = e2;
        e2 = entry(min(u + 3 - base, T - 1));
        if (!(ok = __all_sync(0xffffffffu, wait_ld()))) break;
        start(u & 1, e);
      }
      mma_commit_w(&bar.own_free[o]);
      for (; u < base + T && ok; ++u) {
        if (!(ok = wait_w(&ready[u & 1], u >> 1))) break;
        fence_after();
        finish(u & 1, e0);
        e0 = e1;
      }
      mma_commit_w(&bar.acc_full[1 - o]);
      ld.skip(kOut);
      use.skip(kOut);
      base += T;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.plan_empty[k & 1]);
    }
    mma_commit_w(&bar.mma_done);
    if (first) drain_bar(&bar.mma_done, 0, a.status);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- plans, and the results' way out
    const int total = bhs * tiles * (kCent ? a.splits : 1);
    auto plan = [&](int k) {   // the next tile off the counter into buffer k & 1
      KvTile& in = x.info[k & 1];
      int tile = 0;
      if (lane == 0) tile = atomicAdd(a.counter + (kCent ? 1 : 2), 1);
      tile = __shfl_sync(0xffffffffu, tile, 0);
      if (tile >= total) {
        if (lane == 0) { in.tile = -1; mbar_arrive(&bar.plan_full[k & 1]); }
        return;
      }
      if (!kCent) tile = tile_at(tile, a.B * a.H, tiles, min(tiles, (a.prefix + 127) / 128));
      const int tk = tile % tiles, at = tile / tiles, bh = kCent ? at % bhs : at, split = kCent ? at / bhs : 0;
      int n = 0;
      if (kCent) {   // the range's query blocks that leave any of the tile's key blocks to its centroid
        const int lo = (int)((int64_t)a.nb * split / a.splits), hi = (int)((int64_t)a.nb * (split + 1) / a.splits);
        for (int i = lo; i < hi; i += 32) {
          uint32_t w[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
          if (i + lane < hi) {
            const int* P = a.plan + ((int64_t)bh * ntq + ((i + lane) >> 1)) * plan_ints(mw, a.nb) + 16 + ((i + lane) & 1) * mw;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int first = 128 * tk + 32 * e;
              if (first >= a.nb) continue;
              w[e] = (uint32_t)P[4 * tk + e];
              if (a.nb - first < 32) w[e] |= ~((1u << (a.nb - first)) - 1u);
            }
          }
          const bool live = (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu;
          const uint32_t any = __ballot_sync(0xffffffffu, live);
          if (live) {
            const int at = n + __popc(any & ((1u << lane) - 1u));
            in.list[at] = i + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) in.cword[at][e] = w[e];
          }
          n += __popc(any);
        }
      } else {
        const int* P = a.tplan + (int64_t)tile * tplan_ints(a.nb);
        n = copy_list(in.list, P + 16, P, a.nb, lane);
      }
      if (lane == 0) {
        in.tile = tile; in.n = n;
        in.tk = tk; in.bh = bh; in.h = bh % a.H; in.b = bh / a.H; in.split = split;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.plan_full[k & 1]);
    };
    // The tile's centroid sums: wanted at its end only, so they are read after the
    // previous tile's results are stored (which the loads' ring waits for).
    auto plan_cent = [&](int k) {
      KvTile& in = x.info[k & 1];
      if (in.tile < 0) return;
      const int tk = in.tk;
      const int64_t bh = in.bh;
      if (!kCent && k == 0) griddep_wait();   // launched early: the centroids' pass has to be complete from here on
      if (!kCent && a.centroids) {   // the two blocks' centroid gradients, summed over the query ranges in order
        // (all loads of four ranges in flight together: tiles of few steps wait for this warp)
        float4 sum[D / 32];   // float4s e = lane + 32 i of [gk, gv][half][D]
#pragma unroll
        for (int i = 0; i < D / 32; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int s0 = 0; s0 < a.splits; s0 += 4) {
          float4 q[4][D / 32];
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const int e = lane + 32 * i, d = e % (D / 4), jj = 2 * tk + ((e / (D / 4)) & 1);
              q[s][i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (s0 + s < a.splits && jj < a.nb)
                q[s][i] = reinterpret_cast<const float4*>((e < D / 2 ? a.gk : a.gv) + (((s0 + s) * bhs + bh) * a.nb + jj) * D)[d];
            }
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              sum[i].x += q[s][i].x; sum[i].y += q[s][i].y; sum[i].z += q[s][i].z; sum[i].w += q[s][i].w;
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) reinterpret_cast<float4*>(in.gsum)[lane + 32 * i] = sum[i];
        float cf[4][3];   // the rows' coefficients alpha, beta, gamma
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = 128 * tk + 32 * q + lane, jj = row >> 6;
          const int64_t plane = (int64_t)bhs * 64 * a.nb, at = bh * 64 * a.nb + row;
          const float even = 1.f / (float)min(64, max(1, a.N - 64 * jj));
#pragma unroll
          for (int o = 0; o < 3; ++o) cf[q][o] = row >= a.N ? 0.f : a.mode ? a.coef[o * plane + at] : o == 1 ? 0.f : even;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int o = 0; o < 3; ++o) in.coef[o][32 * q + lane] = cf[q][o];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.plan_cent[k & 1]);
    };
    RingPos<S> pos;
    plan(0);
    plan_cent(0);
    for (int k = 0;; ++k) {
      const KvTile& in = x.info[k & 1];
      if (in.tile < 0) break;
      if (!wait_w(&bar.plan_go, k) || (k >= 1 && !wait_w(&bar.plan_empty[(k + 1) & 1], ((k + 1) >> 1) - 1))) break;
      plan(k + 1);
      if (!kCent) {
        pos.skip(in.n);
        // dV, then dK, each as it is ready; its slot is free (two arrivals) once the store has read it
        const int row0 = 128 * in.tk, h = in.h, b = in.b;
        RingPos<S> q = pos;
        bool ok = true;
        for (int o = 1; o >= 0 && (ok = wait_w(&bar.out_full[o], k)); --o) {
          if (lane == 0) store_rows(o ? &mdv : &mdk, ring + q.s * C::kOTile, row0, h, b);
          q.next();
        }
        if (!ok) break;
        if (lane == 0) {
          for (int o = 0; o < kOut; ++o) {
            if (o == 0) tma_store_wait<1>();
            else tma_store_wait<0>();
            RingPos<S> w = pos;
            w.skip(o);
            mbar_arrive(&bar.empty[w.s]);
            mbar_arrive(&bar.empty[w.s]);
          }
        }
        pos.skip(kOut);
        __syncwarp();
      }
      plan_cent(k + 1);
    }
    if (lane == 0) tma_store_wait<0>();
  } else {
    // ---------------------------------------------------------------- softmax warpgroups
    const int g = (warp >> 2) - 1, sub = warp & 3, r = 32 * sub + lane, hf = r >> 6;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * sub) << 16);
    const uint32_t acc = lane_addr + (g ? C::kDv : C::kDk);   // group 0 brings out dk (gk), group 1 dv (gv)
    const float sl2 = a.scale * kLog2e, sc = g ? 1.f : a.scale;
    const uint64_t sl22 = f2pack(sl2, sl2);
    auto clear = [&](int c) {   // accumulator columns 32c .. from zero
      uint32_t z[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) z[e] = 0u;
      tmem_st32(acc + 32 * c, z);
    };
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) clear(c);
    tmem_wait_st();
    fence_before();
    mbar_arrive(&bar.acc_clear[g]);
    bool ok = true;
    int base = 0;   // steps of the earlier tiles
    RingPos<S> pos;
    for (int k = 0; ok; ++k) {
      if (!(ok = wait_w(&bar.plan_full[k & 1], k >> 1))) break;
      const KvTile& in = x.info[k & 1];
      if (in.tile < 0) break;
      const int T = in.n, tk = in.tk;
      const int64_t bh = in.bh;
      const int j = kCent ? 128 * tk + r : 2 * tk + hf;   // this row's centroid / key block
      const float cadd = kCent && j < a.nb ? a.cbias[bh * a.nb + j] * kLog2e : -INFINITY;
      uint64_t gb2 = 0ull;   // kCent: the sums of ds of even and odd queries
      RingPos<S> at = pos;
      at.skip((base + g) & 1);
      for (int u = base + ((base + g) & 1); u < base + T; u += 2, at.skip(2)) {   // the steps of this group's stage
        const int rs = at.s;
        bool need = true;
        uint64_t add2 = 0ull;
        if (kCent) {
          const float v = (in.cword[u - base][sub] >> lane) & 1u ? -INFINITY : cadd;
          add2 = f2pack(v, v);
        } else {
          need = (in.list[u - base] >> (16 + hf)) & 1;
        }
        ok = __all_sync(0xffffffffu, wait(&bar.full[rs], at.ph) && wait(&bar.s_full[g], u >> 1));
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
            const float4 l4 = reinterpret_cast<const float4*>(x.stat[rs])[c];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint64_t l2 = q ? f2pack(l4.z, l4.w) : f2pack(l4.x, l4.y);
              if (kCent) l2 = fadd2(l2, add2);
              const int i = 4 * c + 2 * q;
              float e0, e1;
              f2unpack(ffma2(f2pack(p[i], p[i + 1]), sl22, l2), e0, e1);
              p[i] = ex2(e0);
              p[i + 1] = ex2(e1);
              pk[2 * c + q] = pack_bf16(p[i], p[i + 1]);
            }
          }
          tmem_st32(st, pk);
          tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[g]);
        if (!(ok = wait_w(&bar.dp_full[g], u >> 1))) break;
        fence_after();
        if (need) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float dp[32];
            tmem_ld32(st + 64 + 32 * hh, dp);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 d4 = reinterpret_cast<const float4*>(x.stat[rs] + 64)[8 * hh + c];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint64_t n2 = q ? f2pack(d4.z, d4.w) : f2pack(d4.x, d4.y);
                const int i = 4 * c + 2 * q;
                float d0, d1;
                const uint64_t d2 = fmul2(f2pack(p[32 * hh + i], p[32 * hh + i + 1]), fadd2(f2pack(dp[i], dp[i + 1]), n2));
                if (kCent) gb2 = fadd2(gb2, d2);
                f2unpack(d2, d0, d1);
                pk[16 * hh + 2 * c + q] = pack_bf16(d0, d1);
              }
            }
          }
          tmem_st32(st + 64, pk);
          tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0 && !withheld(u - base)) mbar_arrive(&bar.ds_full[g]);
      }
      if (!ok) break;
      pos.skip(T);
      base += T;
      // the tile's dk / dv into its ring slot, from where the planning warp stores it (gk / gv: to memory)
      if (!(ok = wait_w(&bar.acc_full[g], k) && wait_w(&bar.plan_cent[k & 1], k >> 1))) break;
      fence_after();
      RingPos<S> out = pos;
      out.skip((1 - g) * (kOut / 2));   // (dV is done first)
      pos.skip(kOut);
      if (kCent) {
        float gbs, odd;
        f2unpack(gb2, gbs, odd);
        gbs += odd;
        if (g == 0) {
          x.gb[k & 1][r] = gbs;
          mbar_arrive(&bar.gb_full[k & 1]);
        } else {
          if (!(ok = wait_w(&bar.gb_full[k & 1], k >> 1))) break;
          if (j < a.nb) a.gb_[((int64_t)in.split * bhs + bh) * a.nb + j] = x.gb[k & 1][r] + gbs;
        }
        // Straight to memory: a row's 32 columns are a line.  (Through ring slots and TMA stores
        // the next tile's first steps waited for these 128 KB, 12,000 clocks from tile to
        // tile; N = 32768, H = 56: 845 us against 800.)
        float* row = (g ? a.gv : a.gk) + (((int64_t)in.split * bhs + bh) * a.nb + j) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          tmem_ld32(acc + 32 * c, v);
          tmem_wait_ld();
          clear(c);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= sc;
          if (j < a.nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) st_global32(row + 32 * c + 8 * e, v + 8 * e);
          }
        }
      } else {
        if (!(ok = wait_w(&bar.full[out.s], out.ph))) break;
        // the row's share of its centroid's gradient, and of the anchor's
        const float mul = in.coef[g ? 2 : 0][r], beta = in.coef[1][r];
        const float4* an = reinterpret_cast<const float4*>(a.anchor + bh * D);
        const float4* gs = reinterpret_cast<const float4*>(in.gsum + (2 * g + hf) * D);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          tmem_ld32(acc + 32 * c, v);
          tmem_wait_ld();
          clear(c);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= sc;
          if (a.centroids) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 q = gs[8 * c + e];
              v[4 * e] = fmaf(mul, q.x, v[4 * e]); v[4 * e + 1] = fmaf(mul, q.y, v[4 * e + 1]);
              v[4 * e + 2] = fmaf(mul, q.z, v[4 * e + 2]); v[4 * e + 3] = fmaf(mul, q.w, v[4 * e + 3]);
            }
            if (a.mode && g == 0) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 q = an[8 * c + e];
                v[4 * e] = fmaf(beta, q.x, v[4 * e]); v[4 * e + 1] = fmaf(beta, q.y, v[4 * e + 1]);
                v[4 * e + 2] = fmaf(beta, q.z, v[4 * e + 2]); v[4 * e + 3] = fmaf(beta, q.w, v[4 * e + 3]);
              }
            }
          }
          put_row<D>(ring + out.s * C::kOTile, r, 2 * c, v);
          put_row<D>(ring + out.s * C::kOTile, r, 2 * c + 1, v + 16);
        }
      }
      tmem_wait_st();
      if (!kCent) fence_async();
      fence_before();
      mbar_arrive(&bar.acc_clear[g]);
      __syncwarp();
      if (lane == 0) {
        if (!kCent) mbar_arrive(&bar.out_full[g]);
        mbar_arrive(&bar.plan_empty[k & 1]);
      }
    }
  }
  fence_before();
  cta_sync();
  if (tid == 0 && x.abort_flag) raise_status(a.status, SOL_ERR_TIMEOUT);
  griddep_wait();   // not complete before the pass in front of it
  if (warp == 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512));
  }
}

// ---- the pooling's gradient (modes 1, 2) -----------------------------------------------------------------
// Per key block: the anchor's weights over its rows again, the rows' coefficients
// (dk_t += alpha_t gk_j + beta_t a, dv_t += gamma_t gv_j) and the block's part of
// the anchor's gradient.  One CTA a block, its K rows held in registers (K read
// once, in mode 2 V too).  N = 8192, H = 56, mode 2: 92 us, 3.2 TB/s (five or six
// CTAs an SM instead of four, by fewer registers or with the rows in shared memory,
// are no faster).
template <int D>
__global__ void __launch_bounds__(256, 4) pool_bwd_kernel(const BwdArgs a) {
  constexpr int LPR = D / 8, G = 256 / LPR, R = 64 / G;   // rows a lane group holds
  __shared__ float sw[64], sh[64], red[G][D], cst[4];
  __shared__ alignas(16) float sg[2][D];
  const int j = blockIdx.y;
  const int64_t bh = blockIdx.x, bhs = (int64_t)a.B * a.H;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H);
  const int c = threadIdx.x % LPR, g = threadIdx.x / LPR, n = min(64, a.N - 64 * j);
  griddep_launch();
  uint4 kr[R], vr[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = g + G * i;
    const int64_t at = (int64_t)b * a.sb + (int64_t)(64 * j + r) * a.sn + (int64_t)h * a.sh + 8 * c;
    kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
    if (r < n) kr[i] = *reinterpret_cast<const uint4*>(a.k + at);
    if (r < n && a.mode == 2) vr[i] = *reinterpret_cast<const uint4*>(a.v + at);
  }
  float an[8], gk[8], gv[8], gb = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 u = *reinterpret_cast<const float4*>(a.anchor + bh * D + 8 * c + i);
    an[i] = u.x; an[i + 1] = u.y; an[i + 2] = u.z; an[i + 3] = u.w;
  }
  griddep_wait();   // the centroids' pass (the rows and the anchor need nothing of it)
  // the block's gk and gv, summed over the query ranges in order (one dim of one of them a thread);
  // the eight ranges' loads and those of gb are in flight together
  {
    const int e = threadIdx.x;
    const float* src = (e < D ? a.gk : a.gv) + (bh * a.nb + j) * D + e % D;
    float part[8], gbp[8], v = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      part[s] = s < a.splits && e < 2 * D ? src[s * bhs * a.nb * D] : 0.f;
      gbp[s] = s < a.splits ? a.gb_[(s * bhs + bh) * a.nb + j] : 0.f;
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) { v += part[s]; gb += gbp[s]; }
    if (e < 2 * D) sg[e / D][e % D] = v;
  }
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
  griddep_launch();
  griddep_wait();
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
constexpr size_t dq_smem() { return 1024 + Cfg<D>::kDqStages * Cfg<D>::kOTile + sizeof(DqExtra); }
template <int D>
constexpr size_t dkv_smem() {
  return 1024 + (2 + Cfg<D>::kStages) * Cfg<D>::kOTile + sizeof(KvExtra);
}
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
bool map_rows(CUtensorMap* m, const __nv_bfloat16* p, const BwdArgs& a, int D, int64_t sb, int64_t sn, int64_t sh, int rows) {
  const cuuint64_t dims[5] = {64, (cuuint64_t)a.N, (cuuint64_t)D / 64, (cuuint64_t)a.H, (cuuint64_t)a.B};
  const cuuint64_t str[4] = {(cuuint64_t)(a.N > 1 ? sn : D) * 2, 128, (cuuint64_t)(a.H > 1 ? sh : D) * 2,
                             (cuuint64_t)(a.B > 1 ? sb : D) * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)D / 64, 1, 1};
  return make_map(m, p, 5, dims, str, box, kSw128);
}
bool map_cent(CUtensorMap* m, const __nv_bfloat16* p, const BwdArgs& a, int D, int rows) {
  const cuuint64_t dims[4] = {64, (cuuint64_t)a.nb, (cuuint64_t)D / 64, (cuuint64_t)a.B * a.H};
  const cuuint64_t str[3] = {(cuuint64_t)D * 2, 128, (cuuint64_t)a.nb * D * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)D / 64, 1};
  return make_map(m, p, 4, dims, str, box, kSw128);
}

template <int D>
cudaError_t launch(const BwdArgs& a, cudaStream_t st) {
  // 64-row boxes where a tile is streamed, 128-row ones (`o`) where it is owned or a result
  CUtensorMap mq, mk, mv, mdo, mkb, mvb, oq, ok, ov, odo, okb, ovb, mdq, mdk, mdv;
  auto in = [&](CUtensorMap* m, CUtensorMap* o, const __nv_bfloat16* p, int64_t sb, int64_t sn, int64_t sh) {
    return map_rows(m, p, a, D, sb, sn, sh, 64) && map_rows(o, p, a, D, sb, sn, sh, 128);
  };
  auto out = [&](CUtensorMap* m, const __nv_bfloat16* p) { return map_rows(m, p, a, D, a.gb, a.gn, a.gh, 128); };
  if (!in(&mq, &oq, a.q, a.sb, a.sn, a.sh) || !in(&mk, &ok, a.k, a.sb, a.sn, a.sh) || !in(&mv, &ov, a.v, a.sb, a.sn, a.sh) ||
      !in(&mdo, &odo, a.d_o, a.ob, a.on, a.oh) || !out(&mdq, a.dq) || !out(&mdk, a.dk) || !out(&mdv, a.dv) ||
      !map_cent(&mkb, a.kbar16, a, D, 64) || !map_cent(&mvb, a.vbar16, a, D, 64) ||
      (a.centroids && (!map_cent(&okb, a.kbar16, a, D, 128) || !map_cent(&ovb, a.vbar16, a, D, 128))))
    return cudaErrorInvalidValue;
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess) return e;
  // Every launch but the first may overlap the one before it.  Who waits for what:
  // the plans need nothing of stat_kernel; tplan_kernel waits for the plans, the
  // centroids' pass for both; behind that pass nothing starts before it has these.
  // Then the keys' pass waits only for the centroids' sums and the rows' coefficients,
  // and dQ's pass for the anchor's gradient (modes 1, 2), at their first tile's end.
  // Each kernel waits for the one before it before it is complete, so the chain
  // ends in order.
  // The keys' plan and the pooling start early only with few key blocks, a CTA of
  // the pooling each: more of them, waiting, keep the passes off the SMs (modes 1, 2;
  // 96 blocks, N = 1000: 41 us early, 47 not; 512, N = 4096: 133 early, 130 not; 7,168,
  // N = 8192: 1,935 early, 1,905 not).
  const bool few = (unsigned)(a.B * a.H) * a.nb <= 2 * kSms;
  e = launch_kernel(stat_kernel<D>, (unsigned)(a.B * a.nb) * (64 / kStatRows) * ((a.H + kStatHeads - 1) / kStatHeads), 256, 0, st, false, a);
  if (e != cudaSuccess) return e;
  AttnArgs pa{};
  pa.row_ptr = a.row_ptr; pa.col_idx = a.col_idx; pa.plan = a.plan; pa.status = a.status;
  pa.B = a.B; pa.H = a.H; pa.N = a.N; pa.nqb = pa.nkb = a.nb; pa.centroids = a.centroids;
  if ((e = launch_plan(pa, st, true)) != cudaSuccess) return e;
  const unsigned bh = (unsigned)(a.B * a.H), tiles = bh * ((a.nb + 1) / 2);
  if ((e = launch_kernel(tplan_kernel, dim3(bh, a.mask_words), kTWarps * 32, 0, st, few, a)) != cudaSuccess) return e;
  if (a.centroids) {
    const unsigned n = std::min(bh * ((a.nb + 127) / 128) * a.splits, kSms);
    e = launch_kernel(dkv_kernel<D, true>, n, kThreads, dkv_smem<D>(), st, true, mq, mdo, okb, ovb, mdk, mdv, a);
    if (e != cudaSuccess) return e;
    if (a.mode) {
      if ((e = launch_kernel(pool_bwd_kernel<D>, dim3(bh, a.nb), 256, 0, st, few, a)) != cudaSuccess) return e;
      if ((e = launch_kernel(anchor_bwd_kernel<D>, bh, 1024, 0, st, true, a)) != cudaSuccess) return e;
    }
  }
  // (the keys' pass, the longer one, first: N = 1000, B = 2, H = 3, mode 2: 41 us, 44 the other way round)
  e = launch_kernel(dkv_kernel<D, false>, std::min(tiles, kSms), kThreads, dkv_smem<D>(), st, a.centroids != 0, mq, mdo, ok, ov, mdk, mdv, a);
  if (e != cudaSuccess) return e;
  return launch_kernel(dq_kernel<D>, std::min(tiles, kSms), kThreads, dq_smem<D>(), st, true, oq, odo, mdq, mk, mv, mkb, mvb, a);
}

}  // namespace

// Query ranges of the centroid pass.  By the length alone, so that a head's
// result does not depend on how many heads a call has.  Up to 32 blocks, where few
// CTAs are at work and a call is as long as one range, four query blocks a range
// (N = 1024, H = 2, D = 64: 11.4 us against 19.7 in one range); beyond, sixteen, which
// is what a tile's way in and out costs (N = 4096, H = 56: 43 us against 61 with
// eight), and at most eight ranges for the partial sums' memory.
int attn_bwd_splits(int nb) { return nb <= 32 ? (nb + 3) / 4 : std::min(8, (nb + 15) / 16); }

#ifdef SOL_FAULT_TEST
cudaError_t set_drop_ds_arrive(int step) {
  return cudaMemcpyToSymbol(g_drop_ds_arrive, &step, sizeof(int));
}
#endif

cudaError_t launch_attn_bwd(const BwdArgs& a, int D, cudaStream_t st) {
  return D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace sol
