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
#include <math.h>

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

// ---- block gradients, fp32 ---------------------------------------------------------------------------
// The simple form of the three passes.  A CTA owns 64 rows (queries, keys or
// centroids) and streams 64-row blocks of the other side through shared memory,
// everything in fp32:
//   kind 0: own = (Q, dO) of query block i; streams its listed (K, V) blocks, then
//           the centroids; acc1 = dq / s
//   kind 1: own = (K, V) of key block j; streams the (Q, dO) blocks that list it;
//           acc1 = dk / s, acc2 = dv
//   kind 2: own = 64 centroids; streams the (Q, dO) blocks of one query range;
//           acc1 = gk / s, acc2 = gv, and gb
template <int D>
struct SimtSmem {
  float own1[64][D + 4], own2[64][D + 4], str1[64][D + 4], str2[64][D + 4];
  float P[64][65], dS[64][65];
  float nl[64], nd[64], add[64], gb[64];
};

template <int D>
__device__ void load_tile(float (*dst)[D + 4], const __nv_bfloat16* src, int64_t sn, int rows) {
  for (int e = threadIdx.x; e < 64 * D / 8; e += 256) {
    const int r = e / (D / 8), c = e % (D / 8);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (r < rows) u = *reinterpret_cast<const uint4*>(src + (int64_t)r * sn + 8 * c);
    unpack8(u, &dst[r][8 * c]);
  }
}

template <int D, int kind>
__global__ void __launch_bounds__(256) simt_kernel(const BwdArgs a) {
  extern __shared__ uint8_t raw[];
  SimtSmem<D>& x = *reinterpret_cast<SimtSmem<D>*>(raw);
  const int own = blockIdx.y;
  const int64_t bh = blockIdx.x;
  const int split = blockIdx.z;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H), tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int ntq = (a.nb + 1) / 2, mw = a.mask_words, pi = plan_ints(mw, a.nb);
  const float sl2 = a.scale * kLog2e;
  auto in = [&](const __nv_bfloat16* p, int n) { return p + (int64_t)b * a.sb + (int64_t)n * a.sn + (int64_t)h * a.sh; };
  auto out = [&](const __nv_bfloat16* p, int n) { return p + (int64_t)b * a.ob + (int64_t)n * a.on + (int64_t)h * a.oh; };
  auto grad = [&](__nv_bfloat16* p, int n) { return p + (int64_t)b * a.gb + (int64_t)n * a.gn + (int64_t)h * a.gh; };
  auto word = [&](int i, int w) {   // exact-block bits of query block i
    return (uint32_t)a.plan[(bh * ntq + (i >> 1)) * pi + 16 + (i & 1) * mw + w];
  };
  const int rows_own = min(64, a.N - 64 * own);
  const int crows = min(64, a.nb - 64 * own);   // kind 2: centroids of this tile
  if (kind == 0) {
    load_tile<D>(x.own1, in(a.q, 64 * own), a.sn, rows_own);
    load_tile<D>(x.own2, out(a.d_o, 64 * own), a.on, rows_own);
    if (tid < 64) { x.nl[tid] = a.nlse[bh * 64 * a.nb + 64 * own + tid]; x.nd[tid] = a.ndelta[bh * 64 * a.nb + 64 * own + tid]; }
  } else if (kind == 1) {
    load_tile<D>(x.own1, in(a.k, 64 * own), a.sn, rows_own);
    load_tile<D>(x.own2, in(a.v, 64 * own), a.sn, rows_own);
  } else {
    load_tile<D>(x.own1, a.kbar16 + (bh * a.nb + 64 * own) * D, D, crows);
    load_tile<D>(x.own2, a.vbar16 + (bh * a.nb + 64 * own) * D, D, crows);
    if (tid < 64) { x.add[tid] = tid < crows ? a.cbias[bh * a.nb + 64 * own + tid] * kLog2e : -INFINITY; x.gb[tid] = 0.f; }
  }
  float acc1[4][D / 16], acc2[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc1[i][j] = acc2[i][j] = 0.f;

  const int ctiles = kind == 0 && a.centroids ? (a.nb + 63) / 64 : 0;
  const int lo = kind == 2 ? (int)((int64_t)a.nb * split / a.splits) : 0;
  const int hi = kind == 2 ? (int)((int64_t)a.nb * (split + 1) / a.splits) : a.nb + ctiles;
  const int* tp = a.tplan + (bh * ntq + (own >> 1)) * tplan_ints(a.nb);
  const int steps = kind == 1 ? tp[0] : hi;
  for (int t = lo; t < steps; ++t) {
    int blk = t;
    bool cent = false;
    if (kind == 0) {
      cent = t >= a.nb;
      if (!cent && !((word(own, t >> 5) >> (t & 31)) & 1u)) continue;
      if (cent) blk = t - a.nb;
    } else if (kind == 1) {
      const int e = tp[16 + t];
      if (!((e >> (16 + (own & 1))) & 1)) continue;
      blk = e & 0xffff;
    }
    __syncthreads();
    if (kind == 0 && !cent) {
      load_tile<D>(x.str1, in(a.k, 64 * blk), a.sn, min(64, a.N - 64 * blk));
      load_tile<D>(x.str2, in(a.v, 64 * blk), a.sn, min(64, a.N - 64 * blk));
      if (tid < 64) x.add[tid] = 64 * blk + tid < a.N ? 0.f : -INFINITY;
    } else if (kind == 0) {
      const int cr = min(64, a.nb - 64 * blk);
      load_tile<D>(x.str1, a.kbar16 + (bh * a.nb + 64 * blk) * D, D, cr);
      load_tile<D>(x.str2, a.vbar16 + (bh * a.nb + 64 * blk) * D, D, cr);
      if (tid < 64) {
        const bool live = tid < cr && !((word(own, 2 * blk + (tid >> 5)) >> (tid & 31)) & 1u);
        x.add[tid] = live ? a.cbias[bh * a.nb + 64 * blk + tid] * kLog2e : -INFINITY;
      }
    } else {
      load_tile<D>(x.str1, in(a.q, 64 * blk), a.sn, min(64, a.N - 64 * blk));
      load_tile<D>(x.str2, out(a.d_o, 64 * blk), a.on, min(64, a.N - 64 * blk));
      if (tid < 64) { x.nl[tid] = a.nlse[bh * 64 * a.nb + 64 * blk + tid]; x.nd[tid] = a.ndelta[bh * 64 * a.nb + 64 * blk + tid]; }
    }
    __syncthreads();
    float S[4][4], dP[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = dP[i][j] = 0.f;
    for (int d = 0; d < D; ++d) {
      float u[4], w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = x.own1[4 * ty + i][d];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = x.str1[tx + 16 * j][d];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = fmaf(u[i], w[j], S[i][j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = x.own2[4 * ty + i][d];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = x.str2[tx + 16 * j][d];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dP[i][j] = fmaf(u[i], w[j], dP[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * ty + i, c = tx + 16 * j;
        float e = S[i][j] * sl2, nd;
        if (kind == 0) { e += x.add[c] + x.nl[r]; nd = x.nd[r]; }
        else { e += x.nl[c]; nd = x.nd[c]; }
        if (kind == 2) {
          const bool live = r < crows && !((word(blk, 2 * own + (r >> 5)) >> (r & 31)) & 1u);
          e = live ? e + x.add[r] : -INFINITY;
        }
        const float p = exp2f(e);
        x.P[r][c] = p;
        x.dS[r][c] = p * (dP[i][j] + nd);
      }
    __syncthreads();
    if (kind == 2 && tid < 64) {
      float s = 0.f;
      for (int c = 0; c < 64; ++c) s += x.dS[tid][c];
      x.gb[tid] += s;
    }
    for (int c = 0; c < 64; ++c) {
      float w1[D / 16], w2[D / 16];
#pragma unroll
      for (int j = 0; j < D / 16; ++j) { w1[j] = x.str1[c][tx + 16 * j]; if (kind != 0) w2[j] = x.str2[c][tx + 16 * j]; }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ds = x.dS[4 * ty + i][c], p = x.P[4 * ty + i][c];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          acc1[i][j] = fmaf(ds, w1[j], acc1[i][j]);
          if (kind != 0) acc2[i][j] = fmaf(p, w2[j], acc2[i][j]);
        }
      }
    }
  }
  __syncthreads();
  const int64_t bhs = (int64_t)a.B * a.H;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i, n = 64 * own + r;
    for (int j = 0; j < D / 16; ++j) {
      const int d = tx + 16 * j;
      float y1 = a.scale * acc1[i][j], y2 = acc2[i][j];
      if (kind == 0 && n < a.N) {
        if (a.da && (n >= a.prefix || a.prefix == a.N)) y1 += a.da[bh * D + d];
        grad(a.dq, n)[d] = __float2bfloat16(y1);
      } else if (kind == 1 && n < a.N) {
        if (a.centroids) {
          float gk = 0.f, gv = 0.f;
          for (int s = 0; s < a.splits; ++s) {
            gk += a.gk[((s * bhs + bh) * a.nb + own) * D + d];
            gv += a.gv[((s * bhs + bh) * a.nb + own) * D + d];
          }
          const int64_t at = bh * 64 * a.nb + n, plane = bhs * 64 * a.nb;
          const float al = a.mode ? a.coef[at] : 1.f / rows_own, ga = a.mode ? a.coef[2 * plane + at] : al;
          y1 += al * gk;
          y2 += ga * gv;
          if (a.mode) y1 += a.coef[plane + at] * a.anchor[bh * D + d];
        }
        grad(a.dk, n)[d] = __float2bfloat16(y1);
        grad(a.dv, n)[d] = __float2bfloat16(y2);
      } else if (kind == 2 && r < crows) {
        const int64_t at = ((split * bhs + bh) * a.nb + n) * D + d;
        a.gk[at] = y1;
        a.gv[at] = y2;
      }
    }
  }
  if (kind == 2 && tid < crows) a.gb_[(split * bhs + bh) * a.nb + 64 * own + tid] = x.gb[tid];
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
  const int j = blockIdx.y;
  const int64_t bh = blockIdx.x, bhs = (int64_t)a.B * a.H;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H);
  const int c = threadIdx.x % LPR, g = threadIdx.x / LPR, n = min(64, a.N - 64 * j);
  float an[8], gk[8], gv[8], gb = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) { an[i] = a.anchor[bh * D + 8 * c + i]; gk[i] = gv[i] = 0.f; }
  for (int s = 0; s < a.splits; ++s) {
    const int64_t at = (s * bhs + bh) * a.nb + j;
    gb += a.gb_[at];
#pragma unroll
    for (int i = 0; i < 8; ++i) { gk[i] += a.gk[at * D + 8 * c + i]; gv[i] += a.gv[at * D + 8 * c + i]; }
  }
  uint4 kr[R], vr[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = g + G * i;
    const int64_t at = (int64_t)b * a.sb + (int64_t)(64 * j + r) * a.sn + (int64_t)h * a.sh + 8 * c;
    kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
    if (r < n) kr[i] = *reinterpret_cast<const uint4*>(a.k + at);
    if (r < n && a.mode == 2) vr[i] = *reinterpret_cast<const uint4*>(a.v + at);
  }
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

template <int D, int kind>
cudaError_t launch_simt(const BwdArgs& a, cudaStream_t st) {
  const int smem = (int)sizeof(SimtSmem<D>);
  cudaError_t e = cudaFuncSetAttribute(simt_kernel<D, kind>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.B * a.H, kind == 2 ? (a.nb + 63) / 64 : a.nb, kind == 2 ? a.splits : 1);
  simt_kernel<D, kind><<<grid, 256, smem, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const BwdArgs& a, cudaStream_t st) {
  stat_kernel<D><<<(unsigned)(a.B * a.nb) * ((a.H + kStatHeads - 1) / kStatHeads), 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  AttnArgs pa{};
  pa.row_ptr = a.row_ptr; pa.col_idx = a.col_idx; pa.plan = a.plan; pa.status = a.status;
  pa.B = a.B; pa.H = a.H; pa.N = a.N; pa.nqb = pa.nkb = a.nb; pa.centroids = a.centroids;
  if ((e = launch_plan(pa, st)) != cudaSuccess) return e;
  tplan_kernel<<<dim3(a.B * a.H, a.mask_words), kTWarps * 32, 0, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.centroids && (e = launch_simt<D, 2>(a, st)) != cudaSuccess) return e;
  if (a.centroids && a.mode) {
    pool_bwd_kernel<D><<<dim3(a.B * a.H, a.nb), 256, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    anchor_bwd_kernel<D><<<a.B * a.H, 1024, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = launch_simt<D, 0>(a, st)) != cudaSuccess) return e;
  return launch_simt<D, 1>(a, st);
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
