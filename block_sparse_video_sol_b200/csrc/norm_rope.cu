// sol_qk_norm_rope and sol_qk_norm_rope_bwd: RMS norm of every query and key
// head and the position rotation, in one pass over Q and K, and its gradient.
//
// Forward, per row x of D dims with weight w:
//   r = 1 / sqrt(mean x^2 + eps),  y = x r w,  z = R y,
// R turning the first rot_dim dims in pairs (i, i + rot_dim/2) or (2i, 2i+1):
//   (a, b) -> (a cos - b sin, b cos + a sin).
// With p(i) the partner of dim i, z_i = r (x_i A_i + x_p(i) B_i), A_i = w_i cos
// and B_i = -/+ w_p(i) sin: A and B depend on the position alone, so a lane
// forms them once and uses them for every head of its item.
//
// Backward, with g = R^T dz and u = w g:
//   dx = r (u - x r^2 sum(u x) / D),  dw = sum over rows of g x r.
//
// Both are HBM-bound (each input element read once, each output written once).
// A row is D/8 lanes of 16 bytes.  A unit is one position of one of Q / K and
// kHeads heads per lane group of a warp; a warp keeps three or four of its units
// in flight with 16-byte asynchronous copies into shared memory, each lane reading
// back only what it copied (no barrier, and no registers held by loads in flight).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "ptx.cuh"   // cp.async

namespace sol {
namespace {

constexpr int kHeads = 4;       // heads per lane group of a unit
constexpr int kWarps = 4;       // warps per CTA
constexpr int kFwdStages = 4, kBwdStages = 3;   // units in flight per warp
constexpr int kFew = 3, kFwdMost = 6, kBwdMost = 4;   // CTAs an SM: see make_plan
constexpr int kSms = 148;
constexpr int kFwdSmem = kWarps * kFwdStages * kHeads * 512;
constexpr int kBwdSmem = kWarps * kBwdStages * 2 * kHeads * 512;

// Eight bf16 as four fp32 pairs, and back.
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(uint64_t f) {
  float lo, hi;
  f2unpack(f, lo, hi);
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const uint64_t* f) {
  return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
__device__ __forceinline__ float sum2(uint64_t f) {
  float lo, hi;
  f2unpack(f, lo, hi);
  return lo + hi;
}

// Eight weights from dim d0 (ones without a weight).
__device__ __forceinline__ void load_weight(const NormRopeArgs& a, int t, int d0, float* w) {
  if (!a.w[t]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (a.w_bf16) {
    uint64_t f[4];
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.w[t]) + d0), f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f2unpack(f[i], w[2 * i], w[2 * i + 1]);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.w[t]) + d0);
    const float4 x = p[0], y = p[1];
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
  }
}

// What a lane (chunk c of a row, dims 8c .. 8c+7) needs to turn its dims at one
// position: cos, the sine with the sign of the forward turn, and the lane
// chunk that holds the partners (its own with interleaved pairs or outside
// the turned dims).  There (c, s) = (1, 0); in the backward kernel with split pairs,
// where a dim is its own partner, halves of it, so that an infinity stays one.
struct Turn {
  float c[8], s[8];
  int partner;
};
template <bool kInter, bool kHalves = false>
__device__ __forceinline__ void load_turn(const NormRopeArgs& a, int b, int n, int c, Turn& t) {
  t.partner = c;
  if (8 * c >= 2 * a.half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { t.c[i] = kHalves ? 0.5f : 1.f; t.s[i] = kHalves ? -0.5f : 0.f; }
    return;
  }
  const int64_t row = (int64_t)b * a.tb + (int64_t)n * a.tn;
  if (kInter) {
    const float4 cs = *reinterpret_cast<const float4*>(a.cos + row + 4 * c);
    const float4 sn = *reinterpret_cast<const float4*>(a.sin + row + 4 * c);
    const float cv[4] = {cs.x, cs.y, cs.z, cs.w}, sv[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.c[2 * i] = t.c[2 * i + 1] = cv[i];
      t.s[2 * i] = -sv[i];
      t.s[2 * i + 1] = sv[i];
    }
  } else {
    const int hc = a.half / 8;
    const bool lo = c < hc;
    t.partner = lo ? c + hc : c - hc;
    const int64_t at = row + 8 * (lo ? c : c - hc);
    const float sg = lo ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 cs = *reinterpret_cast<const float4*>(a.cos + at + i);
      const float4 sn = *reinterpret_cast<const float4*>(a.sin + at + i);
      t.c[i] = cs.x; t.c[i + 1] = cs.y; t.c[i + 2] = cs.z; t.c[i + 3] = cs.w;
      t.s[i] = sg * sn.x; t.s[i + 1] = sg * sn.y; t.s[i + 2] = sg * sn.z; t.s[i + 3] = sg * sn.w;
    }
  }
}

// The partners' eight values of this lane's dims (packed bf16), by shuffle for
// split pairs and by swapping neighbours for interleaved ones.
template <bool kInter, int LPR>
__device__ __forceinline__ void partners(const uint4& u, int partner, uint64_t* f) {
  if (kInter) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2pack(__uint_as_float(w[i] & 0xffff0000u), __uint_as_float(w[i] << 16));
  } else {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, u.x, partner, LPR);
    o.y = __shfl_sync(0xffffffffu, u.y, partner, LPR);
    o.z = __shfl_sync(0xffffffffu, u.z, partner, LPR);
    o.w = __shfl_sync(0xffffffffu, u.w, partner, LPR);
    unpack8(o, f);
  }
}

// The work is cut into jobs (t, b, n, part): one of Q / K, one position, and all
// its head chunks (kHeads heads per lane group each; parts = 1) or one of them
// (parts = chunks).  Job w of the W warps' first round is warp w's, and every
// further one W jobs on, so that all warps read and write in one moving window
// (ranges of their own, one per warp, spread the accesses over every page of the
// tensors at once).  The job index is kept in digits and stepped by W's digits: no
// division per job.
struct Grid {
  int chunks, parts, N, B;
};
struct Pos {
  int p, n, b, t;      // the job
  int chunk, end;      // its next head chunk, and where they end
  int dp, dn, db, dt;  // W in the same digits
  __device__ __forceinline__ static void digits(int j, const Grid& g, int& p, int& n, int& b, int& t) {
    p = j % g.parts;
    j /= g.parts;
    n = j % g.N;
    j /= g.N;
    b = j % g.B;
    t = j / g.B;
  }
  __device__ __forceinline__ Pos(int w, int W, const Grid& g) {
    digits(w, g, p, n, b, t);
    digits(W, g, dp, dn, db, dt);
    open(g);
  }
  __device__ __forceinline__ void open(const Grid& g) {
    chunk = g.parts == 1 ? 0 : p;
    end = g.parts == 1 ? g.chunks : p + 1;
  }
  // to the next head chunk; true at a new job
  __device__ __forceinline__ bool next(const Grid& g) {
    if (++chunk < end) return false;
    p += dp; n += dn; b += db; t += dt;
    if (p >= g.parts) { p -= g.parts; ++n; }
    if (n >= g.N) { n -= g.N; ++b; }
    if (b >= g.B) { b -= g.B; ++t; }
    open(g);
    return true;
  }
};

template <int D, bool kInter, int kCtas>   // kCtas: CTAs an SM, for which registers are allotted
__global__ void __launch_bounds__(kWarps * 32, kCtas) norm_rope_kernel(const NormRopeArgs a, const Grid gr) {
  constexpr int LPR = D / 8, GPW = 32 / LPR, kUnitHeads = GPW * kHeads;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % LPR, g = lane / LPR;
  const int w = blockIdx.x * kWarps + warp, W = gridDim.x * kWarps;
  Pos in(w, W, gr);   // the tensor is the slowest digit: t = 2 is past the last job
  if (in.t >= 2) return;   // whole warp
  Pos at = in;
  uint4* ring = reinterpret_cast<uint4*>(smem) + (warp * kFwdStages * kHeads) * 32 + lane;
  auto row = [&](const __nv_bfloat16* x, const Pos& p, int64_t sb, int64_t sn, int64_t sh) {
    return x + (int64_t)p.b * sb + (int64_t)p.n * sn + (int64_t)g * sh + 8 * c;
  };
  const __nv_bfloat16* xr = row(a.x[in.t], in, a.sb, a.sn, a.sh);
  auto fetch = [&](int stage) {
    if (in.t < 2) {
      const __nv_bfloat16* x = xr + (int64_t)in.chunk * (kUnitHeads * a.sh);
#pragma unroll
      for (int e = 0; e < kHeads; ++e)
        if (in.chunk * kUnitHeads + GPW * e + g < a.H) cp_async16(ring + (stage * kHeads + e) * 32, x + e * (GPW * a.sh));
      if (in.next(gr) && in.t < 2) xr = row(a.x[in.t], in, a.sb, a.sn, a.sh);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kFwdStages; ++s) fetch(s);
  uint64_t A[4], Bp[4];
  __nv_bfloat16* yr = nullptr;
  int partner = c, stage = 0;
  bool fresh = true;   // a new position: its angles and weights
  while (at.t < 2) {
    if (fresh) {   // uniform over the warp
      Turn tr;
      load_turn<kInter>(a, at.b, at.n, c, tr);
      float wt[8];
      load_weight(a, at.t, 8 * c, wt);
#pragma unroll
      for (int e = 0; e < 4; ++e) A[e] = f2pack(wt[2 * e] * tr.c[2 * e], wt[2 * e + 1] * tr.c[2 * e + 1]);
      if (!kInter) load_weight(a, at.t, 8 * tr.partner, wt);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        Bp[e] = f2pack(wt[kInter ? 2 * e + 1 : 2 * e] * tr.s[2 * e], wt[kInter ? 2 * e : 2 * e + 1] * tr.s[2 * e + 1]);
      partner = tr.partner;
      yr = const_cast<__nv_bfloat16*>(row(a.y[at.t], at, a.ob, a.on, a.oh));
    }
    __nv_bfloat16* y = yr + (int64_t)at.chunk * (kUnitHeads * a.oh);
    const int h0 = at.chunk * kUnitHeads + g;
    cp_async_wait<kFwdStages - 1>();
    uint4 u[kHeads];
#pragma unroll
    for (int e = 0; e < kHeads; ++e) u[e] = ring[(stage * kHeads + e) * 32];
    fetch(stage);
    stage = stage + 1 == kFwdStages ? 0 : stage + 1;
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      uint64_t f[4], fp[4], s2 = 0ull;
      unpack8(u[k], f);
      partners<kInter, LPR>(u[k], partner, fp);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = ffma2(f[e], f[e], s2);
      float ss = sum2(s2);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const uint64_t r2 = f2pack(r, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = fmul2(r2, ffma2(f[e], A[e], fmul2(fp[e], Bp[e])));
      if (h0 + GPW * k < a.H) *reinterpret_cast<uint4*>(y + k * (GPW * a.oh)) = pack8(f);
    }
    fresh = at.next(gr);
  }
  cp_async_wait<0>();
}

// Backward.  The CTAs of one tensor (blockIdx.y) share its jobs in a fixed
// order, so each lane's weight-gradient sum has one too; the CTA's sums
// go to part[t][blockIdx.x][D] and dw_kernel adds them in CTA order.
template <int D, bool kInter>
__global__ void __launch_bounds__(kWarps * 32, kBwdMost) norm_rope_bwd_kernel(const NormRopeArgs a, const Grid gr) {
  constexpr int LPR = D / 8, GPW = 32 / LPR, kUnitHeads = GPW * kHeads;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[kWarps * GPW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % LPR, g = lane / LPR;
  const int t = blockIdx.y;
  const int wi = blockIdx.x * kWarps + warp, W = gridDim.x * kWarps;
  Pos in(wi, W, gr);   // one tensor's jobs: t = 1 is past the last
  Pos at = in;
  uint4* ring = reinterpret_cast<uint4*>(smem) + (warp * kBwdStages * 2 * kHeads) * 32 + lane;
  auto row = [&](const __nv_bfloat16* x, const Pos& p, int64_t sb, int64_t sn, int64_t sh) {
    return x + (int64_t)p.b * sb + (int64_t)p.n * sn + (int64_t)g * sh + 8 * c;
  };
  const __nv_bfloat16 *xr = row(a.x[t], in, a.sb, a.sn, a.sh), *zr = row(a.dz[t], in, a.ob, a.on, a.oh);
  auto fetch = [&](int stage) {
    if (in.t == 0) {
      const __nv_bfloat16* x = xr + (int64_t)in.chunk * (kUnitHeads * a.sh);
      const __nv_bfloat16* z = zr + (int64_t)in.chunk * (kUnitHeads * a.oh);
#pragma unroll
      for (int e = 0; e < kHeads; ++e)
        if (in.chunk * kUnitHeads + GPW * e + g < a.H) {
          cp_async16(ring + (stage * 2 * kHeads + 2 * e) * 32, x + e * (GPW * a.sh));
          cp_async16(ring + (stage * 2 * kHeads + 2 * e + 1) * 32, z + e * (GPW * a.oh));
        }
      if (in.next(gr) && in.t == 0) {
        xr = row(a.x[t], in, a.sb, a.sn, a.sh);
        zr = row(a.dz[t], in, a.ob, a.on, a.oh);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kBwdStages; ++s) fetch(s);
  uint64_t w[4], dw[4], cs[4], sn[4];
  {
    float wt[8];
    load_weight(a, t, 8 * c, wt);
#pragma unroll
    for (int i = 0; i < 4; ++i) { w[i] = f2pack(wt[2 * i], wt[2 * i + 1]); dw[i] = 0ull; cs[i] = sn[i] = 0ull; }
  }
  __nv_bfloat16* dxr = nullptr;
  int partner = c, stage = 0;
  bool fresh = true;
  while (at.t == 0) {
    if (fresh) {   // uniform over the warp
      Turn tr;
      load_turn<kInter, !kInter>(a, at.b, at.n, c, tr);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[e] = f2pack(tr.c[2 * e], tr.c[2 * e + 1]);
        sn[e] = f2pack(-tr.s[2 * e], -tr.s[2 * e + 1]);   // the turn back
      }
      partner = tr.partner;
      dxr = const_cast<__nv_bfloat16*>(row(a.y[t], at, a.gb, a.gn, a.gh));
    }
    __nv_bfloat16* dx = dxr + (int64_t)at.chunk * (kUnitHeads * a.gh);
    const int h0 = at.chunk * kUnitHeads + g;
    cp_async_wait<kBwdStages - 1>();
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const bool live = h0 + GPW * k < a.H;
      uint64_t f[4], z[4], zp[4], ss2 = 0ull, sx2 = 0ull;
      // past the last head: a row of ones (r = 1 / sqrt(0) would be infinite) whose dz = 0 adds nothing to dw
      uint4 u = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), v = make_uint4(0, 0, 0, 0);
      if (live) {
        u = ring[(stage * 2 * kHeads + 2 * k) * 32];
        v = ring[(stage * 2 * kHeads + 2 * k + 1) * 32];
      }
      unpack8(u, f);
      unpack8(v, z);
      partners<kInter, LPR>(v, partner, zp);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[e] = ffma2(z[e], cs[e], fmul2(zp[e], sn[e]));   // g = R^T dz
        ss2 = ffma2(f[e], f[e], ss2);
        zp[e] = fmul2(w[e], z[e]);                        // u = w g
        sx2 = ffma2(zp[e], f[e], sx2);
      }
      float ss = sum2(ss2), sx = sum2(sx2);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        sx += __shfl_xor_sync(0xffffffffu, sx, o);
      }
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float q = r * (-1.f / D) * (r * sx);   // (r sx is about |u|; r r overflows below |x| = 5e-20)
      const uint64_t r2 = f2pack(r, r), q2 = f2pack(q, q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dw[e] = ffma2(fmul2(z[e], r2), f[e], dw[e]);
        z[e] = fmul2(r2, ffma2(q2, f[e], zp[e]));
      }
      if (live) *reinterpret_cast<uint4*>(dx + k * (GPW * a.gh)) = pack8(z);
    }
    fetch(stage);
    stage = stage + 1 == kBwdStages ? 0 : stage + 1;
    fresh = at.next(gr);
  }
  cp_async_wait<0>();
  if (!a.dw[t]) return;   // uniform over the CTA
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo2, hi2;
    f2unpack(dw[i], lo2, hi2);
    red[warp * GPW + g][8 * c + 2 * i] = lo2;
    red[warp * GPW + g][8 * c + 2 * i + 1] = hi2;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int i = 0; i < kWarps * GPW; ++i) s += red[i][threadIdx.x];
    a.dw_part[((int64_t)t * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
  }
}

// dw[t] = sum of the CTAs' partial sums: 1024 / D threads a dim take every
// (1024 / D)-th partial, then a fixed-order sum over them.
template <int D>
__global__ void __launch_bounds__(1024) dw_kernel(const NormRopeArgs a, int parts) {
  constexpr int K = 1024 / D;
  __shared__ float red[K][D];
  const int t = blockIdx.x, d = threadIdx.x % D, s = threadIdx.x / D;
  if (!a.dw[t]) return;   // uniform over the CTA
  float v = 0.f;
  for (int i = s; i < parts; i += K) v += a.dw_part[((int64_t)t * parts + i) * D + d];
  red[s][d] = v;
  __syncthreads();
  if (s == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) v += red[i][d];
    a.dw[t][d] = v;
  }
}

// The jobs of `tensors` tensors and the CTAs for them (a tensor's share of `most`
// an SM).  Twelve warps an SM carry the copy rate where a position has several
// head chunks, and more lose some of it (N = 32768, H = 56, D = 128: forward 300 us
// with 12 warps, 343 with 16, 360 with 24; backward 437 / 493 us with 12 / 16).  With
// few heads a position's angles are most of the work and more warps win (H = 8:
// forward 82 us with 12 warps, 66 with 24, backward 103 / 90 us with 12 / 16; the
// two meet at 32 heads of 128 dims, four chunks; one box, the same buffers in every
// call: buffers that change cost 10 to 15% more).  A job is a whole position where every warp
// gets several, else a single head chunk (short calls: more warps at work).
struct Plan {
  Grid g;
  int ctas;
  bool few;
};
Plan make_plan(int B, int N, int H, int D, int tensors, int most) {
  const int heads = 32 / (D / 8) * kHeads, chunks = (H + heads - 1) / heads;
  const bool few = chunks >= 5;
  const int room = kSms * (few ? kFew : most) * tensors / 2;
  Plan r{Grid{chunks, 1, N, B}, 0, few};
  const int64_t positions = (int64_t)tensors * B * N;
  if (positions < 4 * (int64_t)room * kWarps) r.g.parts = chunks;
  r.ctas = (int)std::min<int64_t>((positions * r.g.parts + kWarps - 1) / kWarps, room);
  return r;
}

// Once per device: opt in to the shared memory.
template <int D, bool kInter>
cudaError_t prepare() {
  static std::atomic<int> done[64];   // zero-initialised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire))) return e;
  const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(norm_rope_kernel<D, kInter, kFew>, at, kFwdSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(norm_rope_kernel<D, kInter, kFwdMost>, at, kFwdSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(norm_rope_bwd_kernel<D, kInter>, at, kBwdSmem)) != cudaSuccess) return e;
  if (dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_release);
  return cudaSuccess;
}

template <int D, bool kInter>
cudaError_t fwd(const NormRopeArgs& a, cudaStream_t st) {
  cudaError_t e = prepare<D, kInter>();
  if (e != cudaSuccess) return e;
  const Plan r = make_plan(a.B, a.N, a.H, D, 2, kFwdMost);
  if (r.few) norm_rope_kernel<D, kInter, kFew><<<r.ctas, kWarps * 32, kFwdSmem, st>>>(a, r.g);
  else norm_rope_kernel<D, kInter, kFwdMost><<<r.ctas, kWarps * 32, kFwdSmem, st>>>(a, r.g);
  return cudaGetLastError();
}

template <int D, bool kInter>
cudaError_t bwd(const NormRopeArgs& a, cudaStream_t st) {
  cudaError_t e = prepare<D, kInter>();
  if (e != cudaSuccess) return e;
  const Plan r = make_plan(a.B, a.N, a.H, D, 1, kBwdMost);
  norm_rope_bwd_kernel<D, kInter><<<dim3(r.ctas, 2), kWarps * 32, kBwdSmem, st>>>(a, r.g);
  if ((e = cudaGetLastError()) != cudaSuccess || (!a.dw[0] && !a.dw[1])) return e;
  dw_kernel<D><<<2, 1024, 0, st>>>(a, r.ctas);
  return cudaGetLastError();
}

}  // namespace

int norm_rope_parts(int B, int N, int H, int D) { return make_plan(B, N, H, D, 1, kBwdMost).ctas; }

cudaError_t launch_norm_rope(const NormRopeArgs& a, int D, cudaStream_t st) {
  if (D == 128) return a.inter ? fwd<128, true>(a, st) : fwd<128, false>(a, st);
  return a.inter ? fwd<64, true>(a, st) : fwd<64, false>(a, st);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, int D, cudaStream_t st) {
  if (D == 128) return a.inter ? bwd<128, true>(a, st) : bwd<128, false>(a, st);
  return a.inter ? bwd<64, true>(a, st) : bwd<64, false>(a, st);
}

}  // namespace sol
