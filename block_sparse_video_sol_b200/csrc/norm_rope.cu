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
// A row is D/8 lanes of 16 bytes; a warp takes one position, one of Q / K and
// kHeads heads per lane group, whose loads are all in flight together.
#include "common.cuh"

namespace sol {
namespace {

constexpr int kHeads = 4;      // heads in flight per lane group
constexpr int kFwdWarps = 4;   // warps per CTA (forward)
constexpr int kBwdWarps = 8;   // warps per CTA (backward)

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Eight weights from dim d0 (ones without a weight).
__device__ __forceinline__ void load_weight(const NormRopeArgs& a, int t, int d0, float* w) {
  if (!a.w[t]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  } else if (a.w_bf16) {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.w[t]) + d0), w);
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
// the turned dims, where cos = 1 and sin = 0).
struct Turn {
  float c[8], s[8];
  int partner;
};
template <bool kInter>
__device__ __forceinline__ void load_turn(const NormRopeArgs& a, int b, int n, int c, Turn& t) {
  t.partner = c;
  if (8 * c >= 2 * a.half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { t.c[i] = 1.f; t.s[i] = 0.f; }
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
__device__ __forceinline__ void partners(const uint4& u, int partner, float* f) {
  if (kInter) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] & 0xffff0000u);
      f[2 * i + 1] = __uint_as_float(w[i] << 16);
    }
  } else {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, u.x, partner, LPR);
    o.y = __shfl_sync(0xffffffffu, u.y, partner, LPR);
    o.z = __shfl_sync(0xffffffffu, u.z, partner, LPR);
    o.w = __shfl_sync(0xffffffffu, u.w, partner, LPR);
    unpack8(o, f);
  }
}

// Item it of (b, n, head chunk), chunks fastest, so neighbouring warps read neighbouring heads.
struct Item {
  int b, n, h0;
};
__device__ __forceinline__ Item item_at(const NormRopeArgs& a, int64_t it, int heads) {
  Item r;
  const int chunks = (a.H + heads - 1) / heads;
  r.h0 = (int)(it % chunks) * heads;
  it /= chunks;
  r.n = (int)(it % a.N);
  r.b = (int)(it / a.N);
  return r;
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kFwdWarps * 32) norm_rope_kernel(const NormRopeArgs a, int64_t items) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const int lane = threadIdx.x & 31, c = lane % LPR, g = lane / LPR;
  const int t = blockIdx.y;   // 0: Q, 1: K
  const int64_t it = (int64_t)blockIdx.x * kFwdWarps + (threadIdx.x >> 5);
  if (it >= items) return;    // whole warp
  const Item m = item_at(a, it, GPW * kHeads);
  const __nv_bfloat16* x = a.x[t] + (int64_t)m.b * a.sb + (int64_t)m.n * a.sn + 8 * c;
  __nv_bfloat16* y = a.y[t] + (int64_t)m.b * a.ob + (int64_t)m.n * a.on + 8 * c;
  uint4 u[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = m.h0 + GPW * i + g;
    u[i] = make_uint4(0, 0, 0, 0);
    if (h < a.H) u[i] = *reinterpret_cast<const uint4*>(x + (int64_t)h * a.sh);
  }
  Turn tr;
  load_turn<kInter>(a, m.b, m.n, c, tr);
  float A[8], Bp[8], w[8];
  load_weight(a, t, 8 * c, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) A[i] = w[i] * tr.c[i];
  if (kInter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) Bp[i] = w[i ^ 1] * tr.s[i];
  } else {
    load_weight(a, t, 8 * tr.partner, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) Bp[i] = w[i] * tr.s[i];
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = m.h0 + GPW * i + g;
    float f[8], fp[8], ss = 0.f;
    unpack8(u[i], f);
    partners<kInter, LPR>(u[i], tr.partner, fp);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = r * fmaf(f[e], A[e], fp[e] * Bp[e]);
    if (h < a.H) *reinterpret_cast<uint4*>(y + (int64_t)h * a.oh) = pack8(f);
  }
}

// Backward.  The CTAs of one tensor (blockIdx.y) walk its items in a fixed
// stride, so each lane's weight-gradient sum has a fixed order; the CTA's sums
// go to part[t][blockIdx.x][D] and dw_kernel adds them in CTA order.
template <int D, bool kInter>
__global__ void __launch_bounds__(kBwdWarps * 32) norm_rope_bwd_kernel(const NormRopeArgs a, int64_t items) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  __shared__ float red[kBwdWarps * GPW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % LPR, g = lane / LPR;
  const int t = blockIdx.y;
  float w[8], dw[8];
  load_weight(a, t, 8 * c, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  for (int64_t it = (int64_t)blockIdx.x * kBwdWarps + warp; it < items; it += (int64_t)gridDim.x * kBwdWarps) {
    const Item m = item_at(a, it, GPW * kHeads);
    const __nv_bfloat16* x = a.x[t] + (int64_t)m.b * a.sb + (int64_t)m.n * a.sn + 8 * c;
    const __nv_bfloat16* dz = a.dz[t] + (int64_t)m.b * a.ob + (int64_t)m.n * a.on + 8 * c;
    __nv_bfloat16* dx = a.y[t] + (int64_t)m.b * a.gb + (int64_t)m.n * a.gn + 8 * c;
    uint4 u[kHeads], v[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = m.h0 + GPW * i + g;
      u[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (h < a.H) {
        u[i] = *reinterpret_cast<const uint4*>(x + (int64_t)h * a.sh);
        v[i] = *reinterpret_cast<const uint4*>(dz + (int64_t)h * a.oh);
      }
    }
    Turn tr;
    load_turn<kInter>(a, m.b, m.n, c, tr);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = m.h0 + GPW * i + g;
      float f[8], z[8], zp[8], ss = 0.f, sx = 0.f;
      unpack8(u[i], f);
      unpack8(v[i], z);
      partners<kInter, LPR>(v[i], tr.partner, zp);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[e] = fmaf(z[e], tr.c[e], -(zp[e] * tr.s[e]));   // g = R^T dz
        ss = fmaf(f[e], f[e], ss);
        sx = fmaf(w[e] * z[e], f[e], sx);
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        sx += __shfl_xor_sync(0xffffffffu, sx, o);
      }
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float k = r * r * sx * (1.f / D);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[e] = fmaf(z[e] * r, f[e], dw[e]);
        z[e] = r * fmaf(-k, f[e], w[e] * z[e]);
      }
      if (h < a.H) *reinterpret_cast<uint4*>(dx + (int64_t)h * a.gh) = pack8(z);
    }
  }
  if (!a.dw[t]) return;   // uniform over the CTA
#pragma unroll
  for (int i = 0; i < 8; ++i) red[warp * GPW + g][8 * c + i] = dw[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int i = 0; i < kBwdWarps * GPW; ++i) s += red[i][threadIdx.x];
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

int64_t item_count(const NormRopeArgs& a, int D) {
  const int heads = 32 / (D / 8) * kHeads;
  return (int64_t)a.B * a.N * ((a.H + heads - 1) / heads);
}

template <int D, bool kInter>
cudaError_t fwd(const NormRopeArgs& a, cudaStream_t st) {
  const int64_t items = item_count(a, D);
  const dim3 grid((unsigned)((items + kFwdWarps - 1) / kFwdWarps), 2);
  norm_rope_kernel<D, kInter><<<grid, kFwdWarps * 32, 0, st>>>(a, items);
  return cudaGetLastError();
}

template <int D, bool kInter>
cudaError_t bwd(const NormRopeArgs& a, cudaStream_t st) {
  const int64_t items = item_count(a, D);
  const int parts = norm_rope_parts(a.B, a.N, a.H, D);
  norm_rope_bwd_kernel<D, kInter><<<dim3(parts, 2), kBwdWarps * 32, 0, st>>>(a, items);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.dw[0] && !a.dw[1])) return e;
  dw_kernel<D><<<2, 1024, 0, st>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace

int norm_rope_parts(int B, int N, int H, int D) {
  const int heads = 32 / (D / 8) * kHeads;
  const int64_t items = (int64_t)B * N * ((H + heads - 1) / heads);
  const int64_t ctas = (items + kBwdWarps - 1) / kBwdWarps;
  return (int)(ctas < 2 * 148 ? ctas : 2 * 148);   // two tensors: four CTAs an SM
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, int D, cudaStream_t st) {
  if (D == 128) return a.inter ? fwd<128, true>(a, st) : fwd<128, false>(a, st);
  return a.inter ? fwd<64, true>(a, st) : fwd<64, false>(a, st);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, int D, cudaStream_t st) {
  if (D == 128) return a.inter ? bwd<128, true>(a, st) : bwd<128, false>(a, st);
  return a.inter ? bwd<64, true>(a, st) : bwd<64, false>(a, st);
}

}  // namespace sol
