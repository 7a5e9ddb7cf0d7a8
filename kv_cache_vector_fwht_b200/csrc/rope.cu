// RMS norm of query and key heads with the position rotation, one pass (tq_norm_rope).
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)
//
// Memory bound: every row is read once and written once. Half a warp holds a row of 128
// channels, 8 per lane, as two runs of 4 (one 8- or 16-byte load each) chosen so that both
// channels of a rotary pair sit in the same lane: run A holds the pairs' first channels and run
// B their second ones (interleaved pairs: two adjacent runs), so the rotation needs no
// exchange and the norm four shuffles. A lane's 4 angles depend on the token alone: it
// computes them once and keeps them while it walks the heads of its token, kBatch rows in
// flight at a time.
//
// The angle pos * inv_freq reaches 10^6 rad, where an fp32 product is off by up to 0.03 rad. The
// product of an int32 and an fp32 is taken in fp64 in units of whole turns; only the
// fraction of a turn goes on in fp32 (sincospif), exact to 2e-7 rad for every position.
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kBatch = 4;        // rows a half-warp loads before it uses the first
constexpr int kWarps = 4;

struct RopeArgs {
  const void* src[2];            // 0: queries, 1: keys
  void* dst[2];
  const void* w[2];
  int64_t sb[2], sh[2], st[2];   // strides of the sources and of the outputs, in elements
  int64_t db[2], dh[2], dt[2];
  int n_heads[2];
  int chunks[2];                 // warps that share a token's query / key heads
  const int32_t* pos;
  const float* inv_freq;
  int batch, n_tokens;
  int pairs4;                    // rotary pairs / 4: lanes that hold pairs
  int norm;
  float eps;
  uint8_t axis[kD / 2];
};

template <typename T>
struct Run4;   // 4 consecutive elements as one access
template <>
struct Run4<float> {
  using raw = float4;
  static __device__ void unpack(const raw& r, float* v) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
  static __device__ raw pack(const float* v) { return make_float4(v[0], v[1], v[2], v[3]); }
};
template <>
struct Run4<__nv_bfloat16> {
  using raw = uint2;
  static __device__ void unpack(const raw& r, float* v) {
    v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xffff0000u);
  }
  static __device__ raw pack(const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <>
struct Run4<__half> {
  using raw = uint2;
  static __device__ void unpack(const raw& r, float* v) {
    v[0] = half_lo(r.x); v[1] = half_hi(r.x); v[2] = half_lo(r.y); v[3] = half_hi(r.y);
  }
  static __device__ raw pack(const float* v) {
    const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) k_norm_rope(const __grid_constant__ RopeArgs a) {
  using R = Run4<T>;
  using raw = typename R::raw;
  const int per_token = a.chunks[0] + a.chunks[1];
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t token = warp / per_token;
  if (token >= static_cast<int64_t>(a.batch) * a.n_tokens) return;
  int chunk = static_cast<int>(warp - token * per_token);
  const int side = chunk >= a.chunks[0];
  if (side) chunk -= a.chunks[0];
  const int b = static_cast<int>(token / a.n_tokens), t = static_cast<int>(token - static_cast<int64_t>(b) * a.n_tokens);
  const int lane = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;

  // channels of the lane's two runs; lanes past the pairs hold the channels that do not turn
  const bool turns = lane < a.pairs4;
  const int cA = INTERLEAVED || !turns ? 8 * lane : 4 * lane;
  const int cB = INTERLEAVED || !turns ? cA + 4 : cA + 4 * a.pairs4;

  // this warp's heads, in equal shares of whole rows
  const int heads = a.n_heads[side], share = (heads + a.chunks[side] - 1) / a.chunks[side];
  const int h_end = min(heads, (chunk + 1) * share);
  const T* src = static_cast<const T*>(a.src[side]) + b * a.sb[side] + t * a.st[side];
  T* dst = static_cast<T*>(a.dst[side]) + b * a.db[side] + t * a.dt[side];

  raw xa[kBatch], xb[kBatch];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + 2 * u;
      if (h < h_end) {
        xa[u] = *reinterpret_cast<const raw*>(src + h * a.sh[side] + cA);
        xb[u] = *reinterpret_cast<const raw*>(src + h * a.sh[side] + cB);
      }
    }
  };
  // both halves take the same number of turns, so that every shuffle has the whole warp
  int h0 = chunk * share;
  fetch(h0 + half);   // the first rows are on their way while the angles are computed

  float wA[4] = {1.f, 1.f, 1.f, 1.f}, wB[4] = {1.f, 1.f, 1.f, 1.f};
  if (a.norm && a.w[side] != nullptr) {
    const T* w = static_cast<const T*>(a.w[side]);
    R::unpack(*reinterpret_cast<const raw*>(w + cA), wA);
    R::unpack(*reinterpret_cast<const raw*>(w + cB), wB);
  }
  float co[4], si[4];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int f = 4 * lane + i;
      const int p = a.pos[(static_cast<int64_t>(a.axis[f]) * a.batch + b) * a.n_tokens + t];
      const double whole = static_cast<double>(p) * static_cast<double>(a.inv_freq[f]) * 0.15915494309189533577;  // / 2 pi
      sincospif(2.f * static_cast<float>(whole - rint(whole)), &si[i], &co[i]);
    }
  }

  for (; h0 < h_end; h0 += 2 * kBatch) {
    float va[kBatch][4], vb[kBatch][4];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (h0 + half + 2 * u >= h_end) xa[u] = xb[u] = raw{};
      R::unpack(xa[u], va[u]);
      R::unpack(xb[u], vb[u]);
    }
    if (a.norm) {
      float ss[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        ss[u] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss[u] = fmaf(va[u][i], va[u][i], fmaf(vb[u][i], vb[u][i], ss[u]));
      }
#pragma unroll
      for (int m = 8; m >= 1; m >>= 1)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) ss[u] += __shfl_xor_sync(kFull, ss[u], m);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float r = rsqrtf(ss[u] * (1.f / kD) + a.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          va[u][i] = va[u][i] * r * wA[i];
          vb[u][i] = vb[u][i] * r * wB[i];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + half + 2 * u;
      if (turns) {
        // the pairs: (A[i], B[i]), interleaved (A0 A1) (A2 A3) (B0 B1) (B2 B3)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& y1 = INTERLEAVED ? (i < 2 ? va[u][2 * i] : vb[u][2 * i - 4]) : va[u][i];
          float& y2 = INTERLEAVED ? (i < 2 ? va[u][2 * i + 1] : vb[u][2 * i - 3]) : vb[u][i];
          const float p = y1, q = y2;
          y1 = p * co[i] - q * si[i];
          y2 = q * co[i] + p * si[i];
        }
      }
      if (h < h_end) {
        *reinterpret_cast<raw*>(dst + h * a.dh[side] + cA) = R::pack(va[u]);
        *reinterpret_cast<raw*>(dst + h * a.dh[side] + cB) = R::pack(vb[u]);
      }
    }
    fetch(h0 + half + 2 * kBatch);
  }
}

}  // namespace

tq_status launch_norm_rope(const tq_rope* r, int dtype, int batch, int n_tokens, const int (&n_heads)[2],
                           const tq_heads (&src)[2], const tq_heads (&dst)[2], const void* const (&w)[2],
                           int norm, float eps, cudaStream_t st) {
  RopeArgs a;
  const int64_t tokens = static_cast<int64_t>(batch) * n_tokens;
  for (int s = 0; s < 2; ++s) {
    a.src[s] = src[s].data; a.sb[s] = src[s].stride_b; a.sh[s] = src[s].stride_h; a.st[s] = src[s].stride_t;
    a.dst[s] = dst[s].data; a.db[s] = dst[s].stride_b; a.dh[s] = dst[s].stride_h; a.dt[s] = dst[s].stride_t;
    a.w[s] = w[s];
    a.n_heads[s] = n_heads[s];
    // heads a warp: few where tokens are few (the call is latency), more where the angles'
    // cost is worth sharing
    const int share = tokens * (n_heads[0] + n_heads[1]) >= 148 * 64 * 8 ? 4 * kBatch : 2;
    a.chunks[s] = (n_heads[s] + share - 1) / share;
  }
  a.pos = r->pos_dev;
  a.inv_freq = r->inv_freq_dev;
  a.batch = batch;
  a.n_tokens = n_tokens;
  a.pairs4 = r->rot_dim / 8;
  a.norm = norm;
  a.eps = eps;
  for (int i = 0; i < kD / 2; ++i)
    a.axis[i] = r->axis_of_freq && i < r->rot_dim / 2 ? r->axis_of_freq[i] : 0;
  const int64_t blocks = (tokens * (a.chunks[0] + a.chunks[1]) + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return TQ_EUNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * kWarps);
  const bool il = r->interleaved != 0;
  switch (dtype) {
    case TQ_F32:
      il ? k_norm_rope<float, true><<<grid, block, 0, st>>>(a) : k_norm_rope<float, false><<<grid, block, 0, st>>>(a);
      break;
    case TQ_BF16:
      il ? k_norm_rope<__nv_bfloat16, true><<<grid, block, 0, st>>>(a)
         : k_norm_rope<__nv_bfloat16, false><<<grid, block, 0, st>>>(a);
      break;
    case TQ_F16:
      il ? k_norm_rope<__half, true><<<grid, block, 0, st>>>(a) : k_norm_rope<__half, false><<<grid, block, 0, st>>>(a);
      break;
    default: return TQ_EUNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ECUDA;
}

}  // namespace tq
