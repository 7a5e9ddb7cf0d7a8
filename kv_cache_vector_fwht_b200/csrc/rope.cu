// RMS norm of query and key heads with the position rotation, one pass (tq_norm_rope).
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)
//
// Memory bound: every row is read once and written once. A quarter of a warp holds a row of 128
// channels, 16 per lane, as two runs of 8 (16-byte loads for 16-bit types) chosen so that both
// channels of a rotary pair sit in the same lane: run A holds the pairs' first channels and run B
// their second ones (interleaved pairs: two adjacent runs), so the rotation needs no exchange
// and the norm three shuffles. A block of threads takes up to two tokens and some of their heads:
// 64 threads a token compute its angles' cosines and sines once, while the first rows are on
// their way, and every row of the token reads them from shared memory. 8192 tokens x 72 heads in bf16 (302
// MB read and written) take 56 us, 5.4 TB/s; 8 tokens x 32 heads 2.9 us.
//
// The angle pos * inv_freq reaches 10^6 rad, where an fp32 product is off by up to 0.03 rad. The
// product of an int32 and an fp32 is taken in fp64 in units of whole turns; only the
// fraction of a turn goes on in fp32 (sincospif), exact to 2e-7 rad for every position.
#include <algorithm>
#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kBatch = 2;        // rows a quarter-warp loads before it uses the first
constexpr int kThreads = 128, kQuarters = kThreads / 8;
constexpr int kTokens = 2;       // tokens of a block of threads

struct RopeArgs {
  const void* src[2];            // 0: queries, 1: keys
  void* dst[2];
  const void* w[2];
  int64_t sb[2], sh[2], st[2];   // strides of the sources and of the outputs, in elements
  int64_t db[2], dh[2], dt[2];
  int n_heads[2];
  int chunks, share;             // blocks of threads that share a pair of tokens' heads; heads of each
  const int32_t* pos;
  const float* inv_freq;
  int batch, n_tokens;
  int pairs8;                    // rotary pairs / 8: lanes that hold pairs
  int norm;
  float eps;
  uint8_t axis[kD / 2];
};

template <typename T>
struct Run8;   // 8 consecutive elements
template <>
struct Run8<float> {
  float4 a, b;
  __device__ void load(const float* p) { a = *reinterpret_cast<const float4*>(p); b = *reinterpret_cast<const float4*>(p + 4); }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void unpack(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <typename T>
struct Run16Bit {
  uint4 x;
  __device__ void load(const T* p) { x = *reinterpret_cast<const uint4*>(p); }
  __device__ void zero() { x = make_uint4(0, 0, 0, 0); }
  __device__ void unpack(float* v) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        v[2 * i] = half_lo(w[i]);
        v[2 * i + 1] = half_hi(w[i]);
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  static __device__ void store(T* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Run8<__nv_bfloat16> : Run16Bit<__nv_bfloat16> {};
template <>
struct Run8<__half> : Run16Bit<__half> {};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) k_norm_rope(const __grid_constant__ RopeArgs a) {
  using R = Run8<T>;
  // (cos, sin) of a token's pairs and the weights, as the lanes read them: lane l's pairs 2 j, 2 j + 1 at
  // [j][l], its channels 4 j .. 4 j + 3 (of both runs) at [j][l], so that no two lanes share a bank
  __shared__ float4 turn[kTokens][4][8];
  __shared__ float4 weight[2][4][8];
  const int tid = threadIdx.x, lane = tid & 7, quarter = tid >> 3;
  const int chunk = blockIdx.x % a.chunks;
  const int64_t token0 = static_cast<int64_t>(blockIdx.x / a.chunks) * kTokens, tokens = static_cast<int64_t>(a.batch) * a.n_tokens;
  const int b0 = static_cast<int>(token0 / a.n_tokens), t0 = static_cast<int>(token0 - static_cast<int64_t>(b0) * a.n_tokens);
  const int b1 = t0 + 1 < a.n_tokens ? b0 : b0 + 1, t1 = t0 + 1 < a.n_tokens ? t0 + 1 : 0;   // the second token
  const int h_begin = chunk * a.share, nh = min(a.n_heads[0] + a.n_heads[1], h_begin + a.share) - h_begin;
  const int rows = token0 + 1 < tokens ? 2 * nh : nh;

  // channels of the lane's two runs; lanes past the pairs hold the channels that do not turn
  const bool turns = lane < a.pairs8;
  const int cA = INTERLEAVED || !turns ? 16 * lane : 8 * lane;
  const int cB = INTERLEAVED || !turns ? cA + 8 : cA + 8 * a.pairs8;

  // row r of the block: token r / nh, head h_begin + r % nh (queries, then keys)
  auto place = [&](int r, int& side, int& h, int& b, int& t) {
    const bool second = r >= nh;
    h = h_begin + r - (second ? nh : 0);
    side = h >= a.n_heads[0];
    if (side) h -= a.n_heads[0];
    b = second ? b1 : b0;
    t = second ? t1 : t0;
  };
  wait_for_grid();
  launch_dependents();
  R xa[kBatch], xb[kBatch];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = r0 + kQuarters * u;
      if (r < rows) {
        int side, h, b, t;
        place(r, side, h, b, t);
        const T* p = static_cast<const T*>(a.src[side]) + b * a.sb[side] + h * a.sh[side] + t * a.st[side];
        xa[u].load(p + cA);
        xb[u].load(p + cB);
      } else {
        xa[u].zero();
        xb[u].zero();
      }
    }
  };
  fetch(quarter);   // the first rows are on their way while the angles are computed

  if (a.norm) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      float w = 1.f;
      if (a.w[side] != nullptr) {
        if constexpr (sizeof(T) == 4) w = static_cast<const float*>(a.w[side])[tid];
        else w = static_cast<float>(static_cast<const T*>(a.w[side])[tid]);
      }
      // channel tid's lane, and its place in the lane's 16 channels
      const int rot = 16 * a.pairs8;
      const bool halves = !INTERLEAVED && tid < rot;
      const int c = halves ? tid % (rot / 2) : tid;
      const int l = halves ? c / 8 : tid / 16, o = halves ? c % 8 + (tid >= rot / 2 ? 8 : 0) : tid % 16;
      reinterpret_cast<float*>(&weight[side][o / 4][l])[o % 4] = w;
    }
  }
  {
    const int f = tid & 63, b = tid < 64 ? b0 : b1, t = tid < 64 ? t0 : t1;
    if (f < 8 * a.pairs8 && token0 + (tid >> 6) < tokens) {
      const int p = a.pos[(static_cast<int64_t>(a.axis[f]) * a.batch + b) * a.n_tokens + t];
      const double whole = static_cast<double>(p) * static_cast<double>(a.inv_freq[f]) * 0.15915494309189533577;  // / 2 pi
      float si, co;
      sincospif(2.f * static_cast<float>(whole - rint(whole)), &si, &co);
      reinterpret_cast<float2*>(&turn[tid >> 6][(f % 8) / 2][f / 8])[f % 2] = make_float2(co, si);
    }
  }
  __syncthreads();

  // all threads take the same number of turns, so that every shuffle has the whole warp
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += kQuarters * kBatch) {
    float va[kBatch][8], vb[kBatch][8];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      xa[u].unpack(va[u]);
      xb[u].unpack(vb[u]);
    }
    if (r0 + kQuarters * kBatch < rows) fetch(r0 + kQuarters * kBatch + quarter);
    float ss[kBatch];
    if (a.norm) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        uint64_t s2 = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint64_t p = pk2(va[u][i], va[u][i + 1]), q = pk2(vb[u][i], vb[u][i + 1]);
          s2 = fma2(p, p, fma2(q, q, s2));
        }
        ss[u] = up2(s2).x + up2(s2).y;
      }
#pragma unroll
      for (int m = 4; m >= 1; m >>= 1)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) ss[u] += __shfl_xor_sync(kFull, ss[u], m);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) ss[u] = rsqrtf(ss[u] * (1.f / kD) + a.eps);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = r0 + quarter + kQuarters * u;
      if (r >= rows) continue;
      int side, h, b, t;
      place(r, side, h, b, t);
      if (a.norm) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 p = weight[side][i / 4][lane], q = weight[side][2 + i / 4][lane];
          va[u][i] *= ss[u] * p.x; va[u][i + 1] *= ss[u] * p.y; va[u][i + 2] *= ss[u] * p.z; va[u][i + 3] *= ss[u] * p.w;
          vb[u][i] *= ss[u] * q.x; vb[u][i + 1] *= ss[u] * q.y; vb[u][i + 2] *= ss[u] * q.z; vb[u][i + 3] *= ss[u] * q.w;
        }
      }
      if (turns) {
        // the pairs: (A[i], B[i]), interleaved (A0 A1) (A2 A3) ... (B6 B7)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 c2 = turn[r >= nh][i / 2][lane];
          const float co = i & 1 ? c2.z : c2.x, si = i & 1 ? c2.w : c2.y;
          float& y1 = INTERLEAVED ? (i < 4 ? va[u][2 * i] : vb[u][2 * i - 8]) : va[u][i];
          float& y2 = INTERLEAVED ? (i < 4 ? va[u][2 * i + 1] : vb[u][2 * i - 7]) : vb[u][i];
          const float p = y1, q = y2;
          y1 = p * co - q * si;
          y2 = q * co + p * si;
        }
      }
      T* o = static_cast<T*>(a.dst[side]) + b * a.db[side] + h * a.dh[side] + t * a.dt[side];
      R::store(o + cA, va[u]);
      R::store(o + cB, vb[u]);
    }
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
  }
  // heads of a block of threads: few where tokens are few (the call is latency), all of them where
  // sharing a token's angles counts
  const int heads = n_heads[0] + n_heads[1];
  const int64_t pairs = (tokens + kTokens - 1) / kTokens;
  int device = 0;
  cudaGetDevice(&device);
  a.chunks = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((heads + 15) / 16, sm_count(device) * 8 / pairs)));
  a.share = (heads + a.chunks - 1) / a.chunks;
  a.pos = r->pos_dev;
  a.inv_freq = r->inv_freq_dev;
  a.batch = batch;
  a.n_tokens = n_tokens;
  a.pairs8 = r->rot_dim / 16;
  a.norm = norm;
  a.eps = eps;
  for (int i = 0; i < kD / 2; ++i)
    a.axis[i] = r->axis_of_freq && i < r->rot_dim / 2 ? r->axis_of_freq[i] : 0;
  const int64_t blocks = pairs * a.chunks;
  if (blocks > 0x7fffffff) return TQ_EUNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks));
  void (*kernel)(RopeArgs);
  const bool il = r->interleaved != 0;
  switch (dtype) {
    case TQ_F32: kernel = il ? k_norm_rope<float, true> : k_norm_rope<float, false>; break;
    case TQ_BF16: kernel = il ? k_norm_rope<__nv_bfloat16, true> : k_norm_rope<__nv_bfloat16, false>; break;
    case TQ_F16: kernel = il ? k_norm_rope<__half, true> : k_norm_rope<__half, false>; break;
    default: return TQ_EUNSUPPORTED;
  }
  return launch_early(kernel, grid, kThreads, 0, st, a) == cudaSuccess ? TQ_OK : TQ_ECUDA;
}

}  // namespace tq
