// Block bounds of the packed keys and the choice of blocks for a sparse decode step
// (tq_block_bounds, tq_select_blocks).
#include <algorithm>
#include <cmath>

#include "packed.cuh"

namespace tq {
namespace {

// ------------------------------------------------------------------------------- bounds
// min and max over a block's tokens of n16 c[idx_j] / sqrt(d), channel by channel. Rounding to fp16, the
// type of the result, is monotone: the minimum of the rounded products is the rounded minimum. A NaN norm stays: it
// makes the block's bounds NaN, which the selection puts first. So a
// token's products with the whole codebook are made first (fp32, one rounding: 4 products of a 2-bit
// codebook, 8 of a 3-bit one, the 8 positive ones of a 4-bit one), as byte pools like the codebook's
// own; the token's codes then look up finished fp16 numbers, two to a register, and a value costs its
// lookup and half a minimum and half a maximum. A warp takes a few token blocks of one (sequence, KV
// head): its lanes make the pools of two rows each, then lane = (word of the row, every G-th row) with
// its channels' minima and maxima in registers. The next block's words are loaded before this block's
// results are joined. The lanes that share a word are joined at the end, by exchanges where the row's words
// divide the warp and in shared memory otherwise.
// Bound by instructions of the ALU pipe (lookups, minima): 8 sequences of 8192 to 32768 rows x 4
// KV heads of 2-bit codes (36 bytes a row read, 31 MB) take 15 us, where HBM alone would take 5. With the
// conversions and products of every value in fp32 it was 38.
constexpr int kBW = 4;   // warps of a block of threads

struct BoundsArgs {
  const uint8_t* idx;
  const uint16_t* norms;
  const int32_t* len;
  __half* bounds;
  const DevTables* tab;
  int n_kv_heads, capacity, n_tokens, n_blocks, per_warp, n_norms;
  float scale0, scale1;  // level scale / sqrt(channels of the group)
};

// Two fp16 levels (low bytes in lo, high bytes in hi, selected by sel) times f, rounded once.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t lo, uint32_t hi, uint32_t sel, float f) {
  const uint32_t y = prmt(lo, hi, sel);
  const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&y));
  const __half2 r = __floats2half2_rn(l.x * f, l.y * f);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The pools of a codebook's products with f.
template <int BITS>
__device__ __forceinline__ void scale_levels(const Levels& lv, float f, uint4* dst) {
  if constexpr (BITS == 1) {
    const uint32_t y = scaled_pair(lv.lo[0], 0, 0x3210, f);
    *reinterpret_cast<uint32_t*>(dst) = y;
  } else if constexpr (BITS == 2) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(scaled_pair(lv.lo[0], 0, 0x3210, f), scaled_pair(lv.lo[1], 0, 0x3210, f));
  } else {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t y0 = scaled_pair(lv.lo[i], lv.hi[i], 0x5140, f), y1 = scaled_pair(lv.lo[i], lv.hi[i], 0x7362, f);
      o[2 * i] = prmt(y0, y1, 0x6420);
      o[2 * i + 1] = prmt(y0, y1, 0x7531);
    }
    *dst = make_uint4(o[0], o[1], o[2], o[3]);
  }
}
template <int BITS>
__device__ __forceinline__ Levels scaled_levels(const uint4* src) {
  if constexpr (BITS == 1) return Levels{{*reinterpret_cast<const uint32_t*>(src), 0}, {0, 0}};
  if constexpr (BITS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    return Levels{{v.x, v.y}, {0, 0}};
  }
  const uint4 v = *src;
  return Levels{{v.x, v.z}, {v.y, v.w}};
}

// Two rows' words into the minima and maxima (one three-way minimum takes both).
template <int BITS, int N>
__device__ __forceinline__ void bounds_rows(uint32_t w0, uint32_t w1, const uint4* pool0, const uint4* pool1, __half2 (&v)[N]) {
  constexpr int NP = level_pairs(BITS);
  uint32_t y0[NP], y1[NP];
  unpack_levels<BITS>(w0, scaled_levels<BITS>(pool0), y0);
  unpack_levels<BITS>(w1, scaled_levels<BITS>(pool1), y1);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const __half2 a = *reinterpret_cast<const __half2*>(&y0[i]), b = *reinterpret_cast<const __half2*>(&y1[i]);
    v[i] = __hmin2_nan(__hmin2_nan(v[i], a), b);
    v[N / 2 + i] = __hmax2_nan(__hmax2_nan(v[N / 2 + i], a), b);
  }
}

// Exchange with the lane M away: of N results a lane keeps the half that its bit M names.
template <int M, int N>
__device__ __forceinline__ void join_lanes(__half2* v, int lane) {
  const bool up = lane & M;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __half2 a = v[i], b = v[i + N / 2];
    const __half2 mine = up ? b : a, theirs = up ? a : b;
    v[i] = __hmin2_nan(mine, __shfl_xor_sync(kFull, theirs, M));
  }
}

// B0, B1: code bits of the two channel groups (B1 = 0: one group).
template <int B0, int B1>
__global__ void __launch_bounds__(32 * kBW, B0 == 2 && B1 == 0 ? 8 : 5) k_block_bounds(const __grid_constant__ BoundsArgs a) {
  constexpr bool kGrouped = B1 != 0;
  constexpr int B1x = kGrouped ? B1 : B0;
  constexpr int kWords0 = (kGrouped ? 1 : 4) * storage_width_c(B0);               // 32-bit words of the first group
  constexpr int kWords = kWords0 + (kGrouped ? 3 * storage_width_c(B1x) : 0);
  constexpr int kGroups = 32 / kWords;                                            // lanes that share a word
  constexpr int kRows = (TQ_BLOCK + kGroups - 1) / kGroups;                       // a lane's rows of a block
  constexpr int NP0 = level_pairs(B0), NP1 = level_pairs(B1x), NP = NP0 > NP1 ? NP0 : NP1;
  __shared__ uint4 pools[kBW][kGrouped ? 2 : 1][TQ_BLOCK];
  __shared__ __align__(16) __half2 parts[kBW][kGrouped ? kGroups : 1][2][kD / 2];   // grouped: minima and negated maxima to be joined
  __shared__ __align__(16) __half res_all[kBW][2][kD];
  const int b = blockIdx.z, kv = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_grid();
  launch_dependents();
  const int len = min(a.len[b], a.capacity);
  const int blk0 = max(0, len - a.n_tokens) / TQ_BLOCK + (blockIdx.x * kBW + warp) * a.per_warp;
  const int n_rows = len - blk0 * TQ_BLOCK;
  if (n_rows <= 0) return;
  const int blocks = min(a.per_warp, (n_rows + TQ_BLOCK - 1) / TQ_BLOCK);
  const int64_t pair = static_cast<int64_t>(b) * a.n_kv_heads + kv;
  const int64_t row0 = pair * a.capacity + static_cast<int64_t>(blk0) * TQ_BLOCK;
  // the few lanes beyond groups x words repeat the last group's rows
  const int word = lane % kWords, g = min(lane / kWords, kGroups - 1);
  const bool second = kGrouped && word >= kWords0;
  const Levels lv0 = load_levels(a.tab, 0), lv1 = load_levels(a.tab, kGrouped ? 1 : 0);
  const int n_norms = kGrouped ? 2 : a.n_norms;   // prod rows hold ||r|| too
  const uint32_t* words = reinterpret_cast<const uint32_t*>(a.idx) + row0 * kWords + word;
  const uint16_t* norms = a.norms + row0 * n_norms;
  uint4 (*pool)[TQ_BLOCK] = pools[warp];
  __half* res = &res_all[warp][0][0];
  uint4* out = reinterpret_cast<uint4*>(a.bounds + (pair * a.n_blocks + blk0) * 2 * kD) + lane;
  uint32_t w[kRows];
  uint16_t nr[2][kGrouped ? 2 : 1];
  // a row seen twice changes no minimum: rows past the block's last one are the last one
  auto load_words = [&](int blk) {
    const int last = min(TQ_BLOCK - 1, n_rows - 1 - blk * TQ_BLOCK);
    const uint32_t* p = words + blk * TQ_BLOCK * kWords;
    if (last == TQ_BLOCK - 1 && kGroups * kRows == TQ_BLOCK) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) w[u] = p[(g + kGroups * u) * kWords];
    } else {
#pragma unroll
      for (int u = 0; u < kRows; ++u) w[u] = p[min(g + kGroups * u, last) * kWords];
    }
  };
  auto load_norms = [&](int blk) {
    const int last = min(TQ_BLOCK - 1, n_rows - 1 - blk * TQ_BLOCK);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint16_t* n = norms + (blk * TQ_BLOCK + min(lane + 32 * i, last)) * n_norms;
#pragma unroll
      for (int j = 0; j < (kGrouped ? 2 : 1); ++j) nr[i][j] = n[j];
    }
  };
  load_norms(0);
  load_words(0);
#pragma unroll 1
  for (int blk = 0; blk < blocks; ++blk) {
    __syncwarp();   // the last block's pools and result have been read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      scale_levels<B0>(lv0, __half2float(__ushort_as_half(nr[i][0])) * a.scale0, &pool[0][lane + 32 * i]);
      if constexpr (kGrouped) scale_levels<B1x>(lv1, __half2float(__ushort_as_half(nr[i][1])) * a.scale1, &pool[1][lane + 32 * i]);
    }
    __syncwarp();
    if (blk + 1 < blocks) load_norms(blk + 1);
    __half2 v[2 * NP];   // minima, then maxima
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      v[i] = __half2half2(__ushort_as_half(0x7c00));
      v[NP + i] = __half2half2(__ushort_as_half(0xfc00));
    }
    // rows of the pools past TQ_BLOCK - 1 do not exist; those past the last row repeat it
    auto pool_row = [&](int u) { return kGroups * kRows == TQ_BLOCK ? g + kGroups * u : min(g + kGroups * u, TQ_BLOCK - 1); };
#pragma unroll
    for (int u = 0; u < kRows; u += 2) {
      const int u1 = min(u + 1, kRows - 1);
      const int r0 = pool_row(u), r1 = pool_row(u1);
      if (!second) bounds_rows<B0>(w[u], w[u1], &pool[0][r0], &pool[0][r1], v);
      else if constexpr (kGrouped) bounds_rows<B1x>(w[u], w[u1], &pool[1][r0], &pool[1][r1], v);
    }
    if (blk + 1 < blocks) load_words(blk + 1);
#pragma unroll
    for (int i = 0; i < NP; ++i) v[NP + i] = __hneg2(v[NP + i]);
    if constexpr (!kGrouped) {
      // 4, 8 or 16 words: the lanes that share a word end with 4 of its 2 NP results each
      join_lanes<16, 2 * NP>(v, lane);
      if constexpr (kWords <= 8) join_lanes<8, NP>(v, lane);
      if constexpr (kWords <= 4) join_lanes<4, NP / 2>(v, lane);
      const int at = word * NP + (kWords <= 8 ? (lane >> 3 & 1) * (NP / 2) : 0) + (kWords <= 4 ? (lane >> 2 & 1) * (NP / 4) : 0);
      __half* o = res + (lane >> 4) * kD;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 x = lane >> 4 ? __hneg2(v[i]) : v[i];
        o[level_channel(B0, at + i, 0)] = __low2half(x);
        o[level_channel(B0, at + i, 1)] = __high2half(x);
      }
    } else {
      __half2 (*part)[2][kD / 2] = parts[warp];
      if (lane < kGroups * kWords) {
        const int p = second ? NP0 * kWords0 + (word - kWords0) * NP1 : word * NP0, n = second ? NP1 : NP0;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (i < n) {
            part[g][0][p + i] = v[i];
            part[g][1][p + i] = v[NP + i];
          }
      }
      __syncwarp();
      constexpr int pairs0 = NP0 * kWords0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = lane + 32 * (j & 1), which = j >> 1;
        __half2 x = part[0][which][p];
#pragma unroll
        for (int i = 1; i < kGroups; ++i) x = __hmin2_nan(x, part[i][which][p]);
        if (which) x = __hneg2(x);
        const bool rest = p >= pairs0;
        const int q = rest ? p - pairs0 : p, c0 = which * kD + (rest ? 2 * pairs0 : 0);
        res[c0 + (rest ? level_channel(B1x, q, 0) : level_channel(B0, q, 0))] = __low2half(x);
        res[c0 + (rest ? level_channel(B1x, q, 1) : level_channel(B0, q, 1))] = __high2half(x);
      }
    }
    __syncwarp();
    out[blk * (2 * kD / 8)] = reinterpret_cast<const uint4*>(res)[lane];
  }
}

// ------------------------------------------------------------------------------- selection
// Scores: sum_j max(q_j lo_j, q_j hi_j) = sum_j (q_j (lo_j + hi_j) + |q_j| (hi_j - lo_j)) / 2. q = H (s . q)
// (no 1/sqrt(d): it is the same for every block), all of it in fp64: the operands are exact
// there and the sums are off by 2^-53, so the choice of blocks does not hang on the order of
// a sum, at 1/2 of the fp32 rate for a few million products. A warp holds 4 channels per lane
// of kHG rotated heads in registers and walks its blocks; the bounds are read once, 16 bytes
// a lane; a block of threads walks as many 64-block chunks as leave one round over the SMs, because
// the heads' rotation and the joining cost as much as a chunk. The last block of threads of a
// (sequence, KV head) to finish picks the blocks: the n-th largest key is found by a histogram
// of 1024 equal key ranges, then by ranking the keys of the range that holds it, once they are a warp's
// worth (further histograms inside it until then), and the chosen blocks are written in
// ascending order by ballots. Latency bound: 2048 blocks
// for each of 8 KV heads of 8 heads (8 MB of bounds) take 18 us: rotation and loads, two chunks in fp64 at about 3 us
// each, the joining fence, 2 us of picking.
constexpr int kST = 256, kSW = kST / 32;
constexpr int kHG = 4;       // heads scored at a time
constexpr int kHS = 16;      // rotated heads held in shared memory
constexpr int kBPW = 8;      // blocks a warp scores
constexpr int kBins = 1024;
constexpr int kHeldKeys = 8;   // keys a picking thread holds in registers (2048 blocks: 131072 tokens)
constexpr unsigned long long kAlways = ~0ull;

struct SelectArgs {
  const __half* bounds;
  const void* q;
  const int32_t* len;
  const DevTables* tab;
  int32_t* ids;
  unsigned long long* keys;   // (batch, KV head, n_blocks)
  int* counters;
  int n_kv_heads, capacity, n_q_heads, n_blocks, n_select, n_sink, n_recent;
  int q_dtype, grouped;
  HeadLists heads;
};

__device__ __forceinline__ double shfl_xor_d(double v, int m) { return __shfl_xor_sync(kFull, v, m); }

// A query row with the rotation's signs: lane l holds coordinates 4l .. 4l + 3.
__device__ __forceinline__ void load_row_f64(const SelectArgs& a, int64_t row, int lane, double (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * lane + i;
    const int c = a.grouped ? a.tab->chan[j] : j;
    const float x = load_element(a.q, a.q_dtype, row * kD + c);
    v[i] = (a.tab->sign_bits[j >> 5] >> (j & 31)) & 1u ? -static_cast<double>(x) : static_cast<double>(x);
  }
}

// Its Hadamard transform (unnormalised).
__device__ __forceinline__ void rotate_row_f64(bool grouped, int lane, double (&v)[4]) {
  double t0 = v[0] + v[1], t1 = v[0] - v[1], t2 = v[2] + v[3], t3 = v[2] - v[3];
  v[0] = t0 + t2; v[2] = t0 - t2; v[1] = t1 + t3; v[3] = t1 - t3;
  const int top = grouped ? 4 : 16;   // grouped: 32-point blocks
  for (int m = 1; m <= top; m <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double o = shfl_xor_d(v[i], m);
      v[i] = lane & m ? o - v[i] : v[i] + o;
    }
}

__device__ __forceinline__ unsigned long long order_key(double s) {
  if (isnan(s)) return kAlways - 1;   // above every number, below what is always chosen
  const long long b = __double_as_longlong(s + 0.0);   // -0 and 0 are one value
  return b < 0 ? ~static_cast<unsigned long long>(b) : static_cast<unsigned long long>(b) | (1ull << 63);
}

// The blocks of one (sequence, KV head), by all threads of the block. Warp w looks at the keys
// [w span, (w + 1) span), lane by lane; keys are never 0, which stands for an absent one.
__device__ void pick_blocks(const SelectArgs& a, int pair, int nb) {
  __shared__ __align__(16) uint4 hist4[kBins / 4];
  __shared__ unsigned sums[kSW][2];
  __shared__ int scans[kSW];
  __shared__ unsigned long long few[32];
  __shared__ int s_bin, s_need, s_count, s_few;
  unsigned* hist = reinterpret_cast<unsigned*>(hist4);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const unsigned below = (1u << lane) - 1;
  int32_t* ids = a.ids + static_cast<int64_t>(pair) * a.n_select;
  if (nb <= a.n_select) {
    for (int i = tid; i < a.n_select; i += kST) ids[i] = i < nb ? i : -1;
    return;
  }
  const unsigned long long* keys = a.keys + static_cast<int64_t>(pair) * a.n_blocks;
  const int span = ((nb + kSW - 1) / kSW + 31) & ~31;
  const bool held = span <= 32 * kHeldKeys;
  unsigned long long mine[kHeldKeys];
  if (held) {
#pragma unroll
    for (int j = 0; j < kHeldKeys; ++j) {
      const int i = w * span + 32 * j + lane;
      mine[j] = 32 * j < span && i < nb ? __ldcg(keys + i) : 0;
    }
  }
  auto each = [&](auto f) {   // f(block, key), the warp's lanes together
    if (held) {
#pragma unroll
      for (int j = 0; j < kHeldKeys; ++j)
        if (32 * j < span) f(w * span + 32 * j + lane, mine[j]);
    } else {
      for (int j = 0; j < span; j += 32) {
        const int i = w * span + j + lane;
        f(i, i < nb ? __ldcg(keys + i) : 0ull);
      }
    }
  };
  int need = a.n_select - a.n_sink - a.n_recent;   // nb > n_select: the two ranges do not meet
  unsigned long long T = kAlways;                  // the smallest key chosen ...
  int ties = 0;                                    // ... and how many of its equals
  if (need > 0) {
    unsigned lo32 = ~0u, hi32 = 0;   // of the keys' high words
    each([&](int, unsigned long long k) {
      if (k != 0 && k != kAlways) {
        lo32 = min(lo32, static_cast<unsigned>(k >> 32));
        hi32 = max(hi32, static_cast<unsigned>(k >> 32));
      }
    });
    lo32 = __reduce_min_sync(kFull, lo32);
    hi32 = __reduce_max_sync(kFull, hi32);
    if (lane == 0) { sums[w][0] = lo32; sums[w][1] = hi32; }
    hist4[tid] = make_uint4(0, 0, 0, 0);
    static_assert(kBins == 4 * kST, "four bins a thread");
    __syncthreads();
    for (int i = 0; i < kSW; ++i) { lo32 = min(lo32, sums[i][0]); hi32 = max(hi32, sums[i][1]); }
    unsigned long long lo = static_cast<unsigned long long>(lo32) << 32, hi = static_cast<unsigned long long>(hi32) << 32 | 0xffffffffull;
    while (true) {   // at most 7 turns: each leaves at most a 2^-9 of the key range
      const int width = 64 - __clzll(static_cast<long long>(hi - lo));
      const int s = max(0, width - 10);
      each([&](int, unsigned long long k) {
        if (k >= lo && k <= hi && k != kAlways) atomicAdd(&hist[(k - lo) >> s], 1u);
      });
      __syncthreads();
      // thread t sums the bins [1024 - 4t - 4, 1024 - 4t): a scan from the highest bin down
      const int top = kBins - 1 - 4 * tid;
      const uint4 h4 = hist4[kST - 1 - tid];
      hist4[kST - 1 - tid] = make_uint4(0, 0, 0, 0);   // for the next turn
      const int h[4] = {static_cast<int>(h4.w), static_cast<int>(h4.z), static_cast<int>(h4.y), static_cast<int>(h4.x)};
      const int sum = h[0] + h[1] + h[2] + h[3];
      int upto = sum;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(kFull, upto, m);
        if (lane >= m) upto += o;
      }
      if (lane == 31) scans[w] = upto;
      if (tid == 0) s_few = 0;
      __syncthreads();
      for (int i = 0; i < kSW; ++i) upto += i < w ? scans[i] : 0;
      if (upto >= need && upto - sum < need) {
        int above = upto - sum, i = 0;
        while (above + h[i] < need) above += h[i++];
        s_bin = top - i;
        s_need = need - above;
        s_count = h[i];
      }
      __syncthreads();
      need = s_need;
      const int count = s_count;
      lo += static_cast<unsigned long long>(s_bin) << s;
      hi = lo + min(hi - lo, (1ull << s) - 1);   // the sum may not pass 2^64: a NaN's key is near it
      if (s == 0 || count == need) {
        T = lo;
        ties = s == 0 ? need : nb;   // count == need: everything from lo on, its equals too
        break;
      }
      if (count <= 32) {   // rank them
        each([&](int, unsigned long long k) {
          if (k >= lo && k <= hi && k != kAlways) few[atomicAdd(&s_few, 1)] = k;
        });
        __syncthreads();
        const unsigned long long x = lane < count ? few[lane] : 0;
        int greater = 0, as_great = 0;
        for (int i = 0; i < count; ++i) {
          greater += few[i] > x;
          as_great += few[i] >= x;
        }
        const int src = __ffs(__ballot_sync(kFull, greater < need && need <= as_great)) - 1;
        T = __shfl_sync(kFull, x, src);
        ties = need - __shfl_sync(kFull, greater, src);
        break;
      }
    }
    __syncthreads();   // sums is free
  }
  int more = 0, eq = 0;
  each([&](int, unsigned long long k) {
    more += __popc(__ballot_sync(kFull, k > T || k == kAlways));
    eq += __popc(__ballot_sync(kFull, k == T && k != kAlways));
  });
  if (lane == 0) { sums[w][0] = more; sums[w][1] = eq; }
  __syncthreads();
  int at = 0, seen = 0;   // blocks chosen and equals met before this warp's
  for (int i = 0; i < w; ++i) { at += sums[i][0]; seen += sums[i][1]; }
  at += min(ties, seen);
  each([&](int i, unsigned long long k) {
    const bool is_eq = k == T && k != kAlways;
    const unsigned e = __ballot_sync(kFull, is_eq);
    const bool take = k > T || k == kAlways || (is_eq && seen + __popc(e & below) < ties);
    const unsigned t = __ballot_sync(kFull, take);
    if (take) ids[at + __popc(t & below)] = i;
    at += __popc(t);
    seen += __popc(e);
  });
}

__global__ void __launch_bounds__(kST, 1) k_select_blocks(const __grid_constant__ SelectArgs a) {
  __shared__ double qs[kHS][kD];
  __shared__ bool last;
  const int b = blockIdx.z, kv = blockIdx.y, pair = b * a.n_kv_heads + kv;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int h0 = a.heads.start[kv], nh = a.heads.start[kv + 1] - h0;
  // a row of the KV head's query heads; heads are scored four at a time: an absent one repeats the last
  auto head_row = [&](int r) { return static_cast<int64_t>(b) * a.n_q_heads + a.heads.head[h0 + r]; };
  wait_for_grid();
  launch_dependents();
  double first[4];   // this warp's first row, loaded beside the length
  if (nh) load_row_f64(a, head_row(min(w, min(kHS, nh) - 1)), lane, first);
  const int len = max(0, min(a.len[b], a.capacity));
  const int nb = (len + TQ_BLOCK - 1) / TQ_BLOCK;
  if (nb > a.n_select) {   // else every block is chosen and no score is needed
    int rotated = -1;      // first of the rotated heads in qs
    for (int chunk = blockIdx.x; chunk * kSW * kBPW < nb; chunk += gridDim.x) {
      const int blk0 = (chunk * kSW + w) * kBPW;
      // the bounds are on their way while the heads are rotated; blocks past the last repeat it
      uint2 lo2[kBPW], hi2[kBPW];
#pragma unroll
      for (int i = 0; i < kBPW; ++i) {
        const uint2* p = reinterpret_cast<const uint2*>(
            a.bounds + (static_cast<int64_t>(pair) * a.n_blocks + min(blk0 + i, nb - 1)) * 2 * kD) + lane;
        lo2[i] = p[0];
        hi2[i] = p[32];
      }
      double best = nh ? -INFINITY : 0.0;   // of block blk0 + lane / 4
      for (int r0 = 0; r0 < nh; r0 += kHS) {
        const int nr = min(kHS, nh - r0);
        if (rotated != r0) {
          __syncthreads();
          for (int r = w; r < (nr + kHG - 1) / kHG * kHG; r += kSW) {
            double v[4];
            if (rotated < 0 && r == w) {
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = first[i];
            } else {
              load_row_f64(a, head_row(r0 + min(r, nr - 1)), lane, v);
            }
            rotate_row_f64(a.grouped, lane, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) qs[r][4 * lane + i] = v[i];
          }
          __syncthreads();
          rotated = r0;
        }
        for (int g = 0; g < nr; g += kHG) {
          double q[kHG][4];
#pragma unroll
          for (int h = 0; h < kHG; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) q[h][i] = qs[g + h][4 * lane + i];
          double s[kBPW * kHG];   // (block, head) partial sums of this lane's channels
#pragma unroll
          for (int i = 0; i < kBPW; ++i) {
            const float lo[4] = {half_lo(lo2[i].x), half_hi(lo2[i].x), half_lo(lo2[i].y), half_hi(lo2[i].y)};
            const float hi[4] = {half_lo(hi2[i].x), half_hi(hi2[i].x), half_lo(hi2[i].y), half_hi(hi2[i].y)};
#pragma unroll
            for (int h = 0; h < kHG; ++h) s[i * kHG + h] = 0.0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // fp32 sums of two fp16 numbers would round: fp64 keeps them
              const double l = lo[c], u = hi[c], mid = l + u, rad = u - l;
#pragma unroll
              for (int h = 0; h < kHG; ++h) s[i * kHG + h] = fma(q[h][c], mid, fma(fabs(q[h][c]), rad, s[i * kHG + h]));
            }
          }
          // Sums over the lanes: each exchange halves the results a lane carries, 32 results end in
          // 32 lanes (block lane / 4, head lane % 4) after 31 exchanges that overlap.
          static_assert(kBPW * kHG == 32, "a result per lane");
#pragma unroll
          for (int m = 16, n = 16; m >= 1; m >>= 1, n >>= 1) {
            const bool up = lane & m;
#pragma unroll
            for (int i = 0; i < n; ++i) {
              const double mine = up ? s[i + n] : s[i], theirs = up ? s[i] : s[i + n];
              s[i] = mine + shfl_xor_d(theirs, m);
            }
          }
          // the largest over the four heads; a NaN stays
          double x = s[0];
#pragma unroll
          for (int m = 1; m <= 2; m <<= 1) {
            const double o = shfl_xor_d(x, m);
            x = isnan(o) || o > x ? o : x;
          }
          if (isnan(x) || x > best) best = x;
        }
      }
      const int blk = blk0 + (lane >> 2);
      if ((lane & 3) == 0 && blk < nb)
        a.keys[static_cast<int64_t>(pair) * a.n_blocks + blk] =
            blk < a.n_sink || blk >= nb - a.n_recent ? kAlways : order_key(best);
    }
  }
  // the last block of threads of this (sequence, KV head) picks
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();   // after the barrier: it stands for all threads' keys
    last = atomicAdd(a.counters + pair, 1) == static_cast<int>(gridDim.x) - 1;
    if (last) a.counters[pair] = 0;
  }
  __syncthreads();
  if (last) {
    __threadfence();
    pick_blocks(a, pair, nb);
  }
}

}  // namespace

tq_status launch_block_bounds(const tq_quantizer* q, const tq_kv_cache* c, void* bounds, int n_tokens, cudaStream_t st) {
  BoundsArgs a;
  a.idx = c->keys.idx;
  a.norms = c->keys.norms;
  a.len = c->len_dev;
  a.bounds = static_cast<__half*>(bounds);
  a.tab = q->dev;
  a.n_kv_heads = c->n_kv_heads;
  a.capacity = c->capacity;
  a.n_tokens = n_tokens;
  a.n_blocks = block_count(c->capacity);
  if (q->mode == TQ_MODE_GROUPED) {
    a.scale0 = q->lv_scale[0] / std::sqrt(32.f);
    a.scale1 = q->lv_scale[1] / std::sqrt(96.f);
  } else {
    a.scale0 = q->lv_scale[0] / std::sqrt(static_cast<float>(kD));
    a.scale1 = 0.f;
  }
  a.n_norms = q->layout.n_norms;
  // the blocks that n_tokens tokens can touch, wherever they begin
  const int64_t span = (static_cast<int64_t>(n_tokens) + TQ_BLOCK - 2) / TQ_BLOCK + 1;
  const int64_t most = span < a.n_blocks ? span : a.n_blocks;
  // up to 8 blocks a warp, but several rounds over the SMs so that the last one is short
  const int64_t all = most * c->n_kv_heads * c->batch;
  a.per_warp = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, all / (2 * 32 * std::max(1, sm_count(q->device))))));
  const int64_t per_cta = static_cast<int64_t>(a.per_warp) * kBW;
  const dim3 grid(static_cast<unsigned>((most + per_cta - 1) / per_cta), c->n_kv_heads, c->batch);
  const int bits = q->mode == TQ_MODE_PROD ? q->bits - 1 : q->bits;
  void (*kernel)(BoundsArgs);
  switch (q->mode == TQ_MODE_GROUPED ? 4 + bits : bits) {
    case 1: kernel = k_block_bounds<1, 0>; break;
    case 2: kernel = k_block_bounds<2, 0>; break;
    case 3: kernel = k_block_bounds<3, 0>; break;
    case 4: kernel = k_block_bounds<4, 0>; break;
    case 5: kernel = k_block_bounds<2, 1>; break;
    case 6: kernel = k_block_bounds<3, 2>; break;
    default: kernel = k_block_bounds<4, 3>; break;
  }
  return launch_early(kernel, grid, 32 * kBW, 0, st, a) == cudaSuccess ? TQ_OK : TQ_ECUDA;
}

size_t select_scratch_bytes(const tq_kv_cache* c) {
  return static_cast<size_t>(c->batch) * c->n_kv_heads * block_count(c->capacity) * sizeof(unsigned long long);
}

tq_status launch_select_blocks(const tq_quantizer* q, const tq_kv_cache* c, const void* bounds, const void* query, int q_dtype,
                               int n_q_heads, const int32_t* head_map, int n_select, int n_sink, int n_recent, int32_t* ids,
                               void* workspace, cudaStream_t st) {
  SelectArgs a;
  a.bounds = static_cast<const __half*>(bounds);
  a.q = query;
  a.len = c->len_dev;
  a.tab = q->dev;
  a.ids = ids;
  a.counters = static_cast<int*>(workspace);
  a.keys = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) + kWorkspaceHeader);
  a.n_kv_heads = c->n_kv_heads;
  a.capacity = c->capacity;
  a.n_q_heads = n_q_heads;
  a.n_blocks = block_count(c->capacity);
  a.n_select = n_select;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.q_dtype = q_dtype;
  a.grouped = q->mode == TQ_MODE_GROUPED;
  fill_head_lists(n_q_heads, c->n_kv_heads, head_map, &a.heads);
  const int64_t chunks = (a.n_blocks + kSW * kBPW - 1) / (kSW * kBPW), pairs = static_cast<int64_t>(c->n_kv_heads) * c->batch;
  const int64_t sms = std::max(1, sm_count(q->device)), per = (chunks * pairs + sms - 1) / sms;   // chunks of a block of threads
  const dim3 grid(static_cast<unsigned>((chunks + per - 1) / per), c->n_kv_heads, c->batch);
  return launch_early(k_select_blocks, grid, kST, 0, st, a) == cudaSuccess ? TQ_OK : TQ_ECUDA;
}

}  // namespace tq
