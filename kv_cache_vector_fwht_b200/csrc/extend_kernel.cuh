// Attention of several query tokens over the packed cache on the tensor cores (sm_100a):
// tq_extend_attention, and over listed blocks tq_decode_attention_blocks.
//
// Mathematics. For query row r (one token and one head of a KV head's group) and cached token i
//   s_ri = n16_i ( <q'_r, c[idx_i]> + rho_i <Sq'_r, 2 sigma_i - 1> ) * const,   rho = r16 / n16,
// so a token's packed key is ONE row of a matrix operand: the 128 level values of its codes and
// (prod) 128 signs of size rho, and the token's norm is a factor of its whole row of scores. The
// query side is [q' | Sq'] with q' = H (s . q), Sq' = S_rot q'. Both products of the attention run
// on tcgen05 with the TOKENS along M:
//   S^T [128 tokens x rows] = K' [128 x 128 or 256] . Q'^T      A = K' in tensor memory, B = Q' in shared memory
//   O^T [128 channels x rows] += V^T [128 x 128 tokens] . P      A = V^T, B = P, both in shared memory
// The rows (tokens x heads of the group) are N: a decode step with 8 heads costs an N = 16
// product instead of a 128-row tile padded from 8, and the same kernel serves 1 to 128 rows.
// A token is a lane: its norm, its mask position and its softmax weights live in one thread.
//
// One block of threads per SM works on one KV head, up to 128 query rows and a range of 128-token
// tiles (two 64-token blocks each, listed or consecutive); its warps have roles:
//   loader (1 warp)    packed rows of a tile to a shared ring by bulk copies, several tiles ahead;
//   K (4 or 8 warps)   thread = token: codes to fp16 levels by byte permutes (packed.cuh), signs by
//                      bit arithmetic, written to tensor memory (2 to 4 buffers);
//   V (4 or 8 warps)   thread = token: v = mn16 + code s16 in fp16 (code exact, one rounding), to
//                      shared memory (2 or 3 buffers); tokens past the end are zero rows;
//   MMA (1 thread)     issues S^T of unit u + 2, then O^T of unit u;
//   softmax (2 x 4)    two streams: the even and the odd tiles for up to 64 rows, the lower and the
//                      upper 64 rows beyond. Each has its own score and output columns, reference
//                      maxima and sums, so one's exponentials run under the other's products.
// Softmax in base 2 relative to a reference per row that is raised only when a score exceeds
// it by more than 15 (one vote a unit; then the stream's outputs in tensor memory and its sums
// are scaled), so p <= 2^15 fits fp16. Statistics and sums in fp32. Rounded to fp16 (relative 2^-11
// each): q', Sq' and rho, p, v; the levels are scaled by a common factor that brings them
// within 2^-12.9 of fp16 numbers.
//
// Bounds: a long decode reads 164 bytes a token and KV head (4-bit keys and values) and spends 1240
// thread instructions on it, most of them unpacking: 131072 tokens x 8 KV heads x 8 heads take 68 us (2.5
// TB/s), issue slots 62 % and ALU pipe 58 % busy. A chunk of a prompt (128 rows) is bound by the softmax's
// instructions: 2048 tokens over 16384, 28/4 heads, take 780 us (0.58 PFLOP/s of products, mask counted
// out), issue slots 55 %, tensor pipe 30 %. One short token (333 cached) takes 9.8 us, nearly all latency.
#pragma once

#include <cmath>

#include "packed.cuh"

namespace tq {
namespace ext {

constexpr int kTile = 128;              // tokens of a tile
constexpr int kMaxStages = 6;
constexpr int kMaxKeyBufs = 4, kMaxValueBufs = 3;
constexpr int kMaxList = 64;            // sequences whose block counts are listed one by one
// A reference is raised when a score exceeds it by more than this (base 2): weights reach 2^15 in fp16. It is
// raised to the tile's maximum less reference_gap. At a limit of 8, a tenth of the units of a 64-row stream raised
// (each costs three units' time); at 15 hardly any but a stream's first.
constexpr float kTau = 15.f;
// Weights below 2^-14 are subnormal in fp16 and off by up to 2^-25 each: next to one large weight, a context of n
// tokens that share the rest may lose n 2^-25 of the sum. References are taken so far below the maximum that this
// stays under 2^-11, half a step of fp16, for up to 2^24 tokens of a block's range: not at all for up to 128 tiles (a
// gap of 8 for every length cost the chunk 17 %: references are raised more often).
__device__ __forceinline__ float reference_gap(int tiles) { return static_cast<float>(min(10, max(0, 25 - __clz(tiles - 1)))); }
constexpr float kNoRef = -3e38f;        // reference of a row that has seen nothing: below every finite score
// The query rows of a tile are rounded to fp16 at one common scale (a power of two, by the largest coordinate)
// while their largest coordinates lie within 2^8 of each other: the smallest row's rotated coordinates are then
// 2^-10.5 in the root mean square or more, far above fp16's 2^-14. Beyond that each row has a scale of its own and
// its column of scores a factor, multiplied out in tensor memory by the code that raises references, which every
// unit of such a tile then runs (a factor beside the reference, in every unit's arithmetic, cost the chunk 12 %;
// this costs it 1.4 %).
constexpr int kSpread = 8;
// Logits are S sc - reference in one fused step, which leaves S sc unrounded where the reference is a rounded
// S sc: next to a logit of 2^23 the two are up to a half apart, at 2^30 64. |S| is at most 45 (a query row) x 62 (a
// row of levels) x 2 (prod), 2^12.5, so beyond this score factor a unit that raises rounds S sc first, and its maximum
// has a weight of 1 whatever its size.
constexpr float kLargeFactor = 0x1p10f;
constexpr int kNowhere = 0x40000000;    // position of a token that does not exist
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kPartFloats = 132;        // partial record: m, l, 0, 0, o[128]

struct ExtendArgs {
  const uint8_t* k_idx;
  const uint8_t* k_sgn;
  const uint8_t* k_nrm;
  const uint8_t* v_q;
  const uint8_t* v_par;
  const int32_t* len;
  const int32_t* blocks;    // nullable: (sequence, KV head, n_select) listed blocks
  const DevTables* tab;
  const void* q;
  void* out;
  float* part;              // partial records, slot = block of threads
  int* counters;
  int* err;
  int64_t qb, qh, qt, ob, oh, ot;
  int q_dtype, out_dtype;
  int batch, n_kv_heads, capacity, n_tokens, n_select, n_blocks, causal;
  int row_tiles;            // tiles of N query rows of the KV head with most of them
  int mode, bits0, bits1;   // code bits (grouped: outliers, then the others)
  int idx_bytes, sgn_bytes, nrm_bytes, vq_bytes, vbits;
  int stages, stage_bytes;  // ring of raw tiles
  int key_bufs, value_bufs; // operand buffers: tensor memory, shared memory
  int scal_ring;            // tiles whose score factors are kept (a power of two >= key_bufs + 2)
  float key_scale0, key_scale1;   // level scale / sqrt(channels) of the groups
  float sketch_ratio;       // rho = sketch_ratio * r16 / n16
  float scale_log2;
  int whole;                // no item is split: blocks of threads go by rows, then by sequences
  int uniform_splits;       // batch > kMaxList: splits of every sequence
  int tail_from, tail_splits;   // the last sequence's items from tail_from on have tail_splits splits
  int first[kMaxList + 1];  // first block of threads of each sequence
  int16_t splits[kMaxList];
  HeadLists heads;
};

// Shared-memory plan for N query rows and K columns of the key operand.
__host__ __device__ constexpr int stream_rows(int n) { return n <= 64 ? n : n / 2; }
__host__ __device__ constexpr int p_bytes(int n) { return stream_rows(n) / 8 * 2048; }
// Warpgroups that unpack keys, and as many that unpack values: two each where the softmax threads
// leave them the registers. One warp unpacks at about 5 cycles an instruction (latencies), so a
// decode step (N = 16) is bound by it: 131072 tokens x 8 heads took 93 us with one warpgroup each, 72
// with two; 35 rows (N = 48) 86 and 73 us. From 64 rows on, where the softmax bounds the kernel and
// needs 152 registers a thread, two would have 40 each and lose (a prompt's chunk 849 against 957 us).
__host__ __device__ constexpr int unpack_groups(int n) { return n <= 48 ? 2 : 1; }
// Stages of the raw ring that hold the tiles of group g, those j with j % groups == g: stage g, g + groups, ... A group
// waits for its own tiles alone, so a stage never changes hands: one whose last tile was another group's may still be
// waiting for that tile, and a wait for the next one, of the parity of the tile before it, would pass at once.
__host__ __device__ constexpr int group_stages(int stages, int groups, int g) { return (stages + groups - 1 - g) / groups; }
// K, V, 8 softmax, MMA, loader, and 2 warps that fill the last warpgroup
__host__ __device__ constexpr int block_threads(int n) { return 32 * (8 * unpack_groups(n) + 12); }
constexpr int kVBytes = kTile * kD * 2;
constexpr int kMiscBytes = 2176;
__host__ __device__ constexpr int smem_fixed(int n, int k, int value_bufs, int scal_ring) {
  return n * k * 2 + value_bufs * kVBytes + 2 * p_bytes(n) + kMiscBytes + scal_ring * kTile * 4;
}

struct Misc {
  uint64_t raw_full[kMaxStages], raw_empty[kMaxStages];
  uint64_t k_full[kMaxKeyBufs], k_empty[kMaxKeyBufs], v_full[kMaxValueBufs], v_empty[kMaxValueBufs];
  uint64_t s_full[2], p_full[2], p_empty[2];
  uint64_t hada, q_in, hada_full, rot, sq_in, sq_full, q_full;
  uint32_t tmem;
  int last;
  int poison[4];            // per value group: lowest position of a non-finite cached value
  int sizes[8];             // row sizes of each softmax warp: the largest << 8 | the smallest
  int pos0[16][2];          // first position of a tile's two halves, by tile mod 16
  alignas(16) int limit[128];   // per row: positions it attends to
  alignas(16) float ref[2][64];   // negated references
  alignas(16) float fac[2][64];
  alignas(16) uint8_t size[128];  // row_size of each row
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc fits");

// Place in a ring of n, and the parity of its turn.
struct Ring {
  int i, turn;
  __device__ __forceinline__ Ring(int start) : i(start), turn(0) {}
  __device__ __forceinline__ void step(int by, int n) {
    i += by;
    if (i >= n) { i -= n; turn ^= 1; }
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
// The sizes of K query rows, four coordinates of each a lane: row i's in the lanes with lane / (32 / P) == i, P the power
// of two from K on. A row's size is the exponent (plus 127) of the power of two that brings its largest coordinate
// to 2 .. 4; 0 for a row that sets no scale: all zeros (or next to it), or not finite.
template <int K>
__device__ __forceinline__ int row_sizes(const float (&v)[K][4], int lane) {
  constexpr int P = K <= 2 ? 2 : K <= 4 ? 4 : 8;
  uint32_t m[P] = {};
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) m[i] = max(m[i], __float_as_uint(v[i][k]) & 0x7fffffffu);   // NaN is above infinity
#pragma unroll
  for (int h = P / 2, s = 16; h >= 1; h >>= 1, s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const uint32_t mine = up ? m[i + h] : m[i], theirs = up ? m[i] : m[i + h];
      m[i] = max(mine, __shfl_xor_sync(kFull, theirs, s));
    }
  }
#pragma unroll
  for (int s = 16 / P; s >= 1; s >>= 1) m[0] = max(m[0], __shfl_xor_sync(kFull, m[0], s));
  const int e = static_cast<int>(m[0] >> 23);
  return e == 0 || e == 255 ? 0 : max(67, e - 1);
}
// Registers a thread of this warpgroup may use from here on.
template <int R>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(R)); }
// Barrier of a stream's 128 threads that tells each whether any of them asked.
__device__ __forceinline__ bool named_any(int id, bool ask) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ask)), "r"(id)
      : "memory");
  return r != 0;
}
// One warp's arrival after all of its lanes' writes.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
constexpr uint32_t kBf16AB = (1u << 7) | (1u << 10);       // instruction descriptor: A and B bf16
constexpr uint32_t kMnMajorAB = (1u << 15) | (1u << 16);   // instruction descriptor: A and B M/N-major

// Operand position of rotated coordinate c (the inverse of level_channel) in a run of `bits`-bit codes.
__device__ __forceinline__ int operand_position(int bits, int c) {
  if (bits == 1) {
    const int i = c & 31;
    return (c & ~31) + (i < 16 ? 2 * i : 2 * (i - 16) + 1);
  }
  if (bits == 2) {
    const int i = c & 15;
    return (c & ~15) + 4 * (i & 3) + (i >> 2);
  }
  return c;
}

// Unpack the index words of 32 U channels to 16 U operand pairs in tensor memory; SCALED: times g.
// 32 channels at a time, the next words loaded ahead: the loop is kept rolled, because five roles
// share an SM sub-partition's instruction fetch.
template <int BITS, int U, bool SCALED>
__device__ __forceinline__ void key_units(const uint8_t* row, const Levels& lv, __half2 g, uint32_t tcol) {
  constexpr int NP = level_pairs(BITS), WU = 16 / NP;   // pairs of a word, words of 32 channels
  uint32_t w[WU], n[WU];
  auto load = [&](int u) {
    const uint8_t* p = row + 4 * WU * u;
    if constexpr (!SCALED && WU == 4) {   // rows of 16, 32 or 64 bytes; grouped rows are aligned to words
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      n[0] = x.x; n[1] = x.y; n[2] = x.z; n[3] = x.w;
    } else if constexpr (!SCALED && WU == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      n[0] = x.x; n[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < WU; ++i) n[i] = reinterpret_cast<const uint32_t*>(p)[i];
    }
  };
  load(0);
#pragma unroll 1
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < WU; ++i) w[i] = n[i];
    if (u + 1 < U) load(u + 1);
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < WU; ++i) unpack_levels<BITS>(w[i], lv, *reinterpret_cast<uint32_t(*)[NP]>(r + NP * i));
    if constexpr (SCALED) {
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = h2bits(__hmul2(bits_h2(r[i]), g));
    }
    tmem_st16(tcol + 16 * u, r);
  }
}

// Channel of operand position m of V^T: chunks of 8 positions, pairs (code i, code i + 4) of a
// word of 4-bit codes, (code i, code i + 8) of 2-bit ones.
__device__ __forceinline__ int value_channel(int vbits, int m) {
  const int chunk = m >> 3, p = m & 7;
  if (vbits == 4) return 8 * chunk + (p >> 1) + 4 * (p & 1);
  return 16 * (chunk >> 1) + 4 * (chunk & 1) + (p >> 1) + 8 * (p & 1);
}
// Code pairs of a masked word field as exact fp16 numbers: 1024 + 2^k code, minus 1024, over 2^k.
template <int K>
__device__ __forceinline__ __half2 code_pair(uint32_t w, uint32_t mask) {
  const __half2 t = bits_h2((w & mask) | 0x64006400u);
  if constexpr (K == 0) return __hsub2(t, bits_h2(0x64006400u));
  const __half2 inv = __float2half2_rn(1.f / (1 << K)), off = __float2half2_rn(-1024.f / (1 << K));
  return __hfma2(t, inv, off);
}

// The rows of this thread's 32-token warp reduced: v[i] over the lanes, result i in the lanes
// with lane / 2 == i (16 values in 16 exchanges).
template <typename F>
__device__ __forceinline__ float reduce16(float (&v)[16], int lane, F f) {
#pragma unroll
  for (int h = 8, m = 16; h >= 1; h >>= 1, m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float mine = up ? v[i + h] : v[i], theirs = up ? v[i] : v[i + h];
      v[i] = f(mine, __shfl_xor_sync(kFull, theirs, m));
    }
  }
  return f(v[0], __shfl_xor_sync(kFull, v[0], 1));
}

// Store four channels of a query row's output at element `at`, times f.
__device__ __forceinline__ void store_row(const ExtendArgs& a, int64_t at, float4 v, float f) {
  v.x *= f; v.y *= f; v.z *= f; v.w *= f;
  if (a.out_dtype == TQ_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = v;
  } else if (a.out_dtype == TQ_BF16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(h2bits(__floats2half2_rn(v.x, v.y)), h2bits(__floats2half2_rn(v.z, v.w)));
  }
}

template <int N>
__global__ void __launch_bounds__(block_threads(N), 1) k_extend(const __grid_constant__ ExtendArgs a) {
  constexpr int NS = stream_rows(N);          // rows of a stream
  constexpr bool kByRows = N > 64;            // streams split the rows (else the tiles)
  constexpr int kG = unpack_groups(N);
  constexpr int wV = 4 * kG, wS = 8 * kG, wM = wS + 8, wL = wM + 1;   // first warps of the roles
  // tensor-memory columns: K' buffers (64 or 128 columns each), two of S^T, two of O^T
  constexpr uint32_t kSlot = NS <= 32 ? 32 : 64, kS0 = NS <= 32 ? 384 : 256, kO0 = kS0 + 2 * kSlot;

  extern __shared__ __align__(1024) uint8_t smem[];
  const bool prod = a.mode == TQ_MODE_PROD;
  const int kcols = prod ? 2 * kD : kD;
  const uint32_t kb_cols = kcols / 2;
  uint8_t* sQ = smem;
  uint8_t* sV = sQ + N * kcols * 2;
  uint8_t* sP = sV + a.value_bufs * kVBytes;
  Misc& ms = *reinterpret_cast<Misc*>(sP + 2 * p_bytes(N));
  float* scal = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(&ms) + kMiscBytes);   // [tile mod ring][token]
  uint8_t* sRaw = reinterpret_cast<uint8_t*>(scal + a.scal_ring * kTile);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&ms.raw_full[i], 1);
      mbar_init(&ms.raw_empty[i], 8);
    }
    for (int i = 0; i < kMaxKeyBufs; ++i) {
      mbar_init(&ms.k_full[i], 4);
      mbar_init(&ms.k_empty[i], 1);
    }
    for (int i = 0; i < kMaxValueBufs; ++i) {
      mbar_init(&ms.v_full[i], 4);
      mbar_init(&ms.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_full[i], 4);
      mbar_init(&ms.p_empty[i], 1);
    }
    mbar_init(&ms.hada, 1);
    mbar_init(&ms.q_in, 8);
    mbar_init(&ms.hada_full, 1);
    mbar_init(&ms.rot, 1);
    mbar_init(&ms.sq_in, 8);
    mbar_init(&ms.sq_full, 1);
    mbar_init(&ms.q_full, 8);
    fence_mbar_init();
  }

  // ---- which sequence, KV head, query rows and range of tiles
  int b, local, n_splits;
  const bool whole = a.whole;   // no item is split: the sequences' last rows first, then the rows before them
  if (whole) {
    local = blockIdx.x / a.n_kv_heads;
    b = local % a.batch;
    local = local / a.batch * a.n_kv_heads + blockIdx.x % a.n_kv_heads;
    n_splits = 1;
  } else if (a.batch <= kMaxList) {
    b = 0;
    while (static_cast<int>(blockIdx.x) >= a.first[b + 1]) ++b;
    local = blockIdx.x - a.first[b];
    n_splits = a.splits[b];
  } else {
    const int per = a.n_kv_heads * a.row_tiles * a.uniform_splits;
    b = blockIdx.x / per;
    local = blockIdx.x - b * per;
    n_splits = a.uniform_splits;
  }
  int item = local / n_splits, split = local - item * n_splits;
  if (!whole && b == a.batch - 1 && item >= a.tail_from) {   // the launch's last items, more finely split
    local -= a.tail_from * n_splits;
    n_splits = a.tail_splits;
    item = a.tail_from + local / n_splits;
    split = local % n_splits;
  }
  const int kv = item % a.n_kv_heads;
  // the last rows see most of a causal context: they start first (first chunks of three prompts, where a
  // second round of short items fills what the long ones of the first leave: 55 us by sequences, 47 so)
  const int rt = a.row_tiles - 1 - item / a.n_kv_heads;
  const int head0 = a.heads.start[kv], group = a.heads.start[kv + 1] - head0;
  const int row0 = rt * N;
  const int rows = min(N, group * a.n_tokens - row0);
  wait_for_grid();   // what precedes is done; before the tensor memory is taken, which it may still hold
  if (rows <= 0) return;
  launch_dependents();
  const int len = max(0, min(a.len[b], a.capacity));
  const int shift = a.causal ? a.n_tokens - 1 : 0;
  auto row_limit = [&](int r) {   // positions row r of this tile attends to
    const int t = (row0 + r) / group;
    return max(0, min(len, a.causal ? len - shift + t : len));
  };
  const int top = row_limit(rows - 1), low = row_limit(0);
  const int64_t pair = static_cast<int64_t>(b) * a.n_kv_heads + kv;
  const int32_t* list = a.blocks ? a.blocks + pair * a.n_select : nullptr;
  const int all_tiles = list ? (len > 0 ? (a.n_select + 1) / 2 : 0) : (top + kTile - 1) / kTile;
  const int share = all_tiles / n_splits, more = all_tiles - share * n_splits;
  const int tile0 = split * share + min(split, more);
  const int nt = share + (split < more);

  // The softmax warps read the query rows for the largest norm while the others set up: warp w takes
  // rows w, w + 8, ..., several at a time so that their loads overlap. Up to 32 rows stay in registers;
  // more 16-bit ones wait where their operand rows will be (fp32 rows are read again). Lane l holds
  // channels 4 l .. 4 l + 3 (grouped: in the order of the operand's groups).
  constexpr int kRows = N / 8, kBatch = kRows <= 4 ? kRows : kRows % 4 == 0 ? 4 : 3;
  constexpr bool kKeep = kRows <= 4;
  float qv[kBatch][4] = {};
  auto load_batch = [&](int i0) {
    int64_t at[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {   // rows past the last repeat it
      const int r = row0 + min((warp - wS) + 8 * (i0 + i), rows - 1), t = r / group;
      at[i] = b * a.qb + a.heads.head[head0 + r - t * group] * a.qh + t * a.qt;
    }
    if (a.mode == TQ_MODE_GROUPED) {
      const uchar4 ch = *reinterpret_cast<const uchar4*>(a.tab->chan + 4 * lane);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        qv[i][0] = load_element(a.q, a.q_dtype, at[i] + ch.x);
        qv[i][1] = load_element(a.q, a.q_dtype, at[i] + ch.y);
        qv[i][2] = load_element(a.q, a.q_dtype, at[i] + ch.z);
        qv[i][3] = load_element(a.q, a.q_dtype, at[i] + ch.w);
      }
    } else if (a.q_dtype == TQ_F32) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float4 x = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at[i])[lane];
        qv[i][0] = x.x; qv[i][1] = x.y; qv[i][2] = x.z; qv[i][3] = x.w;
      }
    } else {
      uint2 x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) x[i] = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at[i])[lane];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (a.q_dtype == TQ_BF16) {
          qv[i][0] = __uint_as_float(x[i].x << 16); qv[i][1] = __uint_as_float(x[i].x & 0xffff0000u);
          qv[i][2] = __uint_as_float(x[i].y << 16); qv[i][3] = __uint_as_float(x[i].y & 0xffff0000u);
        } else {
          qv[i][0] = half_lo(x[i].x); qv[i][1] = half_hi(x[i].x); qv[i][2] = half_lo(x[i].y); qv[i][3] = half_hi(x[i].y);
        }
      }
    }
  };
  auto unpack16 = [&](uint2 x, float (&v)[4]) {
    if (a.q_dtype == TQ_BF16) {
      v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
      v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
    } else {
      v[0] = half_lo(x.x); v[1] = half_hi(x.x); v[2] = half_lo(x.y); v[3] = half_hi(x.y);
    }
  };
  const bool stash = !kKeep && a.q_dtype != TQ_F32;
  uint32_t sbits = 0;
  if (warp >= wS && warp < wM) {
    int small = 255, large = 0;
    auto sized = [&](int i0, const auto& v) {   // rows from the i0-th of this warp on; those that attend to nothing set no scale
      constexpr int K = sizeof(v) / sizeof(v[0]), lanes = K <= 2 ? 16 : K <= 4 ? 8 : 4;
      int e = row_sizes(v, lane);
      const int i = lane / lanes, r = (warp - wS) + 8 * (i0 + i);
      if (i < K) {
        if (r >= rows || (low == 0 && row_limit(r) == 0)) e = 0;
        if (e) {
          small = min(small, e);
          large = max(large, e);
        }
        if (lane % lanes == 0) ms.size[r] = static_cast<uint8_t>(e);
      }
    };
    sbits = a.tab->sign_bits[lane >> 3] >> (4 * (lane & 7));
    if (!kKeep && stash) {
      constexpr int kAhead = kRows % 8 == 0 ? 8 : 6;
#pragma unroll 1
      for (int i0 = 0; i0 < kRows; i0 += kAhead) {
        uint2 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {   // rows past the last repeat it
          const int r = row0 + min((warp - wS) + 8 * (i0 + i), rows - 1), t = r / group;
          x[i] = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + b * a.qb +
                                               a.heads.head[head0 + r - t * group] * a.qh + t * a.qt)[lane];
        }
        float v[kAhead][4];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int r = (warp - wS) + 8 * (i0 + i);
          *reinterpret_cast<uint2*>(sQ + (r >> 3) * 16 * kcols + (r & 7) * 16 + (lane >> 1) * 128 + (lane & 1) * 8) = x[i];
          unpack16(x[i], v[i]);
        }
        sized(i0, v);
      }
    } else {
#pragma unroll 1
      for (int i0 = 0; i0 < kRows; i0 += kBatch) {
        if (8 * i0 < rows) load_batch(i0);
        sized(i0, qv);
      }
    }
    small = __reduce_min_sync(kFull, small);
    large = __reduce_max_sync(kFull, large);
    if (lane == 0) ms.sizes[warp - wS] = large << 8 | small;
  }

  if (warp == wM) {
    tmem_alloc(&ms.tmem, 512);
    tmem_relinquish();
  }
  if (tid < 4) ms.poison[tid] = 0x7fffffff;
  if (tid < N) ms.limit[tid] = tid < rows ? row_limit(tid) : 0;
  if (tid < 128) ms.ref[tid >> 6][tid & 63] = -kNoRef;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = ms.tmem;
  const uint32_t tlane = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const int units = kByRows ? 2 * nt : nt;
  bool ok = true;

  // Registers move from the unpacking and issuing warpgroups to the softmax ones, whose threads hold a
  // logit and a sum for each of their stream's rows:
  //   N >= 64: 256 x 64 + 256 x 152 + 128 x 40 = 60416 of the launch's 640 x 96 = 61440
  //   N = 48:  512 x 48 + 256 x 128 + 128 x 40 = 62464 of 896 x 72 = 64512
  //   N = 32:  512 x 64 + 256 x 96 + 128 x 40 = 62464 of 896 x 72
  // A warpgroup changes its share once (a second change would need the warpgroup synchronised in
  // between): what follows the roles is done by the softmax warps.
  constexpr bool kMove = N >= 32;
  if (warp < wV) {
    if (kMove) reg_dec<N == 48 ? 48 : 64>();
    // ------------------------------------------------------------------ K: thread = token
    const Levels lv0 = load_levels(a.tab, 0), lv1 = load_levels(a.tab, 1);
    const int tok = tid & 127;
    const int o_sgn = kTile * a.idx_bytes, o_nrm = o_sgn + kTile * a.sgn_bytes;
    const int grp = kG == 1 ? 0 : warp >> 2, own_stages = group_stages(a.stages, kG, grp);
    Ring st(0), kb(grp);
#pragma unroll 1
    for (int j = grp; j < nt; j += kG, st.step(1, own_stages), kb.step(kG, a.key_bufs)) {
      const int stage = grp + kG * st.i;
      const uint8_t* raw = sRaw + stage * a.stage_bytes;
      if (ok) ok = mbar_wait_ns(&ms.raw_full[stage], st.turn, kWaitNs);
      if (ok && j >= a.key_bufs) ok = mbar_wait_ns(&ms.k_empty[kb.i], kb.turn ^ 1, kWaitNs);
      tc_fence_after();
      const uint32_t tk = tlane + kb_cols * kb.i;
      const uint8_t* row = raw + tok * a.idx_bytes;
      float factor;
      if (a.mode == TQ_MODE_GROUPED) {
        const uint32_t nn = *reinterpret_cast<const uint32_t*>(raw + o_nrm + 4 * tok);
        const float s0 = half_lo(nn) * a.key_scale0, s1 = half_hi(nn) * a.key_scale1;
        factor = fmaxf(s0, s1);
        const float inv = factor > 0.f ? 1.f / factor : 0.f;
        const __half2 g0 = __float2half2_rn(s0 * inv), g1 = __float2half2_rn(s1 * inv);
        const uint8_t* rest = row + 4 * storage_width_c(a.bits0);
        if (a.bits1 == 1) {
          key_units<2, 1, true>(row, lv0, g0, tk);
          key_units<1, 3, true>(rest, lv1, g1, tk + 16);
        } else if (a.bits1 == 2) {
          key_units<3, 1, true>(row, lv0, g0, tk);
          key_units<2, 3, true>(rest, lv1, g1, tk + 16);
        } else {
          key_units<4, 1, true>(row, lv0, g0, tk);
          key_units<3, 3, true>(rest, lv1, g1, tk + 16);
        }
      } else {
        switch (a.bits0) {
          case 1: key_units<1, 4, false>(row, lv0, __half2{}, tk); break;
          case 2: key_units<2, 4, false>(row, lv0, __half2{}, tk); break;
          case 3: key_units<3, 4, false>(row, lv0, __half2{}, tk); break;
          default: key_units<4, 4, false>(row, lv0, __half2{}, tk); break;
        }
        if (prod) {
          const uint32_t nn = *reinterpret_cast<const uint32_t*>(raw + o_nrm + 4 * tok);
          const float n16 = half_lo(nn);
          const uint32_t rho = h2bits(__float2half2_rn(n16 > 0.f ? half_hi(nn) / n16 * a.sketch_ratio : 0.f));
          factor = n16 * a.key_scale0;
          const uint4 sg = *reinterpret_cast<const uint4*>(raw + o_sgn + 16 * tok);
          uint32_t inv[4] = {~sg.x, ~sg.y, ~sg.z, ~sg.w};
#pragma unroll 1
          for (int u = 0; u < 4; ++u) {
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = sign_level(inv[0], i, rho);
            inv[0] = inv[1]; inv[1] = inv[2]; inv[2] = inv[3];
            tmem_st16(tk + 64 + 16 * u, r);
          }
        } else {
          factor = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(raw + o_nrm + 2 * tok))) * a.key_scale0;
        }
      }
      scal[(j & (a.scal_ring - 1)) * kTile + tok] = factor;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.raw_empty[stage]);
        mbar_arrive(&ms.k_full[kb.i]);
      }
    }
  } else if (warp < wS) {
    if (kMove) reg_dec<N == 48 ? 48 : 64>();
    // ------------------------------------------------------------------ V: thread = token
    const int tok = tid & 127;
    const int o_vq = kTile * (a.idx_bytes + a.sgn_bytes + a.nrm_bytes), o_par = o_vq + kTile * a.vq_bytes;
    const int grp = kG == 1 ? 0 : (warp - wV) >> 2, own_stages = group_stages(a.stages, kG, grp);
    Ring st(0), vb(grp);
#pragma unroll 1
    for (int j = grp; j < nt; j += kG, st.step(1, own_stages), vb.step(kG, a.value_bufs)) {
      const int stage = grp + kG * st.i;
      const uint8_t* raw = sRaw + stage * a.stage_bytes;
      if (ok) ok = mbar_wait_ns(&ms.raw_full[stage], st.turn, kWaitNs);
      if (ok && j >= a.value_bufs) ok = mbar_wait_ns(&ms.v_empty[vb.i], vb.turn ^ 1, kWaitNs);
      // until they have been used, the second buffer holds the rotation's matrix and the first the sketch's
      // (without the former: the second)
      if (ok && j == 1 && stash) ok = mbar_wait_ns(&ms.hada_full, 0, kWaitNs);
      if (ok && j == (stash ? 0 : 1) && prod) ok = mbar_wait_ns(&ms.sq_full, 0, kWaitNs);
      const int pos = ms.pos0[j & 15][tok >> 6] + (tok & 63);
      const bool there = pos < len;
      const uint32_t* par = reinterpret_cast<const uint32_t*>(raw + o_par + 16 * tok);
      uint8_t* dst = sV + vb.i * kVBytes + tok * 16;
      const uint8_t* src = raw + o_vq + tok * a.vq_bytes;
      // the lanes take the four groups in different orders, so that eight rows 64 (or 32) bytes
      // apart are read from different banks
      const int turn = a.vbits == 4 ? lane >> 1 : lane >> 2;
#pragma unroll 1
      for (int g0 = 0; g0 < 4; ++g0) {
        const int g = (g0 + turn) & 3;
        uint32_t p = there ? par[g] : 0u;
        if ((p & 0x7c00u) == 0x7c00u || (p & 0x7c000000u) == 0x7c000000u) {
          // inf or NaN: 0 * inf would reach rows that may not see this token, so the product gets
          // zeros and the rows that do see it are set to NaN at the end
          atomicMin(&ms.poison[g], pos);
          p = 0;
        }
        const __half2 mn = __half2half2(__low2half(bits_h2(p))), sc = __half2half2(__high2half(bits_h2(p)));
        if (a.vbits == 4) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(src + 16 * g);
          const uint32_t ws[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w = ws[i], v = w >> 8;
            uint4 o;
            o.x = h2bits(__hfma2(code_pair<0>(w, 0x000f000fu), sc, mn));
            o.y = h2bits(__hfma2(code_pair<4>(w, 0x00f000f0u), sc, mn));
            o.z = h2bits(__hfma2(code_pair<0>(v, 0x000f000fu), sc, mn));
            o.w = h2bits(__hfma2(code_pair<4>(v, 0x00f000f0u), sc, mn));
            *reinterpret_cast<uint4*>(dst + (4 * g + i) * 2048) = o;
          }
        } else {
          const uint2 w2 = *reinterpret_cast<const uint2*>(src + 8 * g);
          const uint32_t ws[2] = {w2.x, w2.y};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = ws[i], v = w >> 8;
            uint4 o;
            o.x = h2bits(__hfma2(code_pair<0>(w, 0x00030003u), sc, mn));
            o.y = h2bits(__hfma2(code_pair<2>(w, 0x000c000cu), sc, mn));
            o.z = h2bits(__hfma2(code_pair<4>(w, 0x00300030u), sc, mn));
            o.w = h2bits(__hfma2(code_pair<6>(w, 0x00c000c0u), sc, mn));
            *reinterpret_cast<uint4*>(dst + (4 * g + 2 * i) * 2048) = o;
            o.x = h2bits(__hfma2(code_pair<0>(v, 0x00030003u), sc, mn));
            o.y = h2bits(__hfma2(code_pair<2>(v, 0x000c000cu), sc, mn));
            o.z = h2bits(__hfma2(code_pair<4>(v, 0x00300030u), sc, mn));
            o.w = h2bits(__hfma2(code_pair<6>(v, 0x00c000c0u), sc, mn));
            *reinterpret_cast<uint4*>(dst + (4 * g + 2 * i + 1) * 2048) = o;
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ms.raw_empty[stage]);
        mbar_arrive(&ms.v_full[vb.i]);
      }
    }
  } else if (warp >= wM) {
    if (kMove) reg_dec<40>();
    if (warp == wL) {
    // ------------------------------------------------------------------ loader
    if (stash && nt > 0 && lane == 0) {
      mbar_expect_tx(&ms.hada, kD * kD * 2);
      bulk_g2s(sV + kVBytes, a.tab->r_umma[a.q_dtype == TQ_BF16], kD * kD * 2, &ms.hada);
    }
    if (prod && nt > 0 && lane == 0) {
      mbar_expect_tx(&ms.rot, kD * kD * 2);
      bulk_g2s(sV + (stash ? 0 : kVBytes), a.tab->s_umma, kD * kD * 2, &ms.rot);
    }
    const int o_sgn = kTile * a.idx_bytes, o_nrm = o_sgn + kTile * a.sgn_bytes, o_vq = o_nrm + kTile * a.nrm_bytes,
              o_par = o_vq + kTile * a.vq_bytes;
    // lane = plane + 5 * half
    const int plane = lane % 5, half = lane / 5;
    const uint8_t* base = plane == 0 ? a.k_idx : plane == 1 ? a.k_sgn : plane == 2 ? a.k_nrm : plane == 3 ? a.v_q : a.v_par;
    const int rb = plane == 0 ? a.idx_bytes : plane == 1 ? a.sgn_bytes : plane == 2 ? a.nrm_bytes : plane == 3 ? a.vq_bytes : 16;
    const int off = plane == 0 ? 0 : plane == 1 ? o_sgn : plane == 2 ? o_nrm : plane == 3 ? o_vq : o_par;
    const int row_bytes = a.idx_bytes + a.sgn_bytes + a.nrm_bytes + a.vq_bytes + 16;
    int j = 0;
    Ring ring(0), next(0);   // of tile j's group and, with two groups, of the other one
    int turn_stages = group_stages(a.stages, kG, 0), next_stages = group_stages(a.stages, kG, kG - 1);
#pragma unroll 1
    for (; j < nt; ++j) {
      const int st = j % kG + kG * ring.i;
      if (j / kG >= turn_stages) ok = mbar_wait_ns(&ms.raw_empty[st], ring.turn ^ 1, kWaitNs);
      if (!ok) break;
      int p[2], n[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 2 * (tile0 + j) + h;
        int blk = i;
        if (list) blk = i < a.n_select ? list[i] : -1;
        const bool in = blk >= 0 && blk < a.n_blocks && blk * TQ_BLOCK < len;
        p[h] = in ? blk * TQ_BLOCK : kNowhere;
        n[h] = in ? min(TQ_BLOCK, (len - blk * TQ_BLOCK + 15) & ~15) : 0;   // within the capacity, a multiple of 16
      }
      if (lane == 0) {
        ms.pos0[j & 15][0] = p[0];
        ms.pos0[j & 15][1] = p[1];
        mbar_expect_tx(&ms.raw_full[st], (n[0] + n[1]) * row_bytes);
      }
      __syncwarp();
      if (p[1] == p[0] + TQ_BLOCK) {   // consecutive blocks: one copy a plane (fewer, larger copies)
        n[0] += n[1];
        n[1] = 0;
      }
      const int mine = half == 0 ? n[0] : n[1], from = half == 0 ? p[0] : p[1];
      if (lane < 10 && mine > 0 && rb > 0)
        bulk_g2s(sRaw + st * a.stage_bytes + off + half * TQ_BLOCK * rb,
                 base + (pair * a.capacity + from) * rb, mine * rb, &ms.raw_full[st]);
      ring.step(1, turn_stages);
      if (kG == 2) {
        const Ring r = ring;
        ring = next;
        next = r;
        const int n = turn_stages;
        turn_stages = next_stages;
        next_stages = n;
      }
    }
    // if another role gave up, wait here for the copies that nothing else will wait for
#pragma unroll 1
    for (int k = max(0, j - kG * kMaxStages); k < j; ++k) {
      const int grp = k % kG, n = group_stages(a.stages, kG, grp), turn = k / kG;
      if (k + kG * n >= j) mbar_wait_ns(&ms.raw_full[grp + kG * (turn % n)], (turn / n) & 1, kWaitNs);   // the stage's last tile
    }
    } else if (warp == wM && nt > 0) {
    // ------------------------------------------------------------------ MMA
    if (elect_one()) {
      const uint32_t qsbo = 16u * kcols;   // bytes of 8 query rows
      const uint64_t q_desc = umma_desc(smem_u32(sQ), 128, qsbo);
      const uint64_t v_desc = umma_desc(smem_u32(sV), 128, 2048), p_desc = umma_desc(smem_u32(sP), 128, 2048);
      if (stash) {
        // H (s . q): D [128 x N] = rotation [128 x 128] . q^T, operands of the query's type (+-1: exact)
        ok = mbar_wait_ns(&ms.hada, 0, kWaitNs);
        if (ok) ok = mbar_wait_ns(&ms.q_in, 0, kWaitNs);
        if (ok) {
          tc_fence_after();
          const uint32_t id = umma_idesc_f16(128, N) | (a.q_dtype == TQ_BF16 ? kBf16AB : 0u);
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_f16(tbase + kS0, v_desc + (kVBytes >> 4) + 16 * k, q_desc + 16 * k, id, k > 0);
          umma_commit(&ms.hada_full);
        }
      }
      if (prod) {
        // S q: D [128 x N] = S_rot [128 x 128] . q'^T, the rows' copy in the sketch's column order
        if (ok) ok = mbar_wait_ns(&ms.rot, 0, kWaitNs);
        if (ok) ok = mbar_wait_ns(&ms.sq_in, 0, kWaitNs);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)   // 16 columns a step: two core matrices of 128 bytes
            umma_f16(tbase + kS0, v_desc + (stash ? 0 : kVBytes >> 4) + 16 * k, p_desc + 16 * k, umma_idesc_f16(128, N), k > 0);
          umma_commit(&ms.sq_full);
        }
      }
      if (ok) ok = mbar_wait_ns(&ms.q_full, 0, kWaitNs);
      Ring kb(0), vb(0);
      // S^T of unit u: its slot was read before the weights of unit u - 2 were complete
      auto scores = [&](int u) {
        const int s = u & 1;
        if (ok && (!kByRows || s == 0)) ok = mbar_wait_ns(&ms.k_full[kb.i], kb.turn, kWaitNs);
        if (!ok) return;
        tc_fence_after();
        const uint64_t bq = q_desc + (kByRows ? s * (NS / 8) * (qsbo >> 4) : 0);
        const uint32_t d = tbase + kS0 + kSlot * s, ak = tbase + kb_cols * kb.i;
#pragma unroll
        for (int k = 0; k < 8; ++k) umma_f16_ts(d, ak + 8 * k, bq + 16 * k, umma_idesc_f16(128, NS), k > 0);
        if (prod) {
#pragma unroll
          for (int k = 8; k < 16; ++k) umma_f16_ts(d, ak + 8 * k, bq + 16 * k, umma_idesc_f16(128, NS), 1);
        }
        umma_commit(&ms.s_full[s]);
        if (!kByRows || s == 1) {   // the tile's last unit
          umma_commit(&ms.k_empty[kb.i]);
          kb.step(1, a.key_bufs);
        }
      };
      // The scores of unit u + 2 are issued before the outputs of unit u, whose stream then waits
      // for one product and not for two.
#pragma unroll 1
      for (int u = -2; u < units && ok; ++u) {
        const int s = u & 1, i = u >> 1;
        if (u >= 0) {
          ok = mbar_wait_ns(&ms.p_full[s], i & 1, kWaitNs);
          if (!ok) break;
          tc_fence_after();
        }
        if (u + 2 < units) scores(u + 2);
        if (u >= 0) {
          if (ok && (!kByRows || s == 0)) ok = mbar_wait_ns(&ms.v_full[vb.i], vb.turn, kWaitNs);
          if (!ok) break;
          tc_fence_after();
          const uint64_t av = v_desc + vb.i * (kVBytes >> 4), bp = p_desc + s * (p_bytes(N) >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_f16(tbase + kO0 + kSlot * s, av + 16 * k, bp + 16 * k, umma_idesc_f16(128, NS) | kMnMajorAB, i > 0 || k > 0);
          umma_commit(&ms.p_empty[s]);
          if (!kByRows || s == 1) {
            umma_commit(&ms.v_empty[vb.i]);
            vb.step(1, a.value_bufs);
          }
        }
      }
    }
    }
  } else {
    // ------------------------------------------------------------------ softmax streams
    if (kMove) reg_inc<N == 32 ? 96 : N == 48 ? 128 : 152>();
    const int s = (warp - wS) >> 2, tok = (warp & 3) * 32 + lane;
    uint8_t* myP = sP + s * p_bytes(N);
    float qscale = 1.f;
    bool apart = false;   // the rows have scales of their own: every unit takes the way of those that raise
    if (nt > 0) {  // ---- the query operand: rotated rows, and S q for prod
      int small = 255, large = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        small = min(small, ms.sizes[i] & 255);
        large = max(large, ms.sizes[i] >> 8);
      }
      apart = large - small > kSpread;
      const int common = large ? large : 127;   // also of the rows that set no scale
      qscale = apart ? a.scale_log2 : a.scale_log2 * __uint_as_float(static_cast<uint32_t>(common) << 23);
      const float unit = __uint_as_float(static_cast<uint32_t>(254 - common) << 23) *
                         (a.mode == TQ_MODE_GROUPED ? 0.17677669529663688f : 0.08838834764831845f);
      auto own_factor = [&](int r) {   // from the common scale to the row's own
        const int own = ms.size[r], more = common - (own ? own : common), half = more >> 1;   // up to 186: in two steps
        return make_float2(__uint_as_float(static_cast<uint32_t>(127 + half) << 23),
                           __uint_as_float(static_cast<uint32_t>(127 + more - half) << 23));
      };
      if (stash) {
        // many 16-bit rows: on the tensor cores, which read them where the operand will be; a thread then
        // holds coordinate tok of its stream's half of the rows
        fence_async_smem();
        warp_arrive(&ms.q_in, lane);
        ok = mbar_wait_ns(&ms.hada_full, 0, kWaitNs);
        tc_fence_after();
        const bool rest = a.mode == TQ_MODE_GROUPED && tok >= 32;
        const int k = rest ? 32 + operand_position(a.bits1, tok - 32) : operand_position(a.bits0, tok);
        const int k2 = tok < 64 ? 2 * tok : 2 * (tok - 64) + 1;   // the sketch matrix's column order
        constexpr int kCols = (N / 2 + 15) / 16 * 16;
#pragma unroll 1
        for (int c = s * kCols; c < min(N, (s + 1) * kCols); c += 16) {
          uint32_t x[16];
          tmem_ld16_sync(tlane + kS0 + c, x);
          if (apart) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 f = own_factor(c + i);
              x[i] = __float_as_uint(__uint_as_float(x[i]) * f.x * f.y);
            }
          }
          uint8_t* col = sQ + (c >> 3) * 16 * kcols + (k >> 3) * 128 + (k & 7) * 2;
          uint8_t* pcol = sP + (c >> 3) * 2048 + (k2 >> 3) * 128 + (k2 & 7) * 2;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const __half h = __float2half_rn(__uint_as_float(x[i]) * unit);
            *reinterpret_cast<__half*>(col + (i >> 3) * 16 * kcols + (i & 7) * 16) = h;
            if (prod) *reinterpret_cast<__half*>(pcol + (i >> 3) * 2048 + (i & 7) * 16) = h;
          }
        }
        tc_fence_before();
      } else {
        const int last_stage = a.mode == TQ_MODE_GROUPED ? 4 : 16;   // grouped: 32-point blocks
        // kRot rows at a time: many rows for the overlap of their shuffles, one at a time (and less code to
        // fetch) where there are few
        constexpr int kRot = kKeep ? 1 : kBatch;
#pragma unroll 1
        for (int i0 = 0; i0 < kRows; i0 += kRot) {
          const int first = (warp - wS) + 8 * i0;
          if (!kKeep && first < rows) load_batch(i0);
          float v[kRot][4];
#pragma unroll
          for (int i = 0; i < kRot; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[i][k] = qv[i][k];
#pragma unroll
              for (int n = 1; kKeep && n < kBatch; ++n) v[i][k] = i0 == n ? qv[n][k] : v[i][k];
              v[i][k] = flip_sign(v[i][k] * unit, sbits, k);
            }
          if (apart) {
#pragma unroll
            for (int i = 0; i < kRot; ++i) {
              const float2 f = own_factor(first + 8 * i);
#pragma unroll
              for (int k = 0; k < 4; ++k) v[i][k] = v[i][k] * f.x * f.y;
            }
          }
          if (first < rows) {
#pragma unroll
            for (int i = 0; i < kRot; ++i) fwht_reg<4>(v[i]);
#pragma unroll
            for (int m = 1; m <= 16; m <<= 1) {
              if (m > last_stage) break;
#pragma unroll
              for (int i = 0; i < kRot; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float o = __shfl_xor_sync(kFull, v[i][k], m);
                  v[i][k] = lane & m ? o - v[i][k] : v[i][k] + o;
                }
            }
          }
#pragma unroll
          for (int i = 0; i < kRot; ++i) {
            const int r = first + 8 * i;
            uint8_t* qrow = sQ + (r >> 3) * 16 * kcols + (r & 7) * 16;
            uint8_t* prow = sP + (r >> 3) * 2048 + (r & 7) * 16;   // in the sketch matrix's column order
            if (r >= rows) {   // zeros: no row, no score above its reference
              if (lane < 16) {
                *reinterpret_cast<uint4*>(qrow + 128 * lane) = make_uint4(0, 0, 0, 0);
                if (prod) *reinterpret_cast<uint4*>(prow + 128 * lane) = make_uint4(0, 0, 0, 0);
              }
              continue;
            }
            const uint32_t h01 = h2bits(__floats2half2_rn(v[i][0], v[i][1])), h23 = h2bits(__floats2half2_rn(v[i][2], v[i][3]));
            if (a.mode != TQ_MODE_GROUPED && a.bits0 >= 3) {   // the operand's order is the coordinates'
              *reinterpret_cast<uint2*>(qrow + (lane >> 1) * 128 + (lane & 1) * 8) = make_uint2(h01, h23);
            } else {
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4) {
                const int c = 4 * lane + k4;
                const bool rest = a.mode == TQ_MODE_GROUPED && c >= 32;
                const int k = rest ? 32 + operand_position(a.bits1, c - 32) : operand_position(a.bits0, c);
                *reinterpret_cast<uint16_t*>(qrow + (k >> 3) * 128 + (k & 7) * 2) =
                    static_cast<uint16_t>((k4 < 2 ? h01 : h23) >> (16 * (k4 & 1)));
              }
            }
            if (prod) {   // columns c, c + 64 side by side: lane l < 16 pairs up with lane l + 16
              const uint32_t o01 = __shfl_xor_sync(kFull, h01, 16), o23 = __shfl_xor_sync(kFull, h23, 16);
              if (lane < 16)
                *reinterpret_cast<uint4*>(prow + 128 * lane) = make_uint4(prmt(h01, o01, 0x5410), prmt(h01, o01, 0x7632),
                                                                          prmt(h23, o23, 0x5410), prmt(h23, o23, 0x7632));
            }
          }
        }
      }
      fence_async_smem();
      if (prod) {
        warp_arrive(&ms.sq_in, lane);
        if (ok) ok = mbar_wait_ns(&ms.sq_full, 0, kWaitNs);
        tc_fence_after();
        // lane = sketch row j; a stream's warps take half of the query rows
        const int k = kD + operand_position(1, tok);
        constexpr int kCols = (N / 2 + 15) / 16 * 16;   // whole chunks of 16; the second stream takes the rest
#pragma unroll 1
        for (int c = s * kCols; c < min(N, (s + 1) * kCols); c += 16) {
          uint32_t x[16];
          tmem_ld16_sync(tlane + kS0 + c, x);
          uint8_t* col = sQ + (c >> 3) * 16 * kcols + (k >> 3) * 128 + (k & 7) * 2;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<__half*>(col + (i >> 3) * 16 * kcols + (i & 7) * 16) =
                __float2half_rn(__uint_as_float(x[i]) * 0.125f);
        }
        tc_fence_before();
        fence_async_smem();
      }
      warp_arrive(&ms.q_full, lane);
    }

    const float tau = apart ? -INFINITY : kTau;
    uint64_t sum[NS / 2];   // packed pairs of fp32 sums
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) sum[i] = 0;
    const int r_first = kByRows ? s * NS : 0;          // this stream's rows of the tile
    const int* limit = ms.limit + r_first;
    float* ref = ms.ref[s];
    const int mine = kByRows ? nt : (nt - s + 1) / 2;  // this stream's units
    // its columns that hold rows, in chunks of 16; the products' other columns are never read
    const int used = max(0, min(NS, ((rows + 15) & ~15) - r_first));
    const uint32_t tS = tlane + kS0 + kSlot * s, tO = tlane + kO0 + kSlot * s;
    const int lowest = kByRows ? row_limit(min(r_first, rows - 1)) : low;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      const int j = kByRows ? i : 2 * i + s;
      if (ok) ok = mbar_wait_ns(&ms.s_full[s], i & 1, kWaitNs);
      tc_fence_after();
      float sc = scal[(j & (a.scal_ring - 1)) * kTile + tok] * qscale;
      const int pos = ms.pos0[j & 15][tok >> 6] + (tok & 63);
      const bool masked = __any_sync(kFull, pos >= lowest);
      // logits (base 2) of all rows, less their references if rel; masked ones -inf
      float x[NS];
      auto logits = [&](bool rel) {
        uint32_t(&y)[NS] = reinterpret_cast<uint32_t(&)[NS]>(x);
#pragma unroll
        for (int c = 0; c < NS; c += 16) tmem_ld16(tS + c, *reinterpret_cast<uint32_t(*)[16]>(y + c));
#pragma unroll
        for (int c = 0; c < NS; c += 16) tmem_ld_wait_tied16(*reinterpret_cast<uint32_t(*)[16]>(y + c));
        const uint64_t sc2 = pk2(sc, sc);
#pragma unroll
        for (int c = 0; c < NS; c += 4) {   // ref holds the negated references
          const ulonglong2 m4 = rel ? *reinterpret_cast<const ulonglong2*>(ref + c) : make_ulonglong2(0, 0);
          const float2 lo = up2(fma2(pk2(x[c], x[c + 1]), sc2, m4.x)), hi = up2(fma2(pk2(x[c + 2], x[c + 3]), sc2, m4.y));
          x[c] = lo.x; x[c + 1] = lo.y; x[c + 2] = hi.x; x[c + 3] = hi.y;
        }
        if (masked) {
#pragma unroll
          for (int c = 0; c < NS; c += 4) {
            const int4 l4 = *reinterpret_cast<const int4*>(limit + c);
            x[c] = pos < l4.x ? x[c] : -INFINITY;
            x[c + 1] = pos < l4.y ? x[c + 1] : -INFINITY;
            x[c + 2] = pos < l4.z ? x[c + 2] : -INFINITY;
            x[c + 3] = pos < l4.w ? x[c + 3] : -INFINITY;
          }
        }
      };
      // no references yet: raised without a look (streams of tiles lose by the branch, 80 to 86 us at 35 rows)
      bool raise = kByRows && i == 0;
      if (!raise) {
        logits(true);
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < NS; c += 2) mx = max3(mx, x[c], x[c + 1]);
        raise = named_any(1 + s, mx > tau);
      }
      bool waited = i == 0;
      if (raise) {
        // raise the references to the tile's maxima
        if (!waited && ok) ok = mbar_wait_ns(&ms.p_empty[s], (i - 1) & 1, kWaitNs);
        waited = true;
        tc_fence_after();
        // scores that x would hold wrongly are multiplied out in tensor memory first, each lane's by itself: the factors
        // of rows past the end are anything, and must not decide how others are rounded
        const bool out = apart || sc > kLargeFactor;
        if (__any_sync(kFull, out)) {
          const float mult = out ? sc : 1.f;
#pragma unroll 1
          for (int c = 0; c < NS; c += 16) {
            uint32_t y[16];
            tmem_ld16_sync(tS + c, y);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float f = apart ? __uint_as_float(static_cast<uint32_t>(ms.size[r_first + c + q]) << 23) : 1.f;
              y[q] = __float_as_uint(__uint_as_float(y[q]) * (f * mult));
            }
            tmem_st16(tS + c, y);
          }
          tmem_st_wait();
          sc = out ? 1.f : sc;
        }
        float* wmax = reinterpret_cast<float*>(myP);   // free: the last product has read it
        float* fac = ms.fac[s];
        logits(false);
#pragma unroll
        for (int c = 0; c < NS; c += 16) {
          const float m = reduce16(*reinterpret_cast<float(*)[16]>(x + c), lane, [](float p, float q) { return fmaxf(p, q); });
          if ((lane & 1) == 0) wmax[(warp & 3) * NS + c + (lane >> 1)] = m;
        }
        named_sync(1 + s, 128);
        if (tok < NS) {
          const float old = -ref[tok];
          const float top = fmaxf(fmaxf(wmax[tok], wmax[NS + tok]), fmaxf(wmax[2 * NS + tok], wmax[3 * NS + tok]));
          const float gap = reference_gap(nt), below = top - gap;   // of scores beyond 2^24 a rounded difference
          const float m = fmaxf(old, top - below == gap ? below : top);
          fac[tok] = old == m ? 1.f : ex2(old - m);
          ref[tok] = -m;
        }
        named_sync(1 + s, 128);
#pragma unroll
        for (int c = 0; c < NS; c += 2) sum[c / 2] = mul2(sum[c / 2], *reinterpret_cast<const uint64_t*>(fac + c));
        if (i > 0) {
#pragma unroll 1
          for (int c = 0; c < used; c += 16) {
            uint32_t o[16];
            tmem_ld16_sync(tO + c, o);
#pragma unroll
            for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * fac[c + q]);
            tmem_st16(tO + c, o);
          }
          tmem_st_wait();
        }
        logits(true);
      }
      if (!waited && ok) ok = mbar_wait_ns(&ms.p_empty[s], (i - 1) & 1, kWaitNs);
#pragma unroll
      for (int c = 0; c < NS; c += 16) {
        uint32_t p[8];
#pragma unroll
        for (int q = 0; q < 16; q += 2) {
          x[c + q] = ex2(x[c + q]);
          x[c + q + 1] = ex2(x[c + q + 1]);
          sum[(c + q) / 2] = add2(sum[(c + q) / 2], pk2(x[c + q], x[c + q + 1]));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) p[q] = h2bits(__floats2half2_rn(x[c + 2 * q], x[c + 2 * q + 1]));
        *reinterpret_cast<uint4*>(myP + (c >> 3) * 2048 + tok * 16) = make_uint4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<uint4*>(myP + ((c >> 3) + 1) * 2048 + tok * 16) = make_uint4(p[4], p[5], p[6], p[7]);
      }
      fence_async_smem();
      tc_fence_before();
      warp_arrive(&ms.p_full[s], lane);
    }

    // ---- join the stream's 128 tokens' sums, then the streams
    if (mine > 0 && ok) ok = mbar_wait_ns(&ms.p_empty[s], (mine - 1) & 1, kWaitNs);
    tc_fence_after();
    float* wsum = reinterpret_cast<float*>(myP);
#pragma unroll
    for (int c = 0; c < NS; c += 16) {
      float y[16];
#pragma unroll
      for (int q = 0; q < 16; q += 2) {
        const float2 v = up2(sum[(c + q) / 2]);
        y[q] = v.x;
        y[q + 1] = v.y;
      }
      const float t = reduce16(y, lane, [](float p, float q) { return p + q; });
      if ((lane & 1) == 0) wsum[(warp & 3) * NS + c + (lane >> 1)] = t;
    }
    named_sync(3, 256);
    // per row: its streams' factors, the joint maximum and sum (by rows: of the row's stream alone)
    float* fac0 = scal;   // free now: two factors, maximum and sum of 128 rows
    float *fac1 = fac0 + kTile, *jm = fac0 + 2 * kTile, *jl = fac0 + 3 * kTile;
    // and 1 / sum and the output's first element, for the rows' loops to spare the divisions
    float* inv = kByRows ? fac0 : jl + kTile / 2;
    int64_t* out_at = reinterpret_cast<int64_t*>(sP + 2 * p_bytes(N)) - N;   // behind the last stream's sums
    if (tok < NS && (kByRows || s == 0)) {
      const int r = r_first + tok, t = (row0 + r) / group;
      if (r < rows) out_at[r] = b * a.ob + a.heads.head[head0 + row0 + r - t * group] * a.oh + t * a.ot;
      const float* w0 = reinterpret_cast<float*>(sP) + tok;
      const float* w1 = reinterpret_cast<float*>(sP + p_bytes(N)) + tok;
      const float l0 = (w0[0] + w0[NS]) + (w0[2 * NS] + w0[3 * NS]);
      const float l1 = (w1[0] + w1[NS]) + (w1[2 * NS] + w1[3 * NS]);
      if (kByRows) {
        const float l = s ? l1 : l0;
        jm[r] = -ref[tok];
        jl[r] = l;
        inv[r] = l == 0.f ? 0.f : 1.f / l;
      } else {
        const float m0 = -ms.ref[0][tok], m1 = -ms.ref[1][tok], m = fmaxf(m0, m1);
        const float f0 = m0 == m ? 1.f : ex2(m0 - m), f1 = m1 == m ? 1.f : ex2(m1 - m);
        fac0[tok] = f0;
        fac1[tok] = f1;
        const float l = l0 * f0 + l1 * f1;
        jm[tok] = m;
        jl[tok] = l;
        inv[tok] = l == 0.f ? 0.f : 1.f / l;
      }
    }
    named_sync(3, 256);
    float* xbuf = reinterpret_cast<float*>(sV) + r_first * kD + value_channel(a.vbits, tok);   // [row][channel]
    const bool both = !kByRows && nt > 1;
    if (nt > 0 && (kByRows || both || s == 0)) {
      const float* f = s ? fac1 : fac0;
      if (both && s == 0) named_sync(3, 256);   // the second stream's outputs first
#pragma unroll 1
      for (int c = 0; c < used; c += 16) {
        uint32_t o[16];
        tmem_ld16_sync(tO + c, o);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float v = __uint_as_float(o[q]);
          if (!kByRows) v *= f[c + q];
          if (both && s == 0) v += xbuf[(c + q) * kD];
          xbuf[(c + q) * kD] = v;
        }
      }
      if (both && s == 1) named_sync(3, 256);
    }
    named_sync(3, 256);
    const int spoilt = ms.poison[lane >> 3];
    constexpr int kOut = kRows % 4 == 0 ? 4 : 2;   // rows whose loads overlap
#pragma unroll 1
    for (int r0 = warp - wS; r0 < rows; r0 += 8 * kOut) {
      float4 v[kOut];
#pragma unroll
      for (int i = 0; i < kOut; ++i) {
        const int r = min(r0 + 8 * i, rows - 1);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);   // no tiles: zeros, or an empty record
        if (nt > 0) v[i] = reinterpret_cast<const float4*>(sV)[r * (kD / 4) + lane];
        if (spoilt < ms.limit[r]) v[i].x = v[i].y = v[i].z = v[i].w = __uint_as_float(0x7fffffffu);
      }
#pragma unroll
      for (int i = 0; i < kOut; ++i) {
        const int r = r0 + 8 * i;
        if (r >= rows) break;
        if (n_splits == 1) {
          store_row(a, out_at[r] + 4 * lane, v[i], inv[r]);
        } else {
          float* rec = a.part + (static_cast<int64_t>(blockIdx.x) * N + r) * kPartFloats;
          reinterpret_cast<float4*>(rec + 4)[lane] = v[i];
          if (lane == 0) *reinterpret_cast<float2*>(rec) = make_float2(jm[r], jl[r]);
        }
      }
    }
    if (n_splits > 1) {
      // the last block of threads of this item joins the splits, in their order
      const int first = blockIdx.x - split;
      named_sync(3, 256);
      if (tid == 32 * wS) {
        __threadfence();   // after the barrier: it stands for all threads' records
        int* counter = a.counters + first;
        ms.last = atomicAdd(counter, 1) == n_splits - 1;
        if (ms.last) *counter = 0;
      }
      named_sync(3, 256);
      if (ms.last) {
        __threadfence();
        // records in batches of 8 loads, of four rows where there are many rows (and few splits)
        constexpr int kRb = N >= 64 ? 4 : 1, kSb = 8 / kRb;
        constexpr int64_t step = static_cast<int64_t>(N) * kPartFloats;
#pragma unroll 1
        for (int r0 = warp - wS; r0 < rows; r0 += 8 * kRb) {
          const float* rec = a.part + (static_cast<int64_t>(first) * N + r0) * kPartFloats;
          float M[kRb], L[kRb];
          float4 O[kRb];
#pragma unroll
          for (int k = 0; k < kRb; ++k) { M[k] = kNoRef; L[k] = 0.f; O[k] = make_float4(0.f, 0.f, 0.f, 0.f); }
#pragma unroll 1
          for (int i0 = 0; i0 < n_splits; i0 += kSb) {
            float2 ml[kRb][kSb];
            float4 o[kRb][kSb];
#pragma unroll
            for (int k = 0; k < kRb; ++k) {
              const int more_rows = min(8 * k, (rows - 1 - r0) & ~7);   // past the last row: an earlier one again
#pragma unroll
              for (int i = 0; i < kSb; ++i) {
                const float* p = rec + more_rows * kPartFloats + min(i0 + i, n_splits - 1) * step;
                ml[k][i] = __ldcg(reinterpret_cast<const float2*>(p));
                o[k][i] = __ldcg(reinterpret_cast<const float4*>(p + 4) + lane);
              }
            }
#pragma unroll
            for (int k = 0; k < kRb; ++k) {
              float m = M[k];
#pragma unroll
              for (int i = 0; i < kSb; ++i) m = fmaxf(m, ml[k][i].x);
              const float g = M[k] == m ? 1.f : ex2(M[k] - m);
              M[k] = m;
              L[k] *= g;
              O[k].x *= g; O[k].y *= g; O[k].z *= g; O[k].w *= g;
#pragma unroll
              for (int i = 0; i < kSb; ++i) {
                if (i0 + i < n_splits) {
                  const float f = ml[k][i].x == m ? 1.f : ex2(ml[k][i].x - m);
                  L[k] = fmaf(f, ml[k][i].y, L[k]);
                  O[k].x = fmaf(f, o[k][i].x, O[k].x); O[k].y = fmaf(f, o[k][i].y, O[k].y);
                  O[k].z = fmaf(f, o[k][i].z, O[k].z); O[k].w = fmaf(f, o[k][i].w, O[k].w);
                }
              }
            }
          }
#pragma unroll
          for (int k = 0; k < kRb; ++k)
            if (r0 + 8 * k < rows) store_row(a, out_at[r0 + 8 * k] + 4 * lane, O[k], L[k] == 0.f ? 0.f : 1.f / L[k]);
        }
      }
    }
  }

  if (!ok) atomicOr(a.err, 1);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == wM) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace ext
}  // namespace tq
