// Packed codebook indices to fp16 level pairs, by byte permutes instead of table lookups in memory.
//
// A codebook of at most 8 values (a level set, or the positive half of a mirrored one) is 8 low and
// 8 high bytes of fp16 numbers: two 8-byte pools, and a byte permute (prmt) looks up four of
// them at once, its selector being four packed 4-bit codes as they stand in the index word.
// A word of eight 3-bit codes takes 9 instructions, against 8 shared-memory lookups. The
// order of the codes in the output ("positions") is whatever is cheapest; level_channel() gives
// the code that a position holds, and users of the output order their other operand by it.
#pragma once

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Byte pools of a codebook (DevTables::lv_lo, lv_hi): the levels over DevTables::lv_scale in fp16
// (4-bit codes: the positive half; 2-bit: lo is the four levels; 1-bit: lo[0] is the positive level twice).
struct Levels {
  uint32_t lo[2], hi[2];
};

__device__ __forceinline__ Levels load_levels(const DevTables* t, int group) {
  return Levels{{t->lv_lo[group][0], t->lv_lo[group][1]}, {t->lv_hi[group][0], t->lv_hi[group][1]}};
}

// fp16 pairs a 32-bit index word of `bits`-bit codes gives
__host__ __device__ constexpr int level_pairs(int bits) { return bits == 1 ? 16 : bits == 2 ? 8 : 4; }

// Element e (0, 1) of pair i of a word: which of the word's codes it is.
__host__ __device__ constexpr int level_code(int bits, int i, int e) {
  return bits == 1 ? i + 16 * e : bits == 2 ? 4 * (2 * (i & 1) + e) + i / 2 : 2 * i + e;
}
// Element e of pair p of a run of words: its channel in the run.
__host__ __device__ constexpr int level_channel(int bits, int p, int e) {
  const int n = level_pairs(bits);
  return p / n * 2 * n + level_code(bits, p % n, e);
}

// Signs of a 32-bit sign word on a positive fp16 pair `mag`: pair i holds bits i and i + 16, a
// set bit is +mag.
__device__ __forceinline__ uint32_t sign_level(uint32_t inv, int i, uint32_t mag) {
  return ((inv << (15 - i)) & 0x80008000u) | mag;
}

template <int BITS>
__device__ __forceinline__ void unpack_levels(uint32_t w, const Levels& t, uint32_t (&out)[level_pairs(BITS)]) {
  if constexpr (BITS == 1) {
    const uint32_t inv = ~w;
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = sign_level(inv, i, t.lo[0]);
  } else if constexpr (BITS == 2) {
    // code c is bytes 2c and 2c + 1 of the four levels: a byte of selectors is 0x22 c + 0x10
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = (w >> (2 * i)) & 0x03030303u;
      const uint32_t sel = c * 0x22u + 0x10101010u;
      out[2 * i] = prmt(t.lo[0], t.lo[1], sel);
      out[2 * i + 1] = prmt(t.lo[0], t.lo[1], sel >> 16);
    }
  } else if constexpr (BITS == 3) {
    const uint32_t c = w & 0x77777777u;   // a selector with bit 3 set would spread the byte's sign
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t sel = i ? c >> 16 : c;
      const uint32_t l = prmt(t.lo[0], t.lo[1], sel), h = prmt(t.hi[0], t.hi[1], sel);
      out[2 * i] = prmt(l, h, 0x5140);
      out[2 * i + 1] = prmt(l, h, 0x7362);
    }
  } else {
    // the mirrored half: code c < 8 is minus level 15 - c, whose magnitude index is 7 - c
    const uint32_t neg = ~w & 0x88888888u;
    const uint32_t c = (w ^ (neg - (neg >> 3))) & 0x77777777u;
    const uint32_t neg4 = neg << 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t sel = i ? c >> 16 : c;
      const uint32_t l = prmt(t.lo[0], t.lo[1], sel);
      // each byte's top bit spread over it: even codes' flags from neg4, odd ones' from neg
      const uint32_t s = prmt(neg4, neg, i ? 0xfbea : 0xd9c8);
      const uint32_t h = prmt(t.hi[0], t.hi[1], sel) ^ (s & 0x80808080u);
      out[2 * i] = prmt(l, h, 0x5140);
      out[2 * i + 1] = prmt(l, h, 0x7362);
    }
  }
}

}  // namespace tq
