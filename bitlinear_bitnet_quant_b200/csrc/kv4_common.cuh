// What the kernels around the 4-bit key/value cache share (sm_100a only).
//
// Cache layout: codes [B][kv_heads][T_cap][d/2] bytes and steps [B][kv_heads][T_cap]
// fp32, for keys and for values: the rows of one sequence's head are contiguous,
// so a block of keys is one run of bytes.  A row stands for code * step.  Of the 8
// codes of a little-endian 32-bit word, code 2j + i (i = 0, 1) sits at bits
// 4j + 16i, two's complement: (word >> 4j) & 0x000F000F is the pair of codes
// (2j, 2j + 1) in the two halves of a register, in order.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace bitnet {

// Where the tokens of a step sit: token l of sequence b is row b * L + l of the
// step's tensors and position t0 + pos[b] + l of its sequence; the first len[b]
// tokens of a sequence are real, the others padding.
struct KvStep {
  const int32_t* pos;                               // [B] or NULL (zeros)
  const int32_t* len;                               // [B] or NULL (L)
  int64_t t0;
  int B, L, T_cap;
  int limit;                                        // positions at or past it lie outside the cache (<= T_cap)
};

BN_DEV int kv_real_tokens(const KvStep& s, int b) {
  if (s.len == nullptr) return s.L;
  const int n = s.len[b];
  return n < 0 ? 0 : (n < s.L ? n : s.L);
}
BN_DEV int64_t kv_first_position(const KvStep& s, int b) {
  return s.t0 + (s.pos == nullptr ? 0 : (int64_t)s.pos[b]);
}

// The append's rows, factors and destinations (fp32 caches or 4-bit ones).
struct RopeTable { double theta[64]; };             // theta_i of the pairs that turn

struct AppendArgs {
  const void *Q, *K, *V;
  int64_t ldq, ldk, ldv;                            // row strides, in values
  const float *gamma_q, *gamma_k;
  float eps;
  int heads, kv_heads, rot_dim, norm, hadamard;
  void* Qo;
  int qo_bf16;
  float *Kc32, *Vc32;                               // fp32 caches [B][T_cap][kv_heads * d]
  uint8_t *Kc4, *Vc4;                               // 4-bit caches
  float *Ks, *Vs;
};

// The attention's operands.
struct AttnArgs {
  const void* Q;                                    // [B * L][heads * d]
  const uint8_t *Kc, *Vc;
  const float *Ks, *Vs;
  void* A;                                          // [B * L][heads * d]
  int heads, kv_heads;
  int window, sinks;                                // window 0: every key up to the query's own
};

// Four code pairs of a word as fp16 pairs, exact: a code's nibble with its sign
// bit flipped is code + 8, which as the low mantissa bits of 1024 (nibbles 0 and
// 2 of each half) or the next four (1 and 3) needs one subtraction, or one
// multiply-add, to become the code.
BN_DEV uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
BN_DEV uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
BN_DEV void codes_to_half2(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t v = w >> 8;
  p[0] = h2_sub((w & 0x000F000Fu) ^ 0x64086408u, 0x64086408u);                 // 1024 + u - 1032
  p[1] = h2_fma((w & 0x00F000F0u) ^ 0x64806480u, 0x2C002C00u, 0xD480D480u);    // (1024 + 16 u) / 16 - 72
  p[2] = h2_sub((v & 0x000F000Fu) ^ 0x64086408u, 0x64086408u);
  p[3] = h2_fma((v & 0x00F000F0u) ^ 0x64806480u, 0x2C002C00u, 0xD480D480u);
}

BN_DEV float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

BN_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What the fp16 pair h leaves of (lo, hi), as another fp16 pair.
BN_DEV uint32_t half2_rest(uint32_t h, float lo, float hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_half2(lo - f.x, hi - f.y);
}

// Pairs of fp32 in one register pair, and operations on both at once.
BN_DEV uint64_t pack_f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
BN_DEV void unpack_f2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
BN_DEV uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
BN_DEV uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
BN_DEV uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
BN_DEV float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
BN_DEV float max_nan(float a, float b) {             // NaN where one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
BN_DEV float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A step's exponent e, at least -24: the append writes steps of 2^-20 and more (or a
// row is empty, step 0, and keeps its weight in the sum).  Together with steps below
// 2^60 no weight p' that counts leaves the range of fp32 (2^-126): 2^(-24 - 60) of
// the largest one, times the weight itself.
BN_DEV int step_exponent(float step) {
  const int e = (int)((__float_as_uint(step) >> 23) & 255u) - 127;
  return e < -24 ? -24 : (e > 126 ? 126 : e);
}
BN_DEV float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// The exponent of a row's largest finite value, so that 2^e and 2^-e are normal numbers.
BN_DEV int row_exponent(float v) {
  const int e = (int)(__float_as_uint(v) >> 23) - 127;
  return e < -100 ? -100 : e;
}

// The key tiles (of KT keys) that some query of positions p_lo .. p_hi sees: those
// of the sinks, then those from the first query's window on.
struct KeyTiles {
  int sink_tiles, first, count;
  BN_DEV int at(int i) const { return i < sink_tiles ? i : first + i - sink_tiles; }
};
template <int KT>
BN_DEV KeyTiles key_tiles(int p_lo, int p_hi, int window, int sinks) {
  KeyTiles k;
  const int hi = p_hi + 1;
  int lo = 0, sk = 0;
  if (window > 0) {
    lo = p_lo - window + 1 > 0 ? p_lo - window + 1 : 0;
    sk = sinks < hi ? sinks : hi;
  }
  k.sink_tiles = (sk + KT - 1) / KT;
  k.first = lo / KT > k.sink_tiles ? lo / KT : k.sink_tiles;
  const int end = (hi + KT - 1) / KT;
  k.count = k.sink_tiles + (end > k.first ? end - k.first : 0);
  return k;
}
BN_DEV bool key_visible(int j, int p, int window, int sinks) {
  return j <= p && (window == 0 || j > p - window || j < sinks);
}

}  // namespace bitnet
