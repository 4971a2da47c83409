// Causal attention over the 4-bit key/value cache for many queries a key head
// (prefill), on tcgen05, in two kernels: the keys and values that the step sees are
// expanded once into fp16 operands (a caller's workspace), then every block of query
// rows streams them through the tensor cores.
#include "kv4_common.cuh"

#include <cuda_bf16.h>

namespace bitnet {

// ---------------------------------------------------------------------------
// Operands.  A tile's keys are code * step * 2^(11 - E) in fp16, E the exponent of the
// tile's largest step, rounded once (half a step of fp16 is 2^-11 of a value, as for
// the weights); its values the same with their exponent F.  A query row is scaled by a
// power of two, bf16 values are then exact in fp16.  A row's score in base-2 exponents
// is acc * c with one factor c a row and tile, and its weight carries the tile's 2^F,
// p' = 2^(acc c + F - m): the output sums p' v 2^(11 - F) over all tiles in one scale,
// and the softmax sum takes 2^-F once a tile.
//
// The workspace holds, for every key head and tile, the two operands as the images that
// shared memory takes (128-byte swizzle), so that a tile is one bulk copy, and c and F.
// Expanding inside the attention kernel, by eight more warps of each block, cost as
// many issue slots as the softmax and read the codes once a block: 4096 causal tokens of
// 8 x 4 heads took 179 us, so 173.
// ---------------------------------------------------------------------------
constexpr int KP_KT = 128;                           // keys a tile
constexpr int KP_POLY = 4;                           // one pair in KP_POLY is raised on the multiply-add units
// 2^r on [-1/2, 1/2], the cubic of least largest relative error (7.5e-05), by linear programming
constexpr float EXP2_C0 = 0.999928073f, EXP2_C1 = 0.693260985f, EXP2_C2 = 0.242611125f, EXP2_C3 = 0.055171670f;

// fp32 rows: of every key of a tile, 4 arrays of KP_KT: the score's factor, the exponent e
// of its value step f 2^e, 2^-e (0 where no query sees the key) and f.
constexpr int KP_KEY_FLOATS = 4 * KP_KT;

template <int D>
struct KpTile {
  static constexpr int BYTES = KP_KT * D * 2;        // keys or values of a tile
  static constexpr int PAIR = 2 * BYTES;             // both
};

// One lane of a warp that runs as a whole.  The compiler knows the lane to be alone
// (unlike a test of the lane's number), so the products' descriptors stay in uniform
// registers: issued from a lane-number branch, a product took 300 cycles instead of 64.
BN_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Instruction descriptor of kind::f16: fp32 accumulator, fp16 operands, A K-major, B
// K-major or (b_mn) with its N dimension contiguous.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Shared-memory descriptors (128-byte swizzle, groups of 8 rows 1024 bytes apart) as a
// low word that a product's offset is added to and a constant high word: the warp that
// issues the products must spend few instructions on each.  K-major operands ignore the
// block distance; with N contiguous it is that of the 64-value column blocks.
constexpr uint32_t KP_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
BN_DEV uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | ((16384u >> 4) << 16); }
BN_DEV void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\t"
               "mov.b64 db, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}"
               :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(KP_DESC_HI) : "memory");
}
BN_DEV void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}"
               :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(KP_DESC_HI) : "memory");
}
// Each lane reads 32 consecutive 32-bit columns of its own tensor-memory lane.
BN_DEV void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr) : "memory");
}

BN_DEV uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
BN_DEV uint32_t both_halves(float v) { return pack_half2(v, v); }

// Part of a sequence that its real queries see.
struct KpSeen {
  int first, last;                                   // positions of the first and last query, inside the cache
  bool any;
};
BN_DEV KpSeen kp_seen(const KvStep& s, int b) {
  const int n = kv_real_tokens(s, b);
  const int64_t pf = kv_first_position(s, b), pl = pf + n - 1;
  KpSeen r;
  r.any = n > 0 && pl >= 0 && pf < s.limit;
  r.first = pf < 0 ? 0 : (int)(pf < s.limit ? pf : s.limit - 1);
  r.last = pl < 0 ? 0 : (int)(pl < s.limit ? pl : s.limit - 1);
  return r;
}

// ---------------------------------------------------------------------------
// Expansion: a block a tile and key head; four warps its keys, four its values.  Bound
// by memory (reads D + 8 bytes a key and head, writes 4 D): 8192 keys of 8 heads in 15 us,
// 3 % of the attention they are for.
// ---------------------------------------------------------------------------
// EXACT (fp32 rows): the images hold the codes themselves, and every key's four factors
// (KP_KEY_FLOATS a tile) are written instead of the tile's.
template <int D, bool EXACT>
__global__ void __launch_bounds__(256)
kv4_expand_kernel(const KvStep s, const AttnArgs a, int head0, int slots, float scale_log2e, uint8_t* images,
                  float* factors) {
  using M = KpTile<D>;
  __shared__ __align__(16) uint32_t step_top[2][4];
  pdl_launch_dependents();
  pdl_wait();                                        // the cache comes from the previous kernel
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, val = warp >> 2, key = tid & 127;
  const int head = head0 + blockIdx.y, b = head / a.kv_heads;
  const KpSeen seen = kp_seen(s, b);
  const KeyTiles tiles = key_tiles<KP_KT>(seen.first, seen.last, a.window, a.sinks);
  const int slot = blockIdx.x;
  if (!seen.any || slot >= tiles.count) return;
  const int j0 = tiles.at(slot) * KP_KT;
  const int seen_lo = a.window > 0 ? seen.first - a.window : -1;       // some row sees the keys past it, and the sinks
  auto is_seen = [&](int j) { return j <= seen.last && (j > seen_lo || j < a.sinks); };
  // a warp's 32 rows are one run of memory: lane i takes 16 bytes of every D / 2-byte row in turn,
  // part i % PARTS of row i / PARTS + RPI q; step factors come from the lane whose number is the row's
  constexpr int PARTS = D / 32, RPI = 32 / PARTS;
  const int part = lane % PARTS, row0 = lane / PARTS, jw = j0 + (key & 96);
  const uint8_t* codes = (val ? a.Vc : a.Kc) + (int64_t)head * s.T_cap * (D / 2);
  uint4 cw[PARTS];
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    const int j = jw + row0 + RPI * q;
    cw[q] = make_uint4(0u, 0u, 0u, 0u);
    if (is_seen(j)) cw[q] = ldg_v4(codes + (int64_t)j * (D / 2) + 16 * part);
  }
  // the tile's largest steps.  A row whose steps are not finite is NaN to the queries that see
  // it, through its key alone: a masked weight of 0 would not hide it in the values
  float kstep = 0.f, vstep = 0.f;
  if (is_seen(j0 + key)) {
    kstep = ldg_f32(a.Ks + (int64_t)head * s.T_cap + j0 + key);
    vstep = ldg_f32(a.Vs + (int64_t)head * s.T_cap + j0 + key);
  }
  const bool bad = !(fabsf(kstep) < INFINITY && fabsf(vstep) < INFINITY);
  const int64_t tile = (int64_t)blockIdx.y * slots + slot;
  uint32_t sh = 0u, sl = 0u;                         // a row's step in two fp16 terms
  if constexpr (EXACT) {
    if (!val) {
      float* f = factors + tile * KP_KEY_FLOATS + key;
      const int e = step_exponent(vstep);
      const float inv = pow2i(-e);
      const bool shown = is_seen(j0 + key);
      f[0] = bad ? NAN : kstep * scale_log2e;
      f[KP_KT] = (float)e;
      f[2 * KP_KT] = bad || !shown ? 0.f : inv;
      f[3 * KP_KT] = bad ? 0.f : vstep * inv;
    }
  } else {
    const uint32_t kt = __reduce_max_sync(0xffffffffu, bad ? 0u : __float_as_uint(fabsf(kstep)));
    const uint32_t vt = __reduce_max_sync(0xffffffffu, bad ? 0u : __float_as_uint(fabsf(vstep)));
    if (warp < 4 && lane == 0) {
      step_top[0][warp] = kt;
      step_top[1][warp] = vt;
    }
    __syncthreads();
    const uint4 k4 = *reinterpret_cast<const uint4*>(step_top[0]), v4 = *reinterpret_cast<const uint4*>(step_top[1]);
    const int E = row_exponent(__uint_as_float(max(max(k4.x, k4.y), max(k4.z, k4.w))));
    const int F = step_exponent(__uint_as_float(max(max(v4.x, v4.y), max(v4.z, v4.w))));
    const float step = val ? vstep * pow2i(11 - F) : kstep * pow2i(11 - E);
    // 8 bits of the step times a code are exact in fp16; the rest of the step joins in one rounding
    const float top = __uint_as_float(__float_as_uint(step) & 0xFFFF0000u);
    sh = bad ? (val ? 0u : 0x7FFF7FFFu) : both_halves(top);
    sl = bad ? 0u : both_halves(step - top);
    if (tid == 0) reinterpret_cast<float2*>(factors)[tile] = make_float2(scale_log2e * pow2i(E - 11), (float)F);
  }
  uint8_t* dst = images + tile * M::PAIR + val * M::BYTES + (key & 96) * 128;
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    const int row = row0 + RPI * q;
    uint32_t rh = 0u, rl = 0u;
    if constexpr (!EXACT) {
      rh = __shfl_sync(0xffffffffu, sh, row);
      rl = __shfl_sync(0xffffffffu, sl, row);
    }
    const uint32_t words[4] = {cw[q].x, cw[q].y, cw[q].z, cw[q].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t v[4];
      codes_to_half2(words[e], v);
      if constexpr (!EXACT) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = h2_fma(v[j], rl, h2_mul(v[j], rh));
      }
      const int chunk = 4 * (part & 1) + e;
      *reinterpret_cast<uint4*>(dst + (part >> 1) * 16384 + row * 128 + ((chunk ^ (row & 7)) << 4)) =
          make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Whether a block's rows are all padding; such blocks of a ragged step leave before they take
// tensor memory, which the next block of their SM would wait for.
BN_DEV bool kp_padding(const KvStep& s, const AttnArgs& a, int head0, int heads_here, int row_tiles, int rows) {
  if (s.len == nullptr) return false;
  pdl_wait();
  const int rt = row_tiles - 1 - (int)(blockIdx.x / heads_here), here = (int)(blockIdx.x % heads_here);
  return rt * rows >= kv_real_tokens(s, (head0 + here) / a.kv_heads) * (a.heads / a.kv_heads);
}

// ---------------------------------------------------------------------------
// Attention.  A block takes 256 rows (token, head of the group) of one key head as two
// streams of 128: one warp copies tiles of 128 keys into shared memory (two stages), one
// issues the products, and four warps a stream turn scores into weights, one row a
// thread.
//   scores  q (shared memory) x keys -> tensor memory, fp32
//   weights written over the scores as fp16, the product's operand in tensor memory
//   output  weights x values (keys as the reduction) -> tensor memory, fp32
// While one stream's weights are computed, the other stream's products run.  A row's 128
// scores are worked on at once, from one load: in parts of 32 or 64 the special-function
// units ran dry at every part's ends.  The running maximum m is that of acc c + F, of the
// tiles for which it was looked for: a tile's weights are computed with the maximum so far,
// and only where their sum passes what one weight may be in fp16 (or a row sees its first
// key) is the tile's maximum found, the output in tensor memory rescaled and the weights
// computed once more.  (Finding every tile's maximum: 522 us for 8192 causal tokens of
// 8 x 4 heads, so 504: 1.1 PFLOP/s, 67 % of a library product's rate, for a call alone with a
// cold L2, and 575 us among others, where the clock is lower.  The rest are the softmax's
// instructions and the filling and draining of 7 blocks an SM.)
// ---------------------------------------------------------------------------
constexpr int KP_THREADS = 320;                      // streams: warps 0-3 and 4-7; products: warp 8; copies: warp 9

template <int D>
struct KpSmem {
  static constexpr int TILE = KpTile<D>::BYTES;      // 128 rows of D 16-bit values
  static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, BYTES = 6 * TILE + 1024;   // 2 of each, + alignment
};

// Bulk copy of `bytes` from global to this block's shared memory, counted on its barrier.
BN_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Wait for a phase, as mbar_wait, for a whole warp; the clock is looked at only after
// many tries (reading it takes longer than most waits here).
BN_DEV bool kp_wait(uint64_t* bar, uint32_t parity, int code) {
  bool ok = false;
  for (int n = 0; n < 1024 && !ok; ++n) ok = mbar_try_wait(bar, parity);
  if (!ok) ok = mbar_wait(bar, parity, code);
  return __all_sync(0xffffffffu, ok);
}

// Every copy that a block issued lands before the block may exit, also after waits that gave up:
// the last N of `issued` copies, which a ring of N barriers counts.  Where the products took the
// tiles the waits return at once.
template <int N>
BN_DEV void kp_copies_done(uint64_t* full, int issued) {
  for (int i = issued > N ? issued - N : 0; i < issued; ++i)
    mbar_wait(&full[i % N], (i / N) & 1, DEV_ERR_TIMEOUT_FULL, false);
}

// Positions of one stream's rows, and what of n keys from j0 on they see.
struct KpRows {
  int n, p_lo, p_hi;                                 // rows; first and last position inside the cache
  bool in;                                           // every row's position lies inside the cache
  BN_DEV bool any(int j0, int keys, int window, int sinks) const {
    return n > 0 && j0 <= p_hi && (window == 0 || j0 + keys - 1 > p_lo - window || j0 < sinks);
  }
  BN_DEV bool full(int j0, int keys, int window, int sinks) const {
    return in && j0 + keys - 1 <= p_lo && (window == 0 || j0 > p_hi - window || j0 + keys <= sinks);
  }
};

// 2^x of a pair on the multiply-add units: x = n + r with r in [-1/2, 1/2] by adding
// 1.5 * 2^23, a cubic for 2^r (relative error 1e-4, a fifth of the fp16 rounding that
// follows), and n into the exponent.  x below -125 counts as -125 (2^-125 rounds to
// zero in fp16).  2^n with n > 127 runs into the sign and means nothing, nor does NaN:
// the caller finds both in `high`, the largest n + 1.5 * 2^23.  (Without that a key far
// above the maximum so far lost its weight; it costs 0.7 % of 8192 causal tokens.)
BN_DEV void exp2_pair(uint64_t x, float& e0, float& e1, float& high) {
  float a, b;
  unpack_f2(x, a, b);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(-125.f));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(-125.f));
  const uint64_t v = pack_f2(a, b);
  const uint64_t big = pack_f2(12582912.f, 12582912.f), nbig = pack_f2(-12582912.f, -12582912.f);
  const uint64_t t = add_f2(v, big);
  const uint64_t n = add_f2(t, nbig);
  const uint64_t r = fma_f2(n, pack_f2(-1.f, -1.f), v);
  uint64_t q = fma_f2(pack_f2(EXP2_C3, EXP2_C3), r, pack_f2(EXP2_C2, EXP2_C2));
  q = fma_f2(q, r, pack_f2(EXP2_C1, EXP2_C1));
  q = fma_f2(q, r, pack_f2(EXP2_C0, EXP2_C0));
  float t0, t1, q0, q1;
  unpack_f2(t, t0, t1);
  high = max3_nan(high, t0, t1);
  unpack_f2(q, q0, q1);
  e0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
  e1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
}

// The weights of a tile's keys for one row, as fp16 pairs, for exponents x f + ref, and
// their sum (infinite where one is not finite or too large for exp2_pair).  Every
// KP_POLY-th pair's exponentials come from the multiply-add units: the special-function
// units alone would take 2048 cycles a tile.
BN_DEV void kp_weights(const float (&x)[KP_KT], float f, float ref, uint32_t (&w)[KP_KT / 2], float& sum) {
  const uint64_t f2 = pack_f2(f, f), ref2 = pack_f2(ref, ref);
  uint64_t s2[4] = {0, 0, 0, 0};
  float high[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < KP_KT / 2; ++c) {
    float e0, e1;
    const uint64_t y = fma_f2(pack_f2(x[2 * c], x[2 * c + 1]), f2, ref2);
    if (c % KP_POLY == KP_POLY - 1) {
      exp2_pair(y, e0, e1, high[(c / KP_POLY) & 1]);
    } else {
      unpack_f2(y, e0, e1);
      e0 = ex2(e0);
      e1 = ex2(e1);
    }
    s2[c & 3] = add_f2(s2[c & 3], pack_f2(e0, e1));
    w[c] = pack_half2(e0, e1);
  }
  float s0, s1;
  unpack_f2(add_f2(add_f2(s2[0], s2[1]), add_f2(s2[2], s2[3])), s0, s1);
  sum = max_nan(high[0], high[1]) <= 12582912.f + 127.f ? s0 + s1 : INFINITY;
}
// The largest score of a row, NaN where one is.
BN_DEV float kp_top(const float (&x)[KP_KT]) {
  float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int c = 4; c < KP_KT; c += 2) mx[(c >> 1) & 3] = max3_nan(mx[(c >> 1) & 3], x[c], x[c + 1]);
  return max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]);
}

// Masks the scores of N columns: those up to hi, and past lo or below sk, stay.  As bits
// of words, two instructions a column.
BN_DEV uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
template <int N>
BN_DEV void kp_mask(float* x, int hi, int lo, int sk) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    const uint32_t seen = bits_below(hi + 1 - c) & (~bits_below(lo + 1 - c) | bits_below(sk - c));
#pragma unroll
    for (int q = 0; q < 32; ++q) x[c + q] = (seen >> q) & 1u ? x[c + q] : -INFINITY;
  }
}

// Completion of this warp's tensor-memory loads; what their use starts from passes
// through, so that the compiler keeps every use behind the wait.
BN_DEV void kp_loads_done(float& ref, float& f) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(ref), "+f"(f) :: "memory");
}

BN_DEV KpRows kp_rows(int r0, int n_rows, int group, int64_t p0, int limit) {
  KpRows r;
  r.n = n_rows - r0 < 0 ? 0 : (n_rows - r0 < 128 ? n_rows - r0 : 128);
  const int64_t pf = p0 + r0 / group, pl = p0 + (r0 + (r.n > 0 ? r.n : 1) - 1) / group;
  r.in = pf >= 0 && pl < limit;
  if (pl < 0 || pf >= limit) r.n = 0;                // no row sees a key
  r.p_lo = pf < 0 ? 0 : (int)(pf < limit ? pf : limit - 1);
  r.p_hi = pl < 0 ? 0 : (int)(pl < limit ? pl : limit - 1);
  return r;
}

template <int D>
__global__ void __launch_bounds__(KP_THREADS, 1)
kv4_prefill_kernel(const KvStep s, const AttnArgs a, int head0, int heads_here, int row_tiles, int slots,
                   const uint8_t* __restrict__ images, const float* __restrict__ tile_factors) {
  const float2* factors = reinterpret_cast<const float2*>(tile_factors);
  using M = KpSmem<D>;
  constexpr float BIAS = 7.f;
  constexpr uint32_t S_COL = 0, O_COL = 256;         // streams: + 128 g
  extern __shared__ uint8_t kp_raw[];
  __shared__ uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2], q_full, s_full[2], p_full[2], all_done;
  __shared__ uint32_t tmem_sh;
  uint8_t* sm = smem_align(kp_raw, 1024);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (kp_padding(s, a, head0, heads_here, row_tiles, 256)) return;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    mbar_init(&q_full, 256);
    mbar_init(&all_done, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&tmem_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  // only once the tensor memory is allocated may the next kernel of the stream be scheduled
  pdl_launch_dependents();
  pdl_wait();                                        // q and the cache come from the previous kernel

  // the longest row tiles first: blocks of the last rows see the most keys
  const int rt = row_tiles - 1 - (int)(blockIdx.x / heads_here);
  const int here = (int)(blockIdx.x % heads_here), b = (head0 + here) / a.kv_heads, h = head0 + here - b * a.kv_heads;
  const int group = a.heads / a.kv_heads;
  const int n_rows = kv_real_tokens(s, b) * group;
  const int r0 = rt * 256;
  const int64_t p0 = kv_first_position(s, b);
  const KpRows rows0 = kp_rows(r0, n_rows, group, p0, s.limit), rows1 = kp_rows(r0 + 128, n_rows, group, p0, s.limit);
  KeyTiles tiles = {0, 0, 0};
  const int first_seen = rows0.n > 0 ? rows0.p_lo : rows1.p_lo, last_seen = rows1.n > 0 ? rows1.p_hi : rows0.p_hi;
  if (rows0.n > 0 || rows1.n > 0) tiles = key_tiles<KP_KT>(first_seen, last_seen, a.window, a.sinks);
  // this block's tiles among the sequence's expanded ones
  const KpSeen seen = kp_seen(s, b);
  const KeyTiles all = key_tiles<KP_KT>(seen.first, seen.last, a.window, a.sinks);
  auto slot = [&](int i) {
    const int j = tiles.at(i);
    return (int64_t)here * slots + (j < all.sink_tiles ? j : j - all.first + all.sink_tiles);
  };

  if (warp < 8) {
    // ------------------------------------------------ a stream: scores to weights, one row a thread
    const int g = warp >> 2, row = tid & 127;
    const KpRows& rows = g == 0 ? rows0 : rows1;
    const int R = r0 + 128 * g + row;
    const bool real = R < n_rows;
    const int tok = R / group;
    const int64_t off = (((int64_t)b * s.L + tok) * a.heads + h * group + R - tok * group) * D;
    const int64_t pr = p0 + tok;
    // (a padding row sees what its tile does)
    const int p = !real ? rows.p_hi : pr >= 0 && pr < s.limit ? (int)pr : -1;
    float row_scale;                               // base-2 score of an accumulator, up to the tile's factor
    {
      // the warp's 32 rows, scaled, K-major with 128-byte swizzle.  RPL rows a load, each a run of
      // lanes
      constexpr int LPR = D / 8, RPL = 32 / LPR;
      const int lane = tid & 31, chunk = lane % LPR;
      uint8_t* dst = sm + M::Q + g * M::TILE + (chunk >> 3) * 16384;
      uint4 v[LPR];
#pragma unroll
      for (int q = 0; q < LPR; ++q) {
        const int from = RPL * q + lane / LPR;
        const int64_t ro = __shfl_sync(0xffffffffu, off, from);
        v[q] = make_uint4(0u, 0u, 0u, 0u);
        if (__shfl_sync(0xffffffffu, (int)real, from))
          v[q] = ldg_v4(static_cast<const __nv_bfloat16*>(a.Q) + ro + 8 * chunk);
      }
      int my_e = 0;
#pragma unroll
      for (int q = 0; q < LPR; ++q) {
        const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = fabsf(bf16lo(w[j])), hi = fabsf(bf16hi(w[j]));
          mx = max3(mx, lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f);
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int e = row_exponent(mx);
        const float up = pow2i(14 - e);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = pack_half2(bf16lo(w[j]) * up, bf16hi(w[j]) * up);
        const int at = (row & 96) + RPL * q + lane / LPR;
        *reinterpret_cast<uint4*>(dst + at * 128 + (((chunk & 7) ^ (at & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
        const int er = __shfl_sync(0xffffffffu, e, (lane % RPL) * LPR);          // of row RPL q + lane % RPL
        if (lane / RPL == q) my_e = er;
      }
      row_scale = pow2i(my_e - 14);
      fence_proxy_async_smem();
      mbar_arrive(&q_full);
    }
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t S = lanes + S_COL + 128u * g, O = lanes + O_COL + 128u * g;
    float m = -INFINITY;
    float l = 0.f;
    bool ok = true;
    int used = 0;                                  // tiles of this stream so far
    for (int i = 0; i < tiles.count && ok; ++i) {
      const int j0 = tiles.at(i) * KP_KT;
      if (!rows.any(j0, KP_KT, a.window, a.sinks)) continue;
      const float2 st = factors[slot(i)];
      ok = kp_wait(&s_full[g], used & 1, DEV_ERR_TIMEOUT_ACC);
      if (!ok) break;
      tc_fence_after();
      const float F = st.y;
      float f = fminf(fmaxf(st.x * row_scale, 0x1p-126f), 0x1p127f);         // finite: 0 f is 0
      const bool full = rows.full(j0, KP_KT, a.window, a.sinks);
      uint32_t w[KP_KT / 2];
      float sum;
      auto weights = [&](bool find_top) {          // with the maximum m; or the largest score
        float x[KP_KT], top = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(S + 32 * c, reinterpret_cast<uint32_t*>(x) + 32 * c);
        float ref = m == -INFINITY ? 0.f : BIAS + F - m;
        kp_loads_done(ref, f);
        if (!full) kp_mask<KP_KT>(x, p - j0, a.window > 0 ? p - a.window - j0 : -1, a.sinks - j0);
        if (find_top) top = kp_top(x);
        else kp_weights(x, f, ref, w, sum);
        return top;
      };
      weights(false);
      // a row that sees its first key, or whose weights may pass fp16: move the maximum
      const int j1 = p < j0 + KP_KT - 1 ? p : j0 + KP_KT - 1;
      const bool sees = p >= j0 && (a.window == 0 || j1 > p - a.window || j0 < a.sinks);
      if (__any_sync(0xffffffffu, !(sum <= 65504.f) || (m == -INFINITY && sees))) {
        const float top = weights(true) * f + F, mn = top > m ? top : m;
        float down = m == -INFINITY ? 0.f : ex2(m - mn), none = 0.f;
        m = mn;
        l *= down;
        if (used > 0) {                            // (every product so far was issued ahead of these scores)
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float v[32];
            tmem_ld32(O + c, reinterpret_cast<uint32_t*>(v));
            kp_loads_done(down, none);
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] *= down;
            tmem_st32(O + c, reinterpret_cast<uint32_t (&)[32]>(v));
          }
        }
        weights(false);
        if (!(top < INFINITY)) sum = NAN;          // a row of such scores
      }
      tmem_st32(S, *reinterpret_cast<uint32_t (*)[32]>(w));          // over scores that have been read
      tmem_st32(S + 32, *reinterpret_cast<uint32_t (*)[32]>(w + 32));
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[g]);
      l += sum * pow2i(-(int)F);
      ++used;
    }
    // ---- the output, divided by the sum ----
    if (ok && used > 0) ok = kp_wait(&all_done, 0, DEV_ERR_TIMEOUT_ACC);
    tc_fence_after();
    // a query outside the cache sees no key: zeros, whatever the masked keys' exponentials (2^-125 where they
    // come from the multiply-add units) left in its sum
    // (a maximum of -inf: scores that are all past the smallest fp32 number, or NaN)
    float inv = p < 0 ? 0.f : m == -INFINITY ? NAN : 0x1p-11f / l;
    // (through the queries' shared memory, free by now, to runs of lanes)
    uint8_t* stage = sm + M::Q + g * M::TILE;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float v[32], none = 0.f;
      if (used > 0) {
        tmem_ld32(O + c, reinterpret_cast<uint32_t*>(v));
        kp_loads_done(inv, none);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y0 = inv == 0.f ? 0.f : v[8 * q + 2 * j] * inv;
          const float y1 = inv == 0.f ? 0.f : v[8 * q + 2 * j + 1] * inv;
          const __nv_bfloat162 hv = __floats2bfloat162_rn(y0, y1);
          o[j] = *reinterpret_cast<const uint32_t*>(&hv);
        }
        const int chunk = c / 8 + q;
        *reinterpret_cast<uint4*>(stage + (chunk >> 3) * 16384 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    __syncwarp();
    {
      constexpr int LPR = D / 8, RPL = 32 / LPR;
      const int lane = tid & 31, chunk = lane % LPR;
#pragma unroll 4
      for (int q = 0; q < LPR; ++q) {
        const int from = RPL * q + lane / LPR, at = (row & 96) + from;
        const int64_t ro = __shfl_sync(0xffffffffu, off, from);
        if (__shfl_sync(0xffffffffu, (int)(real && ok), from))
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.A) + ro + 8 * chunk) =
              *reinterpret_cast<const uint4*>(stage + (chunk >> 3) * 16384 + at * 128 +
                                              (((chunk & 7) ^ (at & 7)) << 4));
      }
    }
    tc_fence_before();
  } else if (warp == 9) {
    // ------------------------------------------------ copies
    bool ok = true;
    int issued[2] = {0, 0};                        // tiles of keys, of values
    for (int i = 0; i < tiles.count && ok; ++i) {
      const uint8_t* src = images + slot(i) * (2 * M::TILE);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint64_t *full = v ? &v_full[i & 1] : &k_full[i & 1], *empty = v ? &v_empty[i & 1] : &k_empty[i & 1];
        if (i >= 2 && ok) ok = kp_wait(empty, ((i >> 1) - 1) & 1, DEV_ERR_TIMEOUT_EMPTY);
        if (ok && elect_one()) {
          mbar_arrive_expect_tx(full, M::TILE);
          bulk_load(sm + (v ? M::V : M::K) + (i & 1) * M::TILE, src + v * M::TILE, M::TILE, full);
        }
        __syncwarp();
        issued[v] += ok;
      }
    }
    kp_copies_done<2>(k_full, issued[0]);
    kp_copies_done<2>(v_full, issued[1]);
  } else {
    if (warp == 8 && tiles.count > 0) {
      // ---------------------------------------------- products
      constexpr uint32_t ID_S = idesc_f16(128, KP_KT, false), ID_O = idesc_f16(128, D, true);
      bool ok = kp_wait(&q_full, 0, DEV_ERR_TIMEOUT_A);
      const uint32_t qd = desc_lo(smem_u32(sm + M::Q));
      const uint32_t kd = desc_lo(smem_u32(sm + M::K)), vd = desc_lo(smem_u32(sm + M::V));
      int used0 = 0, used1 = 0;                    // tiles whose weights were used, by stream
      bool was0 = false, was1 = false;             // the last tile was one of the stream's
      for (int i = 0; i <= tiles.count && ok; ++i) {
        const bool more = i < tiles.count;
        const int j0 = more ? tiles.at(i) * KP_KT : 0;
        const bool now0 = more && rows0.any(j0, KP_KT, a.window, a.sinks);
        const bool now1 = more && rows1.any(j0, KP_KT, a.window, a.sinks);
        const uint32_t kb = kd + (i & 1) * (M::TILE >> 4), vb = vd + ((i - 1) & 1) * (M::TILE >> 4);
        // every wait costs some 200 cycles here, also for what is long there: the copies' ones first,
        // while the weights are still being computed
        if (more) ok = kp_wait(&k_full[i & 1], (i >> 1) & 1, DEV_ERR_TIMEOUT_FULL);
        if (i > 0 && ok) ok = kp_wait(&v_full[(i - 1) & 1], ((i - 1) >> 1) & 1, DEV_ERR_TIMEOUT_FULL);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          int& used = g == 0 ? used0 : used1;
          const bool was = g == 0 ? was0 : was1, now = g == 0 ? now0 : now1;
          if (was && ok) ok = kp_wait(&p_full[g], used & 1, DEV_ERR_TIMEOUT_ACC);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (was) {
#pragma unroll
              for (int k = 0; k < KP_KT / 16; ++k)
                mma_f16_ts(tmem + O_COL + 128u * g, tmem + S_COL + 128u * g + 8 * k, vb + (2048 >> 4) * k, ID_O,
                           k > 0 ? 1u : (uint32_t)used);
            }
            if (now) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                mma_f16_ss(tmem + S_COL + 128u * g,
                           qd + g * (M::TILE >> 4) + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                           kb + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), ID_S, k > 0);
              mma_commit(&s_full[g]);
            }
            if (g == 1 && i > 0) mma_commit(&v_empty[(i - 1) & 1]);
            if (g == 1 && more) mma_commit(&k_empty[i & 1]);
          }
          __syncwarp();
          if (was) ++used;
        }
        was0 = now0;
        was1 = now1;
      }
      // completion of everything issued, also after a wait that gave up
      if (elect_one()) mma_commit(&all_done);
      __syncwarp();
      mbar_wait(&all_done, 0, DEV_ERR_TIMEOUT_ACC, false);
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// fp32 rows.  What the sums may lose is 2^-22 here, so every fp32 operand is two fp16
// terms (22 bits) against the codes, which are exact; the steps stay in the softmax, as
// in the few-query kernel: with step_v = f 2^e a key's exponent takes e, the operand is
// p f, the sum takes p 2^-e.  The tensor cores cut their sums off (measured: 1e-7 of the
// sum a product of 16 values deep, 5e-5 after 512), so a tile's output is summed there
// and the tiles' with rounding outside.
//
// A block takes 128 rows of one key head.  Even and odd key tiles go to two groups of
// four warps, each with its own scores buffer, maximum and sum; a tile's output is
// written to a third buffer of tensor memory and added to the running one, a fourth, by
// four more warps, with the maxima's factors.  Per tile 4 x 8 products of 128 x 128 x 16
// (2048 cycles), which bound long contexts (8192 causal tokens of 32 over 8 heads: 1.09 ms,
// 1000 TFLOP/s of fp16 products); 512 tokens of 16 heads are 64 blocks that spend most of
// their 21 us filling and draining.
// ---------------------------------------------------------------------------
constexpr int KX_THREADS = 448;                      // weights: warps 0-3, 4-7; sums: 8-11; products: 12; copies: 13
constexpr int KX_RING = 4;                           // tiles whose keys' factors are held

template <int D>
struct KxSmem {
  static constexpr int TILE = KpTile<D>::BYTES;
  static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, KEYS = 6 * TILE;             // q: both terms; 2 of K and V
  static constexpr int BYTES = KEYS + KX_RING * KP_KEY_FLOATS * 4 + 1024;
};

template <int D>
__global__ void __launch_bounds__(KX_THREADS, 1)
kv4_prefill_f32_kernel(const KvStep s, const AttnArgs a, int head0, int heads_here, int row_tiles, int slots,
                       const uint8_t* __restrict__ images, const float* __restrict__ factors) {
  using M = KxSmem<D>;
  constexpr float BIAS = 10.f;
  constexpr uint32_t S_COL = 0, PART = 256, SUM = 384;          // scores: + 128 g
  extern __shared__ uint8_t kp_raw[];
  __shared__ uint64_t q_full, k_full[2], v_full[2], k_empty[2], v_empty[2], key_full[KX_RING], s_full[2], p_full[2],
      part_full, part_free, all_done;
  __shared__ uint32_t tmem_sh;
  __shared__ int failed, row_e[128];
  __shared__ float tile_m[4][128], fin_m[2][128], fin_l[2][128];
  uint8_t* sm = smem_align(kp_raw, 1024);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (kp_padding(s, a, head0, heads_here, row_tiles, 128)) return;
  if (tid == 0) {
    mbar_init(&q_full, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    for (int i = 0; i < KX_RING; ++i) mbar_init(&key_full[i], 1);
    mbar_init(&part_full, 1);
    mbar_init(&part_free, 128);
    mbar_init(&all_done, 1);
    failed = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&tmem_sh, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  // only once the tensor memory is allocated may the next kernel of the stream be scheduled
  pdl_launch_dependents();
  pdl_wait();                                        // q, the cache and the images come from the previous kernels

  const int rt = row_tiles - 1 - (int)(blockIdx.x / heads_here);       // the longest row tiles first
  const int here = (int)(blockIdx.x % heads_here), b = (head0 + here) / a.kv_heads, h = head0 + here - b * a.kv_heads;
  const int group = a.heads / a.kv_heads;
  const int n_rows = kv_real_tokens(s, b) * group;
  const int r0 = rt * 128;
  const int64_t p0 = kv_first_position(s, b);
  const KpRows rows = kp_rows(r0, n_rows, group, p0, s.limit);
  KeyTiles tiles = {0, 0, 0};
  if (rows.n > 0) tiles = key_tiles<KP_KT>(rows.p_lo, rows.p_hi, a.window, a.sinks);
  const KpSeen seen = kp_seen(s, b);
  const KeyTiles all = key_tiles<KP_KT>(seen.first, seen.last, a.window, a.sinks);
  auto slot = [&](int i) {
    const int j = tiles.at(i);
    return (int64_t)here * slots + (j < all.sink_tiles ? j : j - all.first + all.sink_tiles);
  };
  const int row = tid & 127;
  const int R = r0 + row, tok = R / group;
  const bool real = R < n_rows;
  const int64_t off = (((int64_t)b * s.L + tok) * a.heads + h * group + R - tok * group) * D;
  const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  bool ok = true;
  float sum_m = -INFINITY;                           // the running output's maximum (warps 8-11)

  if (warp < 8) {
    // ------------------------------------------------ scores to weights, one row a thread
    const int g = warp >> 2;
    const int64_t pr = p0 + tok;
    // (a padding row sees what its tile does)
    const int p = !real ? rows.p_hi : pr >= 0 && pr < s.limit ? (int)pr : -1;
    // queries: 16 rows a warp (32 w + 16 g ..), one a load, a run of lanes
    {
      constexpr int LPR = D / 4, RPL = 32 / LPR;
      const int lane = tid & 31, part = lane % LPR;
      uint8_t* dst = sm + M::Q + (part >> 4) * 16384 + 8 * (part & 1);
#pragma unroll
      for (int q = 0; q < 16 / RPL; ++q) {
        const int from = 16 * g + RPL * q + lane / LPR, at = (row & 96) + from;
        const int64_t ro = __shfl_sync(0xffffffffu, off, from);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (__shfl_sync(0xffffffffu, (int)real, from)) v = ldg_v4(static_cast<const float*>(a.Q) + ro + 4 * part);
        float x[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fabsf(x[j]) < INFINITY ? fabsf(x[j]) : 0.f);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int e = row_exponent(mx);
        const float up = pow2i(14 - e);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] *= up;
        const uint32_t h0 = pack_half2(x[0], x[1]), h1 = pack_half2(x[2], x[3]);
        uint8_t* to = dst + at * 128 + ((((part >> 1) & 7) ^ (at & 7)) << 4);
        *reinterpret_cast<uint2*>(to) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(to + M::TILE) = make_uint2(half2_rest(h0, x[0], x[1]), half2_rest(h1, x[2], x[3]));
        if (part == 0) row_e[at] = e;
      }
      fence_proxy_async_smem();
      mbar_arrive(&q_full);
      ok = kp_wait(&q_full, 0, DEV_ERR_TIMEOUT_A);                     // every row's exponent
    }
    const float row_scale = pow2i(row_e[row] - 14);
    const uint32_t S = lanes + S_COL + 128u * g;
    const uint64_t rs2 = pack_f2(row_scale, row_scale);
    float m = -INFINITY, l = 0.f;
    for (int i = g, n = 0; i < tiles.count && ok; i += 2, ++n) {
      const int j0 = tiles.at(i) * KP_KT;
      const bool masked = !rows.full(j0, KP_KT, a.window, a.sinks);
      const int hi = p - j0, lo = a.window > 0 ? p - a.window - j0 : -1, sk = a.sinks - j0;
      ok = kp_wait(&key_full[i % KX_RING], (i / KX_RING) & 1, DEV_ERR_TIMEOUT_FULL) &&
           kp_wait(&s_full[g], n & 1, DEV_ERR_TIMEOUT_ACC);
      if (!ok) break;
      tc_fence_after();
      const float* ks = reinterpret_cast<const float*>(sm + M::KEYS) + (i % KX_RING) * KP_KEY_FLOATS;
      // 32 scores as base-2 exponents, the value step's among them
      auto scores = [&](int c, float (&x)[32]) {
        float zero = 0.f, one = 0.f;
        tmem_ld32(S + 32 * c, reinterpret_cast<uint32_t*>(x));
        kp_loads_done(zero, one);
        const uint64_t rs = add_f2(rs2, pack_f2(zero, one));           // (after the load)
#pragma unroll
        for (int q = 0; q < 32; q += 4) {
          const ulonglong2 kf = *reinterpret_cast<const ulonglong2*>(ks + 32 * c + q);
          const ulonglong2 ef = *reinterpret_cast<const ulonglong2*>(ks + KP_KT + 32 * c + q);
          unpack_f2(fma_f2(pack_f2(x[q], x[q + 1]), mul_f2(kf.x, rs), ef.x), x[q], x[q + 1]);
          unpack_f2(fma_f2(pack_f2(x[q + 2], x[q + 3]), mul_f2(kf.y, rs), ef.y), x[q + 2], x[q + 3]);
        }
        if (masked) kp_mask<32>(x, hi - 32 * c, lo - 32 * c, sk - 32 * c);
      };
      float top = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float x[32];
        scores(c, x);
#pragma unroll
        for (int q = 0; q < 32; q += 2) top = max3(top, x[q], x[q + 1]);
      }
      const float mn = fmaxf(m, top);
      l *= m == mn ? 1.f : ex2(m - mn);
      m = mn;
      const float ref = m == -INFINITY ? 0.f : BIAS - m;
      const uint64_t ref2 = pack_f2(ref, ref);
      uint64_t l2 = 0;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float x[32];
        uint32_t w[32];                              // 16 pairs, then what they leave
        scores(c, x);
#pragma unroll
        for (int q = 0; q < 32; q += 4) {
          const ulonglong2 inv = *reinterpret_cast<const ulonglong2*>(ks + 2 * KP_KT + 32 * c + q);
          const ulonglong2 vf = *reinterpret_cast<const ulonglong2*>(ks + 3 * KP_KT + 32 * c + q);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float e0, e1, w0, w1;
            unpack_f2(add_f2(pack_f2(x[q + 2 * k], x[q + 2 * k + 1]), ref2), e0, e1);
            const uint64_t e2 = pack_f2(ex2(e0), ex2(e1));
            l2 = fma_f2(e2, k == 0 ? inv.x : inv.y, l2);
            unpack_f2(mul_f2(e2, k == 0 ? vf.x : vf.y), w0, w1);
            w[q / 2 + k] = pack_half2(w0, w1);
            w[16 + q / 2 + k] = half2_rest(w[q / 2 + k], w0, w1);
          }
        }
        tmem_st32(S + 32 * c, w);                    // over the scores they come from
      }
      float l0, l1;
      unpack_f2(l2, l0, l1);
      l += l0 + l1;
      tile_m[i & 3][row] = m;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[g]);
    }
    fin_m[g][row] = m;
    fin_l[g][row] = l;
  } else if (warp < 12) {
    // ------------------------------------------------ the tiles' outputs into the running one
    for (int i = 0; i < tiles.count && ok; ++i) {
      ok = kp_wait(&part_full, i & 1, DEV_ERR_TIMEOUT_ACC);
      if (!ok) break;
      tc_fence_after();
      const float mt = tile_m[i & 3][row], mn = fmaxf(sum_m, mt);
      float keep = sum_m == mn ? 1.f : ex2(sum_m - mn), add = mt == mn ? 1.f : ex2(mt - mn);
      if (mn == -INFINITY) keep = add = 0.f;
      sum_m = mn;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float x[32], y[32];
        tmem_ld32(lanes + PART + c, reinterpret_cast<uint32_t*>(x));
        if (i > 0) tmem_ld32(lanes + SUM + c, reinterpret_cast<uint32_t*>(y));
        kp_loads_done(keep, add);
#pragma unroll
        for (int q = 0; q < 32; ++q) y[q] = i > 0 ? y[q] * keep + x[q] * add : x[q] * add;
        tmem_st32(lanes + SUM + c, reinterpret_cast<uint32_t (&)[32]>(y));
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&part_free);
    }
  } else if (warp == 12 && tiles.count > 0) {
    // ------------------------------------------------ products
    constexpr uint32_t ID_S = idesc_f16(128, KP_KT, false), ID_O = idesc_f16(128, D, true);
    ok = kp_wait(&q_full, 0, DEV_ERR_TIMEOUT_A);
    const uint32_t qd = desc_lo(smem_u32(sm + M::Q));
    const uint32_t kd = desc_lo(smem_u32(sm + M::K)), vd = desc_lo(smem_u32(sm + M::V));
    for (int i = 0; i < tiles.count + 2 && ok; ++i) {
      if (i >= 2) {                                  // tile i - 2's output: its weights lie where tile i's scores go
        const int t = i - 2;
        ok = kp_wait(&v_full[t & 1], (t >> 1) & 1, DEV_ERR_TIMEOUT_FULL) &&
             kp_wait(&p_full[t & 1], (t >> 1) & 1, DEV_ERR_TIMEOUT_ACC) &&
             (t == 0 || kp_wait(&part_free, (t - 1) & 1, DEV_ERR_TIMEOUT_ACC));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t P = tmem + S_COL + 128u * (t & 1), vb = vd + (t & 1) * (M::TILE >> 4);
#pragma unroll
          for (int term = 1; term >= 0; --term)      // the small terms first
#pragma unroll
            for (int k = 0; k < KP_KT / 16; ++k)
              mma_f16_ts(tmem + PART, P + 32 * (k >> 1) + 16 * term + 8 * (k & 1), vb + (2048 >> 4) * k, ID_O,
                         term == 0 || k > 0);
          mma_commit(&part_full);
          mma_commit(&v_empty[t & 1]);
        }
        __syncwarp();
      }
      if (i < tiles.count) {
        ok = kp_wait(&k_full[i & 1], (i >> 1) & 1, DEV_ERR_TIMEOUT_FULL);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t kb = kd + (i & 1) * (M::TILE >> 4);
#pragma unroll
          for (int term = 1; term >= 0; --term)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t o = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
              mma_f16_ss(tmem + S_COL + 128u * (i & 1), qd + term * (M::TILE >> 4) + o, kb + o, ID_S,
                         term == 0 || k > 0);
            }
          mma_commit(&s_full[i & 1]);
          mma_commit(&k_empty[i & 1]);
        }
        __syncwarp();
      }
    }
    // completion of everything issued, also after a wait that gave up
    if (elect_one()) mma_commit(&all_done);
    __syncwarp();
    mbar_wait(&all_done, 0, DEV_ERR_TIMEOUT_ACC, false);
  } else if (warp == 13) {
    // ------------------------------------------------ copies
    int issued_k = 0, issued_v = 0;                  // tiles
    for (int i = 0; i < tiles.count && ok; ++i) {
      const uint8_t* src = images + slot(i) * (2 * M::TILE);
      const int st = i & 1, ring = i % KX_RING;
      if (i >= 2) ok = kp_wait(&k_empty[st], ((i >> 1) - 1) & 1, DEV_ERR_TIMEOUT_EMPTY);
      if (ok && elect_one()) {
        // (tile i - 4's factors: its weights were used before the scores of tile i - 2 were issued)
        mbar_arrive_expect_tx(&key_full[ring], KP_KEY_FLOATS * 4);
        bulk_load(sm + M::KEYS + ring * KP_KEY_FLOATS * 4, factors + slot(i) * KP_KEY_FLOATS, KP_KEY_FLOATS * 4,
                  &key_full[ring]);
        mbar_arrive_expect_tx(&k_full[st], M::TILE);
        bulk_load(sm + M::K + st * M::TILE, src, M::TILE, &k_full[st]);
      }
      __syncwarp();
      issued_k += ok;
      if (i >= 2 && ok) ok = kp_wait(&v_empty[st], ((i >> 1) - 1) & 1, DEV_ERR_TIMEOUT_EMPTY);
      if (ok && elect_one()) {
        mbar_arrive_expect_tx(&v_full[st], M::TILE);
        bulk_load(sm + M::V + st * M::TILE, src + M::TILE, M::TILE, &v_full[st]);
      }
      __syncwarp();
      issued_v += ok;
    }
    kp_copies_done<2>(k_full, issued_k);
    kp_copies_done<KX_RING>(key_full, issued_k);
    kp_copies_done<2>(v_full, issued_v);
  }
  if (!ok) failed = 1;
  __syncthreads();
  if (warp >= 8 && warp < 12 && !failed) {
    tc_fence_after();
    // the two groups' sums in the running output's scale
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < 2; ++g)
      if (fin_m[g][row] != -INFINITY || fin_l[g][row] != 0.f) sum += fin_l[g][row] * ex2(fin_m[g][row] - sum_m);
    // a query outside the cache sees no key: zeros; scores that are all -inf leave 0 / 0
    const int64_t pr = p0 + tok;
    float inv = pr < 0 || pr >= s.limit ? 0.f : 1.0f / sum;
    // (through the queries' shared memory, free by now, to runs of lanes)
    uint8_t* stage = sm + M::Q;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float x[32], none = 0.f;
      if (tiles.count > 0) {
        tmem_ld32(lanes + SUM + c, reinterpret_cast<uint32_t*>(x));
        kp_loads_done(inv, none);
      }
#pragma unroll
      for (int q = 0; q < 32; q += 4) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = inv == 0.f ? 0.f : x[q + j] * inv;
        *reinterpret_cast<float4*>(stage + row * (D * 4) + ((((c + q) >> 2) ^ (row & 7)) << 4)) =
            make_float4(y[0], y[1], y[2], y[3]);
      }
    }
    __syncwarp();
    {
      constexpr int LPR = D / 4, RPL = 32 / LPR;
      const int lane = tid & 31, part = lane % LPR;
#pragma unroll 4
      for (int q = 0; q < LPR; ++q) {
        const int from = RPL * q + lane / LPR, at = (row & 96) + from;
        const int64_t ro = __shfl_sync(0xffffffffu, off, from);
        if (__shfl_sync(0xffffffffu, (int)real, from))
          *reinterpret_cast<float4*>(static_cast<float*>(a.A) + ro + 4 * part) =
              *reinterpret_cast<const float4*>(stage + at * (D * 4) + ((part ^ (at & 7)) << 4));
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Tiles of a sequence that a step's queries can see, at most.
static int64_t kp_slots(const KvStep& s, const AttnArgs& a) {
  const int64_t all = ((int64_t)s.limit + KP_KT - 1) / KP_KT;
  if (a.window == 0) return all;
  const int64_t some = ((int64_t)a.sinks + KP_KT - 1) / KP_KT + ((int64_t)a.window + s.L + KP_KT - 1) / KP_KT + 1;
  return some < all ? some : all;
}
// Workspace of one key head: its tiles' images, then their factors (both in multiples of 16 bytes).
static int64_t kp_head_bytes(const KvStep& s, const AttnArgs& a, int bf16, int d) {
  return kp_slots(s, a) * (2 * KP_KT * d * 2 + (bf16 ? 16 : KP_KEY_FLOATS * 4));
}
// Enough for one launch of every head, or 256 MB: heads are then taken in turns.
size_t kv4_prefill_workspace(const KvStep& s, const AttnArgs& a, int bf16, int d) {
  const int64_t head = kp_head_bytes(s, a, bf16, d), heads = (int64_t)a.kv_heads * s.B, most = (int64_t)256 << 20;
  int64_t turn = most / head;
  turn = turn < 1 ? 1 : (turn < heads ? turn : heads);
  return (size_t)(turn * head);
}
// Heads of a turn in a workspace of `bytes` (at most a grid dimension).
static int kp_turn(const KvStep& s, const AttnArgs& a, int bf16, int d, size_t bytes) {
  const int64_t fit = (int64_t)bytes / kp_head_bytes(s, a, bf16, d), heads = (int64_t)a.kv_heads * s.B;
  const int64_t most = heads < 65535 ? heads : 65535;
  return (int)(fit < most ? fit : most);
}
// Kernels of a call with a workspace of the size above: the expansion and the attention, a turn.
int kv4_prefill_launches(const KvStep& s, const AttnArgs& a, int bf16, int d) {
  const int turn = kp_turn(s, a, bf16, d, kv4_prefill_workspace(s, a, bf16, d));
  return 2 * ((a.kv_heads * s.B + turn - 1) / turn);
}

template <int D, bool EXACT>
static cudaError_t launch_prefill(const KvStep& s, const AttnArgs& a, uint8_t* ws, size_t ws_bytes, cudaStream_t st) {
  auto kern = EXACT ? kv4_prefill_f32_kernel<D> : kv4_prefill_kernel<D>;
  constexpr size_t smem = EXACT ? KxSmem<D>::BYTES : KpSmem<D>::BYTES;
  constexpr int THREADS = EXACT ? KX_THREADS : KP_THREADS, ROWS = EXACT ? 128 : 256;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int row_tiles = (int)(((int64_t)s.L * (a.heads / a.kv_heads) + ROWS - 1) / ROWS);
  const int slots = (int)kp_slots(s, a), heads = a.kv_heads * s.B;
  const int turn = kp_turn(s, a, !EXACT, D, ws_bytes);
  if (turn < 1) return cudaErrorInvalidValue;
  float* factors = reinterpret_cast<float*>(ws + (int64_t)turn * slots * KpTile<D>::PAIR);
  for (int head0 = 0; head0 < heads; head0 += turn) {
    const int n = heads - head0 < turn ? heads - head0 : turn;
    e = launch_pdl(kv4_expand_kernel<D, EXACT>, dim3((unsigned)slots, (unsigned)n), dim3(256), 0, st, 1u, s, a, head0,
                   slots, (float)(1.4426950408889634 / sqrt((double)D)), ws, factors);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)(row_tiles * n)), dim3(THREADS), smem, st, 1u, s, a, head0, n, row_tiles, slots,
                   (const uint8_t*)ws, (const float*)factors);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Whether the step takes this path, by the time either would take (us, fitted to calls with
// a cold L2).  Here a block takes 256 (bf16) or 128 (fp32) rows through the keys at 1.75 or
// 2.2 us a tile behind some 9 us of filling and draining, 148 at a time, after the expansion
// (80 KB a tile and head); the few-query kernel takes 16 rows a warp-tile of 32 keys, which
// cost 2.3 or 3.5 ns of the whole GPU, and 22 ns a block.  Measured, this path and the other: bf16, 128 rows of 8
// heads, 2032 keys 46 and 21; fp32, 128 rows of 16 heads, 2128 keys 58 and 39; 512 causal fp32
// rows of 16 heads 24 and 34; bf16, 8192 causal tokens of 8 x 4 heads 500 and 3800.
bool kv4_prefill_applies(const KvStep& s, const AttnArgs& a, int bf16) {
  const double rows = (double)s.L * (a.heads / a.kv_heads), heads = (double)a.kv_heads * s.B;
  double most = s.limit, mean = s.limit - 0.5 * s.L;                   // keys of a row
  if (mean < 0.5 * s.limit) mean = 0.5 * s.limit;
  if (a.window > 0) {
    const double w = (double)a.window + a.sinks;
    most = w < most ? w : most;
    mean = w < mean ? w : mean;
  }
  const double waves = ceil(rows / (bf16 ? 256.0 : 128.0)) * heads / 148.0;
  const double tiles = (waves <= 1.0 ? most : mean) / KP_KT + 1.0;
  const double here = 10.0 + (waves > 1.0 ? waves : 1.0) * ((bf16 ? 1.75 : 2.2) * tiles + 9.0) +
                      heads * (most / KP_KT + 1.0) * 0.016;
  const double other = 12.0 + ceil(rows / 16.0) * heads * ((mean / 32.0 + 1.0) * (bf16 ? 2.3e-3 : 3.5e-3) + 0.022);
  return rows > 16.0 && here < other;
}

cudaError_t run_kv4_prefill(const KvStep& s, const AttnArgs& a, int bf16, int d, void* ws, size_t ws_bytes,
                            cudaStream_t st) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (d == 128)
    return bf16 ? launch_prefill<128, false>(s, a, w, ws_bytes, st) : launch_prefill<128, true>(s, a, w, ws_bytes, st);
  return bf16 ? launch_prefill<64, false>(s, a, w, ws_bytes, st) : launch_prefill<64, true>(s, a, w, ws_bytes, st);
}

}  // namespace bitnet
