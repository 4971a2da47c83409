// Causal attention over the 4-bit key/value cache for many queries a key head
// (prefill), on tcgen05.  This file is compiled as a whole program, so that its
// warps can share the register file unevenly, and keeps its own copy of the error
// flag.
#define BITNET_OWN_ERROR_FLAG
#include "kv4_common.cuh"

#include <cuda_bf16.h>

namespace bitnet {

// ---------------------------------------------------------------------------
// A block takes 256 rows (token, head of the group) of one key head as two streams
// of 128, which share every tile of 128 keys: four warps unpack a tile from global
// memory into 128-byte swizzled fp16 operands in shared memory (two stages), one
// warp issues the products, and four warps a stream turn scores into weights, one
// row a thread.
//   scores  q (shared memory) x keys -> tensor memory, fp32
//   weights written over the scores as fp16, the product's operand in tensor memory
//   output  weights x values (keys as the reduction) -> tensor memory, fp32
// While one stream's weights are computed, the other stream's products run.
//
// Operands.  A query row is scaled by a power of two (bf16 values are then exact in
// fp16).  A tile's keys are code * step * 2^(11 - E) in fp16, E the exponent of the
// tile's largest step, rounded once (2^-11 of a value, as the weights are); values the
// same with E = F.  A row's score in base-2 exponents is then acc * c with one factor
// c a row and tile, and its weight carries the tile's 2^F, p' = 2^(acc c + F - m): the
// output sums p' v 2^(11 - F) over all tiles in one scale, and the softmax sum takes
// 2^-F once a tile.  The running maximum m is that of acc c + F; it is moved only when
// a row exceeds it by 2^8 (the weights then stay below 2^15), so the output in tensor
// memory is rescaled rarely.  Steps in the softmax instead (a factor, an exponent and
// a reciprocal a key, read from shared memory) took 3000 cycles a stream and tile.
// ---------------------------------------------------------------------------
constexpr int KP_KT = 128;                           // keys a tile
constexpr int KP_STEPS = 4;                          // tiles whose steps are held: a stream may be two tiles behind
constexpr int KP_THREADS = 512;                      // streams: warps 0-3 and 4-7; unpackers 8-11; products: warp 12

template <int D>
struct KpSmem {
  static constexpr int TILE = 128 * D * 2;           // 128 rows of D 16-bit values
  static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, BYTES = 6 * TILE + 1024;   // 2 of each, + alignment
};

// One lane of a warp that runs as a whole.  The compiler knows the lane to be alone
// (unlike a test of the lane's number), so the products' descriptors stay in uniform
// registers: issued from a lane-number branch, a product took 300 cycles instead of 64.
BN_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

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
BN_DEV float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Instruction descriptor of kind::f16: fp32 accumulator, fp16 or bf16 operands, A
// K-major, B K-major or (b_mn) with its N dimension contiguous.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool bf16, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// Shared-memory descriptor, 128-byte swizzle, N contiguous: 64-value column blocks
// `block` bytes apart, groups of 8 reduction rows 1024 bytes apart.
BN_DEV uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((block >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
BN_DEV void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
BN_DEV void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
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

// Positions of one stream's rows, and what of a key tile they see.
struct KpRows {
  int n, p_lo, p_hi;                                 // rows; first and last position inside the cache
  bool in;                                           // every row's position lies inside the cache
  BN_DEV bool any(int j0, int window, int sinks) const {
    return n > 0 && j0 <= p_hi && (window == 0 || j0 + KP_KT - 1 > p_lo - window || j0 < sinks);
  }
  BN_DEV bool full(int j0, int window, int sinks) const {
    return in && j0 + KP_KT - 1 <= p_lo && (window == 0 || j0 > p_hi - window || j0 + KP_KT <= sinks);
  }
};
BN_DEV KpRows kp_rows(int r0, int n_rows, int group, int64_t p0, int T_cap) {
  KpRows r;
  r.n = n_rows - r0 < 0 ? 0 : (n_rows - r0 < 128 ? n_rows - r0 : 128);
  const int64_t pf = p0 + r0 / group, pl = p0 + (r0 + (r.n > 0 ? r.n : 1) - 1) / group;
  r.in = pf >= 0 && pl < T_cap;
  if (pl < 0 || pf >= T_cap) r.n = 0;                // no row sees a key
  r.p_lo = pf < 0 ? 0 : (int)(pf < T_cap ? pf : T_cap - 1);
  r.p_hi = pl < 0 ? 0 : (int)(pl < T_cap ? pl : T_cap - 1);
  return r;
}

template <int D>
__global__ void __launch_bounds__(KP_THREADS, 1)
kv4_prefill_kernel(const KvStep s, const AttnArgs a, float scale_log2e, int row_tiles) {
  using M = KpSmem<D>;
  constexpr float BIAS = 7.f, MOVE = 8.f;
  constexpr uint32_t S_COL = 0, O_COL = 256;         // streams: + 128 g
  extern __shared__ uint8_t kp_raw[];
  __shared__ uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2], q_full, s_full[2], p_full[2], o_full[2];
  __shared__ uint32_t tmem_sh;
  __shared__ __align__(16) uint32_t step_top[2][2][4];        // read as 16 bytes
  __shared__ float2 steps[KP_STEPS];                  // of a tile: the scores' factor, F
  uint8_t* sm = smem_align(kp_raw, 1024);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&v_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&q_full, 256);
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
  pdl_wait();                                        // q and the cache come from the previous kernel

  // the longest row tiles first: blocks of the last rows see the most keys
  const int heads_all = a.kv_heads * s.B;
  const int rt = row_tiles - 1 - (int)(blockIdx.x / heads_all);
  const int hb = (int)(blockIdx.x % heads_all), b = hb / a.kv_heads, h = hb - b * a.kv_heads;
  const int group = a.heads / a.kv_heads;
  const int n_rows = kv_real_tokens(s, b) * group;
  const int r0 = rt * 256;
  const int64_t p0 = kv_first_position(s, b);
  const KpRows rows0 = kp_rows(r0, n_rows, group, p0, s.T_cap), rows1 = kp_rows(r0 + 128, n_rows, group, p0, s.T_cap);
  KeyTiles tiles = {0, 0, 0};
  const int first_seen = rows0.n > 0 ? rows0.p_lo : rows1.p_lo, last_seen = rows1.n > 0 ? rows1.p_hi : rows0.p_hi;
  if (rows0.n > 0 || rows1.n > 0) tiles = key_tiles<KP_KT>(first_seen, last_seen, a.window, a.sinks);
  const int64_t head = (int64_t)b * a.kv_heads + h;

  if (r0 < n_rows) {
    if (warp < 8) {
      // ------------------------------------------------ a stream: scores to weights, one row a thread
      asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
      const int g = warp >> 2, row = tid & 127;
      const KpRows& rows = g == 0 ? rows0 : rows1;
      const int R = r0 + 128 * g + row;
      const bool real = R < n_rows;
      const int tok = R / group;
      const int64_t off = (((int64_t)b * s.L + tok) * a.heads + h * group + R - tok * group) * D;
      const int64_t pr = p0 + tok;
      const int p = real && pr >= 0 && pr < s.T_cap ? (int)pr : -1;
      float row_scale;                               // base-2 score of an accumulator, up to the tile's factor
      {
        // the row's values, scaled, K-major with 128-byte swizzle
        uint8_t* dst = sm + M::Q + g * M::TILE + row * 128;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.Q) + off;
        uint4 v[D / 8];
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          v[c] = make_uint4(0u, 0u, 0u, 0u);
          if (real) v[c] = ldg_v4(src + 8 * c);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = fabsf(bf16lo(w[j])), hi = fabsf(bf16hi(w[j]));
            mx = max3(mx, lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f);
          }
        }
        const int e = row_exponent(mx);
        const float up = pow2i(14 - e);
        row_scale = pow2i(e - 14);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = pack_half2(bf16lo(w[j]) * up, bf16hi(w[j]) * up);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + (((c & 7) ^ (row & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&q_full);
      }
      const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
      const uint32_t S = lanes + S_COL + 128u * g, O = lanes + O_COL + 128u * g;
      float m = -INFINITY;
      float l = 0.f;
      bool started = false, ok = true;
      int seen = 0;
      for (int i = 0; i < tiles.count && ok; ++i) {
        const int j0 = tiles.at(i) * KP_KT;
        if (!rows.any(j0, a.window, a.sinks)) continue;
        ok = mbar_wait_warp(&k_full[i & 1], (i >> 1) & 1, DEV_ERR_TIMEOUT_FULL) &&       // the tile's steps
             mbar_wait_warp(&s_full[g], seen & 1, DEV_ERR_TIMEOUT_ACC);
        ++seen;
        if (!ok) break;
        tc_fence_after();
        const float2 st = steps[i % KP_STEPS];
        const float f = st.x * row_scale, F = st.y;
        float x[KP_KT];
        {
          uint32_t* xr = reinterpret_cast<uint32_t*>(x);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(S + 32 * c, xr + 32 * c);
          tmem_wait_ld();
        }
        if (!rows.full(j0, a.window, a.sinks)) {
          const int hi = p - j0;                                       // columns up to hi, and past lo or below sk
          const int lo = a.window > 0 ? p - a.window - j0 : -1, sk = a.sinks - j0;
#pragma unroll
          for (int c = 0; c < KP_KT; ++c) x[c] = c <= hi && (c > lo || c < sk) ? x[c] : -INFINITY;
        }
        float mx = max3(x[0], x[1], x[2]), my = max3(x[3], x[4], x[5]);
#pragma unroll
        for (int c = 6; c < KP_KT - 2; c += 4) {
          mx = max3(mx, x[c], x[c + 1]);
          my = max3(my, x[c + 2], x[c + 3]);
        }
        mx = max3(mx, my, fmaxf(x[KP_KT - 2], x[KP_KT - 1])) * f + F;
        if (__any_sync(0xffffffffu, mx > m + MOVE || (m == -INFINITY && mx != -INFINITY))) {
          const float mn = fmaxf(m, mx);
          const float down = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= down;
          if (started) {                                               // this stream's products so far are complete
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t v[32];
              tmem_ld32(O + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) * down);
              tmem_st32(O + c, v);
            }
          }
        }
        started = true;
        const float ref = m == -INFINITY ? 0.f : BIAS + F - m;
        const uint64_t ref2 = pack_f2(ref, ref), f2 = pack_f2(f, f);
        uint64_t l2 = 0, l3 = 0;
        uint32_t w[KP_KT / 2];
#pragma unroll
        for (int c = 0; c < KP_KT; c += 4) {
          float e0, e1, e2, e3;
          unpack_f2(fma_f2(pack_f2(x[c], x[c + 1]), f2, ref2), e0, e1);
          unpack_f2(fma_f2(pack_f2(x[c + 2], x[c + 3]), f2, ref2), e2, e3);
          e0 = ex2(e0); e1 = ex2(e1); e2 = ex2(e2); e3 = ex2(e3);
          l2 = add_f2(l2, pack_f2(e0, e1));
          l3 = add_f2(l3, pack_f2(e2, e3));
          w[c / 2] = pack_half2(e0, e1);
          w[c / 2 + 1] = pack_half2(e2, e3);
        }
        {
          float s0, s1;
          unpack_f2(add_f2(l2, l3), s0, s1);
          l += (s0 + s1) * pow2i(-(int)F);
        }
        tmem_st32(S, *reinterpret_cast<uint32_t (*)[32]>(w));
        tmem_st32(S + 32, *reinterpret_cast<uint32_t (*)[32]>(w + 32));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[g]);
      }
      // ---- the output, divided by the sum ----
      if (ok && started) ok = mbar_wait_warp(&o_full[g], 0, DEV_ERR_TIMEOUT_ACC);
      tc_fence_after();
      const float inv = m == -INFINITY ? 0.f : 0x1p-11f / l;           // a query that sees no key: zeros
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.A) + off;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        if (started) {
          tmem_ld32(O + c, v);
          tmem_wait_ld();
        }
        if (real && ok) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float y0 = inv == 0.f ? 0.f : __uint_as_float(v[8 * q + 2 * j]) * inv;
              const float y1 = inv == 0.f ? 0.f : __uint_as_float(v[8 * q + 2 * j + 1]) * inv;
              const __nv_bfloat162 hv = __floats2bfloat162_rn(y0, y1);
              o[j] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            *reinterpret_cast<uint4*>(out + c + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      tc_fence_before();
    } else if (warp < 12) {
      // ------------------------------------------------ codes to operands: one key a thread
      asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
      const int key = tid & 127;
      const uint8_t* kc = a.Kc + head * s.T_cap * (D / 2);
      const uint8_t* vc = a.Vc + head * s.T_cap * (D / 2);
      const float* ks = a.Ks + head * s.T_cap;
      const float* vs = a.Vs + head * s.T_cap;
      uint4 kw[D / 32], vw[D / 32];
      float kstep = 0.f, vstep = 0.f;
      const int seen_lo = a.window > 0 ? first_seen - a.window : -1;   // keys past it, and the sinks, are seen by some row
      auto load_k = [&](int i) {
        const int j = i < tiles.count ? tiles.at(i) * KP_KT + key : s.T_cap;
        kstep = vstep = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) kw[c] = make_uint4(0u, 0u, 0u, 0u);
        if (j <= last_seen && (j > seen_lo || j < a.sinks)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) kw[c] = ldg_v4(kc + (int64_t)j * (D / 2) + 16 * c);
          kstep = ldg_f32(ks + j);
          vstep = ldg_f32(vs + j);
        }
      };
      auto load_v = [&](int i) {
        const int j = i < tiles.count ? tiles.at(i) * KP_KT + key : s.T_cap;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) vw[c] = make_uint4(0u, 0u, 0u, 0u);
        if (j <= last_seen && (j > seen_lo || j < a.sinks)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) vw[c] = ldg_v4(vc + (int64_t)j * (D / 2) + 16 * c);
        }
      };
      load_k(0);
      load_v(0);
      bool ok = true;                                // after a wait that gave up the loop only keeps its barriers
      for (int i = 0; i < tiles.count; ++i) {
        const int st = i & 1;
        // the tile's largest steps.  A row whose steps are not finite is NaN to the queries that
        // see it, through its key alone: a masked weight of 0 would not hide it in the values
        const bool bad = !(fabsf(kstep) < INFINITY && fabsf(vstep) < INFINITY);
        const uint32_t kb = bad ? 0u : __float_as_uint(fabsf(kstep)), vb = bad ? 0u : __float_as_uint(fabsf(vstep));
        const uint32_t kt = __reduce_max_sync(0xffffffffu, kb), vt = __reduce_max_sync(0xffffffffu, vb);
        if ((tid & 31) == 0) {
          step_top[st][0][warp & 3] = kt;
          step_top[st][1][warp & 3] = vt;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const uint4 k4 = *reinterpret_cast<const uint4*>(step_top[st][0]), v4 = *reinterpret_cast<const uint4*>(step_top[st][1]);
        const int E = row_exponent(__uint_as_float(max(max(k4.x, k4.y), max(k4.z, k4.w))));
        const int F = step_exponent(__uint_as_float(max(max(v4.x, v4.y), max(v4.z, v4.w))));
        const float kx = kstep * pow2i(11 - E);
        // 8 bits of the step times a code are exact in fp16; the rest of the step joins in one rounding
        const float k_top = __uint_as_float(__float_as_uint(kx) & 0xFFFF0000u);
        const uint32_t kh = bad ? 0x7FFF7FFFu : both_halves(k_top), kl = both_halves(kx - k_top);
        const uint32_t vh = bad ? 0u : both_halves(vstep * pow2i(11 - F));
        // the scores of tile i - 2 are complete, so both streams are done with the steps of tile i - 3
        if (i >= 2 && ok) ok = mbar_wait(&k_empty[st], ((i >> 1) - 1) & 1, DEV_ERR_TIMEOUT_EMPTY);
        uint8_t* kd = sm + M::K + st * M::TILE + key * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 q = kw[c >> 2];
          const uint32_t word = (c & 3) == 0 ? q.x : (c & 3) == 1 ? q.y : (c & 3) == 2 ? q.z : q.w;
          uint32_t v[4];
          codes_to_half2(word, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = h2_fma(v[j], kl, h2_mul(v[j], kh));
          *reinterpret_cast<uint4*>(kd + (c >> 3) * 16384 + (((c & 7) ^ (key & 7)) << 4)) =
              make_uint4(v[0], v[1], v[2], v[3]);
        }
        if (key == 0) steps[i % KP_STEPS] = make_float2(scale_log2e * pow2i(E - 11), (float)F);
        fence_proxy_async_smem();
        mbar_arrive(&k_full[st]);
        load_k(i + 1);
        if (i >= 2 && ok) ok = mbar_wait(&v_empty[st], ((i >> 1) - 1) & 1, DEV_ERR_TIMEOUT_EMPTY);
        uint8_t* vd = sm + M::V + st * M::TILE + key * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 q = vw[c >> 2];
          const uint32_t word = (c & 3) == 0 ? q.x : (c & 3) == 1 ? q.y : (c & 3) == 2 ? q.z : q.w;
          uint32_t v[4];
          codes_to_half2(word, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = h2_mul(v[j], vh);
          *reinterpret_cast<uint4*>(vd + (c >> 3) * 16384 + (((c & 7) ^ (key & 7)) << 4)) =
              make_uint4(v[0], v[1], v[2], v[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&v_full[st]);
        load_v(i + 1);
      }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
      if (warp == 12 && tiles.count > 0) {
        // ---------------------------------------------- products
        constexpr uint32_t ID_S = idesc_f16(128, KP_KT, false, false), ID_O = idesc_f16(128, D, false, true);
        bool ok = mbar_wait_warp(&q_full, 0, DEV_ERR_TIMEOUT_A);
        int used0 = 0, used1 = 0;                    // weight tiles used, by stream
        const uint32_t smq = smem_u32(sm + M::Q), smk = smem_u32(sm + M::K), smv = smem_u32(sm + M::V);
        for (int i = 0; i <= tiles.count && ok; ++i) {
          const bool more = i < tiles.count;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const KpRows& rows = g == 0 ? rows0 : rows1;
            int& used = g == 0 ? used0 : used1;
            if (i > 0 && ok && rows.any(tiles.at(i - 1) * KP_KT, a.window, a.sinks)) {
              ok = mbar_wait_warp(&p_full[g], used & 1, DEV_ERR_TIMEOUT_ACC) &&
                   mbar_wait_warp(&v_full[(i - 1) & 1], ((i - 1) >> 1) & 1, DEV_ERR_TIMEOUT_FULL);
              if (ok) {
                tc_fence_after();
                const uint32_t vb = smv + ((i - 1) & 1) * M::TILE;
                if (elect_one()) {
#pragma unroll
                  for (int k = 0; k < KP_KT / 16; ++k)
                    mma_f16_ts(tmem + O_COL + 128u * g, tmem + S_COL + 128u * g + 8 * k,
                               smem_desc_mn_sw128(vb + 2048 * k, 16384), ID_O, used > 0 || k > 0);
                }
                __syncwarp();
                ++used;
              }
            }
            // (a stream's wait also covers a tile that only the other stream sees)
            if (more && ok) ok = mbar_wait_warp(&k_full[i & 1], (i >> 1) & 1, DEV_ERR_TIMEOUT_FULL);
            if (more && ok && rows.any(tiles.at(i) * KP_KT, a.window, a.sinks)) {
              const uint32_t qb = smq + g * M::TILE, kb = smk + (i & 1) * M::TILE;
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  mma_f16_ss(tmem + S_COL + 128u * g, smem_desc_k_sw128(qb + (k >> 2) * 16384 + (k & 3) * 32),
                             smem_desc_k_sw128(kb + (k >> 2) * 16384 + (k & 3) * 32), ID_S, k > 0);
                mma_commit(&s_full[g]);
              }
              __syncwarp();
            }
          }
          if (!ok) break;
          if (elect_one()) {
            if (i > 0) mma_commit(&v_empty[(i - 1) & 1]);
            if (more) mma_commit(&k_empty[i & 1]);
          }
          __syncwarp();
        }
        // completion of everything issued, also after a wait that gave up
        if (elect_one()) {
          mma_commit(&o_full[0]);
          mma_commit(&o_full[1]);
        }
        __syncwarp();
        mbar_wait(&o_full[1], 0, DEV_ERR_TIMEOUT_ACC, false);
      }
    }
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
template <int D>
static cudaError_t launch_prefill(const KvStep& s, const AttnArgs& a, cudaStream_t st) {
  auto kern = kv4_prefill_kernel<D>;
  constexpr size_t smem = KpSmem<D>::BYTES;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int row_tiles = (int)(((int64_t)s.L * (a.heads / a.kv_heads) + 255) / 256);
  return launch_pdl(kern, dim3((unsigned)(row_tiles * a.kv_heads * s.B)), dim3(KP_THREADS), smem, st, 1u, s, a,
                    (float)(1.4426950408889634 / sqrt((double)D)), row_tiles);
}

cudaError_t run_kv4_prefill(const KvStep& s, const AttnArgs& a, int d, cudaStream_t st) {
  return d == 128 ? launch_prefill<128>(s, a, st) : launch_prefill<64>(s, a, st);
}

// Reads and clears this unit's error flag on the current device.
cudaError_t kv4_prefill_error(int* code) {
  int zero = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(code, g_device_error, sizeof(int));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}

}  // namespace bitnet
