// Norm, rotation and append: the pass between the Q/K/V projections and the
// attention over a key/value cache held in fp32 or in 4 bits, and the way back
// from the 4-bit cache to values.
//
// Per head row x of d values at position p:
//   norm      y = x / sqrt(mean(x^2) + eps) * gamma       (queries and keys)
//   rotation  the pairs (y[2i], y[2i+1]), i < rot_dim / 2, turn by p theta_i,
//             theta_i = base^(-2i / rot_dim)              (queries and keys)
//   Hadamard  y H / sqrt(d), H the Sylvester matrix       (queries and keys: it
//             leaves every q . k as it is and spreads wide channels of the keys
//             over the row before it is held in 4 bits, as H-BitLinear does for
//             activations [P1 방법론])
//   4 bits    t = fp32(y), s = 7 / max(max|t|, 1e-5), code = clamp(rint(t s), -8, 7),
//             step = 1 / s: the framework's absmax rule for int4 codes
// Precision: y is computed in fp64 and rounded once to fp32 where a code follows
// (keys of the 4-bit cache), so a code never depends on the order of a sum; in
// fp32, with cosine and sine from fp64 angles, where it does not (queries, fp32
// caches).  Values are not turned.
//
// What bounds it: without the Hadamard transform memory (8000 bf16 tokens of 32 + 8 + 8
// heads with norm into fp32 caches, 61 us, 74 % of a copy's rate); with it the instruction
// issue (69 % of the cycles), half of a query's instructions being the transform's exchanges
// between lanes (32768 such tokens into the 4-bit cache, 215 us, 3.3 TB/s).  Every input is
// read once and every output written once.
// 8 values a lane (one 16-byte load of bf16 rows): 16 lanes (d = 128) or 8 (d = 64)
// hold a head, a warp 2 or 4 heads of one token.  The cosines lie in shared memory in
// the order the lanes read them.
#include "kv4_common.cuh"

#include <cuda_bf16.h>

#include <type_traits>

namespace bitnet {

constexpr int KVA_WARPS = 8;

// A lane's 8 values of a row, as loaded: fp32 rows take two registers of 16 bytes.
template <typename XT>
struct Raw8 { uint4 v[sizeof(XT) / 2]; };
template <typename XT>
BN_DEV void load8(const XT* p, Raw8<XT>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(XT) / 2; ++i) r.v[i] = ldg_v4(p + i * (16 / (int)sizeof(XT)));
}
BN_DEV void values8(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x); x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z); x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
BN_DEV void values8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int j = 0; j < 4; ++j) { x[2 * j] = bf16lo(w[j]); x[2 * j + 1] = bf16hi(w[j]); }
}

BN_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
BN_DEV void store8_f32(float* p, const float (&t)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(t[0], t[1], t[2], t[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(t[4], t[5], t[6], t[7]);
}
BN_DEV void store8_bf16(__nv_bfloat16* p, const float (&t)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(t[0], t[1]), pack_bf16(t[2], t[3]), pack_bf16(t[4], t[5]), pack_bf16(t[6], t[7]));
}

// Cosine and sine of pair 4 q + i of a head lie at i * (D / 8) + q.
BN_DEV void turn_pair(const double2 w, double& a, double& b) {
  const double x = a, y = b;
  a = x * w.x - y * w.y;
  b = x * w.y + y * w.x;
}
BN_DEV void turn_pair(const float2 w, float& a, float& b) {
  const float x = a, y = b;
  a = x * w.x - y * w.y;
  b = x * w.y + y * w.x;
}

// Hadamard transform of a head's row, 8 values a lane: strides 1, 2, 4 in the lane, the
// others across lanes (y = +-y + the partner's).
template <int D>
BN_DEV void hadamard_row(double (&y)[8], int q) {
#pragma unroll
  for (int st = 1; st < 8; st <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((i & st) == 0) {
        const double a = y[i], b = y[i + st];
        y[i] = a + b;
        y[i + st] = a - b;
      }
    }
  }
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) {
    const double sign = (q & o) ? -1.0 : 1.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * sign + __shfl_xor_sync(0xffffffffu, y[i], o);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] *= D == 128 ? 0.08838834764831844055 : 0.125;      // 1 / sqrt(d)
}
// In fp32 on pairs: half the instructions.
template <int D>
BN_DEV void hadamard_row(float (&y)[8], int q) {
  uint64_t v[4];
  const uint64_t neg = pack_f2(-1.f, -1.f), alt = pack_f2(1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 4; ++i)                        // stride 1: (a + b, a - b)
    v[i] = fma_f2(pack_f2(y[2 * i + 1], y[2 * i + 1]), alt, pack_f2(y[2 * i], y[2 * i]));
#pragma unroll
  for (int st = 1; st < 4; st <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((i & st) == 0) {
        const uint64_t a = v[i], b = v[i + st];
        v[i] = add_f2(a, b);
        v[i + st] = fma_f2(b, neg, a);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) {
    const float sign = (q & o) ? -1.f : 1.f;
    const uint64_t sign2 = pack_f2(sign, sign);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpack_f2(v[i], a, b);
      v[i] = fma_f2(v[i], sign2, pack_f2(__shfl_xor_sync(0xffffffffu, a, o), __shfl_xor_sync(0xffffffffu, b, o)));
    }
  }
  const float f = D == 128 ? 0.08838834764831844055f : 0.125f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack_f2(v[i], a, b);
    y[2 * i] = a * f;
    y[2 * i + 1] = b * f;
  }
}

// Norm, rotation and Hadamard of a head's row, in CT arithmetic: 8 values of the row a
// lane, dimensions 8 q .. 8 q + 7 for lane q of the head's LPH lanes.
template <typename CT, typename CS, int D>
BN_DEV void turn_row(const float (&x)[8], float (&t)[8], int q, int norm, const float* gamma, float eps, int rot_dim,
                     const CS* cs, int hadamard) {
  constexpr int LPH = D / 8;
  CT y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = (CT)x[i];
  if (norm) {
    CT ss = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const CT r = (CT)1 / sqrt(ss / (CT)D + (CT)eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= r;
    if (gamma != nullptr) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + 8 * q + 4 * i));
        y[4 * i] *= (CT)g.x; y[4 * i + 1] *= (CT)g.y; y[4 * i + 2] *= (CT)g.z; y[4 * i + 3] *= (CT)g.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (8 * q + 2 * i < rot_dim) turn_pair(cs[i * LPH + q], y[2 * i], y[2 * i + 1]);
  if (hadamard) hadamard_row<D>(y, q);
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = (float)y[i];
}

// A lane's 8 values of a row to a word of codes; every lane of the row gets the step.
// rint(t s) + 8 stands in the low bits of t s + (1.5 * 2^23 + 8), rounded to nearest even;
// the shifted sum of eight such words, less that of their constant parts (modulo 2^32),
// is the word of biased codes.  |t s| <= 7 up to its rounding, so that no code needs the
// clamp to -8 .. 7.  A row with a value that is not finite gets the step NaN, whatever its
// codes: it stands for NaN, as the rule's inf * 0 and NaN do.
template <int D>
BN_DEV uint32_t row_to_codes(const float (&t)[8], float& step) {
  constexpr int LPH = D / 8;
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) mx = max3_nan(mx, fabsf(t[i]), fabsf(t[i + 1]));
#pragma unroll
  for (int o = 1; o < LPH; o <<= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float s = __fdiv_rn(7.0f, fmaxf(mx, 1e-5f));
  step = mx < INFINITY ? __fdiv_rn(1.0f, s) : NAN;
  uint32_t w = 0u, constant = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = 4 * (i >> 1) + 16 * (i & 1);
    w += __float_as_uint(__fadd_rn(__fmul_rn(t[i], s), 12582920.f)) << at;
    constant += 0x4B400000u << at;
  }
  return (w - constant) ^ 0x88888888u;
}

// Grid: x over groups of `tokens` rows of the step.  A unit is one warp's heads of K, V
// or Q of one token.  tokens == KVA_WARPS: a warp takes every unit of its token;
// tokens == 1: the token's units over the warps of the y blocks, one each.
template <int D, typename XT, bool FOUR>
__global__ void __launch_bounds__(32 * KVA_WARPS, 4)
append_kernel(const KvStep s, const AppendArgs a, const __grid_constant__ RopeTable rope, int tokens) {
  constexpr int LPH = D / 8, HPW = 32 / LPH, PAIRS = D / 2;
  extern __shared__ double2 cs64[];                  // [tokens][PAIRS] cosine, sine; then the same in fp32
  float2* cs32 = reinterpret_cast<float2*>(cs64 + tokens * PAIRS);
  pdl_launch_dependents();
  pdl_wait();                                        // the rows come from the previous kernel
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rows = (uint32_t)s.B * (uint32_t)s.L;
  const uint32_t r0 = blockIdx.x * (uint32_t)tokens;
  const int nr = rows - r0 < (uint32_t)tokens ? (int)(rows - r0) : tokens;
  const int pairs = a.rot_dim >> 1;
  for (int e = tid; e < nr * pairs; e += 32 * KVA_WARPS) {
    const int tk = e / pairs, i = e - tk * pairs;
    const uint32_t b = (r0 + tk) / (uint32_t)s.L;
    const int64_t p = kv_first_position(s, (int)b) + (r0 + tk - b * (uint32_t)s.L);
    double sn, c;
    sincos((double)p * rope.theta[i], &sn, &c);
    const int at = tk * PAIRS + (i & 3) * LPH + (i >> 2);
    cs64[at] = make_double2(c, sn);
    cs32[at] = make_float2((float)c, (float)sn);
  }
  __syncthreads();
  const int tk = tokens == 1 ? 0 : warp;
  const uint32_t row = r0 + tk;
  if (row >= rows) return;
  const int b = (int)(row / (uint32_t)s.L), l = (int)(row - (uint32_t)b * (uint32_t)s.L);
  if (l >= kv_real_tokens(s, b)) return;
  const int64_t p = kv_first_position(s, b) + l;
  const bool in = p >= 0 && p < s.T_cap;             // a row outside the cache is not appended
  const int q = lane % LPH, hw = lane / LPH;
  const int uk = (a.kv_heads + HPW - 1) / HPW, uq = (a.heads + HPW - 1) / HPW;
  const double2* c64 = cs64 + tk * PAIRS;
  const float2* c32 = cs32 + tk * PAIRS;

  // `count` units of one kind (0 keys, 1 values, 2 queries) from head h0 on, the next unit's rows
  // loaded while one is worked on
  auto units = [&](auto kind_c, const void* base, int64_t ld, int n_heads, int h0, int count) {
    constexpr int KIND = decltype(kind_c)::value;
    int h = h0 + hw;
    const XT* src = static_cast<const XT*>(base) + (int64_t)row * ld + h * D + 8 * q;
    auto load = [&](bool real, Raw8<XT>& r) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(XT) / 2; ++i) r.v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (real) load8<XT>(src, r);
      src += HPW * D;
    };
    Raw8<XT> next;
    load(h < n_heads, next);
    // where a row goes: Qo, or the caches at the token's position
    int64_t at = KIND == 2 ? ((int64_t)row * a.heads + h) * D + 8 * q
                 : FOUR    ? ((int64_t)b * a.kv_heads + h) * s.T_cap + p
                           : (((int64_t)b * s.T_cap + p) * a.kv_heads + h) * D + 8 * q;
    const int64_t step_at = KIND != 2 && FOUR ? (int64_t)HPW * s.T_cap : HPW * D;
    for (int v = 0; v < count; ++v, h += HPW, at += step_at) {
      float x[8], t[8];
      values8(next, x);
      if (v + 1 < count) load(h + HPW < n_heads, next);
      const bool real = h < n_heads;
      if constexpr (KIND == 2) {
        turn_row<float, float2, D>(x, t, q, a.norm, a.gamma_q, a.eps, a.rot_dim, c32, a.hadamard);
        if (real) {
          if (a.qo_bf16) store8_bf16(static_cast<__nv_bfloat16*>(a.Qo) + at, t);
          else store8_f32(static_cast<float*>(a.Qo) + at, t);
        }
      } else {
        if constexpr (KIND == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = x[i];
        } else if constexpr (FOUR) {
          turn_row<double, double2, D>(x, t, q, a.norm, a.gamma_k, a.eps, a.rot_dim, c64, a.hadamard);
        } else {
          turn_row<float, float2, D>(x, t, q, a.norm, a.gamma_k, a.eps, a.rot_dim, c32, 0);
        }
        if constexpr (FOUR) {
          float step;
          const uint32_t w = row_to_codes<D>(t, step);
          if (real && in) {
            *reinterpret_cast<uint32_t*>((KIND == 0 ? a.Kc4 : a.Vc4) + at * (D / 2) + 4 * q) = w;
            if (q == 0) (KIND == 0 ? a.Ks : a.Vs)[at] = step;
          }
        } else if (real && in) {
          store8_f32((KIND == 0 ? a.Kc32 : a.Vc32) + at, t);
        }
      }
    }
  };
  using Keys = std::integral_constant<int, 0>;
  using Values = std::integral_constant<int, 1>;
  using Queries = std::integral_constant<int, 2>;
  int first = 0, count = 0x7fffffff;                 // this warp's units among K, V, Q in turn
  if (tokens == 1) {
    first = (int)blockIdx.y * KVA_WARPS + warp;
    count = 1;
  }
  auto part = [&](int lo, int n, int& f, int& k) {   // of units lo .. lo + n - 1
    f = first > lo ? first - lo : 0;
    const int64_t end = (int64_t)first + count - lo;
    k = (int)(end < n ? end : n) - f;
    return k > 0;
  };
  int f, k;
  if (part(0, uk, f, k)) units(Keys(), a.K, a.ldk, a.kv_heads, f * HPW, k);
  if (part(uk, uk, f, k)) units(Values(), a.V, a.ldv, a.kv_heads, f * HPW, k);
  if (part(2 * uk, uq, f, k)) units(Queries(), a.Q, a.ldq, a.heads, f * HPW, k);
}

// ---------------------------------------------------------------------------
// 4-bit rows back to values: a thread writes 16 bytes of a key row and of the value
// row (half a word's codes as fp32, a word's as bf16), so that a warp's stores are one
// run of memory.  Bound by the instructions that take the codes apart (they issue in two
// thirds of the cycles): 32768 tokens of 8 heads to fp32 in 70 us, 4.3 TB/s.
// ---------------------------------------------------------------------------
BN_DEV float code_value(uint32_t w, int i, float step) {   // code i of a word
  const int c = (int)(w << (28 - 4 * (i >> 1) - 16 * (i & 1))) >> 28;
  return __fmul_rn((float)c, step);
}
template <bool BF16>
BN_DEV void write_values(void* base, int64_t off, uint32_t w, int first, float step) {
  if (BF16) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_bf16(code_value(w, 2 * j, step), code_value(w, 2 * j + 1, step));
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    w >>= 2 * first;                                 // codes 4 .. 7 lie 8 bits above 0 .. 3
    *reinterpret_cast<float4*>(static_cast<float*>(base) + off) =
        make_float4(code_value(w, 0, step), code_value(w, 1, step), code_value(w, 2, step), code_value(w, 3, step));
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256)
read_kernel(const KvStep s, int kv_heads, const uint8_t* __restrict__ Kc, const float* __restrict__ Ks,
            const uint8_t* __restrict__ Vc, const float* __restrict__ Vs, void* K, void* V) {
  constexpr int N = BF16 ? 8 : 4, PARTS = D / N;     // values a thread, threads a head
  pdl_launch_dependents();
  pdl_wait();                                        // the cache comes from the previous kernel
  const uint32_t per_row = (uint32_t)kv_heads * PARTS;
  const uint64_t idx = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (uint64_t)s.B * s.L * per_row) return;
  const uint32_t row = (uint32_t)(idx / per_row), e = (uint32_t)(idx - (uint64_t)row * per_row);
  const int h = (int)(e / PARTS), part = (int)(e % PARTS);
  const int b = (int)(row / (uint32_t)s.L), l = (int)(row - (uint32_t)b * (uint32_t)s.L);
  if (l >= kv_real_tokens(s, b)) return;
  const int64_t p = kv_first_position(s, b) + l;
  if (p < 0 || p >= s.T_cap) return;
  const int64_t cr = ((int64_t)b * kv_heads + h) * s.T_cap + p;
  const int64_t word = cr * (D / 8) + N * part / 8, off = (int64_t)idx * N;
  const uint32_t kw = K != nullptr ? reinterpret_cast<const uint32_t*>(Kc)[word] : 0u;
  const uint32_t vw = V != nullptr ? reinterpret_cast<const uint32_t*>(Vc)[word] : 0u;
  if (K != nullptr) write_values<BF16>(K, off, kw, N * part % 8, Ks[cr]);
  if (V != nullptr) write_values<BF16>(V, off, vw, N * part % 8, Vs[cr]);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int D, typename XT, bool FOUR>
static cudaError_t launch_append(const KvStep& s, const AppendArgs& a, const RopeTable& rope, cudaStream_t st) {
  constexpr int HPW = 32 / (D / 8);
  const int64_t rows = (int64_t)s.B * s.L;
  const int units = 2 * ((a.kv_heads + HPW - 1) / HPW) + (a.heads + HPW - 1) / HPW;
  // few tokens: one a block and its units over blocks, one unit a warp; many: a token a warp
  const int tokens = rows >= 8 * 148 ? KVA_WARPS : 1;
  const int gy = tokens == 1 ? (units + KVA_WARPS - 1) / KVA_WARPS : 1;
  const size_t smem = (size_t)tokens * (D / 2) * (sizeof(double2) + sizeof(float2));
  return launch_pdl(append_kernel<D, XT, FOUR>, dim3((unsigned)((rows + tokens - 1) / tokens), (unsigned)gy),
                    dim3(32 * KVA_WARPS), smem, st, 1u, s, a, rope, tokens);
}

cudaError_t run_append(const KvStep& s, const AppendArgs& a, int x_bf16, int d, double base, cudaStream_t st) {
  RopeTable rope;
  for (int i = 0; i < 64; ++i)
    rope.theta[i] = 2 * i < a.rot_dim ? exp2(-(2.0 * i / a.rot_dim) * log2(base)) : 0.0;
  const bool four = a.Kc4 != nullptr;
  using bf = __nv_bfloat16;
  if (d == 128) {
    if (four && x_bf16) return launch_append<128, bf, true>(s, a, rope, st);
    if (four) return launch_append<128, float, true>(s, a, rope, st);
    return x_bf16 ? launch_append<128, bf, false>(s, a, rope, st) : launch_append<128, float, false>(s, a, rope, st);
  }
  if (four && x_bf16) return launch_append<64, bf, true>(s, a, rope, st);
  if (four) return launch_append<64, float, true>(s, a, rope, st);
  return x_bf16 ? launch_append<64, bf, false>(s, a, rope, st) : launch_append<64, float, false>(s, a, rope, st);
}

cudaError_t run_kv4_read(const KvStep& s, int kv_heads, int d, const uint8_t* Kc, const float* Ks, const uint8_t* Vc,
                         const float* Vs, void* K, void* V, int bf16, cudaStream_t st) {
  const int64_t threads = (int64_t)s.B * s.L * kv_heads * (d / (bf16 ? 8 : 4));
  const dim3 grid((unsigned)((threads + 255) / 256));
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(256), 0, st, 1u, s, kv_heads, Kc, Ks, Vc, Vs, K, V);
  };
  if (d == 128) return bf16 ? go(read_kernel<128, true>) : go(read_kernel<128, false>);
  return bf16 ? go(read_kernel<64, true>) : go(read_kernel<64, false>);
}

}  // namespace bitnet
