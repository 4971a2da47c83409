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
// What bounds it: memory; every input is read once and every output written once.
// 16 values a lane: 8 lanes (d = 128) or 4 (d = 64) hold a head, a warp 4 or 8
// heads of one token, so that norm and Hadamard cross few lanes.
#include "kv4_common.cuh"

#include <cuda_bf16.h>

namespace bitnet {

constexpr int KVA_WARPS = 8;

template <typename XT>
BN_DEV void load16(const XT* p, float (&x)[16]);
template <>
BN_DEV void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 u = ldg_v4(p + 4 * i);
    x[4 * i] = __uint_as_float(u.x); x[4 * i + 1] = __uint_as_float(u.y);
    x[4 * i + 2] = __uint_as_float(u.z); x[4 * i + 3] = __uint_as_float(u.w);
  }
}
template <>
BN_DEV void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = ldg_v4(p + 8 * i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { x[8 * i + 2 * j] = bf16lo(w[j]); x[8 * i + 2 * j + 1] = bf16hi(w[j]); }
  }
}

BN_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

BN_DEV void store16_f32(float* p, const float (&t)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(p + 4 * i) = make_float4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
}
BN_DEV void store16_bf16(__nv_bfloat16* p, const float (&t)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint4*>(p + 8 * i) =
        make_uint4(pack_bf16(t[8 * i], t[8 * i + 1]), pack_bf16(t[8 * i + 2], t[8 * i + 3]),
                   pack_bf16(t[8 * i + 4], t[8 * i + 5]), pack_bf16(t[8 * i + 6], t[8 * i + 7]));
}

// Norm, rotation and Hadamard of a head's row, in CT arithmetic: 16 values of
// the row a lane, dimensions 16 q .. 16 q + 15 for lane q of the head's LPH lanes.
template <typename CT, int D>
BN_DEV void turn_row(const float (&x)[16], float (&t)[16], int q, int norm, const float* gamma, float eps,
                     int rot_dim, const double2* cs, int hadamard) {
  constexpr int LPH = D / 16;
  CT y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = (CT)x[i];
  if (norm) {
    CT ss = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss += y[i] * y[i];
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const CT r = (CT)1 / sqrt(ss / (CT)D + (CT)eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] *= r;
    if (gamma != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + 16 * q + 4 * i));
        y[4 * i] *= (CT)g.x; y[4 * i + 1] *= (CT)g.y; y[4 * i + 2] *= (CT)g.z; y[4 * i + 3] *= (CT)g.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (16 * q + 2 * i < rot_dim) {
      const double2 w = cs[8 * q + i];
      const CT c = (CT)w.x, s = (CT)w.y, a = y[2 * i], b = y[2 * i + 1];
      y[2 * i] = a * c - b * s;
      y[2 * i + 1] = a * s + b * c;
    }
  }
  if (hadamard) {
#pragma unroll
    for (int st = 1; st < 16; st <<= 1) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if ((i & st) == 0) {
          const CT a = y[i], b = y[i + st];
          y[i] = a + b;
          y[i + st] = a - b;
        }
      }
    }
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const CT z = __shfl_xor_sync(0xffffffffu, y[i], o);
        y[i] = (q & o) ? z - y[i] : y[i] + z;
      }
    }
    const CT f = (CT)(D == 128 ? 0.08838834764831844055 : 0.125);    // 1 / sqrt(d)
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] *= f;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = (float)y[i];
}

// A lane's 16 values of a row to codes; every lane of the row gets the step.
template <int D>
BN_DEV uint2 row_to_codes(const float (&t)[16], float& step) {
  constexpr int LPH = D / 16;
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(t[i]));
#pragma unroll
  for (int o = 1; o < LPH; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float s = __fdiv_rn(7.0f, fmaxf(mx, 1e-5f));
  step = __fdiv_rn(1.0f, s);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    int c = __float2int_rn(__fmul_rn(t[i], s));
    c = c < -8 ? -8 : (c > 7 ? 7 : c);
    w[i >> 3] |= (uint32_t)(c & 15) << (4 * ((i & 7) >> 1) + 16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}

// Grid: x over groups of `tokens` rows of the step, y over the units of a token (a
// unit is one warp's heads of Q, K or V).
template <int D, typename XT, bool FOUR>
__global__ void __launch_bounds__(32 * KVA_WARPS)
append_kernel(const KvStep s, const AppendArgs a, const __grid_constant__ RopeTable rope, int tokens) {
  constexpr int LPH = D / 16, HPW = 32 / LPH;
  extern __shared__ double2 cs[];                    // [tokens][rot_dim / 2] cosine, sine
  pdl_launch_dependents();
  pdl_wait();                                        // the rows come from the previous kernel
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rows = (int64_t)s.B * s.L;
  const int64_t r0 = (int64_t)blockIdx.x * tokens;
  const int nr = rows - r0 < tokens ? (int)(rows - r0) : tokens;
  const int pairs = a.rot_dim >> 1;
  for (int e = tid; e < nr * pairs; e += 32 * KVA_WARPS) {
    const int tk = e / pairs, i = e - tk * pairs;
    const int b = (int)((r0 + tk) / s.L);
    const int64_t p = kv_first_position(s, b) + (r0 + tk - (int64_t)b * s.L);
    double sn, c;
    sincos((double)p * rope.theta[i], &sn, &c);
    cs[e] = make_double2(c, sn);
  }
  __syncthreads();
  const int q = lane % LPH, hw = lane / LPH;
  const int uk = (a.kv_heads + HPW - 1) / HPW, uq = (a.heads + HPW - 1) / HPW;
  const int units = 2 * uk + uq;
  for (int64_t e = (int64_t)blockIdx.y * KVA_WARPS + warp; e < (int64_t)nr * units; e += (int64_t)gridDim.y * KVA_WARPS) {
    const int tk = (int)(e / units);
    const int u = (int)(e - (int64_t)tk * units);
    const int64_t row = r0 + tk;
    const int b = (int)(row / s.L), l = (int)(row - (int64_t)b * s.L);
    const int64_t p = kv_first_position(s, b) + l;
    if (l >= kv_real_tokens(s, b)) continue;
    const bool in = p >= 0 && p < s.T_cap;           // a row outside the cache is not appended
    const int kind = u < uk ? 0 : (u < 2 * uk ? 1 : 2);                       // K, V, Q
    const int h = (kind == 0 ? u : kind == 1 ? u - uk : u - 2 * uk) * HPW + hw;
    const bool real = h < (kind == 2 ? a.heads : a.kv_heads);
    const XT* src = static_cast<const XT*>(kind == 0 ? a.K : kind == 1 ? a.V : a.Q) +
                    row * (kind == 0 ? a.ldk : kind == 1 ? a.ldv : a.ldq) + (int64_t)h * D + 16 * q;
    float x[16], t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    if (real) load16<XT>(src, x);
    const double2* rcs = cs + (size_t)tk * pairs;
    if (kind == 2) {
      turn_row<float, D>(x, t, q, a.norm, a.gamma_q, a.eps, a.rot_dim, rcs, a.hadamard);
      if (real) {
        const int64_t off = row * a.heads * D + (int64_t)h * D + 16 * q;
        if (a.qo_bf16) store16_bf16(static_cast<__nv_bfloat16*>(a.Qo) + off, t);
        else store16_f32(static_cast<float*>(a.Qo) + off, t);
      }
    } else {
      if (kind == 0) {
        if (FOUR) turn_row<double, D>(x, t, q, a.norm, a.gamma_k, a.eps, a.rot_dim, rcs, a.hadamard);
        else turn_row<float, D>(x, t, q, a.norm, a.gamma_k, a.eps, a.rot_dim, rcs, 0);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = x[i];
      }
      if (FOUR) {
        float step;
        const uint2 c = row_to_codes<D>(t, step);
        if (real && in) {
          const int64_t cr = ((int64_t)b * a.kv_heads + h) * s.T_cap + p;
          *reinterpret_cast<uint2*>((kind == 0 ? a.Kc4 : a.Vc4) + cr * (D / 2) + 8 * q) = c;
          if (q == 0) (kind == 0 ? a.Ks : a.Vs)[cr] = step;
        }
      } else if (real && in) {
        float* dst = (kind == 0 ? a.Kc32 : a.Vc32) + ((int64_t)b * s.T_cap + p) * a.kv_heads * D + (int64_t)h * D + 16 * q;
        store16_f32(dst, t);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// 4-bit rows back to values: a thread takes one word (8 codes) of a key row and
// the same word of the value row.
// ---------------------------------------------------------------------------
BN_DEV void word_to_values(uint32_t w, float step, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = (int)(w << (28 - 4 * j - 16 * i)) >> 28;
      v[2 * j + i] = __fmul_rn((float)c, step);
    }
  }
}

template <bool BF16>
BN_DEV void store8(void* base, int64_t off, const float (&v)[8]) {
  if (BF16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256)
read_kernel(const KvStep s, int kv_heads, const uint8_t* __restrict__ Kc, const float* __restrict__ Ks,
            const uint8_t* __restrict__ Vc, const float* __restrict__ Vs, void* K, void* V) {
  constexpr int WPR = D / 8;                         // words a row
  pdl_launch_dependents();
  pdl_wait();                                        // the cache comes from the previous kernel
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t hr = idx / WPR;                      // (row, head)
  const int w = (int)(idx - hr * WPR);
  const int64_t row = hr / kv_heads;
  const int h = (int)(hr - row * kv_heads);
  if (row >= (int64_t)s.B * s.L) return;
  const int b = (int)(row / s.L), l = (int)(row - (int64_t)b * s.L);
  if (l >= kv_real_tokens(s, b)) return;
  const int64_t p = kv_first_position(s, b) + l;
  if (p < 0 || p >= s.T_cap) return;
  const int64_t cr = ((int64_t)b * kv_heads + h) * s.T_cap + p;
  float v[8];
  const int64_t off = hr * D + 8 * w;
  if (K != nullptr) {
    word_to_values(*reinterpret_cast<const uint32_t*>(Kc + cr * (D / 2) + 4 * w), Ks[cr], v);
    store8<BF16>(K, off, v);
  }
  if (V != nullptr) {
    word_to_values(*reinterpret_cast<const uint32_t*>(Vc + cr * (D / 2) + 4 * w), Vs[cr], v);
    store8<BF16>(V, off, v);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int D, typename XT, bool FOUR>
static cudaError_t launch_append(const KvStep& s, const AppendArgs& a, const RopeTable& rope, cudaStream_t st) {
  constexpr int HPW = 32 / (D / 16);
  const int64_t rows = (int64_t)s.B * s.L;
  const int units = 2 * ((a.kv_heads + HPW - 1) / HPW) + (a.heads + HPW - 1) / HPW;
  // few tokens: one a block and its units over blocks, one unit a warp; many: 8 tokens a block
  const int tokens = rows >= 8 * 148 ? 8 : 1;
  const int gy = tokens == 1 ? (units + KVA_WARPS - 1) / KVA_WARPS : 1;
  const size_t smem = (size_t)tokens * (a.rot_dim / 2) * sizeof(double2);
  return launch_pdl(append_kernel<D, XT, FOUR>, dim3((unsigned)((rows + tokens - 1) / tokens), (unsigned)gy),
                    dim3(32 * KVA_WARPS), smem, st, 1u, s, a, rope, tokens);
}

cudaError_t run_append(const KvStep& s, const AppendArgs& a, int x_bf16, int d, double base, cudaStream_t st) {
  RopeTable rope;
  for (int i = 0; i < 64; ++i)
    rope.theta[i] = 2 * i < a.rot_dim ? exp2(-(2.0 * i / a.rot_dim) * log2(base)) : 0.0;
  const bool four = a.Kc4 != nullptr;
  using bf = __nv_bfloat16;
  if (d == 128)
    return four ? (x_bf16 ? launch_append<128, bf, true>(s, a, rope, st) : launch_append<128, float, true>(s, a, rope, st))
                : (x_bf16 ? launch_append<128, bf, false>(s, a, rope, st) : launch_append<128, float, false>(s, a, rope, st));
  return four ? (x_bf16 ? launch_append<64, bf, true>(s, a, rope, st) : launch_append<64, float, true>(s, a, rope, st))
              : (x_bf16 ? launch_append<64, bf, false>(s, a, rope, st) : launch_append<64, float, false>(s, a, rope, st));
}

cudaError_t run_kv4_read(const KvStep& s, int kv_heads, int d, const uint8_t* Kc, const float* Ks, const uint8_t* Vc,
                         const float* Vs, void* K, void* V, int bf16, cudaStream_t st) {
  const int64_t threads = (int64_t)s.B * s.L * kv_heads * (d / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(256), 0, st, 1u, s, kv_heads, Kc, Ks, Vc, Vs, K, V);
  };
  if (d == 128) return bf16 ? go(read_kernel<128, true>) : go(read_kernel<128, false>);
  return bf16 ? go(read_kernel<64, true>) : go(read_kernel<64, false>);
}

}  // namespace bitnet
