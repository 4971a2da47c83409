// Causal softmax attention over the 4-bit key/value cache, optionally through a
// sliding window with a few first keys that stay visible.
//
//   score  s_j = (q . code_kj) step_kj / sqrt(d)
//   output sum_j e^(s_j) step_vj code_vj / sum_j e^(s_j)
//   over the keys j <= p with window == 0 or j > p - window or j < sinks.
//
// Codes are small integers, exact in fp16, so both products run on the tensor
// cores with fp16 operands and fp32 sums:
//   - q is scaled by a power of two for each row (its largest value then lies in
//     [2^14, 2^15)); bf16 queries are then exact in fp16, fp32 queries are split into
//     two fp16 terms (22 bits);
//   - the value step is folded into the weight: with step_v = f 2^e the weight's
//     exponent takes e, p'_j = 2^(s_j log2(e) + e_j - m), the operand is p'_j f_j in
//     fp16 (two terms for fp32 outputs) and the sum takes p'_j 2^(-e_j).  The running
//     maximum m is that of s_j log2(e) + e_j, so the operand's largest value is near
//     2^10 whatever the steps' range, and what fp16 cannot hold is 2^-34 of it.
// The softmax runs in one pass over the keys (running maximum and sum, fp32).
#include "kv4_common.cuh"

#include <cuda_bf16.h>

namespace bitnet {

// ---------------------------------------------------------------------------
// few queries a key head: warp-level products (m16n8k16), keys as the 16 rows and
// queries as the 8 columns, so that up to 8 queries (the heads that share a key
// head, times a few tokens) cost one product.  A warp takes every (warps)-th tile
// of 32 keys through its own ring of asynchronous copies; scores, weights and the
// output stay in its registers.  Taking the codes apart costs more than reading them
// (16 bf16 sequences of 2048 to 32768 keys, 32 over 8 heads: 113 us, of which the memory
// needs 46), by too few warps to fill the issue slots (59 %); a single short sequence is
// latency (513 keys, 16 heads: 7 us in a graph).  The warps' partial softmaxes are merged
// in shared memory; where several blocks share a row tile's keys, over distributed shared
// memory of a cluster, or (many blocks a row tile) through the workspace by a second kernel.
// ---------------------------------------------------------------------------
constexpr int KD_WARPS = 4;
constexpr int KD_STAGES = 3;
constexpr int KD_KT = 32;                            // keys a tile

template <int D>
struct KdTile {                                      // one stage of a warp's ring, in bytes
  static constexpr int CODES = KD_KT * D / 2;
  static constexpr int BYTES = 2 * CODES + 2 * KD_KT * 4;
};

BN_DEV void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
BN_DEV uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
BN_DEV float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// A tile's codes and steps into one stage: a tile is one run of memory, lane i copies
// every 32nd 16 bytes.  Keys past the cache's end are zero.  Value rows 2t of each 8 lie
// first, then rows 2t + 1: the product's lanes read rows 2t (t = 0..3) at once, then
// without bank conflicts.
template <int D>
BN_DEV void kd_stage(const uint8_t* kc, const float* ks, const uint8_t* vc, const float* vs, int j0, int T_cap,
                     uint32_t dst, int lane) {
  constexpr int CPR = D / 32;                        // 16-byte chunks a row
  const int64_t off = (int64_t)j0 * (D / 2) + 16 * lane;
  const int c = lane & 7;                            // 4 steps a chunk (T_cap is a multiple of 16)
  const float* steps = (lane < 8 ? ks : vs) + j0 + 4 * c;
  const uint32_t steps_dst = dst + 2 * KdTile<D>::CODES + (lane < 8 ? 0 : KD_KT * 4) + 16 * c;
#pragma unroll
  for (int i = 0; i < CPR; ++i) {
    const int r = (lane + 32 * i) / CPR, cc = (lane + 32 * i) % CPR;
    const int vr = (r & ~7) | ((r & 7) >> 1) | ((r & 1) << 2);
    const uint32_t kd = dst + 16 * (lane + 32 * i), vd = dst + KdTile<D>::CODES + vr * (D / 2) + 16 * cc;
    if (j0 + KD_KT <= T_cap) {
      cp_async_16(kd, kc + off + 512 * i, 16u);
      cp_async_16(vd, vc + off + 512 * i, 16u);
    } else {
      const bool in = j0 + r < T_cap;
      cp_async_16(kd, in ? kc + off + 512 * i : kc, in ? 16u : 0u);
      cp_async_16(vd, in ? vc + off + 512 * i : vc, in ? 16u : 0u);
    }
  }
  if (lane < 16) {
    const bool in = j0 + 4 * c < T_cap;
    cp_async_16(steps_dst, in ? steps : ks, in ? 16u : 0u);
  }
}

// Four blocks to an SM where a warp holds 8 query rows (32 fp32 sequences of 513 keys, 16 heads: 26.6 us, in
// as many registers as the compiler takes, two blocks, 30.7); 16 rows do not fit so few registers.
template <int D, int NT, typename XT>
__global__ void __launch_bounds__(32 * KD_WARPS, NT == 1 ? 4 : 1)
kv4_decode_kernel(const KvStep s, const AttnArgs a, float scale_log2e, int splits, float* parts) {
  constexpr bool SPLIT = sizeof(XT) == 4;            // fp32: two fp16 terms for q and for the weights
  constexpr int ROWS = 8 * NT;
  constexpr int KW = D / 32, VW = D / 64;            // words of a key row, of a value row, a lane holds
  constexpr int MT = D / 16;                         // 16-dimension tiles of the output
  constexpr float BIAS = 10.f;
  extern __shared__ __align__(16) uint8_t kd_smem[];
  __shared__ float w_m[KD_WARPS][ROWS], w_l[KD_WARPS][ROWS];
  __shared__ float c_m[ROWS], c_l[ROWS];
  float* c_o = reinterpret_cast<float*>(kd_smem + KD_WARPS * KD_STAGES * KdTile<D>::BYTES);   // [ROWS][D]
  pdl_launch_dependents();
  pdl_wait();                                        // q and the cache come from the previous kernel
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  // block crank of the csize that share a row tile: of a cluster, or with parts of the grid
  const uint32_t csize = (uint32_t)splits, crank = blockIdx.x % csize;
  const int group = a.heads / a.kv_heads;
  const int b = blockIdx.z, h = blockIdx.y;
  const int r0 = (int)(blockIdx.x / csize) * ROWS;   // first row (token * group + head of the group)
  const int n_rows = kv_real_tokens(s, b) * group;
  if (r0 >= n_rows) return;                          // the same for the whole cluster
  const int nr = n_rows - r0 < ROWS ? n_rows - r0 : ROWS;
  const int64_t p0 = kv_first_position(s, b);
  const int64_t pf = p0 + r0 / group, pl = p0 + (r0 + nr - 1) / group;
  const int p_lo = pf < 0 ? 0 : (pf < s.limit ? (int)pf : s.limit);
  const int p_hi = pl < 0 ? -1 : (pl < s.limit ? (int)pl : s.limit - 1);
  KeyTiles tiles = key_tiles<KD_KT>(p_lo, p_hi, a.window, a.sinks);
  if (p_lo > p_hi) tiles.count = 0;                  // every query lies outside the cache

  // ---- queries: row g of each 8 (scaled by a power of two), dimensions (D / 4) t .. ----
  uint32_t qh[NT][2 * KW * 2], ql[SPLIT ? NT : 1][SPLIT ? 4 * KW : 1];
  float unscale[NT][2];                              // of rows 2t, 2t + 1
  int pos[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int rr = 8 * n + g;
    const bool real = rr < nr;
    const int R = r0 + rr;
    const int l = R / group, hd = h * group + R - l * group;
    const XT* src = static_cast<const XT*>(a.Q) + (((int64_t)b * s.L + l) * a.heads + hd) * D + (D / 4) * t;
    float x[8 * KW];
#pragma unroll
    for (int i = 0; i < 8 * KW; ++i) x[i] = 0.f;
    if (real) {
      if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < 2 * KW; ++i) {
          const uint4 u = ldg_v4(src + 4 * i);
          x[4 * i] = __uint_as_float(u.x); x[4 * i + 1] = __uint_as_float(u.y);
          x[4 * i + 2] = __uint_as_float(u.z); x[4 * i + 3] = __uint_as_float(u.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const uint4 u = ldg_v4(src + 8 * i);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) { x[8 * i + 2 * j] = bf16lo(w[j]); x[8 * i + 2 * j + 1] = bf16hi(w[j]); }
        }
      }
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * KW; ++i) {
      const float v = fabsf(x[i]);
      mx = fmaxf(mx, v < INFINITY ? v : 0.f);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = row_exponent(mx);
    const float up = pow2i(14 - e);
#pragma unroll
    for (int i = 0; i < 4 * KW; ++i) {
      const float lo = x[2 * i] * up, hi = x[2 * i + 1] * up;
      qh[n][i] = pack_half2(lo, hi);
      if constexpr (SPLIT) ql[n][i] = half2_rest(qh[n][i], lo, hi);
    }
    const float down = pow2i(e - 14) * scale_log2e;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unscale[n][i] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + i));
      const int rc = 8 * n + 2 * t + i < nr ? 8 * n + 2 * t + i : nr - 1;
      const int64_t p = p0 + (r0 + rc) / group;
      pos[n][i] = p >= 0 && p < s.limit ? (int)p : -1;
    }
  }
  const bool rows_in = pf >= 0 && pl < s.limit;

  const int64_t head = (int64_t)b * a.kv_heads + h;
  const uint8_t* kc = a.Kc + head * s.T_cap * (D / 2);
  const uint8_t* vc = a.Vc + head * s.T_cap * (D / 2);
  const float* ks = a.Ks + head * s.T_cap;
  const float* vs = a.Vs + head * s.T_cap;
  uint8_t* ring = kd_smem + warp * KD_STAGES * KdTile<D>::BYTES;
  const uint32_t ring_a = smem_u32(ring);

  float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[n][i][c] = 0.f;
  }
  const int first = (int)crank * KD_WARPS + warp, stride = (int)csize * KD_WARPS;
  const int mine = tiles.count > first ? (tiles.count - first + stride - 1) / stride : 0;
#pragma unroll
  for (int i = 0; i < KD_STAGES - 1; ++i) {
    if (i < mine)
      kd_stage<D>(kc, ks, vc, vs, tiles.at(first + i * stride) * KD_KT, s.T_cap, ring_a + i * KdTile<D>::BYTES, lane);
    cp_async_commit();
  }
  int slot = 0, nslot = KD_STAGES - 1;               // stages of this tile and of the one that is fetched
#pragma unroll 1
  for (int it = 0, at = first; it < mine; ++it, at += stride) {
    asm volatile("cp.async.wait_group %0;" :: "n"(KD_STAGES - 2) : "memory");
    __syncwarp();                                    // this tile is in place, and every lane is done with the last one
    if (it + KD_STAGES - 1 < mine)
      kd_stage<D>(kc, ks, vc, vs, tiles.at(at + (KD_STAGES - 1) * stride) * KD_KT, s.T_cap,
                  ring_a + nslot * KdTile<D>::BYTES, lane);
    cp_async_commit();
    const uint8_t* stage = ring + slot * KdTile<D>::BYTES;
    slot = slot + 1 == KD_STAGES ? 0 : slot + 1;
    nslot = nslot + 1 == KD_STAGES ? 0 : nslot + 1;
    const float* kst = reinterpret_cast<const float*>(stage + 2 * KdTile<D>::CODES);
    const float* vst = kst + KD_KT;
    const int j0 = tiles.at(at) * KD_KT;
    // ---- scores of keys 16 x + g, + 8 (rows) and queries 2t, 2t + 1 (columns) ----
    // (fp32: the products of the second terms are summed apart, so that the first ones' sum is cut
    // off half as often)
    float sc[2][NT][4], sl[SPLIT ? 2 : 1][SPLIT ? NT : 1][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sc[x][n][c] = 0.f;
          if constexpr (SPLIT) sl[x][n][c] = 0.f;
        }
      const uint8_t* kr = stage + (16 * x + g) * (D / 2) + 4 * KW * t;
      uint32_t w0[KW], w1[KW];
      if constexpr (KW == 4) {
        const uint4 u0 = *reinterpret_cast<const uint4*>(kr), u1 = *reinterpret_cast<const uint4*>(kr + 8 * (D / 2));
        w0[0] = u0.x; w0[1] = u0.y; w0[2] = u0.z; w0[3] = u0.w;
        w1[0] = u1.x; w1[1] = u1.y; w1[2] = u1.z; w1[3] = u1.w;
      } else {
        const uint2 u0 = *reinterpret_cast<const uint2*>(kr), u1 = *reinterpret_cast<const uint2*>(kr + 8 * (D / 2));
        w0[0] = u0.x; w0[1] = u0.y;
        w1[0] = u1.x; w1[1] = u1.y;
      }
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint32_t k0[4], k1[4];
        codes_to_half2(w0[i], k0);
        codes_to_half2(w1[i], k1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            mma_f16(sc[x][n], k0[2 * u], k1[2 * u], k0[2 * u + 1], k1[2 * u + 1], qh[n][4 * i + 2 * u],
                    qh[n][4 * i + 2 * u + 1]);
            if constexpr (SPLIT)
              mma_f16(sl[x][n], k0[2 * u], k1[2 * u], k0[2 * u + 1], k1[2 * u + 1], ql[n][4 * i + 2 * u],
                      ql[n][4 * i + 2 * u + 1]);
          }
        }
      }
    }
    // ---- steps: scores in base-2 exponents, plus the value step's exponent ----
    float f[2][2], inv[2][2];
    const bool full = rows_in && j0 + KD_KT - 1 <= p_lo &&
                      (a.window == 0 || j0 > p_hi - a.window || j0 + KD_KT <= a.sinks);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int key = 16 * x + 8 * y + g;
        // a step that is not finite is NaN to the queries that see the key, through the score (inf 0 = NaN),
        // and finite in the operand, where a hidden key's weight is zero
        const float vstep = vst[key], both = fmaf(vstep, 0.f, kst[key]), kstep = fmaf(both, 0.f, both);
        // the exponent field, clamped as in step_exponent; as a float through the low bits of 2^23
        int e = (int)(__float_as_uint(vstep) >> 23);
        e = e < 103 ? 103 : (e > 253 ? 253 : e);
        const float ef = __uint_as_float(0x4B000000u + (uint32_t)e) - 8388735.f;
        inv[x][y] = __uint_as_float((uint32_t)(254 - e) << 23);
        f[x][y] = fminf(fabsf(vstep) * inv[x][y], 2.f);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float acc = sc[x][n][2 * y + i];
            if constexpr (SPLIT) acc += sl[x][n][2 * y + i];
            sc[x][n][2 * y + i] = acc * (kstep * unscale[n][i]) + ef;
          }
        if (!full) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& v = sc[x][n][2 * y + i];
              v = key_visible(j0 + key, pos[n][i], a.window, a.sinks) ? v : -INFINITY;
            }
        }
      }
    // ---- running maximum (a query's keys lie in the 8 lanes of one t), weights, sums ----
    bool moved = false;
    float last[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmaxf(sc[0][n][i], sc[0][n][2 + i]), fmaxf(sc[1][n][i], sc[1][n][2 + i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        last[n][i] = m[n][i];
        m[n][i] = fmaxf(mx, m[n][i]);
        moved |= m[n][i] != last[n][i];
      }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float corr = m[n][i] == last[n][i] ? 1.f : ex2(last[n][i] - m[n][i]);
          l[n][i] *= corr;
#pragma unroll
          for (int q = 0; q < MT; ++q) { o[n][q][i] *= corr; o[n][q][2 + i] *= corr; }
        }
    }
    uint32_t ph[2][NT][2], pr[SPLIT ? 2 : 1][SPLIT ? NT : 1][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float ref0 = m[n][0] == -INFINITY ? 0.f : m[n][0] - BIAS;
      const float ref1 = m[n][1] == -INFINITY ? 0.f : m[n][1] - BIAS;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float e0 = ex2(sc[x][n][2 * y] - ref0), e1 = ex2(sc[x][n][2 * y + 1] - ref1);
          l[n][0] += e0 * inv[x][y];
          l[n][1] += e1 * inv[x][y];
          const float w0 = e0 * f[x][y], w1 = e1 * f[x][y];
          const uint32_t hi = pack_half2(w0, w1);
          ph[x][n][y] = transpose8x8(hi);
          if constexpr (SPLIT) pr[x][n][y] = transpose8x8(half2_rest(hi, w0, w1));
        }
    }
    // ---- output: dimensions as the 16 rows, queries as the columns ----
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t w[4][VW];                             // keys 2t, 2t + 1, 2t + 8, 2t + 9 of the 16
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* vr = stage + KdTile<D>::CODES + (16 * x + 8 * (k >> 1) + 4 * (k & 1) + t) * (D / 2) + 4 * VW * g;
        if constexpr (VW == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(vr);
          w[k][0] = u.x; w[k][1] = u.y;
        } else {
          w[k][0] = *reinterpret_cast<const uint32_t*>(vr);
        }
      }
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        uint32_t a0[4], a1[4], a2[4], a3[4];         // even and odd dimensions of the key pairs
        codes_to_half2(__byte_perm(w[0][i], w[1][i], 0x5410), a0);
        codes_to_half2(__byte_perm(w[0][i], w[1][i], 0x7632), a1);
        codes_to_half2(__byte_perm(w[2][i], w[3][i], 0x5410), a2);
        codes_to_half2(__byte_perm(w[2][i], w[3][i], 0x7632), a3);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (SPLIT) {
              // the tensor cores cut their sums off: 16 keys' products are summed there, the output with
              // rounding here
              float part[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(part, a0[j], a1[j], a2[j], a3[j], pr[x][n][0], pr[x][n][1]);
              mma_f16(part, a0[j], a1[j], a2[j], a3[j], ph[x][n][0], ph[x][n][1]);
#pragma unroll
              for (int c = 0; c < 4; ++c) o[n][4 * i + j][c] += part[c];
            } else {
              mma_f16(o[n][4 * i + j], a0[j], a1[j], a2[j], a3[j], ph[x][n][0], ph[x][n][1]);
            }
          }
      }
    }
  }
  cp_async_wait_all();
  // ---- the warps' states into shared memory, merged over the warps ----
  __syncthreads();                                   // every ring is free
  float* w_o = reinterpret_cast<float*>(kd_smem);    // [KD_WARPS][ROWS][D]
  static_assert(ROWS * D * 4 <= KD_STAGES * KdTile<D>::BYTES, "the partial outputs fit the rings");
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[n][i];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int row = 8 * n + 2 * t + i;
      if (g == 0) { w_m[warp][row] = m[n][i]; w_l[warp][row] = sum; }
      float* dst = w_o + ((size_t)warp * ROWS + row) * D + (D / 8) * g;     // dimensions (D / 8) g + 2 q, + 1
#pragma unroll
      for (int q = 0; q < MT; ++q) *reinterpret_cast<float2*>(dst + 2 * q) = make_float2(o[n][q][i], o[n][q][2 + i]);
    }
  __syncthreads();
  if (tid < ROWS) {
    float mx = w_m[0][tid];
#pragma unroll
    for (int w = 1; w < KD_WARPS; ++w) mx = fmaxf(mx, w_m[w][tid]);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < KD_WARPS; ++w) {
      const float c = w_m[w][tid] == -INFINITY && w_l[w][tid] == 0.f ? 0.f : ex2(w_m[w][tid] - mx);
      sum += w_l[w][tid] * c;
      w_m[w][tid] = c;                               // the warp's factor
    }
    c_m[tid] = mx;
    c_l[tid] = sum;
  }
  __syncthreads();
  for (int e = tid; e < ROWS * D / 4; e += 32 * KD_WARPS) {
    const int row = e / (D / 4);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < KD_WARPS; ++w) {
      const float c = w_m[w][row];
      const float4 v = *reinterpret_cast<const float4*>(w_o + (size_t)w * ROWS * D + 4 * e);
      acc.x += c * v.x; acc.y += c * v.y; acc.z += c * v.z; acc.w += c * v.w;
    }
    *reinterpret_cast<float4*>(c_o + 4 * e) = acc;
  }
  if (parts != nullptr) {
    // this block's state: ROWS maxima, ROWS sums, ROWS outputs
    __syncthreads();
    float* out = parts + ((((int64_t)b * a.kv_heads + h) * gridDim.x + blockIdx.x) * (ROWS * (D + 2)));
    if (tid < ROWS) {
      out[tid] = c_m[tid];
      out[ROWS + tid] = c_l[tid];
    }
    for (int e = tid; e < ROWS * D / 4; e += 32 * KD_WARPS)
      *reinterpret_cast<float4*>(out + 2 * ROWS + 4 * e) = *reinterpret_cast<const float4*>(c_o + 4 * e);
    return;
  }
  // ---- merged over the cluster: each block takes a share of the outputs ----
  cluster_arrive();
  cluster_wait();
  const uint32_t m_a = smem_u32(c_m), l_a = smem_u32(c_l), o_a = smem_u32(c_o);
  for (int e = (int)crank * 32 * KD_WARPS + tid; e < nr * (D / 2); e += (int)csize * 32 * KD_WARPS) {
    const int row = e / (D / 2), dim = 2 * (e - row * (D / 2));
    float mx = -INFINITY;
    for (uint32_t c = 0; c < csize; ++c) mx = fmaxf(mx, ld_cluster_f32(cluster_map(m_a + 4 * row, c)));
    float sum = 0.f, x0 = 0.f, x1 = 0.f;
    for (uint32_t c = 0; c < csize; ++c) {
      const float mc = ld_cluster_f32(cluster_map(m_a + 4 * row, c));
      const float lc = ld_cluster_f32(cluster_map(l_a + 4 * row, c));
      const float w = mc == -INFINITY && lc == 0.f ? 0.f : ex2(mc - mx);
      sum += w * lc;
      const uint32_t oa = cluster_map(o_a + 4 * (row * D + dim), c);
      x0 += w * ld_cluster_f32(oa);
      x1 += w * ld_cluster_f32(oa + 4);
    }
    const int R = r0 + row, tok = R / group;
    // a query outside the cache sees no key: zeros; scores that are all -inf leave 0 / 0
    const float r = p0 + tok < 0 || p0 + tok >= s.limit ? 0.f : 1.0f / sum;
    const int64_t off = (((int64_t)b * s.L + tok) * a.heads + h * group + R - tok * group) * D + dim;
    if constexpr (SPLIT) {
      *reinterpret_cast<float2*>(static_cast<float*>(a.A) + off) = make_float2(x0 * r, x1 * r);
    } else {
      *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.A) + off) =
          __floats2bfloat162_rn(x0 * r, x1 * r);
    }
  }
  cluster_arrive();
  cluster_wait();                                    // no block leaves while another reads its shared memory
}

// The second kernel merges the parts, a block a row: the parts' weights first, then the
// outputs, two dimensions a thread, the parts shared between 512 / D groups of threads
// and the groups' sums added in their order.  Bound by latency: the parts lie in L2.
constexpr int KD_MAX_SPLITS = 3 * 148;
template <int D, int ROWS, typename XT>
__global__ void __launch_bounds__(256)
kv4_merge_kernel(const KvStep s, const AttnArgs a, int splits, const float* parts) {
  constexpr int PAIRS = D / 2, GROUPS = 256 / PAIRS, PART = ROWS * (D + 2);
  __shared__ float w_part[KD_MAX_SPLITS], l_part[KD_MAX_SPLITS];
  __shared__ float2 x_part[GROUPS][PAIRS];
  pdl_launch_dependents();
  pdl_wait();                                        // the parts come from the previous kernel
  const int group = a.heads / a.kv_heads, b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int tile = blockIdx.x / ROWS, row = blockIdx.x % ROWS, R = tile * ROWS + row;
  if (R >= kv_real_tokens(s, b) * group) return;
  const float* p = parts + (((int64_t)b * a.kv_heads + h) * (gridDim.x / ROWS) + tile) * splits * PART;
  for (int c = tid; c < splits; c += 256) {
    w_part[c] = p[(int64_t)c * PART + row];
    l_part[c] = p[(int64_t)c * PART + ROWS + row];
  }
  __syncthreads();
  float mx = -INFINITY;
  for (int c = lane; c < splits; c += 32) mx = fmaxf(mx, w_part[c]);
  mx = warp_max(mx);
  __syncthreads();
  for (int c = tid; c < splits; c += 256)
    w_part[c] = w_part[c] == -INFINITY && l_part[c] == 0.f ? 0.f : ex2(w_part[c] - mx);
  __syncthreads();
  const int g = tid / PAIRS, pair = tid % PAIRS;
  float2 x = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int c = g; c < splits; c += GROUPS) {
    const float2 v = *reinterpret_cast<const float2*>(p + (int64_t)c * PART + 2 * ROWS + row * D + 2 * pair);
    x.x += w_part[c] * v.x;
    x.y += w_part[c] * v.y;
  }
  x_part[g][pair] = x;
  __syncthreads();
  if (g != 0) return;
  float sum = 0.f;
  for (int c = 0; c < splits; ++c) sum += w_part[c] * l_part[c];
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) {
    x.x += x_part[i][pair].x;
    x.y += x_part[i][pair].y;
  }
  const int tok = R / group;
  // a query outside the cache sees no key: zeros; scores that are all -inf leave 0 / 0
  const int64_t at = kv_first_position(s, b) + tok;
  const float r = at < 0 || at >= s.limit ? 0.f : 1.0f / sum;
  const int64_t off = (((int64_t)b * s.L + tok) * a.heads + h * group + R - tok * group) * D + 2 * pair;
  if constexpr (sizeof(XT) == 4) {
    *reinterpret_cast<float2*>(static_cast<float*>(a.A) + off) = make_float2(x.x * r, x.y * r);
  } else {
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.A) + off) =
        __floats2bfloat162_rn(x.x * r, x.y * r);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// How a step's row tiles are split over blocks.
struct KdSplit {
  int rows;                                          // a tile
  int64_t row_tiles;
  int splits;                                        // blocks a row tile
  bool parts;                                        // merged through the workspace (else in a cluster)
};
static KdSplit kd_split(const KvStep& s, const AttnArgs& a) {
  KdSplit d;
  const int64_t rows = (int64_t)s.L * (a.heads / a.kv_heads);
  d.rows = rows <= 8 ? 8 : 16;
  d.row_tiles = (rows + d.rows - 1) / d.rows;
  const int64_t blocks = d.row_tiles * a.kv_heads * s.B;
  int64_t keys = s.limit;
  if (a.window > 0 && (int64_t)a.window + a.sinks + s.L < keys) keys = (int64_t)a.window + a.sinks + s.L;
  const int64_t per_tile = KD_WARPS * KD_KT;         // keys a block takes with one tile a warp
  // Few row tiles with long contexts: three blocks to an SM, of two tiles a warp at least, merged by a
  // second kernel.  (One sequence of 32000 keys, 16 key heads, bf16: 35 us, in clusters of 8 58 us.)
  const int64_t fill = KD_MAX_SPLITS / blocks, most = keys / (2 * per_tile);
  const int64_t n = fill < most ? fill : most;
  d.parts = n > 8;
  d.splits = (int)n;
  if (d.parts) return d;
  // A cluster: until the blocks fill the GPU (three to an SM) with two tiles a warp at least, and, as
  // sequences may be of very different lengths, until no warp has more than 16 tiles.  (16 sequences of
  // 2048 to 32768 keys, 8 key heads: two blocks a cluster 179 us, four 133, eight 117, sixteen 123.)
  d.splits = 1;
  while (d.splits < 8 && ((blocks * d.splits * 2 <= 3 * 148 && keys > d.splits * per_tile * 2) ||
                          keys > d.splits * per_tile * 16))
    d.splits *= 2;
  return d;
}
// Bytes of the parts (0: none).
size_t kv4_decode_workspace(const KvStep& s, const AttnArgs& a, int d) {
  const KdSplit k = kd_split(s, a);
  return k.parts ? (size_t)(k.row_tiles * a.kv_heads * s.B * k.splits * k.rows * (d + 2)) * sizeof(float) : 0;
}

template <int D, int NT, typename XT>
static cudaError_t launch_decode(const KvStep& s, const AttnArgs& a, const KdSplit& k, void* ws, cudaStream_t st) {
  auto kern = kv4_decode_kernel<D, NT, XT>;
  const size_t smem = (size_t)KD_WARPS * KD_STAGES * KdTile<D>::BYTES + (size_t)8 * NT * D * 4;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  float* parts = k.parts ? static_cast<float*>(ws) : nullptr;
  const unsigned cluster = k.parts ? 1u : (unsigned)k.splits;
  e = launch_pdl(kern, dim3((unsigned)(k.row_tiles * k.splits), (unsigned)a.kv_heads, (unsigned)s.B),
                 dim3(32 * KD_WARPS), smem, st, dim3(cluster, 1, 1), s, a,
                 (float)(1.4426950408889634 / sqrt((double)D)), k.splits, parts);
  if (e != cudaSuccess || !k.parts) return e;
  return launch_pdl(kv4_merge_kernel<D, 8 * NT, XT>,
                    dim3((unsigned)(k.row_tiles * 8 * NT), (unsigned)a.kv_heads, (unsigned)s.B), dim3(256), 0,
                    st, 1u, s, a, k.splits, (const float*)parts);
}

template <int D, typename XT>
static cudaError_t launch_attention(const KvStep& s, const AttnArgs& a, void* ws, cudaStream_t st) {
  const KdSplit k = kd_split(s, a);
  return k.rows == 8 ? launch_decode<D, 1, XT>(s, a, k, ws, st) : launch_decode<D, 2, XT>(s, a, k, ws, st);
}

cudaError_t run_kv4_decode(const KvStep& s, const AttnArgs& a, int bf16, int d, void* ws, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (d == 128) return bf16 ? launch_attention<128, bf>(s, a, ws, st) : launch_attention<128, float>(s, a, ws, st);
  return bf16 ? launch_attention<64, bf>(s, a, ws, st) : launch_attention<64, float>(s, a, ws, st);
}

}  // namespace bitnet
