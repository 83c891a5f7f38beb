// The gated delta rule over packed requests with their states in slots.
//
// Per request and value head, token t with gate a_t and strength b_t (FP32 state S [d_k][d_v]):
//     S <- a_t S + b_t k_t (v_t - a_t S^T k_t)^T,     o_t = scale S^T q_t.
// Over a chunk of C tokens from state S0, with g_i = a_1 ... a_i (all of U's, R's and O's columns, one
// per column of S, are independent):
//     N[i][j] = g_i / g_j b_j k_i . k_j  (j < i)      T = (I + N)^-1
//     R = V - g K S0,  U = T R                        M[i][j] = g_i / g_j b_j q_i . k_j  (j <= i)
//     O = scale (g Q S0 + M U)                        S = g_C S0 + K^T diag(b_j g_C / g_j) U
// The ratios g_i / g_j are products a_(j+1) ... a_i, not quotients: a gate of zero ends a memory
// without a division by zero.
//
// Three kernels here, chosen on the host by the most new tokens of a request: delta_step_kernel (up to 3) streams the
// state once through registers, delta_block_kernel (up to 32, or 24 of d_k = 256) takes 8 tokens at a time,
// delta_chunk_kernel chunks of 32 of prompts with d_k = 256; prompts of d_k 64 and 128 are delta_wide_kernel's.
#include "vq3_internal.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(delta_batch)
}
#include "delta_common.cuh"

namespace vq3 {
namespace {

// ---------------------------------------------------------------- chunks of 32 tokens, d_k = 256
//
// A CTA takes one request, one value head and 64 of its columns and walks the chunks in order. Each of
// its four consumer warps owns 16 columns for the whole call: S^T [16][d_k] stays in registers as the
// accumulators of m16n8k16 tiles, which is also the A operand's layout of the next product S^T [K; Q]^T,
// and R^T, U^T follow in the same way, so no state and no intermediate passes through shared memory.
// Three producer warps take turns with the chunks: they copy K and Q, form T and M, which do not depend on
// the state, and hand them over through a ring of three stages (named barriers, no spinning).
//
// Numbers: the tensor cores multiply FP16. K and Q enter exactly (BF16 rows are brought to a largest entry of 2^14
// by a power of two, which the factors of the token take back: exact down to 2^-31 of the largest entry, smaller ones
// lose bits to FP16's subnormals, 2^-39 of the largest at most). Every FP32 operand (S, R, U,
// T, M) enters as two FP16 parts, hi and what hi leaves, scaled by a power of two per row of the product
// so that neither part leaves FP16's range: some 22 bits, for either type: a BF16 output made from hi
// alone (11 bits) may be rounded the other way (one prompt of 8,192 tokens: 670 us instead of 720).
//
// mma.sync: a state of 256 x 128 with its two parts, the chunk's products and [K; Q] K^T would take 768 of the 512
// columns of tensor memory. (d_k = 128, before BF16 outputs took both parts: 16 ragged prompts 415 us here, 321 by the
// wide kernel; one prompt of 8,192 tokens 648 us here, whose 96 CTAs fill more SMs, 668 there: not worth a
// second kernel for one case that is as fast.) One prompt of 1,024 tokens, 48 heads of 256 x 128, BF16: 155 us (139 with
// outputs from hi alone and no look at the values' range; then 148 with two producers: a chunk's T and M take a warp as
// long as two chunks of the consumers). A chunk gone through token by token: some 36 us.
constexpr int kConsumers = 4, kProducers = 3, kStages = 3;
constexpr int kChunkThreads = 32 * (kConsumers + kProducers);
constexpr int kWarpCols = 16, kCtaCols = kWarpCols * kConsumers;
// Named barriers: per stage and consumer warp "filled" (the warps do not wait for one another), per stage "free".
constexpr int kFullBar = 1, kEmptyBar = kFullBar + kStages * kConsumers;
constexpr int kFullThreads = 64, kEmptyThreads = 32 * (kConsumers + 1);
static_assert(kEmptyBar + kStages <= 16, "named barriers");

constexpr int KS = 16, NN = 4;  // steps of 16 of d_k, blocks of 8 tokens
struct Stage {
  static constexpr int DK = 16 * KS, C = 8 * NN;
  static constexpr int RS = DK + 8;                              // row of K and Q in halves: 16 bytes past 128
  static constexpr int TS = 40;                                  // row of T and M: ldmatrix without conflicts
  static constexpr int VS = kCtaCols + 8;                        // row of V
  static constexpr int kK = 0, kQ = kK + C * RS * 2, kV = kQ + C * RS * 2, kT = kV + C * VS * 2;
  static constexpr int NS = C + 4;                               // column of N in floats
  // T: hi, then lo; before, in the same place, N
  static constexpr int kM = kT + (2 * TS * 2 > NS * 4 ? 2 * TS * 2 : NS * 4) * C, kC = kM + 2 * C * TS * 2;  // M: hi, lo
  static constexpr int kBytes = (kC + (6 * C + 4) * 4 + 127) / 128 * 128;
  // factors per token: of V in R, of K S0 in R, of Q S0 and of M U in O, of U in the state; then g_C, and whether T has
  // grown too large; gates
  static constexpr int kFv = 0, kFk = C, kFq = 2 * C, kFm = 3 * C, kFw = 4 * C, kFg = 5 * C, kFt = kFg + 1, kFa = 5 * C + 4;
};

__device__ __forceinline__ uint32_t smem_of(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(b0));
}
// Four 8 x 8 matrices; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// Rows g and g + 8 of NT accumulator tiles: the largest magnitude over the row (lanes of one g).
template <int NT>
__device__ __forceinline__ void row_max(const float (&x)[NT][4], float& m0, float& m1) {
  m0 = m1 = 0.f;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m0 = fmaxf(m0, fmaxf(fabsf(x[n][0]), fabsf(x[n][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(x[n][2]), fabsf(x[n][3])));
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
  }
}

// ---- producer: one chunk's K, Q, T, M and factors
//
// One warp, so everything is a chain of latencies: the copies land while the ratios are formed, the
// ratios and N are kept by columns (lane j's 16-byte stores and loads do not conflict), and the
// substitution goes column by column: once x_m is known every later row takes its part, 31 - m
// independent products, where row by row each x_m waits for a sum (2,000 -> 700 cycles at C = 32).
template <bool BF16>
__device__ __forceinline__ void produce(const DeltaArgs& a, const DeltaRequest& rq, int h, int col0, int t0,
                                        unsigned char* st, int lane) {
  using L = Stage;
  constexpr int C = L::C, RS = L::RS, DK = L::DK, TS = L::TS, NS = L::NS;
  const int nt = rq.n - t0 < C ? rq.n - t0 : C;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t sk = smem_of(st + L::kK), sq = smem_of(st + L::kQ);
  float* const ratio = reinterpret_cast<float*>(st + L::kT);  // [column j][row i], then N; T takes its place
  // gates, lane = token
  float al = 1.f, be = 0.f;
  if (lane < nt && VQ3_IN(rq.first + t0 + lane, a.tokens, 2)) {
    al = __ldg(a.alpha + (long long)(rq.first + t0 + lane) * a.alpha_token + h);
    be = __ldg(a.beta + (long long)(rq.first + t0 + lane) * a.beta_token + h);
  }
  // rows of K and Q, tokens past the last zero: a lane takes one 16-byte column
  {
    static_assert(DK / 8 == 32, "a lane per column");
    const int hq = h / a.group, c = lane;
    const uint16_t* kp = static_cast<const uint16_t*>(a.k) + (rq.first + t0) * a.k_token + hq * a.k_head + c * 8;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (rq.first + t0) * a.q_token + hq * a.q_head + c * 8;
    const uint32_t off = (uint32_t)(c * 8) * 2u;
#pragma unroll 2
    for (int row = 0; row < C; ++row) {
      const uint32_t at = off + (uint32_t)(row * RS) * 2u;
      // bytes read: 16, or none past the last token (zeros are written)
      const int bytes = row < nt && VQ3_IN(rq.first + t0 + row, a.tokens, 1) ? 16 : 0;
      const long long from = bytes ? row : 0;  // an address inside the rows
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sk + at), "l"(kp + from * a.k_token), "r"(bytes) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sq + at), "l"(qp + from * a.q_token), "r"(bytes) : "memory");
    }
    // V: 8 lanes a row; columns behind the last are not used
    const int rv = lane >> 3, cv = (lane & 7) * 8;
    const bool some = col0 + cv < a.d_v;
    const uint16_t* vp = static_cast<const uint16_t*>(a.v) + (rq.first + t0) * a.v_token + h * a.v_head + (some ? col0 + cv : 0);
    const uint32_t sv = smem_of(st + L::kV) + (uint32_t)(rv * L::VS + cv) * 2u;
#pragma unroll 2
    for (int i = 0; i < C / 4; ++i) {
      const int row = 4 * i + rv;
      const int bytes = some && row < nt && VQ3_IN(rq.first + t0 + row, a.tokens, 4) ? 16 : 0;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sv + (uint32_t)(4 * i * L::VS) * 2u),
                   "l"(vp + (bytes ? row : 0) * a.v_token), "r"(bytes) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // ratios D[i][j] = a_(j+1) ... a_i (lane = j), the running product g_i, and g_C / g_j
  float* const f = reinterpret_cast<float*>(st + L::kC);
  f[L::kFv + lane] = al;
  f[L::kFa + lane] = al;
  __syncwarp();
  float r = 1.f, gam = 1.f, gi = 1.f;
#pragma unroll
  for (int i = 0; i < C; i += 4) {
    const float4 a4 = *reinterpret_cast<const float4*>(f + L::kFv + i);
    const float av[4] = {a4.x, a4.y, a4.z, a4.w};
    float d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gam *= av[e];
      gi = i + e == lane ? gam : gi;
      r *= i + e > lane ? av[e] : 1.f;
      d[e] = r;
    }
    *reinterpret_cast<float4*>(ratio + lane * NS + i) = make_float4(d[0], d[1], d[2], d[3]);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  // BF16 rows to FP16, each scaled by a power of two (lane = row: 16 bytes past 128 a row, no conflicts)
  float kb = 1.f, qb = 1.f;
  if constexpr (BF16) {
#pragma unroll 1
    for (int m = 0; m < 2; ++m) {
      {
        uint4* row = reinterpret_cast<uint4*>(st + (m ? L::kQ : L::kK) + lane * RS * 2);
        __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll 4
        for (int c = 0; c < DK / 8; ++c) {
          const uint4 w = row[c];
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e])));
        }
        const Scale s = scale_of(fmaxf(__low2float(top), __high2float(top)));
        const __nv_bfloat162 fs = __float2bfloat162_rn(s.to);
#pragma unroll 4
        for (int c = 0; c < DK / 8; ++c) {
          const uint4 w = row[c];
          uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e]), fs);
            const float2 y = delta_unpack2<true>(*reinterpret_cast<const uint32_t*>(&x));
            ws[e] = pack_f16(y.x, y.y);
          }
          row[c] = make_uint4(ws[0], ws[1], ws[2], ws[3]);
        }
        (m ? qb : kb) = s.back;
      }
    }
    __syncwarp();
  }
  // [K; Q] K^T by blocks of 8 tokens: rows g of a tile are k_i . k_j, rows g + 8 q_i . k_j; j-block n <= i-block b
  constexpr int kTiles = NN * (NN + 1) / 2;
  float kq[kTiles][4];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) kq[i][0] = kq[i][1] = kq[i][2] = kq[i][3] = 0.f;
#pragma unroll 2
  for (int s = 0; s < KS; ++s) {
    uint32_t kf[NN][4];
#pragma unroll
    for (int b = 0; b < NN; ++b)  // matrices: K columns 0-7, 8-15 of the step, Q the same
      ldsm4(kf[b], (lane < 16 ? sk : sq) + (uint32_t)((8 * b + (lane & 7)) * RS + 16 * s + ((lane >> 3) & 1) * 8) * 2u);
    int i = 0;
#pragma unroll
    for (int b = 0; b < NN; ++b) {
      const uint32_t af[4] = {kf[b][0], kf[b][2], kf[b][1], kf[b][3]};
#pragma unroll
      for (int n = 0; n <= b; ++n, ++i) mma16(kq[i], af, kf[n][0], kf[n][1]);
    }
  }
  // N over the ratios (each thread where it read them); M, rows scaled, as FP16 parts
  uint16_t* mhi = reinterpret_cast<uint16_t*>(st + L::kM);
  uint16_t* mlo = mhi + C * TS;
  const float bk = be * kb;  // b_j and the factor of k_j
  float fm = 0.f;
  float bj[NN][2];
#pragma unroll
  for (int n = 0; n < NN; ++n) {
    bj[n][0] = __shfl_sync(0xffffffffu, bk, 8 * n + 2 * t);
    bj[n][1] = __shfl_sync(0xffffffffu, bk, 8 * n + 2 * t + 1);
  }
  int i = 0;
#pragma unroll
  for (int b = 0; b < NN; ++b) {
    const float ki = __shfl_sync(0xffffffffu, kb, 8 * b + g);
    float m[NN][2];
    float top = 0.f;
#pragma unroll
    for (int n = 0; n <= b; ++n, ++i) {
      const int row = 8 * b + g, col = 8 * n + 2 * t;
      float* at0 = ratio + col * NS + row;
      float* at1 = at0 + NS;
      const float d0 = *at0 * bj[n][0], d1 = *at1 * bj[n][1];
      *at0 = col < row ? -d0 * ki * kq[i][0] : 0.f;
      *at1 = col + 1 < row ? -d1 * ki * kq[i][1] : 0.f;
      m[n][0] = col <= row ? d0 * kq[i][2] : 0.f;
      m[n][1] = col + 1 <= row ? d1 * kq[i][3] : 0.f;
      top = fmaxf(top, fmaxf(fabsf(m[n][0]), fabsf(m[n][1])));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const Scale s = scale_of(top);
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      // the block above the diagonal that the last 16-token step of the row block reads is zero
      if (n > (b | 1)) continue;
      uint32_t hi = 0u, lo = 0u;
      if (n <= b) split2(m[n][0] * s.to, m[n][1] * s.to, hi, lo);
      *reinterpret_cast<uint32_t*>(mhi + (8 * b + g) * TS + 8 * n + 2 * t) = hi;
      *reinterpret_cast<uint32_t*>(mlo + (8 * b + g) * TS + 8 * n + 2 * t) = lo;
    }
    const float back = __shfl_sync(0xffffffffu, s.back, (lane & 7) * 4);  // of row 8 b + lane % 8
    if (lane >> 3 == b) fm = back;
  }
  __syncwarp();
  // T = (I + N)^-1 by forward substitution, lane = column of T; -N is in `ratio` by columns. Rows in pairs.
  float2 x[C / 2];
#pragma unroll
  for (int k = 0; k < C / 2; ++k) x[k] = make_float2(2 * k == lane ? 1.f : 0.f, 2 * k + 1 == lane ? 1.f : 0.f);
#pragma unroll
  for (int m = 0; m < C - 1; ++m) {
    const float xm = m & 1 ? x[m / 2].y : x[m / 2].x;
#pragma unroll
    for (int k = (m + 1) / 4 * 4; k < C; k += 4) {  // rows up to m hold zeros (the diagonal block's)
      const float4 nv = *reinterpret_cast<const float4*>(ratio + m * NS + k);
      if (k + 1 > m) x[k / 2] = fma_pair(make_float2(nv.x, nv.y), xm, x[k / 2]);
      x[k / 2 + 1] = fma_pair(make_float2(nv.z, nv.w), xm, x[k / 2 + 1]);
    }
  }
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < C / 2; ++k) top = fmaxf(top, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
  const Scale ts = scale_of(top);
  __syncwarp();  // every lane has read N
  {  // column j of T as row j
    uint4* thi = reinterpret_cast<uint4*>(st + L::kT + lane * TS * 2);
    uint4* tlo = reinterpret_cast<uint4*>(st + L::kT + (C + lane) * TS * 2);
#pragma unroll
    for (int k = 0; k < C; k += 8) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(x[k / 2 + e].x * ts.to, x[k / 2 + e].y * ts.to, hi[e], lo[e]);
      thi[k / 8] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      tlo[k / 8] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    f[L::kFv + lane] = ts.back;
    f[L::kFk + lane] = gi * kb * ts.back;
    f[L::kFq + lane] = a.scale * gi * qb;
    f[L::kFm + lane] = a.scale * qb * fm;
    f[L::kFw + lane] = bk * r;
    const bool grown = __any_sync(0xffffffffu, !(top < kGrown));
    if (lane == 0) {
      f[L::kFg] = gam;
      f[L::kFt] = grown ? 1.f : 0.f;
    }
  }
  __syncwarp();
}

// ---- tokens one at a time, by a warp with 16 columns of S in its accumulators (row(n, e) of S: entry e of tile n)
template <int NT, bool BF16, class Row>
__device__ __forceinline__ void warp_steps(const DeltaArgs& a, int h, long long row0, int nt, int col, float (&acc)[NT][4],
                                           Row row) {
  const int hq = h / a.group, t = threadIdx.x & 3;
  for (int j = 0; j < nt && VQ3_IN(row0 + j, a.tokens, 16); ++j) {
    const long long at = row0 + j;
    const uint16_t* kp = static_cast<const uint16_t*>(a.k) + at * a.k_token + hq * a.k_head;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + at * a.q_token + hq * a.q_head;
    float s[5] = {0.f, 0.f, 0.f, 0.f, 0.f};  // k . S of two columns, q . S of them, k . q
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 k = delta_unpack2<BF16>(__ldg(reinterpret_cast<const uint32_t*>(kp + row(n, 0))));
      const float2 q = delta_unpack2<BF16>(__ldg(reinterpret_cast<const uint32_t*>(qp + row(n, 0))));
      s[0] = fmaf(k.x, acc[n][0], fmaf(k.y, acc[n][1], s[0]));
      s[1] = fmaf(k.x, acc[n][2], fmaf(k.y, acc[n][3], s[1]));
      s[2] = fmaf(q.x, acc[n][0], fmaf(q.y, acc[n][1], s[2]));
      s[3] = fmaf(q.x, acc[n][2], fmaf(q.y, acc[n][3], s[3]));
      s[4] = fmaf(k.x, q.x, fmaf(k.y, q.y, s[4]));
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      s[i] += __shfl_xor_sync(0xffffffffu, s[i], 1);
      s[i] += __shfl_xor_sync(0xffffffffu, s[i], 2);
    }
    const float al = __ldg(a.alpha + at * a.alpha_token + h), be = __ldg(a.beta + at * a.beta_token + h);
    const float2 v = delta_unpack2<BF16>(__ldg(
        reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.v) + at * a.v_token + h * a.v_head + col)));
    const float u0 = be * (v.x - al * s[0]), u1 = be * (v.y - al * s[1]);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 k = delta_unpack2<BF16>(__ldg(reinterpret_cast<const uint32_t*>(kp + row(n, 0))));
      acc[n][0] = fmaf(k.x, u0, al * acc[n][0]);
      acc[n][1] = fmaf(k.y, u0, al * acc[n][1]);
      acc[n][2] = fmaf(k.x, u1, al * acc[n][2]);
      acc[n][3] = fmaf(k.y, u1, al * acc[n][3]);
    }
    if (t == 0)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at * a.o_token + h * a.o_head + col) =
          delta_pack2<BF16>(a.scale * fmaf(s[4], u0, al * s[2]), a.scale * fmaf(s[4], u1, al * s[3]));
  }
}
// Least of a column's sizes over the lanes that share it.
__device__ __forceinline__ float seen_least(float m) {
  m = fminf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fminf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
// The least that a token finds in its two columns, from `size` on and with earlier tokens' R as the gates leave them
// (nothing at all needs no bits): for the few chunks whose least R alone, or a zero, would have had them gone through again.
template <int NB, class Gate>
__device__ __forceinline__ float2 least_found(const float (&r)[NB][4], float2 size, Gate gate) {
  const int quad = threadIdx.x & 28;
  float2 least = both(INFINITY);
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y0 = fabsf(__shfl_sync(0xffffffffu, r[n][i & 1], quad + i / 2));
      const float y1 = fabsf(__shfl_sync(0xffffffffu, r[n][2 + (i & 1)], quad + i / 2));
      const float a = fabsf(gate(8 * n + i));
      size = make_float2(fmaxf(a * size.x, y0), fmaxf(a * size.y, y1));
      if (size.x > 0.f) least.x = fminf(least.x, size.x);
      if (size.y > 0.f) least.y = fminf(least.y, size.y);
    }
  return least;
}

// ---- consumer: one chunk against this warp's 16 columns; acc: S^T, row g column 2g, row g + 8 column 2g + 1.
// False, with S as it was: the chunk has to be gone through token by token.
template <bool BF16>
__device__ __forceinline__ bool consume(float (&acc)[2 * KS][4], const unsigned char* st, float (&o)[NN][4], int nt, int warp,
                                        int lane) {
  using L = Stage;
  constexpr int C = L::C, RS = L::RS, TS = L::TS;
  constexpr int K2 = NN / 2;  // steps of 16 tokens
  const int g = lane >> 2, t = lane & 3;
  const uint32_t sk = smem_of(st + L::kK), sq = smem_of(st + L::kQ), sT = smem_of(st + L::kT), sM = smem_of(st + L::kM);
  const float* f = reinterpret_cast<const float*>(st + L::kC);

  float m0, m1;
  row_max<2 * KS>(acc, m0, m1);
  const Scale s0 = scale_of(m0), s1 = scale_of(m1);
  float xk[NN][4], xq[NN][4];
#pragma unroll
  for (int n = 0; n < NN; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) xk[n][e] = xq[n][e] = 0.f;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      split2(acc[2 * s + p][0] * s0.to, acc[2 * s + p][1] * s0.to, hi[2 * p], lo[2 * p]);
      split2(acc[2 * s + p][2] * s1.to, acc[2 * s + p][3] * s1.to, hi[2 * p + 1], lo[2 * p + 1]);
    }
#pragma unroll
    for (int n = 0; n < NN; n += 2) {
      const uint32_t off = (uint32_t)((8 * n + (lane & 7) + (lane >> 4) * 8) * RS + 16 * s + ((lane >> 3) & 1) * 8) * 2u;
      uint32_t b[4];
      ldsm4(b, sk + off);
      mma16(xk[n], hi, b[0], b[1]);
      mma16(xk[n + 1], hi, b[2], b[3]);
      mma16(xk[n], lo, b[0], b[1]);
      mma16(xk[n + 1], lo, b[2], b[3]);
      ldsm4(b, sq + off);
      mma16(xq[n], hi, b[0], b[1]);
      mma16(xq[n + 1], hi, b[2], b[3]);
      mma16(xq[n], lo, b[0], b[1]);
      mma16(xq[n + 1], lo, b[2], b[3]);
    }
  }
#pragma unroll
  for (int n = 0; n < NN; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      xk[n][e] *= e < 2 ? s0.back : s1.back;
      xq[n][e] *= e < 2 ? s0.back : s1.back;
    }
  // R^T = V^T - X_K, times the factor of T's column
  const unsigned char* sv = st + L::kV + ((2 * t) * L::VS + warp * kWarpCols + 2 * g) * 2;
  float seen0 = INFINITY, seen1 = INFINITY;  // of the request's tokens
#pragma unroll
  for (int n = 0; n < NN; ++n) {
    const float2 fv = *reinterpret_cast<const float2*>(f + L::kFv + 8 * n + 2 * t);
    const float2 fk = *reinterpret_cast<const float2*>(f + L::kFk + 8 * n + 2 * t);
    const float2 va = delta_unpack2<BF16>(*reinterpret_cast<const uint32_t*>(sv + 8 * n * L::VS * 2));
    const float2 vb = delta_unpack2<BF16>(*reinterpret_cast<const uint32_t*>(sv + (8 * n + 1) * L::VS * 2));
    xk[n][0] = va.x * fv.x - fk.x * xk[n][0];
    xk[n][1] = vb.x * fv.y - fk.y * xk[n][1];
    xk[n][2] = va.y * fv.x - fk.x * xk[n][2];
    xk[n][3] = vb.y * fv.y - fk.y * xk[n][3];
    if (8 * n + 2 * t < nt) {
      seen0 = fminf(seen0, fmaxf(fabsf(va.x * fv.x), fabsf(xk[n][0])));
      seen1 = fminf(seen1, fmaxf(fabsf(va.y * fv.x), fabsf(xk[n][2])));
    }
    if (8 * n + 2 * t + 1 < nt) {
      seen0 = fminf(seen0, fmaxf(fabsf(vb.x * fv.y), fabsf(xk[n][1])));
      seen1 = fminf(seen1, fmaxf(fabsf(vb.y * fv.y), fabsf(xk[n][3])));
    }
  }
  seen0 = seen_least(seen0);
  seen1 = seen_least(seen1);
  // U^T = R^T T^T
  float top0, top1;
  row_max<NN>(xk, top0, top1);
  const Scale r0 = scale_of(top0), r1 = scale_of(top1);
  float u[NN][4];
#pragma unroll
  for (int n = 0; n < NN; ++n) u[n][0] = u[n][1] = u[n][2] = u[n][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < K2; ++ks) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      split2(xk[2 * ks + p][0] * r0.to, xk[2 * ks + p][1] * r0.to, hi[2 * p], lo[2 * p]);
      split2(xk[2 * ks + p][2] * r1.to, xk[2 * ks + p][3] * r1.to, hi[2 * p + 1], lo[2 * p + 1]);
    }
#pragma unroll
    for (int n = 2 * ks; n < NN; ++n) {
      // matrices: tokens 0-7, 8-15 of the step (rows) at block n (columns), hi, then lo
      uint32_t b[4];
      ldsm4t(b, sT + (uint32_t)(((lane >> 4) * C + 16 * ks + (lane & 15)) * TS + 8 * n) * 2u);
      mma16(u[n], hi, b[0], b[1]);
      mma16(u[n], lo, b[0], b[1]);
      mma16(u[n], hi, b[2], b[3]);
    }
  }
#pragma unroll
  for (int n = 0; n < NN; ++n) {
    u[n][0] *= r0.back;
    u[n][1] *= r0.back;
    u[n][2] *= r1.back;
    u[n][3] *= r1.back;
  }
  float um0, um1;
  row_max<NN>(u, um0, um1);
  {
    float all = 0.f;
#pragma unroll
    for (int n = 0; n < NN; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) all += fabsf(u[n][e]);
    // (R and what it comes from have T's factor of 2^-14)
    if (__any_sync(0xffffffffu, !(all < INFINITY)) || f[L::kFt] != 0.f) return false;
    const float need0 = fmaxf(top0, 0x1p-14f * um0) * kRange, need1 = fmaxf(top1, 0x1p-14f * um1) * kRange;
    if (__any_sync(0xffffffffu, need0 > seen0 || need1 > seen1)) {
      const float2 least = least_found<NN>(xk, make_float2(0x1p-17f * m0, 0x1p-17f * m1), [f](int i) { return f[L::kFa + i]; });
      if (__any_sync(0xffffffffu, need0 > least.x || need1 > least.y)) return false;
    }
  }
  // S^T <- g_C S^T + (U diag(w))^T K
  {
    float w[NN][4];
#pragma unroll
    for (int n = 0; n < NN; ++n) {
      const float2 fw = *reinterpret_cast<const float2*>(f + L::kFw + 8 * n + 2 * t);
      w[n][0] = u[n][0] * fw.x;
      w[n][1] = u[n][1] * fw.y;
      w[n][2] = u[n][2] * fw.x;
      w[n][3] = u[n][3] * fw.y;
    }
    row_max<NN>(w, m0, m1);
    const Scale w0 = scale_of(m0), w1 = scale_of(m1);
    uint32_t hi[K2][4], lo[K2][4];
#pragma unroll
    for (int ks = 0; ks < K2; ++ks)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        split2(w[2 * ks + p][0] * w0.to, w[2 * ks + p][1] * w0.to, hi[ks][2 * p], lo[ks][2 * p]);
        split2(w[2 * ks + p][2] * w1.to, w[2 * ks + p][3] * w1.to, hi[ks][2 * p + 1], lo[ks][2 * p + 1]);
      }
    const float gC = f[L::kFg];
#pragma unroll
    for (int n = 0; n < 2 * KS; n += 2) {
      float d[2][4];
#pragma unroll
      for (int p = 0; p < 2; ++p) d[p][0] = d[p][1] = d[p][2] = d[p][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < K2; ++ks) {
        uint32_t b[4];  // matrices: tokens 0-7, 8-15 of the step (rows) at d_k 8n, then at 8(n + 1)
        ldsm4t(b, sk + (uint32_t)((16 * ks + (lane & 15)) * RS + 8 * n + (lane >> 4) * 8) * 2u);
        mma16(d[0], hi[ks], b[0], b[1]);
        mma16(d[1], hi[ks], b[2], b[3]);
        mma16(d[0], lo[ks], b[0], b[1]);
        mma16(d[1], lo[ks], b[2], b[3]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        acc[n + p][0] = fmaf(w0.back, d[p][0], gC * acc[n + p][0]);
        acc[n + p][1] = fmaf(w0.back, d[p][1], gC * acc[n + p][1]);
        acc[n + p][2] = fmaf(w1.back, d[p][2], gC * acc[n + p][2]);
        acc[n + p][3] = fmaf(w1.back, d[p][3], gC * acc[n + p][3]);
      }
    }
  }
  // O^T = X_Q + U^T M^T
  const Scale u0 = scale_of(um0), u1 = scale_of(um1);
#pragma unroll
  for (int n = 0; n < NN; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < K2; ++ks) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      split2(u[2 * ks + p][0] * u0.to, u[2 * ks + p][1] * u0.to, hi[2 * p], lo[2 * p]);
      split2(u[2 * ks + p][2] * u1.to, u[2 * ks + p][3] * u1.to, hi[2 * p + 1], lo[2 * p + 1]);
    }
#pragma unroll
    for (int n = 2 * ks; n < NN; ++n) {
      // matrices: block n (rows) at tokens 0-7, 8-15 of the step, hi, then lo
      uint32_t b[4];
      ldsm4(b, sM + (uint32_t)(((lane >> 4) * C + 8 * n + (lane & 7)) * TS + 16 * ks + ((lane >> 3) & 1) * 8) * 2u);
      mma16(o[n], hi, b[0], b[1]);
      mma16(o[n], lo, b[0], b[1]);
      mma16(o[n], hi, b[2], b[3]);
    }
  }
#pragma unroll
  for (int n = 0; n < NN; ++n) {
    const float2 fq = *reinterpret_cast<const float2*>(f + L::kFq + 8 * n + 2 * t);
    const float2 fm = *reinterpret_cast<const float2*>(f + L::kFm + 8 * n + 2 * t);
    o[n][0] = fq.x * xq[n][0] + fm.x * (u0.back * o[n][0]);
    o[n][1] = fq.y * xq[n][1] + fm.y * (u0.back * o[n][1]);
    o[n][2] = fq.x * xq[n][2] + fm.x * (u1.back * o[n][2]);
    o[n][3] = fq.y * xq[n][3] + fm.y * (u1.back * o[n][3]);
  }
  return true;
}

template <bool BF16>
__global__ void __launch_bounds__(kChunkThreads, 1) delta_chunk_kernel(const __grid_constant__ DeltaArgs a) {
  using L = Stage;
  constexpr int C = L::C;
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y;
  const DeltaRequest rq = delta_request(a, blockIdx.z, h);
  const int chunks = (rq.n + C - 1) / C;

  if (warp >= kConsumers) {
    for (int c = warp - kConsumers; c < chunks; c += kProducers) {
      const int s = c % kStages;
      if (c >= kStages) bar_sync(kEmptyBar + s, kEmptyThreads);  // the consumers are done with chunk c - kStages
      produce<BF16>(a, rq, h, blockIdx.x * kCtaCols, c * C, smem + s * L::kBytes, lane);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) bar_arrive(kFullBar + s * kConsumers + w, kFullThreads);
    }
    return;
  }

  // a consumer without columns (d_v is a multiple of 16 only) goes along for the barriers
  const int c0 = blockIdx.x * kCtaCols + warp * kWarpCols;
  const bool on = c0 < a.d_v;
  const int col = c0 + 2 * g;
  const size_t n_state = (size_t)a.d_k * a.d_v;
  float acc[2 * KS][4];
#pragma unroll
  for (int n = 0; n < 2 * KS; ++n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const size_t at = (size_t)(8 * n + 2 * t + e) * a.d_v + col;
      float2 s = make_float2(0.f, 0.f);
      if (on && rq.in && VQ3_IN(at + 1, n_state, 3)) s = *reinterpret_cast<const float2*>(rq.in + at);
      acc[n][e] = s.x;
      acc[n][2 + e] = s.y;
    }
  }
  uint16_t* op = static_cast<uint16_t*>(a.out) + rq.first * a.o_token + h * a.o_head + col;
  for (int c = 0; c < chunks; ++c) {
    const int s = c % kStages;
    bar_sync(kFullBar + s * kConsumers + warp, kFullThreads);
    float o[NN][4];
    const bool done = on && consume<BF16>(acc, smem + s * L::kBytes, o, rq.n - c * C, warp, lane);
    if (c + kStages < chunks) bar_arrive(kEmptyBar + s, kEmptyThreads);
    if (on && !done) {
      warp_steps<2 * KS, BF16>(a, h, rq.first + c * C, min(rq.n - c * C, C), col, acc, [t](int n, int e) { return 8 * n + 2 * t + e; });
    } else if (on) {
#pragma unroll
      for (int n = 0; n < NN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = c * C + 8 * n + 2 * t + e;
          if (tok < rq.n && VQ3_IN(rq.first + tok, a.tokens, 5))
            *reinterpret_cast<uint32_t*>(op + tok * a.o_token) = delta_pack2<BF16>(o[n][e], o[n][2 + e]);
        }
    }
  }
  if (on && rq.out && (chunks || rq.out != rq.in)) {
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const size_t at = (size_t)(8 * n + 2 * t + e) * a.d_v + col;
        if (VQ3_IN(at + 1, n_state, 6)) *reinterpret_cast<float2*>(rq.out + at) = make_float2(acc[n][e], acc[n][2 + e]);
      }
  }
}

template <bool BF16>
cudaError_t launch_chunk(const DeltaArgs& a, cudaStream_t st) {
  constexpr int smem = kStages * Stage::kBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(delta_chunk_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.d_v + kCtaCols - 1) / kCtaCols), (unsigned)a.v_heads, (unsigned)a.requests);
  delta_chunk_kernel<BF16><<<grid, kChunkThreads, smem, st>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- a few tokens
//
// Verify steps: blocks of 8 tokens, the mathematics and numbers of a chunk, but every warp by itself, with 16 columns of
// a head's state in registers and no barrier: bound by the state's bytes, it lives from many warps that each wait for
// their own loads. K and Q are loaded as the B operand of S^T [K; Q]^T, which is also both operands of [K; Q] K^T and,
// transposed by movmatrix, K's part of the state's product. The order of d_k within a product is free: a lane loads 16
// bytes of a row, two pairs of entries for each of two steps, and the state's rows follow (block_row). N goes through
// 64 floats of shared memory to lanes that each solve for a column of T. 16 requests x 8 tokens, 48 heads of 128 x 128:
// 27.9 us (56% of a copy's rate), some 1,550 instructions a warp at three warps a scheduler. When it took 27.2: 28.8 us as
// chunks of 8 whose T and M two warps made for four; 29.0 us with four warps a scheduler, which spill; 27.0 us, but 5.0
// instead of 4.6 for one request, with the next task's state on its way into shared memory; 41 us in FP32 on CUDA cores,
// bound by the reads of k and q from shared memory.
constexpr int kBlockTokens = 8, kBlockThreads = 128;

template <bool BF16>
__device__ __forceinline__ void row_to_f16(uint32_t* x, int n, float& back) {  // a row's entries in 4 lanes
  if constexpr (BF16) {
    __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < n; ++i) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x[i])));
    float m = fmaxf(__low2float(top), __high2float(top));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const Scale s = scale_of(m);
    const __nv_bfloat162 f = __float2bfloat162_rn(s.to);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), f);
      const float2 z = delta_unpack2<true>(*reinterpret_cast<const uint32_t*>(&y));
      x[i] = pack_f16(z.x, z.y);
    }
    back = s.back;
  }
}
// The row of the state at entry e of lane t in tile n: 8-entry tiles 4 i .. 4 i + 3 hold the 32 rows from 32 i on, 8 to a lane.
__device__ __forceinline__ int block_row(int n, int t, int e) { return 32 * (n >> 2) + 8 * t + 2 * (n & 3) + e; }
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int KS, bool BF16>
__global__ void __launch_bounds__(kBlockThreads, KS <= 8 ? 3 : 2) delta_block_kernel(const __grid_constant__ DeltaArgs a) {
  constexpr int B = kBlockTokens;
  __shared__ float solve[kBlockThreads / 32][B][B];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, hq = h / a.group, c0 = blockIdx.x * kCtaCols + warp * kWarpCols;
  if (c0 >= a.d_v) return;  // (no barrier of the block's follows)
  const DeltaRequest rq = delta_request(a, blockIdx.z, h);
  const int col = c0 + 2 * g;
  const size_t n_state = (size_t)a.d_k * a.d_v;
  float(*const sn)[B] = solve[warp];
  float acc[2 * KS][4];
#pragma unroll
  for (int n = 0; n < 2 * KS; ++n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const size_t at = (size_t)block_row(n, t, e) * a.d_v + col;
      float2 s = make_float2(0.f, 0.f);
      if (rq.in && VQ3_IN(at + 1, n_state, 10)) s = __ldcs(reinterpret_cast<const float2*>(rq.in + at));
      acc[n][e] = s.x;
      acc[n][2 + e] = s.y;
    }
  }
  for (int t0 = 0; t0 < rq.n; t0 += B) {
    const int nt = rq.n - t0 < B ? rq.n - t0 : B;
    const long long row0 = rq.first + t0;
    // K, Q of token g; tokens past the last: zeros, a gate of 1, a strength of 0
    uint32_t kf[2 * KS], qf[2 * KS];
    {
      const bool in = g < nt && VQ3_IN(row0 + g, a.tokens, 11);
      const uint16_t* kp = static_cast<const uint16_t*>(a.k) + (row0 + (in ? g : 0)) * a.k_token + hq * a.k_head + 8 * t;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (row0 + (in ? g : 0)) * a.q_token + hq * a.q_head + 8 * t;
#pragma unroll
      for (int i = 0; i < 2 * KS; i += 4) {
        uint4 k = make_uint4(0u, 0u, 0u, 0u), q = k;
        if (in) {
          k = __ldg(reinterpret_cast<const uint4*>(kp + 8 * i));
          q = __ldg(reinterpret_cast<const uint4*>(qp + 8 * i));
        }
        kf[i] = k.x;
        kf[i + 1] = k.y;
        kf[i + 2] = k.z;
        kf[i + 3] = k.w;
        qf[i] = q.x;
        qf[i + 1] = q.y;
        qf[i + 2] = q.z;
        qf[i + 3] = q.w;
      }
    }
    uint32_t vw[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int tok = 2 * t + e;
      vw[e] = tok < nt && VQ3_IN(row0 + tok, a.tokens, 12)
                  ? __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.v) + (row0 + tok) * a.v_token + h * a.v_head + col))
                  : 0u;
    }
    float al = 1.f, be = 0.f;
    if (lane < nt && VQ3_IN(row0 + lane, a.tokens, 13)) {
      al = __ldg(a.alpha + (row0 + lane) * a.alpha_token + h);
      be = __ldg(a.beta + (row0 + lane) * a.beta_token + h);
    }
    // d0, d1: a_(j+1) ... a_g of j = 2 t, 2 t + 1; of those tokens: a_1 ... a_j and a_(j+1) ... a_8
    float d0 = 1.f, d1 = 1.f, g0 = 1.f, g1 = 1.f, e0 = 1.f, e1 = 1.f, g8 = 1.f;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const float ai = __shfl_sync(0xffffffffu, al, i);
      g8 *= ai;
      (i <= 2 * t ? g0 : e0) *= ai;
      (i <= 2 * t + 1 ? g1 : e1) *= ai;
      if (i <= g) {
        d0 *= i > 2 * t ? ai : 1.f;
        d1 *= i > 2 * t + 1 ? ai : 1.f;
      }
    }
    float kb = 1.f, qb = 1.f;  // of token g
    row_to_f16<BF16>(kf, 2 * KS, kb);
    row_to_f16<BF16>(qf, 2 * KS, qb);
    const float bk = __shfl_sync(0xffffffffu, be, g) * kb;
    const float bk0 = __shfl_sync(0xffffffffu, bk, 8 * t), bk1 = __shfl_sync(0xffffffffu, bk, 8 * t + 4);
    const float kb0 = __shfl_sync(0xffffffffu, kb, 8 * t), kb1 = __shfl_sync(0xffffffffu, kb, 8 * t + 4);
    const float qb0 = __shfl_sync(0xffffffffu, qb, 8 * t), qb1 = __shfl_sync(0xffffffffu, qb, 8 * t + 4);
    float kq[4] = {0.f, 0.f, 0.f, 0.f};  // k_g . k_j, q_g . k_j of j = 2 t, 2 t + 1
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t af[4] = {kf[2 * s], qf[2 * s], kf[2 * s + 1], qf[2 * s + 1]};
      mma16(kq, af, kf[2 * s], kf[2 * s + 1]);
    }
    sn[g][2 * t] = 2 * t < g ? d0 * bk0 * kb * kq[0] : 0.f;
    sn[g][2 * t + 1] = 2 * t + 1 < g ? d1 * bk1 * kb * kq[1] : 0.f;
    const float m0 = 2 * t <= g ? d0 * bk0 * kq[2] : 0.f, m1 = 2 * t + 1 <= g ? d1 * bk1 * kq[3] : 0.f;
    __syncwarp();
    // T by forward substitution, lane % 8 = column
    float x[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      x[i] = i == (lane & 7) ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) x[i] = fmaf(-sn[i][m], x[m], x[i]);
    }
    __syncwarp();
    if (lane < B)
#pragma unroll
      for (int i = 0; i < B; ++i) sn[i][lane] = x[i];
    __syncwarp();
    const float2 tr = *reinterpret_cast<const float2*>(&sn[g][2 * t]);
    __syncwarp();
    const auto over_t = [](float m) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    };
    const Scale ts = scale_of(over_t(fmaxf(fabsf(tr.x), fabsf(tr.y)))), ms = scale_of(over_t(fmaxf(fabsf(m0), fabsf(m1))));
    uint32_t th, tl, mh, ml;
    split2(tr.x * ts.to, tr.y * ts.to, th, tl);
    split2(m0 * ms.to, m1 * ms.to, mh, ml);
    const float tb0 = __shfl_sync(0xffffffffu, ts.back, 8 * t), tb1 = __shfl_sync(0xffffffffu, ts.back, 8 * t + 4);
    const float mb0 = __shfl_sync(0xffffffffu, ms.back, 8 * t), mb1 = __shfl_sync(0xffffffffu, ms.back, 8 * t + 4);

    // X^T = S^T [K; Q]^T
    float top0, top1;
    row_max<2 * KS>(acc, top0, top1);
    const float2 size = make_float2(0.125f * top0, 0.125f * top1);
    const Scale s0 = scale_of(top0), s1 = scale_of(top1);
    float xk[1][4] = {{0.f, 0.f, 0.f, 0.f}}, xq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        split2(acc[2 * s + p][0] * s0.to, acc[2 * s + p][1] * s0.to, hi[2 * p], lo[2 * p]);
        split2(acc[2 * s + p][2] * s1.to, acc[2 * s + p][3] * s1.to, hi[2 * p + 1], lo[2 * p + 1]);
      }
      mma16(xk[0], hi, kf[2 * s], kf[2 * s + 1]);
      mma16(xq, hi, qf[2 * s], qf[2 * s + 1]);
      mma16(xk[0], lo, kf[2 * s], kf[2 * s + 1]);
      mma16(xq, lo, qf[2 * s], qf[2 * s + 1]);
    }
    // R^T, U^T
    {
      const float2 va = delta_unpack2<BF16>(vw[0]), vb = delta_unpack2<BF16>(vw[1]);
      xk[0][0] = va.x - g0 * kb0 * (s0.back * xk[0][0]);
      xk[0][1] = vb.x - g1 * kb1 * (s0.back * xk[0][1]);
      xk[0][2] = va.y - g0 * kb0 * (s1.back * xk[0][2]);
      xk[0][3] = vb.y - g1 * kb1 * (s1.back * xk[0][3]);
    }
    uint32_t hi[4], lo[4];
    float seen0, seen1;
    {
      const float2 va = delta_unpack2<BF16>(vw[0]), vb = delta_unpack2<BF16>(vw[1]);
      const float a0 = 2 * t < nt ? 0.f : INFINITY, b0 = 2 * t + 1 < nt ? 0.f : INFINITY;  // tokens past the last count for nothing
      seen0 = seen_least(fminf(fmaxf(fmaxf(fabsf(va.x), fabsf(xk[0][0])), a0), fmaxf(fmaxf(fabsf(vb.x), fabsf(xk[0][1])), b0)));
      seen1 = seen_least(fminf(fmaxf(fmaxf(fabsf(va.y), fabsf(xk[0][2])), a0), fmaxf(fmaxf(fabsf(vb.y), fabsf(xk[0][3])), b0)));
    }
    row_max<1>(xk, top0, top1);
    const Scale r0 = scale_of(top0), r1 = scale_of(top1);
    split2(xk[0][0] * r0.to, xk[0][1] * r0.to, hi[0], lo[0]);
    split2(xk[0][2] * r1.to, xk[0][3] * r1.to, hi[1], lo[1]);
    float u[1][4] = {{0.f, 0.f, 0.f, 0.f}};
    mma8(u[0], hi, th);
    mma8(u[0], lo, th);
    mma8(u[0], hi, tl);
    u[0][0] *= r0.back * tb0;
    u[0][1] *= r0.back * tb1;
    u[0][2] *= r1.back * tb0;
    u[0][3] *= r1.back * tb1;
    {
      float um0, um1;
      row_max<1>(u, um0, um1);
      const float need0 = fmaxf(top0, um0) * kRange, need1 = fmaxf(top1, um1) * kRange;
      bool lost = __any_sync(0xffffffffu, !(fabsf(u[0][0]) + fabsf(u[0][1]) + fabsf(u[0][2]) + fabsf(u[0][3]) < INFINITY));
      if (__any_sync(0xffffffffu, need0 > seen0 || need1 > seen1)) {
        const float2 least = least_found<1>(xk, size, [al](int i) { return __shfl_sync(0xffffffffu, al, i); });
        lost |= __any_sync(0xffffffffu, need0 > least.x || need1 > least.y) != 0;
      }
      if (lost) {
        warp_steps<2 * KS, BF16>(a, h, row0, nt, col, acc, [t](int n, int e) { return block_row(n, t, e); });
        continue;
      }
      top0 = um0;
      top1 = um1;
    }
    // O^T = X_Q + U^T M^T
    {
      const Scale u0 = scale_of(top0), u1 = scale_of(top1);
      split2(u[0][0] * u0.to, u[0][1] * u0.to, hi[0], lo[0]);
      split2(u[0][2] * u1.to, u[0][3] * u1.to, hi[1], lo[1]);
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      mma8(o, hi, mh);
      mma8(o, lo, mh);
      mma8(o, hi, ml);
      const float f0 = a.scale * qb0, f1 = a.scale * qb1;
      uint16_t* op = static_cast<uint16_t*>(a.out) + row0 * a.o_token + h * a.o_head + col;
      if (2 * t < nt && VQ3_IN(row0 + 2 * t, a.tokens, 14))
        *reinterpret_cast<uint32_t*>(op + 2 * t * a.o_token) =
            delta_pack2<BF16>(f0 * (g0 * (s0.back * xq[0]) + mb0 * (u0.back * o[0])), f0 * (g0 * (s1.back * xq[2]) + mb0 * (u1.back * o[2])));
      if (2 * t + 1 < nt && VQ3_IN(row0 + 2 * t + 1, a.tokens, 14))
        *reinterpret_cast<uint32_t*>(op + (2 * t + 1) * a.o_token) =
            delta_pack2<BF16>(f1 * (g1 * (s0.back * xq[1]) + mb1 * (u0.back * o[1])), f1 * (g1 * (s1.back * xq[3]) + mb1 * (u1.back * o[3])));
    }
    // S^T <- g_8 S^T + (U diag w)^T K
    u[0][0] *= bk0 * e0;
    u[0][1] *= bk1 * e1;
    u[0][2] *= bk0 * e0;
    u[0][3] *= bk1 * e1;
    row_max<1>(u, top0, top1);
    const Scale w0 = scale_of(top0), w1 = scale_of(top1);
    split2(u[0][0] * w0.to, u[0][1] * w0.to, hi[0], lo[0]);
    split2(u[0][2] * w1.to, u[0][3] * w1.to, hi[1], lo[1]);
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n) {
      const uint32_t kt = transposed(kf[n]);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma8(d, hi, kt);
      mma8(d, lo, kt);
      acc[n][0] = fmaf(w0.back, d[0], g8 * acc[n][0]);
      acc[n][1] = fmaf(w0.back, d[1], g8 * acc[n][1]);
      acc[n][2] = fmaf(w1.back, d[2], g8 * acc[n][2]);
      acc[n][3] = fmaf(w1.back, d[3], g8 * acc[n][3]);
    }
  }
  if (rq.out && (rq.n || rq.out != rq.in)) {
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const size_t at = (size_t)block_row(n, t, e) * a.d_v + col;
        if (VQ3_IN(at + 1, n_state, 15)) __stcs(reinterpret_cast<float2*>(rq.out + at), make_float2(acc[n][e], acc[n][2 + e]));
      }
  }
}

template <int DK, bool BF16>
cudaError_t launch_block(const DeltaArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.d_v + kCtaCols - 1) / kCtaCols), (unsigned)a.v_heads, (unsigned)a.requests);
  delta_block_kernel<DK / 16, BF16><<<grid, kBlockThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- single tokens
//
// A CTA takes one request, one value head and 64 columns.
constexpr int kStepThreads = 128;
constexpr int kGroups = kStepThreads / 16;

template <int ROWS, bool BF16>  // d_k = 8 * ROWS
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const __grid_constant__ DeltaArgs a) {
  __shared__ StepShared<ROWS, kGroups, 16> sm;
  delta_steps<ROWS, kGroups, 16, BF16>(a, delta_request(a, blockIdx.z, blockIdx.y), blockIdx.y, blockIdx.x * 64, sm);
}

template <int ROWS, bool BF16>
cudaError_t launch_step(const DeltaArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.d_v + 63) / 64), (unsigned)a.v_heads, (unsigned)a.requests);
  delta_step_kernel<ROWS, BF16><<<grid, kStepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int DK, bool BF16>
cudaError_t launch_of(const DeltaArgs& a, cudaStream_t st) {
  // (without rows states are copied at most, and there is nothing for a tensor map to describe)
  if (!a.tokens || (a.max_new > 0 && a.max_new <= kDeltaStepTokens)) return launch_step<DK / kGroups, BF16>(a, st);
  if (a.max_new > 0 && a.max_new <= (DK == 256 ? kDeltaBlockTokens256 : kDeltaBlockTokens)) return launch_block<DK, BF16>(a, st);
  if constexpr (DK <= 128)
    return launch_delta_wide(a, BF16, st);
  else
    return launch_chunk<BF16>(a, st);
}
template <bool BF16>
cudaError_t launch_delta_type(const DeltaArgs& a, cudaStream_t st) {
  if (a.d_k == 64) return launch_of<64, BF16>(a, st);
  if (a.d_k == 128) return launch_of<128, BF16>(a, st);
  return launch_of<256, BF16>(a, st);
}

}  // namespace

cudaError_t launch_delta_batch(const DeltaArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_delta_type<true>(a, st) : launch_delta_type<false>(a, st);
}

}  // namespace vq3
