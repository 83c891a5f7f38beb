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
// Two kernels, chosen on the host: delta_chunk_kernel for chunks of 8, 16 or 32 tokens on tensor
// cores, delta_step_kernel for one or a few tokens, which streams the state once through registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vq3_internal.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(delta_batch)
namespace {

// ---------------------------------------------------------------- requests

struct Request {
  int first, n;              // its rows, inside the batch whatever the starts are
  const float* in;           // its state of this head, or null: zeros
  float* out;                // or null: not written
};

__device__ __forceinline__ Request delta_request(const DeltaArgs& a, int r, int h) {
  Request q;
  int s = __ldg(a.q_start + r), e = __ldg(a.q_start + r + 1);
  s = s < 0 ? 0 : (s > a.tokens ? a.tokens : s);
  e = e < s ? s : (e > a.tokens ? a.tokens : e);
  q.first = s;
  q.n = e - s;
  const int in = a.slot_in ? __ldg(a.slot_in + r) : -1, out = a.slot_out ? __ldg(a.slot_out + r) : -1;
  const long long head = (long long)h * a.d_k * a.d_v;
  q.in = in >= 0 && in < a.slots ? a.states + in * a.state_slot + head : nullptr;
  q.out = out >= 0 && out < a.slots ? a.states + out * a.state_slot + head : nullptr;
  return q;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (!BF16) return pack_f16(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- chunks on tensor cores
//
// A CTA takes one request, one value head and 64 of its columns and walks the chunks in order. Each of
// its four consumer warps owns 16 columns for the whole call: S^T [16][d_k] stays in registers as the
// accumulators of m16n8k16 tiles, which is also the A operand's layout of the next product S^T [K; Q]^T,
// and R^T, U^T follow in the same way, so no state and no intermediate passes through shared memory.
// Two producer warps take turns with the chunks: they copy K and Q, form T and M, which do not depend on
// the state, and hand them over through a ring of three stages (named barriers, no spinning).
//
// Numbers: the tensor cores multiply FP16. K and Q enter exactly (BF16 rows are brought to a largest
// entry of 2^8 by a power of two, which the factors of the token take back). Every FP32 operand (S, R, U,
// T, M) enters as two FP16 parts, hi and what hi leaves, scaled by a power of two per row of the product
// so that neither part leaves FP16's range: some 22 bits. Where only the 16-bit output depends on
// a product (Q S0, M U) and the type is BF16, hi alone is used: 11 bits under an output of 8.
//
// mma.sync and not tcgen05: at 64 columns (N) the latter takes 48 cycles for 128 x 64 x 16, so a chunk
// of 64 tokens would take 1,900 cycles of products and three trips through tensor and shared memory
// where these four warps take 3,000 and none.
constexpr int kConsumers = 4, kProducers = 2, kStages = 3;
constexpr int kChunkThreads = 32 * (kConsumers + kProducers);
constexpr int kWarpCols = 16, kCtaCols = kWarpCols * kConsumers;
constexpr int kFullBar = 1, kEmptyBar = kFullBar + kStages;
constexpr int kBarThreads = 32 * (kConsumers + 1);

template <int KS, int NN>
struct Stage {
  static constexpr int DK = 16 * KS, C = 8 * NN;
  static constexpr int RS = DK + 8;                              // row of K and Q in halves: 16 bytes past 128
  static constexpr int TS = NN == 4 ? 40 : (NN == 2 ? 24 : 8);   // row of T and M: ldmatrix without conflicts
  static constexpr int kK = 0, kQ = kK + C * RS * 2, kT = kQ + C * RS * 2;
  static constexpr int kM = kT + 2 * C * TS * 2, kC = kM + 2 * C * TS * 2;  // hi, then lo
  static constexpr int kBytes = (kC + (5 * C + 4) * 4 + 127) / 128 * 128;
  // factors per token: of V in R, of K S0 in R, of Q S0 and of M U in O, of U in the state; then g_C
  static constexpr int kFv = 0, kFk = C, kFq = 2 * C, kFm = 3 * C, kFw = 4 * C, kFg = 5 * C;
  static constexpr int NS = C + 4;                               // row of N in floats
  static constexpr int kScratch = C * NS * 4;                    // per producer: ratios, then N
  static constexpr int kTotal = kStages * kBytes + kProducers * kScratch;
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
__device__ __forceinline__ uint32_t ldsm1t(uint32_t at) {
  uint32_t r;
  asm volatile("ldmatrix.sync.aligned.m8n8.x1.trans.shared.b16 {%0}, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t ldsm1(uint32_t at) {
  uint32_t r;
  asm volatile("ldmatrix.sync.aligned.m8n8.x1.shared.b16 {%0}, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}

// The power of two that brings m >= 0 to [2^8, 2^9), and its inverse; exponents are kept inside FP32's
// normal range (an infinite or NaN m gives finite factors: the values themselves carry it on).
struct Scale {
  float to, back;
};
__device__ __forceinline__ Scale scale_of(float m) {
  int e = (int)(__float_as_uint(m) >> 23);
  e = e < 9 ? 9 : e;
  return Scale{__uint_as_float((uint32_t)(262 - e) << 23), __uint_as_float((uint32_t)(e - 8) << 23)};
}
// Two FP32 values as FP16 pairs: hi, and what hi leaves.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16(x, y);
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  lo = pack_f16(x - h.x, y - h.y);
}
// Rows g and g + 8 of NN accumulator tiles: the largest magnitude over the row (lanes of one g).
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
template <int KS, int NN, bool BF16>
__device__ __forceinline__ void produce(const DeltaArgs& a, const Request& rq, int h, int t0, unsigned char* st,
                                        float* scratch, int lane) {
  using L = Stage<KS, NN>;
  constexpr int C = L::C, RS = L::RS, DK = L::DK, TS = L::TS, NS = L::NS;
  const int nt = rq.n - t0 < C ? rq.n - t0 : C;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t sk = smem_of(st + L::kK), sq = smem_of(st + L::kQ);
  // rows of K and Q, tokens past the last zero
  const int hq = h / a.group;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + (long long)(rq.first + t0) * a.k_token + hq * a.k_head;
  const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (long long)(rq.first + t0) * a.q_token + hq * a.q_head;
#pragma unroll 4
  for (int i = lane; i < C * (DK / 8); i += 32) {
    const int row = i / (DK / 8), c = i % (DK / 8);
    const uint32_t off = (uint32_t)(row * RS + c * 8) * 2u;
    if (row < nt && VQ3_IN(rq.first + t0 + row, a.tokens, 1)) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sk + off), "l"(kp + row * a.k_token + c * 8) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sq + off), "l"(qp + row * a.q_token + c * 8) : "memory");
    } else {
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sk + off), "r"(0u) : "memory");
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(sq + off), "r"(0u) : "memory");
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  float al = 1.f, be = 0.f;  // lane = token
  if (lane < nt && VQ3_IN(rq.first + t0 + lane, a.tokens, 2)) {
    al = __ldg(a.alpha + (long long)(rq.first + t0 + lane) * a.alpha_token + h);
    be = __ldg(a.beta + (long long)(rq.first + t0 + lane) * a.beta_token + h);
  }
  // ratios D[i][j] = a_(j+1) ... a_i (lane = j), the running product g_i, and g_C / g_j
  float r = 1.f, gam = 1.f, gi = 1.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const float ai = __shfl_sync(0xffffffffu, al, i);
    gam *= ai;
    if (i == lane) gi = gam;
    if (i > lane) r *= ai;
    if (lane < C) scratch[i * NS + lane] = r;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  // BF16 rows to FP16, each scaled by a power of two (lane = row: 16 bytes past 128 a row, no conflicts)
  float kb = 1.f, qb = 1.f;
  if constexpr (BF16) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (lane < C) {
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
        const __nv_bfloat162 f = __float2bfloat162_rn(s.to);
#pragma unroll 4
        for (int c = 0; c < DK / 8; ++c) {
          const uint4 w = row[c];
          uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e]), f);
            const float2 y = unpack2<true>(*reinterpret_cast<const uint32_t*>(&x));
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
    uint32_t kf[NN][2], qf[NN][2];
#pragma unroll
    for (int b = 0; b < NN; ++b) {
      // matrices: K columns 0-7, 8-15 of the step, Q the same
      uint32_t f[4];
      ldsm4(f, (lane < 16 ? sk : sq) + (uint32_t)((8 * b + (lane & 7)) * RS + 16 * s + ((lane >> 3) & 1) * 8) * 2u);
      kf[b][0] = f[0];
      kf[b][1] = f[1];
      qf[b][0] = f[2];
      qf[b][1] = f[3];
    }
    int i = 0;
#pragma unroll
    for (int b = 0; b < NN; ++b) {
      const uint32_t af[4] = {kf[b][0], qf[b][0], kf[b][1], qf[b][1]};
#pragma unroll
      for (int n = 0; n <= b; ++n, ++i) mma16(kq[i], af, kf[n][0], kf[n][1]);
    }
  }
  // N over the ratios in scratch (each thread where it read them); M, rows scaled, as FP16 parts
  uint16_t* mhi = reinterpret_cast<uint16_t*>(st + L::kM);
  uint16_t* mlo = mhi + C * TS;
  const float bk = be * kb;  // b_j and the factor of k_j
  float fm = 0.f;
  int i = 0;
#pragma unroll
  for (int b = 0; b < NN; ++b) {
    const float ki = __shfl_sync(0xffffffffu, kb, 8 * b + g);
    float m[NN][2];
    float top = 0.f;
#pragma unroll
    for (int n = 0; n <= b; ++n, ++i) {
      const int row = 8 * b + g, col = 8 * n + 2 * t;
      const float b0 = __shfl_sync(0xffffffffu, bk, col), b1 = __shfl_sync(0xffffffffu, bk, col + 1);
      float2* at = reinterpret_cast<float2*>(scratch + row * NS + col);
      const float2 d = *at;
      const float d0 = d.x * b0, d1 = d.y * b1;
      *at = make_float2(col < row ? d0 * ki * kq[i][0] : 0.f, col + 1 < row ? d1 * ki * kq[i][1] : 0.f);
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
      if constexpr (!BF16) *reinterpret_cast<uint32_t*>(mlo + (8 * b + g) * TS + 8 * n + 2 * t) = lo;
    }
    const float back = __shfl_sync(0xffffffffu, s.back, (lane & 7) * 4);  // of row 8 b + lane % 8
    if (lane >> 3 == b) fm = back;
  }
  __syncwarp();
  // T = (I + N)^-1 by forward substitution, lane = column
  float x[C];
#pragma unroll
  for (int k = 0; k < C; ++k) x[k] = 0.f;
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int m = 0; m < k; m += 4) {
      const float4 nv = *reinterpret_cast<const float4*>(scratch + k * NS + m);
      s0 = fmaf(nv.x, x[m], s0);
      s1 = fmaf(nv.y, x[m + 1], s1);
      s2 = fmaf(nv.z, x[m + 2], s2);
      s3 = fmaf(nv.w, x[m + 3], s3);
    }
    x[k] = (k == lane ? 1.f : 0.f) - ((s0 + s1) + (s2 + s3));
    top = fmaxf(top, fabsf(x[k]));
  }
  const Scale ts = scale_of(top);
  if (lane < C) {  // column j of T as row j
    uint4* thi = reinterpret_cast<uint4*>(st + L::kT + lane * TS * 2);
    uint4* tlo = reinterpret_cast<uint4*>(st + L::kT + (C + lane) * TS * 2);
#pragma unroll
    for (int k = 0; k < C; k += 8) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(x[k + 2 * e] * ts.to, x[k + 2 * e + 1] * ts.to, hi[e], lo[e]);
      thi[k / 8] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      tlo[k / 8] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    float* f = reinterpret_cast<float*>(st + L::kC);
    f[L::kFv + lane] = ts.back;
    f[L::kFk + lane] = gi * kb * ts.back;
    f[L::kFq + lane] = a.scale * gi * qb;
    f[L::kFm + lane] = a.scale * qb * fm;
    f[L::kFw + lane] = bk * r;
    if (lane == 0) f[L::kFg] = gam;
  }
  __syncwarp();
}

// ---- consumer: one chunk against this warp's 16 columns; acc: S^T, row g column 2g, row g + 8 column 2g + 1
template <int KS, int NN, bool BF16>
__device__ __forceinline__ void consume(float (&acc)[2 * KS][4], const uint32_t (&vw)[NN][2], const unsigned char* st,
                                        float (&o)[NN][4], int lane) {
  using L = Stage<KS, NN>;
  constexpr int C = L::C, RS = L::RS, TS = L::TS;
  constexpr int K2 = NN == 1 ? 1 : NN / 2;  // steps of 16 tokens (one of 8 for NN = 1)
  const int t = lane & 3;
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
    if constexpr (NN == 1) {
      // matrices: K columns 0-7, 8-15 of the step, Q the same
      uint32_t b[4];
      ldsm4(b, (lane < 16 ? sk : sq) + (uint32_t)((lane & 7) * RS + 16 * s + ((lane >> 3) & 1) * 8) * 2u);
      mma16(xk[0], hi, b[0], b[1]);
      mma16(xq[0], hi, b[2], b[3]);
      mma16(xk[0], lo, b[0], b[1]);
      if constexpr (!BF16) mma16(xq[0], lo, b[2], b[3]);
    } else {
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
        if constexpr (!BF16) {
          mma16(xq[n], lo, b[0], b[1]);
          mma16(xq[n + 1], lo, b[2], b[3]);
        }
      }
    }
  }
  // R^T = V^T - X_K, times the factor of T's column
#pragma unroll
  for (int n = 0; n < NN; ++n) {
    const float2 fv = *reinterpret_cast<const float2*>(f + L::kFv + 8 * n + 2 * t);
    const float2 fk = *reinterpret_cast<const float2*>(f + L::kFk + 8 * n + 2 * t);
    const float2 va = unpack2<BF16>(vw[n][0]), vb = unpack2<BF16>(vw[n][1]);
    xk[n][0] = va.x * fv.x - fk.x * (s0.back * xk[n][0]);
    xk[n][1] = vb.x * fv.y - fk.y * (s0.back * xk[n][1]);
    xk[n][2] = va.y * fv.x - fk.x * (s1.back * xk[n][2]);
    xk[n][3] = vb.y * fv.y - fk.y * (s1.back * xk[n][3]);
  }
  // U^T = R^T T^T
  row_max<NN>(xk, m0, m1);
  const Scale r0 = scale_of(m0), r1 = scale_of(m1);
  float u[NN][4];
#pragma unroll
  for (int n = 0; n < NN; ++n) u[n][0] = u[n][1] = u[n][2] = u[n][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < K2; ++ks) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int p = 0; p < (NN == 1 ? 1 : 2); ++p) {
      split2(xk[2 * ks + p][0] * r0.to, xk[2 * ks + p][1] * r0.to, hi[2 * p], lo[2 * p]);
      split2(xk[2 * ks + p][2] * r1.to, xk[2 * ks + p][3] * r1.to, hi[2 * p + 1], lo[2 * p + 1]);
    }
    if constexpr (NN == 1) {
      const uint32_t bh = ldsm1t(sT + (lane & 7) * TS * 2), bl = ldsm1t(sT + (C + (lane & 7)) * TS * 2);
      mma8(u[0], hi, bh);
      mma8(u[0], lo, bh);
      mma8(u[0], hi, bl);
    } else {
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
  }
#pragma unroll
  for (int n = 0; n < NN; ++n) {
    u[n][0] *= r0.back;
    u[n][1] *= r0.back;
    u[n][2] *= r1.back;
    u[n][3] *= r1.back;
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
      for (int p = 0; p < (NN == 1 ? 1 : 2); ++p) {
        split2(w[2 * ks + p][0] * w0.to, w[2 * ks + p][1] * w0.to, hi[ks][2 * p], lo[ks][2 * p]);
        split2(w[2 * ks + p][2] * w1.to, w[2 * ks + p][3] * w1.to, hi[ks][2 * p + 1], lo[ks][2 * p + 1]);
      }
    const float gC = f[L::kFg];
    if constexpr (NN == 1) {
#pragma unroll
      for (int n = 0; n < 2 * KS; n += 4) {
        uint32_t b[4];  // matrices: 8 tokens (rows) at d_k 8n, 8(n + 1), ...
        ldsm4t(b, sk + (uint32_t)((lane & 7) * RS + 8 * n + (lane >> 3) * 8) * 2u);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma8(d, hi[0], b[p]);
          mma8(d, lo[0], b[p]);
          acc[n + p][0] = fmaf(w0.back, d[0], gC * acc[n + p][0]);
          acc[n + p][1] = fmaf(w0.back, d[1], gC * acc[n + p][1]);
          acc[n + p][2] = fmaf(w1.back, d[2], gC * acc[n + p][2]);
          acc[n + p][3] = fmaf(w1.back, d[3], gC * acc[n + p][3]);
        }
      }
    } else {
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
  }
  // O^T = X_Q + U^T M^T
  row_max<NN>(u, m0, m1);
  const Scale u0 = scale_of(m0), u1 = scale_of(m1);
#pragma unroll
  for (int n = 0; n < NN; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < K2; ++ks) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int p = 0; p < (NN == 1 ? 1 : 2); ++p) {
      split2(u[2 * ks + p][0] * u0.to, u[2 * ks + p][1] * u0.to, hi[2 * p], lo[2 * p]);
      split2(u[2 * ks + p][2] * u1.to, u[2 * ks + p][3] * u1.to, hi[2 * p + 1], lo[2 * p + 1]);
    }
    if constexpr (NN == 1) {
      const uint32_t bh = ldsm1(sM + (lane & 7) * TS * 2);
      mma8(o[0], hi, bh);
      if constexpr (!BF16) {
        mma8(o[0], lo, bh);
        mma8(o[0], hi, ldsm1(sM + (C + (lane & 7)) * TS * 2));
      }
    } else {
#pragma unroll
      for (int n = 2 * ks; n < NN; ++n) {
        // matrices: block n (rows) at tokens 0-7, 8-15 of the step, hi, then lo
        uint32_t b[4];
        ldsm4(b, sM + (uint32_t)((((BF16 ? 0 : lane >> 4)) * C + 8 * n + (lane & 7)) * TS + 16 * ks + ((lane >> 3) & 1) * 8) * 2u);
        mma16(o[n], hi, b[0], b[1]);
        if constexpr (!BF16) {
          mma16(o[n], lo, b[0], b[1]);
          mma16(o[n], hi, b[2], b[3]);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NN; ++n) {
    const float2 fq = *reinterpret_cast<const float2*>(f + L::kFq + 8 * n + 2 * t);
    const float2 fm = *reinterpret_cast<const float2*>(f + L::kFm + 8 * n + 2 * t);
    o[n][0] = fq.x * (s0.back * xq[n][0]) + fm.x * (u0.back * o[n][0]);
    o[n][1] = fq.y * (s0.back * xq[n][1]) + fm.y * (u0.back * o[n][1]);
    o[n][2] = fq.x * (s1.back * xq[n][2]) + fm.x * (u1.back * o[n][2]);
    o[n][3] = fq.y * (s1.back * xq[n][3]) + fm.y * (u1.back * o[n][3]);
  }
}

template <int KS, int NN, bool BF16>
__global__ void __launch_bounds__(kChunkThreads, KS <= 8 ? 2 : 1) delta_chunk_kernel(const __grid_constant__ DeltaArgs a) {
  using L = Stage<KS, NN>;
  constexpr int C = L::C;
  extern __shared__ __align__(128) unsigned char sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y;
  const Request rq = delta_request(a, blockIdx.z, h);
  const int chunks = (rq.n + C - 1) / C;

  if (warp >= kConsumers) {
    const int p = warp - kConsumers;
    float* scratch = reinterpret_cast<float*>(sm + kStages * L::kBytes + p * L::kScratch);
    for (int c = p; c < chunks; c += kProducers) {
      const int s = c % kStages;
      if (c >= kStages) bar_sync(kEmptyBar + s, kBarThreads);  // the consumers are done with chunk c - kStages
      produce<KS, NN, BF16>(a, rq, h, c * C, sm + s * L::kBytes, scratch, lane);
      bar_arrive(kFullBar + s, kBarThreads);
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
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + (long long)rq.first * a.v_token + h * a.v_head + col;
  uint16_t* op = static_cast<uint16_t*>(a.out) + (long long)rq.first * a.o_token + h * a.o_head + col;
  uint32_t vw[NN][2];
  const auto load_v = [&](int t0) {
#pragma unroll
    for (int n = 0; n < NN; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = t0 + 8 * n + 2 * t + e;
        vw[n][e] = on && tok < rq.n && VQ3_IN(rq.first + tok, a.tokens, 4)
                       ? __ldg(reinterpret_cast<const uint32_t*>(vp + tok * a.v_token)) : 0u;
      }
  };
  load_v(0);
  for (int c = 0; c < chunks; ++c) {
    const int s = c % kStages;
    bar_sync(kFullBar + s, kBarThreads);
    if (on) {
      float o[NN][4];
      consume<KS, NN, BF16>(acc, vw, sm + s * L::kBytes, o, lane);
#pragma unroll
      for (int n = 0; n < NN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = c * C + 8 * n + 2 * t + e;
          if (tok < rq.n && VQ3_IN(rq.first + tok, a.tokens, 5))
            *reinterpret_cast<uint32_t*>(op + tok * a.o_token) = pack2<BF16>(o[n][e], o[n][2 + e]);
        }
      load_v((c + 1) * C);
    }
    if (c + kStages < chunks) bar_arrive(kEmptyBar + s, kBarThreads);
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

template <int KS, int NN, bool BF16>
cudaError_t launch_chunk(const DeltaArgs& a, cudaStream_t st) {
  constexpr int smem = Stage<KS, NN>::kTotal;
  const cudaError_t e =
      cudaFuncSetAttribute(delta_chunk_kernel<KS, NN, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.d_v + kCtaCols - 1) / kCtaCols), (unsigned)a.v_heads, (unsigned)a.requests);
  delta_chunk_kernel<KS, NN, BF16><<<grid, kChunkThreads, smem, st>>>(a);
  return cudaGetLastError();
}
template <int KS, bool BF16>
cudaError_t launch_chunk_of(const DeltaArgs& a, cudaStream_t st) {
  if (a.max_new > 0 && a.max_new <= 8) return launch_chunk<KS, 1, BF16>(a, st);
  if (a.max_new > 0 && a.max_new <= 16) return launch_chunk<KS, 2, BF16>(a, st);
  return launch_chunk<KS, 4, BF16>(a, st);
}

// ---------------------------------------------------------------- single tokens
//
// A CTA takes one request, one value head and 64 columns: 8 groups of 16 lanes hold every eighth row of S,
// 4 columns a lane, in registers. With x = S^T k and y = S^T q of the OLD state both products need one pass
// over it and one exchange between the groups:
//     u = b (v - a x),   S <- a S + k u^T,   o = scale (a y + (k . q) u).
// All in FP32. Bound by the state's bytes, read once and written once.
constexpr int kStepThreads = 128;
constexpr int kGroups = kStepThreads / 16;

template <int ROWS, bool BF16>  // d_k = 8 * ROWS
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const __grid_constant__ DeltaArgs a) {
  constexpr int DK = kGroups * ROWS;
  __shared__ float2 kqs[2][DK];                              // (k, q) of the token
  __shared__ float4 part[2][2][kStepThreads / 32][16];       // x and y by warp
  __shared__ float dots[2][kStepThreads / 32];               // k . q by warp
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = tid >> 4, cl = tid & 15;
  const int h = blockIdx.y, hq = h / a.group;
  const Request rq = delta_request(a, blockIdx.z, h);
  const int col = blockIdx.x * 64 + cl * 4;
  const bool on = col < a.d_v;
  const size_t n_state = (size_t)a.d_k * a.d_v;
  float4 S[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const size_t at = (size_t)(i * kGroups + grp) * a.d_v + col;
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on && rq.in && VQ3_IN(at + 3, n_state, 7)) S[i] = __ldcs(reinterpret_cast<const float4*>(rq.in + at));
  }
  for (int t = 0; t < rq.n; ++t) {
    const int b = t & 1;
    const long long row = rq.first + t;
    const bool in = VQ3_IN(row, a.tokens, 8);
    const uint16_t* kp = static_cast<const uint16_t*>(a.k) + row * a.k_token + hq * a.k_head;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + row * a.q_token + hq * a.q_head;
    float dot = 0.f;
    for (int d = tid * 2; d < DK; d += 2 * kStepThreads) {
      const float2 k2 = in ? unpack2<BF16>(__ldg(reinterpret_cast<const uint32_t*>(kp + d))) : make_float2(0.f, 0.f);
      const float2 q2 = in ? unpack2<BF16>(__ldg(reinterpret_cast<const uint32_t*>(qp + d))) : make_float2(0.f, 0.f);
      kqs[b][d] = make_float2(k2.x, q2.x);
      kqs[b][d + 1] = make_float2(k2.y, q2.y);
      dot += k2.x * q2.x + k2.y * q2.y;
    }
    const float al = in ? __ldg(a.alpha + row * a.alpha_token + h) : 1.f;
    const float be = in ? __ldg(a.beta + row * a.beta_token + h) : 0.f;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (on && in) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.v) + row * a.v_token + h * a.v_head + col));
      const float2 v0 = unpack2<BF16>(w.x), v1 = unpack2<BF16>(w.y);
      v[0] = v0.x;
      v[1] = v0.y;
      v[2] = v1.x;
      v[3] = v1.y;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (lane == 0) dots[b][warp] = dot;
    __syncthreads();
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float2 kq = kqs[b][i * kGroups + grp];
      x.x = fmaf(kq.x, S[i].x, x.x);
      x.y = fmaf(kq.x, S[i].y, x.y);
      x.z = fmaf(kq.x, S[i].z, x.z);
      x.w = fmaf(kq.x, S[i].w, x.w);
      y.x = fmaf(kq.y, S[i].x, y.x);
      y.y = fmaf(kq.y, S[i].y, y.y);
      y.z = fmaf(kq.y, S[i].z, y.z);
      y.w = fmaf(kq.y, S[i].w, y.w);
    }
    const auto both = [](float f) { return f + __shfl_xor_sync(0xffffffffu, f, 16); };
    x = make_float4(both(x.x), both(x.y), both(x.z), both(x.w));
    y = make_float4(both(y.x), both(y.y), both(y.z), both(y.w));
    if (lane < 16) {
      part[b][0][warp][cl] = x;
      part[b][1][warp][cl] = y;
    }
    __syncthreads();
    x = y = make_float4(0.f, 0.f, 0.f, 0.f);
    float kq = 0.f;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) {
      const float4 px = part[b][0][w][cl], py = part[b][1][w][cl];
      x = make_float4(x.x + px.x, x.y + px.y, x.z + px.z, x.w + px.w);
      y = make_float4(y.x + py.x, y.y + py.y, y.z + py.z, y.w + py.w);
      kq += dots[b][w];
    }
    const float4 u = make_float4(be * (v[0] - al * x.x), be * (v[1] - al * x.y), be * (v[2] - al * x.z), be * (v[3] - al * x.w));
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float k = kqs[b][i * kGroups + grp].x;
      S[i] = make_float4(fmaf(k, u.x, al * S[i].x), fmaf(k, u.y, al * S[i].y), fmaf(k, u.z, al * S[i].z),
                         fmaf(k, u.w, al * S[i].w));
    }
    if (grp == 0 && on && in) {
      const uint2 w = make_uint2(pack2<BF16>(a.scale * fmaf(kq, u.x, al * y.x), a.scale * fmaf(kq, u.y, al * y.y)),
                                 pack2<BF16>(a.scale * fmaf(kq, u.z, al * y.z), a.scale * fmaf(kq, u.w, al * y.w)));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.o_token + h * a.o_head + col) = w;
    }
  }
  if (on && rq.out && (rq.n || rq.out != rq.in)) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const size_t at = (size_t)(i * kGroups + grp) * a.d_v + col;
      if (VQ3_IN(at + 3, n_state, 9)) __stcs(reinterpret_cast<float4*>(rq.out + at), S[i]);
    }
  }
}

template <int ROWS, bool BF16>
cudaError_t launch_step(const DeltaArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.d_v + 63) / 64), (unsigned)a.v_heads, (unsigned)a.requests);
  delta_step_kernel<ROWS, BF16><<<grid, kStepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_delta_type(const DeltaArgs& a, cudaStream_t st) {
  const bool step = a.max_new > 0 && a.max_new <= kDeltaStepTokens;
  switch (a.d_k) {
    case 64: return step ? launch_step<8, BF16>(a, st) : launch_chunk_of<4, BF16>(a, st);
    case 128: return step ? launch_step<16, BF16>(a, st) : launch_chunk_of<8, BF16>(a, st);
    default: return step ? launch_step<32, BF16>(a, st) : launch_chunk_of<16, BF16>(a, st);
  }
}

}  // namespace

cudaError_t launch_delta_batch(const DeltaArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_delta_type<true>(a, st) : launch_delta_type<false>(a, st);
}

}  // namespace vq3
