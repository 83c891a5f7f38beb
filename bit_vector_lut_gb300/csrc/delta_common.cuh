// What the delta-rule kernels for packed requests share: a request's rows and state, number formats, and the
// single-token step. A file that includes it defines its bounds-check record first.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vq3_internal.h"

namespace vq3 {

struct DeltaRequest {
  int first, n;              // its rows, inside the batch whatever the starts are
  const float* in;           // its state of this head, or null: zeros
  float* out;                // or null: not written
};

__device__ __forceinline__ int2 delta_request_rows(const DeltaArgs& a, int r) {  // the first and how many
  int s = __ldg(a.q_start + r), e = __ldg(a.q_start + r + 1);
  s = s < 0 ? 0 : (s > a.tokens ? a.tokens : s);
  e = e < s ? s : (e > a.tokens ? a.tokens : e);
  return make_int2(s, e - s);
}
__device__ __forceinline__ DeltaRequest delta_request(const DeltaArgs& a, int r, int h) {
  DeltaRequest q;
  const int2 rows = delta_request_rows(a, r);
  q.first = rows.x;
  q.n = rows.y;
  const int in = a.slot_in ? __ldg(a.slot_in + r) : -1, out = a.slot_out ? __ldg(a.slot_out + r) : -1;
  const long long head = (long long)h * a.d_k * a.d_v;
  q.in = in >= 0 && in < a.slots ? a.states + in * a.state_slot + head : nullptr;
  q.out = out >= 0 && out < a.slots ? a.states + out * a.state_slot + head : nullptr;
  return q;
}

template <bool BF16>
__device__ __forceinline__ float2 delta_unpack2(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t delta_pack2(float lo, float hi) {
  if constexpr (!BF16) return pack_f16(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The power of two that brings m >= 0 to [2^TO, 2^(TO + 1)), and its inverse: at 2^14 two FP16 parts hold what is above
// 2^-17 of the largest value with 22 bits, the rest to 2^-39 of it; exponents are kept inside FP32's
// normal range (an infinite or NaN m gives finite factors: the values themselves carry it on).
struct Scale {
  float to, back;
};
template <int TO = 14>
__device__ __forceinline__ Scale scale_of(float m) {
  int e = (int)(__float_as_uint(m) >> 23);
  e = e < TO + 1 ? TO + 1 : e;
  return Scale{__uint_as_float((uint32_t)(254 + TO - e) << 23), __uint_as_float((uint32_t)(e - TO) << 23)};
}
// Where tokens of a chunk share a power of two, what a token adds has to be seen beside what its column holds already (of
// the values, the state and earlier tokens, as the gates leave them), or tokens behind it, which it cannot see, cost it
// its bits (T's and M's entries share one, too: nothing new behind a small gate is as bad as something small);
// and matrix products bring infinities and NaN of later tokens to earlier ones as 0 * inf. So a chunk is gone through again
// token by token where R or U has a value of 2^20 times that size, or one that is not finite: each is right to 2^-19 of what
// the token sees. Seldom: not for values of like size, nor for small ones behind large ones.
constexpr float kRange = 0x1p-20f;
// Entries of T = (I + N)^-1 are below this for keys and strengths that do not let the state grow; its columns share
// a power of two, too.
constexpr float kGrown = 4.f;
// Two FP32 operations an instruction.
__device__ __forceinline__ unsigned long long pair_bits(float2 x) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
  return r;
}
__device__ __forceinline__ float2 bits_pair(unsigned long long r) {
  float2 y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(y.x), "=f"(y.y) : "l"(r));
  return y;
}
__device__ __forceinline__ unsigned long long mul_bits(unsigned long long x, unsigned long long y) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ unsigned long long fma_bits(unsigned long long x, unsigned long long y, unsigned long long a) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(a));
  return r;
}
__device__ __forceinline__ float2 mul_pair(float2 x, float2 y) { return bits_pair(mul_bits(pair_bits(x), pair_bits(y))); }
__device__ __forceinline__ float2 fma_pair(float2 x, float2 y, float2 a) {
  return bits_pair(fma_bits(pair_bits(x), pair_bits(y), pair_bits(a)));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mul_pair(float2 x, float m) { return mul_pair(x, both(m)); }
__device__ __forceinline__ float2 fma_pair(float2 x, float m, float2 a) { return fma_pair(x, both(m), a); }
__device__ __forceinline__ float max_pair(float m, float2 x) { return fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y))); }
// Two FP32 values as FP16 pairs: hi, and what hi leaves.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16(x.x, x.y);
  const float2 l = fma_pair(__half22float2(*reinterpret_cast<const __half2*>(&hi)), -1.f, x);
  lo = pack_f16(l.x, l.y);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) { split2(make_float2(x, y), hi, lo); }

// ---------------------------------------------------------------- single tokens
//
// GROUPS groups of LANES lanes; a lane holds 4 columns of every GROUPS-th row of S in registers. With x = S^T k and
// y = S^T q of the OLD state both products need one pass over it and one exchange between the groups:
//     u = b (v - a x),   S <- a S + k u^T,   o = scale (a y + (k . q) u).
// All in FP32. Bound by the state's bytes, read once and written once: 64 users' single tokens, 48 heads of 128 x 128,
// 60.5 us (99% of a copy's rate).
template <int ROWS, int GROUPS, int LANES>
struct StepShared {
  static constexpr int kWarps = GROUPS * LANES / 32;
  float2 kq[2][GROUPS * ROWS];       // (k, q) of the token
  float4 part[2][2][kWarps][LANES];  // x and y by warp
  float dots[2][kWarps];             // k . q by warp
};
template <int ROWS, int GROUPS, int LANES, bool BF16>
__device__ __forceinline__ void delta_steps(const DeltaArgs& a, const DeltaRequest& rq, int h, int col0,
                                            StepShared<ROWS, GROUPS, LANES>& sm) {
  constexpr int DK = GROUPS * ROWS, kThreads = GROUPS * LANES, kWarps = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = tid / LANES, cl = tid % LANES;
  const int hq = h / a.group, col = col0 + cl * 4;
  const bool on = col < a.d_v;
  const size_t n_state = (size_t)a.d_k * a.d_v;
  float4 S[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const size_t at = (size_t)(i * GROUPS + grp) * a.d_v + col;
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
    for (int d = tid * 2; d < DK; d += 2 * kThreads) {
      const float2 k2 = in ? delta_unpack2<BF16>(__ldg(reinterpret_cast<const uint32_t*>(kp + d))) : make_float2(0.f, 0.f);
      const float2 q2 = in ? delta_unpack2<BF16>(__ldg(reinterpret_cast<const uint32_t*>(qp + d))) : make_float2(0.f, 0.f);
      sm.kq[b][d] = make_float2(k2.x, q2.x);
      sm.kq[b][d + 1] = make_float2(k2.y, q2.y);
      dot += k2.x * q2.x + k2.y * q2.y;
    }
    const float al = in ? __ldg(a.alpha + row * a.alpha_token + h) : 1.f;
    const float be = in ? __ldg(a.beta + row * a.beta_token + h) : 0.f;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (on && in) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.v) + row * a.v_token + h * a.v_head + col));
      const float2 v0 = delta_unpack2<BF16>(w.x), v1 = delta_unpack2<BF16>(w.y);
      v[0] = v0.x;
      v[1] = v0.y;
      v[2] = v1.x;
      v[3] = v1.y;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (lane == 0) sm.dots[b][warp] = dot;
    __syncthreads();
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float2 kq = sm.kq[b][i * GROUPS + grp];
      x.x = fmaf(kq.x, S[i].x, x.x);
      x.y = fmaf(kq.x, S[i].y, x.y);
      x.z = fmaf(kq.x, S[i].z, x.z);
      x.w = fmaf(kq.x, S[i].w, x.w);
      y.x = fmaf(kq.y, S[i].x, y.x);
      y.y = fmaf(kq.y, S[i].y, y.y);
      y.z = fmaf(kq.y, S[i].z, y.z);
      y.w = fmaf(kq.y, S[i].w, y.w);
    }
#pragma unroll
    for (int d = LANES; d < 32; d <<= 1) {
      const auto sum = [d](float f) { return f + __shfl_xor_sync(0xffffffffu, f, d); };
      x = make_float4(sum(x.x), sum(x.y), sum(x.z), sum(x.w));
      y = make_float4(sum(y.x), sum(y.y), sum(y.z), sum(y.w));
    }
    if (lane < LANES) {
      sm.part[b][0][warp][cl] = x;
      sm.part[b][1][warp][cl] = y;
    }
    __syncthreads();
    x = y = make_float4(0.f, 0.f, 0.f, 0.f);
    float kq = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 px = sm.part[b][0][w][cl], py = sm.part[b][1][w][cl];
      x = make_float4(x.x + px.x, x.y + px.y, x.z + px.z, x.w + px.w);
      y = make_float4(y.x + py.x, y.y + py.y, y.z + py.z, y.w + py.w);
      kq += sm.dots[b][w];
    }
    const float4 u = make_float4(be * (v[0] - al * x.x), be * (v[1] - al * x.y), be * (v[2] - al * x.z), be * (v[3] - al * x.w));
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float k = sm.kq[b][i * GROUPS + grp].x;
      S[i] = make_float4(fmaf(k, u.x, al * S[i].x), fmaf(k, u.y, al * S[i].y), fmaf(k, u.z, al * S[i].z),
                         fmaf(k, u.w, al * S[i].w));
    }
    if (grp == 0 && on && in) {
      const uint2 w =
          make_uint2(delta_pack2<BF16>(a.scale * fmaf(kq, u.x, al * y.x), a.scale * fmaf(kq, u.y, al * y.y)),
                     delta_pack2<BF16>(a.scale * fmaf(kq, u.z, al * y.z), a.scale * fmaf(kq, u.w, al * y.w)));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.o_token + h * a.o_head + col) = w;
    }
  }
  if (on && rq.out && (rq.n || rq.out != rq.in)) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const size_t at = (size_t)(i * GROUPS + grp) * a.d_v + col;
      if (VQ3_IN(at + 3, n_state, 9)) __stcs(reinterpret_cast<float4*>(rq.out + at), S[i]);
    }
  }
}

}  // namespace vq3
