// The cache append with the position rotation on the way: pairs (x1, x2) of the first 2 * half entries of every
// query and key head are turned by position * freq,
//     (x1 cos - x2 sin, x2 cos + x1 sin),
// queries to their output, keys and values into the pages.
//
// Angles: freq / (2 pi) as a 64-bit fraction of a turn (from two FP64 parts), times the position modulo one turn in
// integers: right for any position, where an FP32 product is off by whole radians from some 10^7 on (by 2^-8 radians at
// 10^5), and for any frequency up to 2^40, where FP64 alone would be off by 2^-25 of a turn per radian a position.
//
// A CTA takes 4 tokens (one where tokens are few), makes their table of (cos, sin) once for all heads, and walks
// the heads' items: 2 x 16 bytes a thread, both partners of 8 pairs, so that a row may be turned in place. Bound by
// HBM: some 16,000 tokens of 32 + 8 heads of 128, BF16, 65 us (90% of a copy's rate).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vq3_internal.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(rotary)
namespace {

constexpr int kRotThreads = 256;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 ldg_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

template <int TILE, bool BF16>
__global__ void __launch_bounds__(kRotThreads, 4) kv_append_rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ unsigned long long turns[128];
  __shared__ float2 table[TILE][128];  // (cos, sin)
  __shared__ int pos[TILE];
  __shared__ long long slot[TILE];
  const int tid = threadIdx.x, t0 = blockIdx.x * TILE;
  const AppendArgs& kv = a.kv;
  const long long limit = (long long)kv.n_pages << kv.page_shift;
  if (tid < a.half) {
    // freq / (2 pi) in two FP64 parts, their distance from a whole number as 64-bit fractions
    constexpr double kInv = 0.15915494309189535, kRest = -9.839338337591243e-18, kOne = 18446744073709551616.0;
    const double f = (double)__ldg(a.freq + tid), x = f * kInv, rest = fma(f, kInv, -x) + f * kRest;
    turns[tid] = (unsigned long long)(long long)((x - rint(x)) * kOne) + (unsigned long long)(long long)(rest * kOne);
  }
  if (tid < TILE) {
    const bool in = t0 + tid < kv.tokens;
    pos[tid] = in ? __ldg(a.positions + t0 + tid) : -1;
    slot[tid] = in ? __ldg(kv.slots + t0 + tid) : -1;
  }
  __syncthreads();
  for (int i = tid; i < TILE * a.half; i += kRotThreads) {
    const int t = i / a.half, f = i - t * a.half;
    const unsigned long long phase = turns[f] * (unsigned long long)(unsigned)pos[t];
    float s, c;
    sincospif((float)(int)(phase >> 32) * 4.656612873077393e-10f, &s, &c);  // half turns: / 2^31
    table[t][f] = make_float2(c, s);
  }
  __syncthreads();
  // An item is both chunks of 8 pairs of a head; a thread takes the same one of many heads, so that it reads the table
  // once. Items of a head side by side, then heads.
  const int item_shift = kv.chunk_shift - 1, items = tid >> item_shift;
  const int p = tid & ((1 << item_shift) - 1), step = (kRotThreads / TILE) >> item_shift, t = items / step;
  const int units = a.heads + 2 * kv.kv_heads, tok = t0 + t;
  if (pos[t] < 0 || !VQ3_IN(tok, kv.tokens, 1)) return;
  const bool turns_here = p < a.half >> 3, apart = turns_here && !a.interleaved;
  float4 cs[4];  // (c0, s0, c1, s1), ...
  if (turns_here)
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = reinterpret_cast<const float4*>(&table[t][8 * p])[e];
  const long long sl = slot[t], page = sl >> kv.page_shift, in = sl & ((1 << kv.page_shift) - 1);
  const bool kept = sl >= 0 && sl < limit && VQ3_IN(page, kv.n_pages, 2);
  // both chunks: halves half apart where the rotation pairs them so, neighbours otherwise (values are never turned)
  const int d0 = apart ? 8 * p : 16 * p, d1 = apart ? a.half + 8 * p : 16 * p + 8;
  struct Item {
    uint4 x, y;
    uint16_t *to, *to2;
  };
  const auto fetch = [&](int unit, Item& it) {
    it.to = nullptr;
    const uint16_t* src;
    bool value = false;
    if (unit < a.heads) {
      src = a.q + tok * a.q_token + unit * a.q_head;
      it.to = a.q_out + tok * a.o_token + unit * a.o_head;
    } else if (kept && unit < units) {
      const int h = unit - a.heads, hv = h - kv.kv_heads;
      value = hv >= 0;
      src = value ? kv.v_rows + tok * kv.v_row + hv * kv.v_row_head : kv.k_rows + tok * kv.k_row + h * kv.k_row_head;
      it.to = value ? kv.v_pages + page * kv.v_page + in * kv.v_token + hv * kv.v_head
                    : kv.k_pages + page * kv.k_page + in * kv.k_token + h * kv.k_head;
    }
    if (!it.to) return;
    const int a0 = value ? 16 * p : d0, a1 = value ? 16 * p + 8 : d1;
    it.x = ldg_once(src + a0);
    it.y = ldg_once(src + a1);
    it.to2 = it.to + a1;
    it.to += a0;
  };
  const auto finish = [&](int unit, Item& it) {
    if (!it.to) return;
    if (turns_here && unit < a.heads + kv.kv_heads) {
      uint32_t xs[4] = {it.x.x, it.x.y, it.x.z, it.x.w}, ys[4] = {it.y.x, it.y.y, it.y.z, it.y.w};
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 c = cs[e >> 1], d = cs[2 + (e >> 1)];
          const float2 v = unpack2<BF16>(xs[e]), w = unpack2<BF16>(ys[e]);
          const float c0 = e & 1 ? c.z : c.x, s0 = e & 1 ? c.w : c.y, c1 = e & 1 ? d.z : d.x, s1 = e & 1 ? d.w : d.y;
          xs[e] = pack2<BF16>(v.x * c0 - v.y * s0, v.y * c0 + v.x * s0);
          ys[e] = pack2<BF16>(w.x * c1 - w.y * s1, w.y * c1 + w.x * s1);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 c = cs[e];
          const float2 v = unpack2<BF16>(xs[e]), w = unpack2<BF16>(ys[e]);
          xs[e] = pack2<BF16>(v.x * c.x - w.x * c.y, v.y * c.z - w.y * c.w);
          ys[e] = pack2<BF16>(w.x * c.x + v.x * c.y, w.y * c.z + v.y * c.w);
        }
      }
      it.x = make_uint4(xs[0], xs[1], xs[2], xs[3]);
      it.y = make_uint4(ys[0], ys[1], ys[2], ys[3]);
    }
    *reinterpret_cast<uint4*>(it.to) = it.x;
    *reinterpret_cast<uint4*>(it.to2) = it.y;
  };
  constexpr int kInFlight = 2;
  for (int unit = items - t * step; unit < units; unit += kInFlight * step) {
    Item it[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) fetch(unit + u * step, it[u]);
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) finish(unit + u * step, it[u]);
  }
}

template <bool BF16>
cudaError_t launch_type(const RotaryArgs& a, cudaStream_t st) {
  const int n = a.kv.tokens;
  // a token | 4 tokens a CTA, 32 + 8 heads of 128, us: 64 tokens 2.8 | 4.0, 256 tokens 3.3 | 4.0, 600 tokens 4.6 | 4.7,
  // 1,200 tokens 8.1 | 6.6, some 16,000 tokens 86 | 64 (with three CTAs an SM instead of four 67, with five 73)
  if (n < 5 * device_sm_count())
    kv_append_rotary_kernel<1, BF16><<<n, kRotThreads, 0, st>>>(a);
  else
    kv_append_rotary_kernel<4, BF16><<<(n + 3) / 4, kRotThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append_rotary(const RotaryArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? launch_type<true>(a, st) : launch_type<false>(a, st);
}

}  // namespace vq3
