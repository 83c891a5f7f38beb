// Short causal depthwise convolution over packed requests, with the inputs before a request's first token in
// a slot, SiLU, and the heads of the leading channels brought to unit length:
//     y_t[c] = bias[c] + sum_j w[c][j] x_(t - W + 1 + j)[c],  z = y / (1 + e^-y),  out = z / sqrt(sum z^2 + eps).
//
// A thread takes 8 channels and up to L tokens of one request, the last W - 1 inputs in registers. Tiles begin
// at a request's first token, and L >= W - 1, so that only a request's first tile reads its slot; that tile's
// threads write the new state, too, behind their own reads, and the slot read and the slot written may be the
// same. Bound by HBM: an input is read by its own tile and, from L2, by the next one (3 rows of L). What it took: the
// next inputs on their way while four tokens are worked on (104 -> 86 us for 8,921 tokens x 10,240 channels of 4, FP16),
// SiLU by ex2 and rcp of some 2^-22 under an output of 2^-11 (80), whole rows of channels at about the same time (79.6),
// the sums of four tokens exchanged together and two channels an instruction (67: 5.5 TB/s, 81% of a copy's rate).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vq3_internal.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(conv)
namespace {

constexpr int kConvThreads = 128;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16) {
      f[2 * e] = __uint_as_float(ws[e] << 16);
      f[2 * e + 1] = __uint_as_float(ws[e] & 0xffff0000u);
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&ws[e]));
      f[2 * e] = x.x;
      f[2 * e + 1] = x.y;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
    else
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r[e]) : "f"(f[2 * e + 1]), "f"(f[2 * e]));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ unsigned long long pair_of(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ unsigned long long fma_two(unsigned long long x, unsigned long long y, unsigned long long a) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(a));
  return r;
}
__device__ __forceinline__ unsigned long long mul_two(unsigned long long x, unsigned long long y) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ void split_pair(unsigned long long v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int start_of(const ConvArgs& a, int r) {
  const int s = __ldg(a.q_start + r);
  return s < 0 ? 0 : (s > a.tokens ? a.tokens : s);
}

// Tile i of the launch: request r's tiles begin at index first_r / L + r, which leaves room for all of them
// (ceil(n / L) <= (first + n) / L - first / L + 1), whatever the lengths are.
// U: tokens worked on, and fetched, together.
template <int W, int U, bool BF16>
__global__ void __launch_bounds__(kConvThreads, U == 1 ? 6 : 4) short_conv_kernel(const __grid_constant__ ConvArgs a, int shift,
                                                                   int blocks) {
  __shared__ int counts[kConvThreads / 32];
  const int tile = blockIdx.x / blocks, tid = threadIdx.x, L = 1 << shift;
  const int c = ((blockIdx.x - tile * blocks) * kConvThreads + tid) * 8;
  // threads behind the last channel stay: the lanes of a head exchange sums
  const bool on = c < a.channels;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 ws[W], bs = none;
  const auto weights = [&] {
#pragma unroll
    for (int j = 0; j < W; ++j) ws[j] = on ? __ldg(reinterpret_cast<const uint4*>(a.weight + (long long)c * W) + j) : none;
    if (on && a.bias) bs = __ldg(reinterpret_cast<const uint4*>(a.bias + c));
  };
  if constexpr (U == 1)
    if (a.tokens) weights();  // under the search for the request; without rows there may be none
  int before = 0;  // requests whose tiles begin at or before this one
  for (int i = tid; i < a.requests; i += kConvThreads) before += (start_of(a, i) >> shift) + i <= tile;
  before = __reduce_add_sync(0xffffffffu, before);
  if ((tid & 31) == 0) counts[tid >> 5] = before;
  __syncthreads();
  int r = -1;
#pragma unroll
  for (int w = 0; w < kConvThreads / 32; ++w) r += counts[w];
  if (r < 0) return;
  const int s = start_of(a, r), e = max(s, start_of(a, r + 1)), n = e - s;
  const int t0 = (tile - (s >> shift) - r) << shift;  // from the request's first token
  if (t0 < 0 || (t0 >= n && t0 > 0)) return;
  const uint16_t* x = a.x + (long long)s * a.x_token + c;
  const auto row = [&](int t) {
    return on && VQ3_IN(s + t, a.tokens, 1) ? __ldg(reinterpret_cast<const uint4*>(x + t * a.x_token)) : none;
  };

  const int in = t0 == 0 && a.slot_in ? __ldg(a.slot_in + r) : -1, out = t0 == 0 && a.slot_out ? __ldg(a.slot_out + r) : -1;
  const int end = min(t0 + L, n);
  // the next inputs are on their way while the last ones are worked on
  uint4 next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) next[u] = t0 + u < end ? row(t0 + u) : none;
  uint4 last[W - 1];  // the inputs before t0
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    last[j] = none;
    if (t0)
      last[j] = row(t0 - (W - 1) + j);
    else if (on && in >= 0 && in < a.slots && VQ3_IN(c + 7, a.channels, 2))
      last[j] = *reinterpret_cast<const uint4*>(a.states + in * a.state_slot + j * a.state_row + c);
  }
  if (on && out >= 0 && out < a.slots && (n || out != in)) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      // input n + j of the line (old state, new tokens)
      uint4 w = none;
      if (n + j >= W - 1) {
        w = row(n + j - (W - 1));
      } else {
#pragma unroll
        for (int i = j; i < W - 1; ++i)
          if (n + j == i) w = last[i];
      }
      if (VQ3_IN(c + 7, a.channels, 3)) *reinterpret_cast<uint4*>(a.states + out * a.state_slot + j * a.state_row + c) = w;
    }
  }
  if (n == 0) return;
  if constexpr (U > 1) weights();
  unsigned long long w[W][4], bias[4];  // pairs of channels
  {
    float f[W * 8];
#pragma unroll
    for (int j = 0; j < W; ++j) unpack8<BF16>(ws[j], reinterpret_cast<float(&)[8]>(f[8 * j]));
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[j][i] = pair_of(f[2 * i * W + j], f[(2 * i + 1) * W + j]);
    float g[8];
    unpack8<BF16>(bs, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = pair_of(g[2 * i], g[2 * i + 1]);
  }
  const bool unit = c < a.unit_channels;  // the same for all lanes of a head
  const bool units = __any_sync(0xffffffffu, unit);
  uint16_t* o = a.out + (long long)(s + t0) * a.o_token + c;
  const uint16_t* ahead = x + (t0 + U) * a.x_token;
  for (int t = t0; t < end; t += U) {
    uint4 line[W - 1 + U];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) line[j] = last[j];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      line[W - 1 + u] = next[u];
      next[u] = on && t + U + u < end && VQ3_IN(s + t + U + u, a.tokens, 5) ? __ldg(reinterpret_cast<const uint4*>(ahead)) : none;
      ahead += a.x_token;
    }
    unsigned long long y[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[u][i] = bias[i];
#pragma unroll
    for (int j = 0; j < W - 1 + U; ++j) {
      float f[8];
      unpack8<BF16>(line[j], f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned long long x2 = pair_of(f[2 * i], f[2 * i + 1]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j - u >= 0 && j - u < W) y[u][i] = fma_two(w[j - u < 0 || j - u >= W ? 0 : j - u][i], x2, y[u][i]);
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) last[j] = line[U + j];
    if (a.silu)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float e0, e1;
          // a quarter of 1 + e^-y, so that its reciprocal is no subnormal number while e^-y is below 2^128
          split_pair(fma_two(y[u][i], pair_of(-1.4426950408889634f, -1.4426950408889634f), pair_of(-2.f, -2.f)), e0, e1);
          y[u][i] = mul_two(mul_two(y[u][i], pair_of(0.25f, 0.25f)), pair_of(rcp(0.25f + ex2(e0)), rcp(0.25f + ex2(e1))));
        }
    if (units) {
      float sum[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        unsigned long long two = mul_two(y[u][0], y[u][0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) two = fma_two(y[u][i], y[u][i], two);
        float odd;
        split_pair(two, sum[u], odd);
        sum[u] += odd;
      }
      for (int d = 1; d < a.head_chunks; d <<= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], d);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = unit ? rsqrtf(sum[u] + a.eps) : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[u][i] = mul_two(y[u][i], pair_of(f, f));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float z[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) split_pair(y[u][i], z[2 * i], z[2 * i + 1]);
      if (on && t + u < end && VQ3_IN(s + t + u, a.tokens, 4)) *reinterpret_cast<uint4*>(o) = pack8<BF16>(z);
      o += a.o_token;
    }
  }
}

template <int W>
cudaError_t launch_width(const ConvArgs& a, bool bf16, cudaStream_t st) {
  const int blocks = (a.channels / 8 + kConvThreads - 1) / kConvThreads;
  // Tokens of a tile: 4 to 32, the most that still give every SM 4 CTAs, 32 where they give it 8. Tiles of 4 | 8 | 16 |
  // 32 tokens at 10,240 channels, us: 512 tokens 7.4 | 6.7 | 7.2 | 9.8, 1,024 tokens 14.0 | 11.5 | 11.3 | 14.9, 2,048
  // tokens 25.3 | 20.5 | 19.1 | 20.5, 8,960 tokens 100 | 77 | 69 | 67.
  int shift = 2;
  while (shift < 5 && (long long)blocks * (a.tokens >> (shift + 1)) >= (shift < 4 ? 4LL : 8LL) * device_sm_count()) ++shift;
  // a tile's blocks of channels side by side: whole rows are read and written at about the same time
  const long long tiles = (long long)((a.tokens >> shift) + a.requests) * blocks;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)tiles;
  // One token at a time where there is hardly more than one a request: 64 users' tokens of 10,240 channels 5.9 -> 4.1 us.
  const auto run = [&](auto* kernel) { kernel<<<grid, kConvThreads, 0, st>>>(a, shift, blocks); };
  if (a.tokens <= a.requests)
    run(bf16 ? short_conv_kernel<W, 1, true> : short_conv_kernel<W, 1, false>);
  else
    run(bf16 ? short_conv_kernel<W, 4, true> : short_conv_kernel<W, 4, false>);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_short_conv(const ConvArgs& a, int width, bool bf16, cudaStream_t st) {
  switch (width) {
    case 2: return launch_width<2>(a, bf16, st);
    case 3: return launch_width<3>(a, bf16, st);
    default: return launch_width<4>(a, bf16, st);
  }
}

}  // namespace vq3
