// Short causal depthwise convolution over packed requests, with the inputs before a request's first token in
// a slot, SiLU, and the heads of the leading channels brought to unit length:
//     y_t[c] = bias[c] + sum_j w[c][j] x_(t - W + 1 + j)[c],  z = y / (1 + e^-y),  out = z / sqrt(sum z^2 + eps).
//
// A thread takes 8 channels and up to L tokens of one request, the last W - 1 inputs in registers. Tiles begin
// at a request's first token, and L >= W - 1, so that only a request's first tile reads its slot; that tile's
// threads write the new state, too, behind their own reads, and the slot read and the slot written may be the
// same. Bound by HBM: an input is read by its own tile and, from L2, by the next one (3 rows of L).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vq3_internal.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(conv)
namespace {

constexpr int kConvThreads = 128;
constexpr int kUnroll = 4;  // tokens whose loads are in flight together

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

__device__ __forceinline__ int start_of(const ConvArgs& a, int r) {
  const int s = __ldg(a.q_start + r);
  return s < 0 ? 0 : (s > a.tokens ? a.tokens : s);
}

// Tile i of the launch: request r's tiles begin at index first_r / L + r, which leaves room for all of them
// (ceil(n / L) <= (first + n) / L - first / L + 1), whatever the lengths are.
template <int W, bool BF16>
__global__ void __launch_bounds__(kConvThreads) short_conv_kernel(const __grid_constant__ ConvArgs a, int shift) {
  __shared__ int counts[kConvThreads / 32];
  const int tile = blockIdx.x, tid = threadIdx.x, L = 1 << shift;
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
  const int c = (blockIdx.y * kConvThreads + tid) * 8;
  // threads behind the last channel stay: the lanes of a head exchange sums
  const bool on = c < a.channels;
  const uint16_t* x = a.x + (long long)s * a.x_token + c;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const auto row = [&](int t) {
    return on && VQ3_IN(s + t, a.tokens, 1) ? __ldg(reinterpret_cast<const uint4*>(x + t * a.x_token)) : none;
  };

  uint4 last[W - 1];  // the inputs before t0
  if (t0 == 0) {
    const int in = a.slot_in ? __ldg(a.slot_in + r) : -1, out = a.slot_out ? __ldg(a.slot_out + r) : -1;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      last[j] = none;
      if (on && in >= 0 && in < a.slots && VQ3_IN(c + 7, a.channels, 2))
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
  } else {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) last[j] = row(t0 - (W - 1) + j);
  }

  float w[W][8], bias[8];
  {
    uint4 ws[W];
#pragma unroll
    for (int j = 0; j < W; ++j)
      ws[j] = on ? __ldg(reinterpret_cast<const uint4*>(a.weight + (long long)c * W) + j) : none;
    float f[W * 8];
#pragma unroll
    for (int j = 0; j < W; ++j) unpack8<BF16>(ws[j], reinterpret_cast<float(&)[8]>(f[8 * j]));
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) w[j][i] = f[i * W + j];
    unpack8<BF16>(on && a.bias ? __ldg(reinterpret_cast<const uint4*>(a.bias + c)) : none, bias);
  }
  const int end = min(t0 + L, n);
  const bool unit = c < a.unit_channels;  // the same for all lanes of a head
  uint16_t* o = a.out + (long long)s * a.o_token + c;
  for (int t = t0; t < end; t += kUnroll) {
    uint4 line[W - 1 + kUnroll];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) line[j] = last[j];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) line[W - 1 + u] = t + u < end ? row(t + u) : none;
    float y[kUnroll][8];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[u][i] = bias[i];
#pragma unroll
    for (int j = 0; j < W - 1 + kUnroll; ++j) {
      float f[8];
      unpack8<BF16>(line[j], f);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (j - u >= 0 && j - u < W)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[u][i] = fmaf(w[j - u < 0 || j - u >= W ? 0 : j - u][i], f[i], y[u][i]);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) last[j] = line[kUnroll + j];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (t + u >= end) break;
      if (a.silu)
#pragma unroll
        for (int i = 0; i < 8; ++i) y[u][i] = __fdividef(y[u][i], 1.f + __expf(-y[u][i]));
      if (a.unit_channels) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(y[u][i], y[u][i], sum);
        for (int d = 1; d < a.head_chunks; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float f = unit ? rsqrtf(sum + a.eps) : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[u][i] *= f;
      }
      if (on && VQ3_IN(s + t + u, a.tokens, 4)) *reinterpret_cast<uint4*>(o + (t + u) * a.o_token) = pack8<BF16>(y[u]);
    }
  }
}

template <int W>
cudaError_t launch_width(const ConvArgs& a, bool bf16, cudaStream_t st) {
  const int blocks = (a.channels / 8 + kConvThreads - 1) / kConvThreads;
  // tokens of a tile: 4 to 32, the longest that still gives every SM 16 CTAs
  int shift = 2;
  while (shift < 5 && (long long)blocks * (a.tokens >> (shift + 1)) >= 16LL * device_sm_count()) ++shift;
  const dim3 grid((unsigned)((a.tokens >> shift) + a.requests), (unsigned)blocks);
  if (bf16)
    short_conv_kernel<W, true><<<grid, kConvThreads, 0, st>>>(a, shift);
  else
    short_conv_kernel<W, false><<<grid, kConvThreads, 0, st>>>(a, shift);
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
