// The gated delta rule over packed requests, prompts: chunks of 64 tokens on the 5th-generation tensor cores
// (mathematics and names as in delta_batch.cu; d_k 64 or 128).
//
// A CTA takes one request, one value head and up to 128 of its columns. Everything is kept transposed, one column
// of the state to a lane of tensor memory, so that every product has M = 128 and its FP32 operand comes from tensor
// memory, where it was made, and every power of two that scales a row is a number of its thread:
//     X^T = S^T [K; Q]^T                  two products of N = 64
//     R^T = V^T - X_K^T g,  U^T = R^T T^T
//     dS^T = (U diag w)^T K,  S^T <- g_C S^T + dS^T   (S in registers, FP32)
//     O^T = X_Q^T g + U^T M^T
//   warps 0-7    the state: two threads a column, each half of d_k and half of a chunk's tokens
//   warps 8-11   rows: K and Q as FP16, and N, M from [K; Q] K^T, one row of a product a thread; the output
//   warps 12-13  T = (I + N)^-1, one column a lane: the two 32 x 32 blocks by substitution, then
//                T21 = -T22 N21 T11
//   warp 14      issues the products of the state
//   warp 15      copies K, Q and V by TMA and issues [K; Q] K^T
// The chain of a chunk is X_K, R, U, U w, dS, S; what is not on it (X_Q, O and its output of the chunk before, the
// next chunks' rows and T) runs under it. FP32 operands enter as two FP16 parts as in delta_batch.cu. The scale of S
// has to be known before dS is: it is made from a bound, |g_C| max |S| + sum |u w| max |k|, which is some 2^5 above
// what comes out and leaves 17 bits of FP16's range below it. A chunk with values that cannot share a power of two
// (kRange, kGrown) goes on as it is, but its dS and its output are not used: the state's warps, whose S is still the
// chunk's first, step through its tokens in FP32: 74 us instead of 5.8. Looking for such values costs the others 4 to 6% (the
// loop over R under the wait for U).
// Bound by that chain and by the row warps, which are both busy some 11,000 cycles a chunk, a third of them waiting for
// products of 50 to 70 cycles for 128 x 64 x 16 (32 where they have the SM to themselves): 5.8 us a chunk of 64 tokens,
// 0.77 ms for one prompt of 8,192 tokens (48 heads of 128 x 128, BF16, 48 CTAs), 0.34 ms for 16 of 1 to 1,100 tokens.
// (When both took 0.67 and 0.32 ms, with BF16 outputs from 11 bits: without the copying warp, with code of 165 KB, 1,622
// and 611 us; the output by the state's warps while U is made: the same for one prompt, 336 us for 16; the output's
// copies by the copying warp: 728 us.)
// All waits are bounded: one that runs out ends the CTA's work and sets the caller's status word, or the device's.
#include "vq3_internal.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(delta_wide)
}
#include "delta_common.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace vq3 {
namespace {

constexpr int kC = 64;           // tokens of a chunk
constexpr int kCols = 128;       // columns of a CTA
// Tokens up to which a request is stepped through instead (16 requests of 48 heads, one request: 5 tokens 71, 10.4 us
// against 89, 15.0; 6 tokens 80, 12.0 against 90, 15.2; 8 tokens 96, 14.9 against 90, 15.2).
constexpr int kStepMost = 6;
constexpr int kWideThreads = 512;
constexpr int kRowWarp = 8, kInvWarp = 12, kIssueWarp = 14;
// Registers per thread: 128 at launch; the state's warps take what the others give up.
constexpr int kRegsState = 152, kRegsRows = 104, kRegsOther = 104;
static_assert(2 * kRegsState + kRegsRows + kRegsOther == 4 * 128, "register shares");

// Columns of tensor memory.
constexpr uint32_t kTmShi = 0, kTmSlo = 64;      // S, two parts, 2 values a column
constexpr uint32_t kTmW = 0;                     // U w, hi at 0 and lo at 32, once X_Q is done
constexpr uint32_t kTmX = 128;                   // X_K, then U
constexpr uint32_t kTmQ = 192;                   // X_Q
constexpr uint32_t kTmR = 256;                   // R, hi and lo; then U for the output
constexpr uint32_t kTmD = 320;                   // dS (128 columns), then U M in the first 64
constexpr uint32_t kTmKK = 448;                  // [K; Q] K^T

template <int DK, bool BF16>
struct Wide {
  static constexpr int KB = DK / 64;             // 64-column blocks of K and Q
  static constexpr int SD = DK / 2;              // rows of S a thread
  static constexpr int NS = kC + 4;              // row of N in floats
  // [K; Q] by 64-column blocks, T and M in the 128-byte swizzle; V; the output; factors
  static constexpr int kBlock = 2 * kC * 128, kTile = kC * 128;
  // (a place of T holds N first)
  static constexpr int kKQBytes = KB * kBlock, kTBytes = kC * NS * 4, kMBytes = 2 * kTile;
  static constexpr int kVBytes = kC * kCols * 2, kFBytes = 2048;
  static_assert(kTBytes >= 2 * kTile && kTBytes % 1024 == 0, "N and T");
  static constexpr int kKQ = 0, kT = kKQ + 3 * kKQBytes, kM = kT + 2 * kTBytes, kV = kM + 2 * kMBytes, kOut = kV + 2 * kVBytes;
  static constexpr int kF = kOut + kVBytes;
  // factors per token: of V and of X_K in R, of X_Q and of U M in O, of U in dS, the largest |k|, its gate; then g_C
  static constexpr int kFv = 0, kFk = 64, kFq = 128, kFm = 192, kFw = 256, kKm = 320, kFa = 384, kG = 448;
  // exchange of the column's halves: float2 [2][128], float4 [2][128]; scales for the output: float2 [2][128]; rows: gates
  // and factors; barriers
  static constexpr int kX1 = kF + 3 * kFBytes, kX2 = kX1 + 2048, kXO = kX2 + 4096, kRow = kXO + 2048, kMax = kRow + 1024, kBar = kMax + 256;
  static constexpr int kSmem = kBar + 512;
  static_assert(kSmem + 1024 <= 227 * 1024, "shared memory per CTA");
};

// Barriers, in order. Who arrives at one for a later use has waited for something that every waiter of the use before
// did behind its wait, so that a phase is neither filled by the next one's arrivals nor missed.
enum {
  kbKQFull = 0,   // [3] K and Q copied
  kbKQ = 3,       // [3] as FP16
  kbKQFree = 6,   // [3]
  kbVFull = 9,    // [2]
  kbVFree = 11,   // [2]
  kbTM = 13,      // [2] T and the factors
  kbTFree = 15,   // [2]
  kbM = 17,       // [2]
  kbMFree = 19,   // [2]
  kbN = 21,       // [2]
  kbKK = 23,
  kbS = 24,       // [4] S stored: half of d_k, half of that
  kbXK = 28, kbR, kbU, kbXQ, kbW,
  kbD = 33,       // [2]
  kbO = 35, kbORead, kbDrain,
  kbPair,         // [4] the two warps of 32 columns, while they step
  kBars = kbPair + 4
};

__device__ int g_delta_status;  // of the calls without a status word of their own; vq3_delta_status reads it

struct DeltaMaps {
  CUtensorMap k, q, v, out;
};

__device__ __forceinline__ float2 bits2(const uint32_t* r, int i) {
  return make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
}
__device__ __forceinline__ uint32_t swz(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }
__device__ __forceinline__ void sync_threads(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void st_shared4(uint32_t at, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// A wait tries so often, each try sleeping so long at most: a second in all.
constexpr int kTries = 200000;
constexpr uint32_t kTryNs = 5000;
constexpr int kPolls = 4000000;  // of the copying warp, with 100 ns between two
__device__ __forceinline__ bool try_wait_for(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kTryNs)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool is_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}

// The request whose turn it is: by classes of length, a power of two each, the longest first, and by their places in a
// class. The CTAs that come last are short ones then, and the SMs end together. More requests than threads come as
// they are.
__device__ __forceinline__ int request_in_turn(const DeltaArgs& a, int turn, int* s) {
  if (a.requests == 1 || a.requests > kWideThreads) return turn;
  const int r = threadIdx.x, warp = r >> 5, lane = r & 31;
  const bool is = r < a.requests;
  const int cls = is ? 32 - __clz(delta_request_rows(a, r).y) : 0;  // 0 .. 31
  const auto before = [&](int& v) {  // v of the lanes before this one, summed; v with them
    const int own = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += o;
    }
    return v - own;
  };
  if (r < 32) s[r] = 0;
  __syncthreads();
  if (is) atomicAdd(s + cls, 1);
  __syncthreads();
  int upto = s[31 - lane];
  const int longer = before(upto);
  const int at = __ffs(__ballot_sync(0xffffffffu, upto > turn)) - 1;
  const int place = turn - __shfl_sync(0xffffffffu, longer, at);  // in class 31 - at
  const uint32_t peers = __ballot_sync(0xffffffffu, is && cls == 31 - at);
  if (lane == 0) s[32 + warp] = __popc(peers);
  __syncthreads();
  int in_warp = lane < kWideThreads / 32 ? s[32 + lane] : 0;
  const int in_front = __shfl_sync(0xffffffffu, before(in_warp), warp) + __popc(peers & ((1u << lane) - 1u));
  if (is && cls == 31 - at && in_front == place) s[48] = r;
  __syncthreads();
  return s[48];
}

template <int DK, bool BF16>
__global__ void __launch_bounds__(kWideThreads, 1) delta_wide_kernel(const __grid_constant__ DeltaArgs a,
                                                                    const __grid_constant__ DeltaMaps maps) {
  using L = Wide<DK, BF16>;
  constexpr int KB = L::KB, SD = L::SD;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, col0 = blockIdx.x * kCols;
  __shared__ int turns[64];
  const DeltaRequest rq = delta_request(a, request_in_turn(a, blockIdx.z, turns), h);
  if (rq.n <= kStepMost) {
    using Steps = StepShared<DK / 16, 16, 32>;
    static_assert(sizeof(Steps) <= L::kSmem, "shared memory of the steps");
    delta_steps<DK / 16, 16, 32, BF16>(a, rq, h, col0, *reinterpret_cast<Steps*>(smem));
    return;
  }
  const int chunks = (rq.n + kC - 1) / kC;
  const uint32_t base = smem_u32(smem), bar0 = base + L::kBar;
  const auto bar = [&](int i) { return bar0 + 8u * i; };
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(smem + L::kBar + 8 * kBars);
  volatile int* const abort = reinterpret_cast<volatile int*>(smem + L::kBar + 8 * kBars + 4);
  // of the last four chunks: its number + 1 if it has to be gone through token by token
  volatile int* const again = abort + 1;
  static_assert(8 * kBars + 24 <= 512, "barriers");

  if (tid < kBars) {
    // arrivals: a copy, a product's completion or a warp each
    constexpr int n[kBars] = {1, 1, 1, 4, 4, 4, 1, 1, 1, 1, 1, 8, 8, 6, 6, 1, 1, 2, 2, 1, 1, 2, 2, 1, 4, 4, 4, 4, 1, 8, 1, 1, 8, 1, 1, 1, 4, 1, 2, 2, 2, 2};
    mbar_init(bar(tid), KB == 1 && tid >= kbS && tid < kbS + 4 ? 8 : n[tid]);
    if (tid == 0) *abort = 0;
    if (tid < 4) again[tid] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *s_tmem;
  bool dead = false;  // a wait gave up (the same for the whole warp): the warp issues nothing more
  const auto wait = [&](int i, int use) {  // for the end of use `use` of a barrier
    int left = kTries;
    bool ok;
#pragma unroll 1
    while (!(ok = try_wait_for(bar(i), (uint32_t)(use & 1))) && --left && !*abort) {
    }
    if (__all_sync(0xffffffffu, ok)) return;
    dead = true;
    *abort = 1;
  };
  const auto arrive = [&](int i) {  // behind everything this warp has read and written
    tc_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };
  constexpr uint32_t id_k = idesc(64, false, false), id_mn = idesc(64, false, true);

  if (warp < kRowWarp) {
    // ------------------------------------------------------------ the state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
    const int sub = warp & 3, hf = warp >> 2, c = sub * 32 + lane, col = col0 + c;
    const bool on = col < a.d_v;
    const uint32_t tm = tmem + ((uint32_t)(sub * 32) << 16);
    const size_t n_state = (size_t)DK * a.d_v;
    float2* const x1 = reinterpret_cast<float2*>(smem + L::kX1);
    float4* const x2 = reinterpret_cast<float4*>(smem + L::kX2);
    const auto pair_sync = [&] { sync_threads(1 + sub, 64); };
    float2 S[SD / 2];
    float mS = 0.f;
#pragma unroll
    for (int i = 0; i < SD / 2; ++i) {
      const size_t at = (size_t)(hf * SD + 2 * i) * a.d_v + col;
      S[i] = make_float2(0.f, 0.f);
      if (on && rq.in && VQ3_IN(at + a.d_v, n_state, 1)) S[i] = make_float2(__ldcs(rq.in + at), __ldcs(rq.in + at + a.d_v));
      mS = max_pair(mS, S[i]);
    }
    x1[hf * 128 + c] = make_float2(mS, 0.f);
    pair_sync();
    Scale ss = scale_of(fmaxf(mS, x1[(hf ^ 1) * 128 + c].x)), ws{0.f, 0.f};
    float gC = 1.f;
    // S over a chunk token by token, with its output: delta_steps with two threads a column. S goes through tensor memory,
    // where its parts are otherwise, a slice at a time: in registers it cost the loop around it some 100 spilled ones.
    int n_met = 0;
    const auto met = [&] {
      arrive(kbPair + sub);
      wait(kbPair + sub, n_met++);
    };
    const auto steps = [&](int ch) {
      const int nt = rq.n - ch * kC < kC ? rq.n - ch * kC : kC, hq = h / a.group;
      const uint32_t at = tm + kTmShi + (uint32_t)(hf * SD);
#pragma unroll
      for (int i = 0; i < SD; i += 16) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(e & 1 ? S[(i + e) / 2].y : S[(i + e) / 2].x);
        tmem_st16(at + (uint32_t)i, w);
      }
      tc_wait_st();
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        const long long row = rq.first + ch * kC + j;
        if (!VQ3_IN(row, a.tokens, 5)) break;
        const uint4* kp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) + row * a.k_token + hq * a.k_head + hf * SD);
        const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + row * a.q_token + hq * a.q_head + hf * SD);
        float2 x = both(0.f), y = x, kq = x;
#pragma unroll 1
        for (int i = 0; i < SD; i += 32) {
          uint32_t s[32];
          tmem_ld32(at + (uint32_t)i, s);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4 kw = __ldg(kp + i / 8 + e), qw = __ldg(qp + i / 8 + e);
            const uint32_t k4[4] = {kw.x, kw.y, kw.z, kw.w}, q4[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
            for (int l = 0; l < 4; ++l) {
              const float2 k2 = delta_unpack2<BF16>(k4[l]), q2 = delta_unpack2<BF16>(q4[l]), s2 = bits2(s, 8 * e + 2 * l);
              x = fma_pair(k2, s2, x);
              y = fma_pair(q2, s2, y);
              kq = fma_pair(k2, q2, kq);
            }
          }
        }
        const float4 own = make_float4(x.x + x.y, y.x + y.y, kq.x + kq.y, 0.f);
        x2[hf * 128 + c] = own;
        met();
        const float4 other = x2[(hf ^ 1) * 128 + c];
        met();
        const float al = __ldg(a.alpha + row * a.alpha_token + h), be = __ldg(a.beta + row * a.beta_token + h);
        const float v = on ? delta_unpack2<BF16>(__ldg(static_cast<const uint16_t*>(a.v) + row * a.v_token + h * a.v_head + col)).x : 0.f;
        const float u = be * (v - al * (own.x + other.x));
#pragma unroll 1
        for (int i = 0; i < SD; i += 32) {
          uint32_t s[32], w[16];
          tmem_ld32(at + (uint32_t)i, s);
          tc_wait_ld();
#pragma unroll
          for (int n = 0; n < 32; n += 16) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 kw = __ldg(kp + (i + n) / 8 + e);
              const uint32_t k4[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
              for (int l = 0; l < 4; ++l) {
                const float2 s2 = fma_pair(delta_unpack2<BF16>(k4[l]), u, mul_pair(bits2(s, n + 8 * e + 2 * l), al));
                w[8 * e + 2 * l] = __float_as_uint(s2.x);
                w[8 * e + 2 * l + 1] = __float_as_uint(s2.y);
              }
            }
            tmem_st16(at + (uint32_t)(i + n), w);
          }
        }
        tc_wait_st();
        if (on && hf == 0)
          static_cast<uint16_t*>(a.out)[row * a.o_token + h * a.o_head + col] =
              (uint16_t)delta_pack2<BF16>(a.scale * fmaf(own.z + other.z, u, al * (own.y + other.y)), 0.f);
      }
      mS = 0.f;
#pragma unroll
      for (int i = 0; i < SD; i += 32) {
        uint32_t s[32];
        tmem_ld32(at + (uint32_t)i, s);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          S[(i + e) / 2] = bits2(s, e);
          mS = max_pair(mS, S[(i + e) / 2]);
        }
      }
      x1[hf * 128 + c] = make_float2(mS, 0.f);
      met();
      ss = scale_of(fmaxf(mS, x1[(hf ^ 1) * 128 + c].x));
    };
    for (int ch = 0;; ++ch) {
      // S <- g_C S + dS, and its parts for the products, half by half
      if (ch) {
        wait(kbD + (KB == 2 ? hf : 0), ch - 1);
        if constexpr (KB == 2) wait(kbD + (hf ^ 1), ch - 1);  // every product has read U w, whose place S takes
        tc_after();
        mS = 0.f;
      }
      // every warp's word on it came before its arrival for U w; only where a wait gave up the two warps of a column may
      // see different ones, and so steps() has no barrier that is not bounded
      const bool stepped = ch && again[(ch - 1) & 3] == ch;
      if (stepped) steps(ch - 1);
#pragma unroll
      for (int i = 0; i < SD; i += 32) {
        if (ch && !stepped) {
          uint32_t x[32];
          tmem_ld32(tm + kTmD + (uint32_t)(hf * SD + i), x);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2& y = S[(i + e) / 2];
            y = fma_pair(bits2(x, e), ws.back, mul_pair(y, gC));
            mS = max_pair(mS, y);
          }
        }
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) split2(mul_pair(S[i / 2 + e], ss.to), hi[e], lo[e]);
        tmem_st16(tm + kTmShi + (uint32_t)((hf * SD + i) / 2), hi);
        tmem_st16(tm + kTmSlo + (uint32_t)((hf * SD + i) / 2), lo);
        tc_wait_st();
        // behind the last chunk, too: U M goes where dS was, once everyone has read it
        arrive(kbS + (KB == 2 ? 2 * hf : 0) + i / 32);
      }
      if (ch == chunks) break;
      const float* f = reinterpret_cast<const float*>(smem + L::kF + (ch % 3) * L::kFBytes);
      // R^T = V^T - X_K^T, times the factor of T's column
      wait(kbVFull + (ch & 1), ch >> 1);
      uint32_t x[32];
      float2 r[16];
      float top = 0.f;
      uint16_t vw[32];
      {
        const uint16_t* v = reinterpret_cast<const uint16_t*>(smem + L::kV + (ch & 1) * L::kVBytes) + 32 * hf * kCols + c;
#pragma unroll
        for (int j = 0; j < 32; ++j) vw[j] = v[j * kCols];
        const int left = rq.n - ch * kC - 32 * hf;  // rows behind the request's last are another's
        if (left < 32)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j >= left) vw[j] = 0;
      }
      arrive(kbVFree + (ch & 1));
      wait(kbTM + (ch & 1), ch >> 1);
      wait(kbXK, ch);
      tc_after();
      tmem_ld32(tm + kTmX + 32u * hf, x);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 fv = *reinterpret_cast<const float4*>(f + L::kFv + 32 * hf + j);
        const float4 fk = *reinterpret_cast<const float4*>(f + L::kFk + 32 * hf + j);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 v2 = delta_unpack2<BF16>((uint32_t)vw[j + e] | (uint32_t)vw[j + e + 1] << 16);
          float2& y = r[(j + e) / 2];
          y = mul_pair(v2, e ? make_float2(fv.z, fv.w) : make_float2(fv.x, fv.y));
          y = fma_pair(mul_pair(bits2(x, j + e), -ss.back), e ? make_float2(fk.z, fk.w) : make_float2(fk.x, fk.y), y);
          top = max_pair(top, y);
        }
      }
      x1[hf * 128 + c] = make_float2(top, mS);
      pair_sync();
      const float2 o1 = x1[(hf ^ 1) * 128 + c];
      const float topr = fmaxf(top, o1.x);
      const Scale rs = scale_of(topr);
      const float mS_all = fmaxf(mS, o1.y);
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) split2(mul_pair(r[e], rs.to), hi[e], lo[e]);
      if (ch) {  // U M of the chunk before has read U
        wait(kbO, ch - 1);
        tc_after();
      }
      tmem_st16(tm + kTmR + 16u * hf, hi);
      tmem_st16(tm + kTmR + 32u + 16u * hf, lo);
      tc_wait_st();
      arrive(kbR);
      // (under U) the least that a token of this half finds in its column, its own R with it: from the state on in the first
      // half (with T's factor of 2^-14, as R, and less, for keys that are no unit vectors)
      const float need = topr * (4.f * kRange);
      float found = hf ? 0.f : 0x1p-17f * mS_all, least = INFINITY, worst = INFINITY;
      const auto scan = [&](auto each) {
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 fa = *reinterpret_cast<const float4*>(f + L::kFa + 32 * hf + j);
          const float av[4] = {fa.x, fa.y, fa.z, fa.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            found = fmaxf(fabsf(av[e] * found), fabsf(e & 1 ? r[(j + e) / 2].y : r[(j + e) / 2].x));
            each(av[e]);
          }
        }
      };
      scan([&](float) { least = fminf(least, found); });
      if (hf && __any_sync(0xffffffffu, least < need)) {  // what the gates up to such a token leave of the first half's
        float kept = 1.f;
        found = 0.f;
        scan([&](float a) {
          kept *= a;
          if (found < need) worst = fminf(worst, fabsf(kept));
        });
      }
      // U^T, as it is for the output and times w for dS
      wait(kbU, ch);
      tc_after();
      tmem_ld32(tm + kTmX + 32u * hf, x);
      tc_wait_ld();
      float topu = 0.f, l1 = 0.f;
      top = 0.f;
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        const float4 fw = *reinterpret_cast<const float4*>(f + L::kFw + 32 * hf + j);
        const float4 km = *reinterpret_cast<const float4*>(f + L::kKm + 32 * hf + j);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float2& u = r[(j + e) / 2];
          u = mul_pair(bits2(x, j + e), rs.back);
          const float2 w = mul_pair(u, e ? make_float2(fw.z, fw.w) : make_float2(fw.x, fw.y));
          topu = max_pair(topu, u);
          top = max_pair(top, w);
          l1 = fmaf(fabsf(w.x), e ? km.z : km.x, fmaf(fabsf(w.y), e ? km.w : km.y, l1));
        }
      }
      x2[hf * 128 + c] = make_float4(topu, top, l1, found);
      pair_sync();
      const float4 o2 = x2[(hf ^ 1) * 128 + c];
      const Scale us = scale_of(fmaxf(topu, o2.x));
      ws = scale_of(fmaxf(top, o2.y));
      gC = f[L::kG];
      if (hf == 0) reinterpret_cast<float2*>(smem + L::kXO)[(ch & 1) * 128 + c] = make_float2(ss.back, us.back);
      ss = scale_of(fabsf(gC) * mS_all + (l1 + o2.z));
      {
        // (l1 is not finite if a U is not; U is up to twice R, whose factor of T is 2^-14 or 2^-13)
        const bool lost = !(l1 + o2.z < INFINITY) || 0x1p-14f * fmaxf(topu, o2.x) > 4.f * topr ||
                          (hf ? worst < INFINITY && o2.w * worst < need : least < need);
        if (__any_sync(0xffffffffu, lost) && lane == 0) again[ch & 3] = ch + 1;
      }
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float4 fw = *reinterpret_cast<const float4*>(f + L::kFw + 32 * hf + 2 * e);
        split2(mul_pair(mul_pair(r[e], make_float2(fw.x, fw.y)), ws.to), hi[e], lo[e]);
        split2(mul_pair(mul_pair(r[e + 1], make_float2(fw.z, fw.w)), ws.to), hi[e + 1], lo[e + 1]);
      }
      wait(kbXQ, ch);  // X_Q has read S, whose place this takes
      tc_after();
      tmem_st16(tm + kTmW + 16u * hf, hi);
      tmem_st16(tm + kTmW + 32u + 16u * hf, lo);
      tc_wait_st();
      arrive(kbW);
#pragma unroll
      for (int e = 0; e < 16; ++e) split2(mul_pair(r[e], us.to), hi[e], lo[e]);
      tmem_st16(tm + kTmR + 16u * hf, hi);  // (kbS comes behind these stores, and U M behind kbS)
      tmem_st16(tm + kTmR + 32u + 16u * hf, lo);
      tc_wait_st();
    }
    if (on && rq.out && !dead) {
#pragma unroll
      for (int i = 0; i < SD / 2; ++i) {
        const size_t at = (size_t)(hf * SD + 2 * i) * a.d_v + col;
        if (VQ3_IN(at + a.d_v, n_state, 3)) {
          __stcs(rq.out + at, S[i].x);
          __stcs(rq.out + at + a.d_v, S[i].y);
        }
      }
    }
  } else if (warp < kInvWarp) {
    // ------------------------------------------------------------ rows
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRows));
    const int p = tid - kRowWarp * 32, i = p & 63;
    const bool is_k = p < 64;
    float* const gate = reinterpret_cast<float*>(smem + L::kRow);  // a_(j + 1); b_j and the factor of k_j; g_C / g_j; a_0
    float *const bks = gate + 64, *const rest = bks + 64, *const gate0 = rest + 64;
    float al = 1.f, be = 0.f;  // of the next chunk
    const auto load_gates = [&](int t0) {
      al = 1.f;
      be = 0.f;
      if (is_k && t0 + p < rq.n && VQ3_IN(rq.first + t0 + p, a.tokens, 4)) {
        al = __ldg(a.alpha + (long long)(rq.first + t0 + p) * a.alpha_token + h);
        be = __ldg(a.beta + (long long)(rq.first + t0 + p) * a.beta_token + h);
      }
    };
    // Output of a chunk, this warp's 32 columns (lane = column), through shared memory.
    const int sub = warp - kRowWarp;
    const int row_bytes = 2 * (a.d_v - col0 < kCols ? a.d_v - col0 : kCols);
    const auto output = [&](int ch) {
      const uint32_t tm = tmem + ((uint32_t)(sub * 32) << 16), tile = base + (uint32_t)L::kOut;
      const float* f = reinterpret_cast<const float*>(smem + L::kF + (ch % 3) * L::kFBytes);
      wait(kbO, ch);
      tc_after();
      const float2 back = reinterpret_cast<const float2*>(smem + L::kXO)[(ch & 1) * 128 + sub * 32 + lane];
#pragma unroll 1
      for (int j0 = 0; j0 < kC; j0 += 32) {
        uint32_t xq[32], um[32];
        tmem_ld32(tm + kTmQ + (uint32_t)j0, xq);
        tmem_ld32(tm + kTmD + (uint32_t)j0, um);
        tc_wait_ld();
        if (j0) arrive(kbORead);
        const uint32_t at = tile + (uint32_t)(j0 * kCols + sub * 32 + lane) * 2u;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 fq = *reinterpret_cast<const float4*>(f + L::kFq + j0 + j);
          const float4 fm = *reinterpret_cast<const float4*>(f + L::kFm + j0 + j);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const float2 q = mul_pair(bits2(xq, j + e), back.x), u = mul_pair(bits2(um, j + e), back.y);
            const float2 y = fma_pair(e ? make_float2(fm.z, fm.w) : make_float2(fm.x, fm.y), u,
                                      mul_pair(e ? make_float2(fq.z, fq.w) : make_float2(fq.x, fq.y), q));
            const uint32_t two = delta_pack2<BF16>(y.x, y.y);
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + (uint32_t)((j + e) * kCols * 2)), "h"((uint16_t)two) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + (uint32_t)((j + e + 1) * kCols * 2)), "h"((uint16_t)(two >> 16)) : "memory");
          }
        }
      }
      const bool skip = *abort || again[ch & 3] == ch + 1;  // written by the state's warps in that case
      fence_async();
      sync_threads(9, 128);  // whole rows
      if (rq.n - ch * kC >= kC) {
        if (p == 0 && !skip && VQ3_IN(rq.first + ch * kC + kC - 1, a.tokens, 2))
          asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                           reinterpret_cast<uint64_t>(&maps.out)),
                       "r"(col0), "r"(h), "r"(rq.first + ch * kC), "r"(tile)
                       : "memory");
      } else {  // the rows behind the request's last are another's: row by row, up to 256 bytes
        const int t = 16 * sub + lane;
        if (lane < 16 && ch * kC + t < rq.n && !skip && VQ3_IN(rq.first + ch * kC + t, a.tokens, 2)) {
          const uint16_t* to = static_cast<const uint16_t*>(a.out) + (rq.first + ch * kC + t) * a.o_token + h * a.o_head + col0;
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(tile + (uint32_t)(t * kCols * 2)),
                       "r"(row_bytes) : "memory");
        }
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    };
    const auto output_read = [&] { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); };
    load_gates(0);
    for (int ch = 0; ch < chunks + 3; ++ch) {
      if (ch > 2) output(ch - 3);  // (chunk ch's factors go where those of ch - 3 were)
      if (ch >= chunks) {
        output_read();
        sync_threads(9, 128);
        continue;
      }
      const int t0 = ch * kC, nt = rq.n - t0 < kC ? rq.n - t0 : kC, s3 = ch % 3;
      const uint32_t kq = base + (uint32_t)(L::kKQ + s3 * L::kKQBytes);
      float* const f = reinterpret_cast<float*>(smem + L::kF + s3 * L::kFBytes);
      if (ch > 2) output_read();
      sync_threads(9, 128);  // the last chunk's gates have been read
      if (is_k) {
        f[L::kFa + p] = al;
        if (p)
          gate[p - 1] = al;
        else
          gate[63] = 1.f, *gate0 = al;
      }
      const float b_i = be;
      load_gates(t0 + kC);
      wait(kbKQFull + s3, ch / 3);
      // thread = row of [K; Q]: its largest entry; BF16 to FP16, scaled by a power of two; rows behind the last are zero
      float back = 1.f, largest = 0x1p15f;
      {
        const uint32_t row = kq + (is_k ? 0u : kC * 128u);
        const auto at = [&](int q) { return row + (uint32_t)((q >> 3) * L::kBlock) + swz(i, q & 7); };
        if (i >= nt) {
          const uint32_t zero[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
          for (int q = 0; q < DK / 8; ++q) st_shared4(at(q), zero);
        } else if constexpr (BF16) {
          uint4 w[DK / 8];
          __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
          for (int q = 0; q < DK / 8; ++q) w[q] = ld_shared4(at(q));
#pragma unroll
          for (int q = 0; q < DK / 8; ++q) {
            const uint32_t ws[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e])));
          }
          const Scale sc = scale_of(fmaxf(__low2float(top), __high2float(top)));
          const __nv_bfloat162 fs = __float2bfloat162_rn(sc.to);
#pragma unroll
          for (int q = 0; q < DK / 8; ++q) {
            uint32_t ws[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&ws[e]), fs);
              const float2 y = delta_unpack2<true>(*reinterpret_cast<const uint32_t*>(&x));
              ws[e] = pack_f16(y.x, y.y);
            }
            st_shared4(at(q), ws);
          }
          back = sc.back;
        } else if (is_k) {
          __half2 top = __float2half2_rn(0.f);
#pragma unroll 8
          for (int q = 0; q < DK / 8; ++q) {
            const uint4 w = ld_shared4(at(q));
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __hmax2(top, __habs2(*reinterpret_cast<const __half2*>(&ws[e])));
          }
          largest = fmaxf(__low2float(top), __high2float(top));
        }
      }
      const float bk = b_i * back;
      if (is_k) {
        bks[p] = bk;
        f[L::kKm + p] = largest;
      }
      fence_async();
      arrive(kbKQ + s3);  // (KK of the last chunk has been read)
      sync_threads(9, 128);
      // a_(j + 1) ... a_i for j < i, 1 from there on
      float r[kC], run = 1.f;
#pragma unroll
      for (int j = kC - 4; j >= 0; j -= 4) {
        const float4 g4 = *reinterpret_cast<const float4*>(gate + j);
        const float g[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          run *= j + e < i ? g[e] : 1.f;
          r[j + e] = run;
        }
      }
      const float gi = run * *gate0;
      if (p == 63) {
#pragma unroll
        for (int j = 0; j < kC; j += 4) *reinterpret_cast<float4*>(rest + j) = make_float4(r[j], r[j + 1], r[j + 2], r[j + 3]);
        f[L::kG] = gi;
      }
      // (all four: an arrival at kbTM for this chunk must not count for the chunk before the last)
      if (ch >= 2) wait(kbTFree + (ch & 1), (ch >> 1) - 1);
      wait(kbKK, ch);
      tc_after();
      float top = 0.f;
      const int lim = is_k ? i : i + 1;         // N is strictly lower, M has its diagonal
      const float sign = is_k ? -back : 1.f;    // -N, with the factor of k_i
#pragma unroll
      for (int j0 = 0; j0 < kC; j0 += 32) {
        uint32_t x[32];
        tmem_ld32(tmem + ((uint32_t)((warp - kRowWarp) * 32) << 16) + kTmKK + (uint32_t)j0, x);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 b4 = *reinterpret_cast<const float4*>(bks + j0 + j);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int jj = j0 + j + e;
            const float2 y = mul_pair(mul_pair(make_float2(r[jj], r[jj + 1]), mul_pair(bits2(x, j + e), sign)),
                                      e ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y));
            r[jj] = jj < lim ? y.x : 0.f;
            r[jj + 1] = jj + 1 < lim ? y.y : 0.f;
            top = fmaxf(top, fmaxf(fabsf(r[jj]), fabsf(r[jj + 1])));
          }
        }
      }
      if (is_k) {
        float* const n_col = reinterpret_cast<float*>(smem + L::kT + (ch & 1) * L::kTBytes) + i;
#pragma unroll
        for (int j = 0; j < kC; ++j)
          if (j < 32 || i >= 32) n_col[j * L::NS] = r[j];
        f[L::kFk + p] = gi * back;
        sync_threads(11, 64);
        f[L::kFw + p] = bk * rest[p];
        arrive(kbN + (ch & 1));
        arrive(kbTM + (ch & 1));
      } else {
        const Scale sc = scale_of(top);
        f[L::kFq + i] = a.scale * gi * back;
        f[L::kFm + i] = a.scale * back * sc.back;
        arrive(kbTM + (ch & 1));
        if (ch >= 2) wait(kbMFree + (ch & 1), (ch >> 1) - 1);
        const uint32_t m = base + (uint32_t)(L::kM + (ch & 1) * L::kMBytes);
#pragma unroll
        for (int q = 0; q < kC / 8; ++q) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(r[8 * q + 2 * e] * sc.to, r[8 * q + 2 * e + 1] * sc.to, hi[e], lo[e]);
          st_shared4(m + swz(i, q), hi);
          st_shared4(m + L::kTile + swz(i, q), lo);
        }
        fence_async();
        arrive(kbM + (ch & 1));
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp < kIssueWarp) {
      // ---------------------------------------------------------- T, -N by columns
      const int w = warp - kInvWarp;
      float* const tops = reinterpret_cast<float*>(smem + L::kMax);
      constexpr int NS = L::NS;
      for (int ch = 0; ch < chunks; ++ch) {
        wait(kbN + (ch & 1), ch >> 1);
        float* const n = reinterpret_cast<float*>(smem + L::kT + (ch & 1) * L::kTBytes);
        // a 32 x 32 block of the diagonal; rows in pairs
        float2 x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = make_float2(2 * k == lane ? 1.f : 0.f, 2 * k + 1 == lane ? 1.f : 0.f);
        const float* nd = n + w * (32 * NS + 32);
        // step m needs rows m + 1 .. of column m (up to m: zeros); the next column's are on their way meanwhile
        float4 v[2][8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[0][q] = *reinterpret_cast<const float4*>(nd + 4 * q);
#pragma unroll
        for (int m = 0; m < 31; ++m) {
          if (m < 30)
#pragma unroll
            for (int q = (m + 2) / 4; q < 8; ++q) v[(m + 1) & 1][q] = *reinterpret_cast<const float4*>(nd + (m + 1) * NS + 4 * q);
          const float xm = m & 1 ? x[m / 2].y : x[m / 2].x;
#pragma unroll
          for (int q = (m + 1) / 4; q < 8; ++q) {
            const float4 t = v[m & 1][q];
            if (4 * q + 1 > m) x[2 * q] = fma_pair(make_float2(t.x, t.y), xm, x[2 * q]);
            x[2 * q + 1] = fma_pair(make_float2(t.z, t.w), xm, x[2 * q + 1]);
          }
        }
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
        __syncwarp();
        if (w == 0) {  // T11 by rows, in the place of N11
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            n[(2 * k) * NS + lane] = x[k].x;
            n[(2 * k + 1) * NS + lane] = x[k].y;
          }
        } else {  // T22 by columns, in the place of N22
#pragma unroll
          for (int k = 0; k < 16; k += 2)
            *reinterpret_cast<float4*>(n + (32 + lane) * NS + 32 + 2 * k) = make_float4(x[k].x, x[k].y, x[k + 1].x, x[k + 1].y);
        }
        sync_threads(10, 64);
        // rows 16 w .. of -N21 T11, then of T21 = T22 (-N21 T11)
        float2 y[8];
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = make_float2(0.f, 0.f);
          const float* right = n + half * (32 * NS);
          const float* left = right + 32 + 16 * w;
#pragma unroll 8
          for (int m = 0; m < 32; ++m) {
            const float t = right[m * NS + lane];
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 v = *reinterpret_cast<const float4*>(left + m * NS + k);
              y[k / 2] = fma_pair(make_float2(v.x, v.y), t, y[k / 2]);
              y[k / 2 + 1] = fma_pair(make_float2(v.z, v.w), t, y[k / 2 + 1]);
            }
          }
          if (half == 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              n[(32 + 16 * w + 2 * k) * NS + lane] = y[k].x;
              n[(32 + 16 * w + 2 * k + 1) * NS + lane] = y[k].y;
            }
            sync_threads(10, 64);
          }
        }
        float topy = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) topy = fmaxf(topy, fmaxf(fabsf(y[k].x), fabsf(y[k].y)));
        tops[w * 32 + lane] = w == 0 ? fmaxf(top, topy) : topy;
        sync_threads(10, 64);
        const float top0 = fmaxf(tops[lane], tops[32 + lane]);
        const Scale s0 = scale_of(top0), s1 = scale_of(top);  // column lane; 32 + lane
        if (__any_sync(0xffffffffu, !(fmaxf(top0, top) < kGrown)) && lane == 0) again[ch & 3] = ch + 1;
        const uint32_t t = base + (uint32_t)(L::kT + (ch & 1) * L::kTBytes);
        const auto put = [&](int j, int q, const float2* v, float to) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(v[e].x * to, v[e].y * to, hi[e], lo[e]);
          st_shared4(t + swz(j, q), hi);
          st_shared4(t + L::kTile + swz(j, q), lo);
        };
        float* const f = reinterpret_cast<float*>(smem + L::kF + (ch % 3) * L::kFBytes);
        const Scale sx = w ? s1 : s0;
#pragma unroll
        for (int q = 0; q < 4; ++q) put(32 * w + lane, 4 * w + q, x + 4 * q, sx.to);
        f[L::kFv + 32 * w + lane] = sx.back;
        f[L::kFk + 32 * w + lane] *= sx.back;
        if (w) {
          const uint32_t zero[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            st_shared4(t + swz(32 + lane, q), zero);
            st_shared4(t + L::kTile + swz(32 + lane, q), zero);
          }
        }
        put(lane, 4 + 2 * w, y, s0.to);
        put(lane, 5 + 2 * w, y + 4, s0.to);
        fence_async();
        arrive(kbTM + (ch & 1));
      }
    } else if (warp == kIssueWarp) {
      // ---------------------------------------------------------- products of the state
      const auto kq_at = [&](int ch, int b) { return base + (uint32_t)(L::kKQ + (ch % 3) * L::kKQBytes + b * L::kBlock); };
      for (int ch = 0;; ++ch) {
        if (ch < chunks) wait(kbKQ + ch % 3, ch / 3);
#pragma unroll 1
        for (int i = 0; i < (KB == 2 ? 2 : 1); ++i) {   // X_K as the parts of S come: of each half of d_k 32, then 32
#pragma unroll 1
          for (int b = 0; b < KB; ++b) {
            wait(kbS + 2 * b + i, ch);  // behind the last chunk: dS has been read
            tc_after();
            if (ch < chunks && !dead) {
              const uint64_t k = desc_sw128(kq_at(ch, b), 16) + 4u * i;
#pragma unroll 1
              for (uint32_t part = 0; part < 2; ++part)
                mma_ts2<2>(tmem + kTmX, tmem + (part ? kTmSlo : kTmShi) + 32u * b + 16u * i, k, id_k, i + b + part > 0);
            }
          }
        }
        if constexpr (KB == 1) {
          if (ch < chunks && !dead) {
            const uint64_t k = desc_sw128(kq_at(ch, 0), 16) + 4u;
#pragma unroll 1
            for (uint32_t part = 0; part < 2; ++part)
              mma_ts2<2>(tmem + kTmX, tmem + (part ? kTmSlo : kTmShi) + 16u, k, id_k, 1);
          }
        }
        if (ch < chunks && !dead) mma_commit(bar(kbXK));
        if (ch) {  // O of the chunk before
          const int was = ch - 1;
          wait(kbM + (was & 1), was >> 1);
          if (!dead) {
            const uint64_t m = desc_sw128(base + (uint32_t)(L::kM + (was & 1) * L::kMBytes), 16);
            // U hi by M hi, U lo by M hi, U hi by M lo
#pragma unroll 1
            for (uint32_t part = 0; part < 3; ++part)
              mma_ts4<2>(tmem + kTmD, tmem + kTmR + (part == 1 ? 32u : 0u), m + (part == 2 ? (uint64_t)(L::kTile >> 4) : 0u), id_k,
                         part > 0);
            mma_commit(bar(kbO));
            mma_commit(bar(kbMFree + (was & 1)));
          }
        }
        if (ch == chunks) break;
        wait(kbTM + (ch & 1), ch >> 1);
        wait(kbR, ch);
        tc_after();
        if (!dead) {  // R hi and lo by T hi, R hi by T lo
          const uint64_t t = desc_sw128(base + (uint32_t)(L::kT + (ch & 1) * L::kTBytes), 16);
#pragma unroll 1
          for (uint32_t part = 0; part < 3; ++part)
            mma_ts4<128>(tmem + kTmX, tmem + kTmR + (part == 1 ? 32u : 0u), t + (part == 2 ? (uint64_t)(L::kTile >> 4) : 0u), id_mn,
                         part > 0);
          mma_commit(bar(kbU));
          mma_commit(bar(kbTFree + (ch & 1)));
        }
        if (ch) {
          wait(kbORead, ch - 1);
          tc_after();
        }
        if (!dead) {
#pragma unroll 1
          for (int b = 0; b < KB; ++b) {
            const uint64_t q = desc_sw128(kq_at(ch, b) + kC * 128u, 16);
#pragma unroll 1
            for (uint32_t part = 0; part < 2; ++part)
              mma_ts4<2>(tmem + kTmQ, tmem + (part ? kTmSlo : kTmShi) + 32u * b, q, id_k, b + part > 0);
          }
          mma_commit(bar(kbXQ));
        }
        wait(kbW, ch);
        tc_after();
        if (!dead) {
#pragma unroll 1
          for (int b = 0; b < KB; ++b) {
            const uint64_t k = desc_sw128(kq_at(ch, b), 16);
#pragma unroll 1
            for (uint32_t part = 0; part < 2; ++part)
              mma_ts4<128>(tmem + kTmD + 64u * b, tmem + kTmW + 32u * part, k, id_mn, part);
            mma_commit(bar(kbD + b));
          }
          mma_commit(bar(kbKQFree + ch % 3));
        }
      }
      mma_commit(bar(kbDrain));
      mbar_drain(bar(kbDrain), 0);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- copies; rows behind the request's last come along
      if (lane < 4) {
        const CUtensorMap* const m = &maps.k + lane;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
      }
      const int hq = h / a.group;
      int n_kq = 0, n_v = 0, n_kk = 0;  // begun
      const auto done = [&](int i, int use) { return __all_sync(0xffffffffu, is_done(bar(i), (uint32_t)(use & 1))); };
      // Each as soon as its place is free and its operands are there; the tries without any are bounded.
      for (int tries = 0; (n_kq < chunks || n_v < chunks || n_kk < chunks) && tries < kPolls && !*abort; ++tries) {
        if (n_kq < chunks && (n_kq < 3 || done(kbKQFree + n_kq % 3, n_kq / 3 - 1))) {
          if (lane == 0) {
            const int s = n_kq % 3;
            const uint32_t kq = base + (uint32_t)(L::kKQ + s * L::kKQBytes);
            mbar_expect_tx(bar(kbKQFull + s), (uint32_t)L::kKQBytes);
#pragma unroll 1
            for (int b = 0; b < KB; ++b) {
              tma_3d(kq + (uint32_t)(b * L::kBlock), &maps.k, 64 * b, hq, rq.first + n_kq * kC, bar(kbKQFull + s));
              tma_3d(kq + (uint32_t)(b * L::kBlock) + kC * 128u, &maps.q, 64 * b, hq, rq.first + n_kq * kC, bar(kbKQFull + s));
            }
          }
          __syncwarp();
          ++n_kq;
          tries = 0;
        }
        if (n_v < chunks && (n_v < 2 || done(kbVFree + (n_v & 1), (n_v >> 1) - 1))) {
          if (lane == 0) {
            const int s = n_v & 1;
            mbar_expect_tx(bar(kbVFull + s), (uint32_t)L::kVBytes);
            tma_3d(base + (uint32_t)(L::kV + s * L::kVBytes), &maps.v, col0, h, rq.first + n_v * kC, bar(kbVFull + s));
          }
          __syncwarp();
          ++n_v;
          tries = 0;
        }
        if (n_kk < chunks && done(kbKQ + n_kk % 3, n_kk / 3)) {  // [K; Q] K^T
          tc_after();
#pragma unroll 1
          for (int b = 0; b < KB; ++b) {
            const uint64_t d = desc_sw128(base + (uint32_t)(L::kKQ + (n_kk % 3) * L::kKQBytes + b * L::kBlock), 16);
            mma_ss4(tmem + kTmKK, d, d, id_k, b > 0);
          }
          mma_commit(bar(kbKK));
          ++n_kk;
          tries = 0;
        }
        __nanosleep(100);
      }
      if (n_kk < chunks || n_v < chunks) *abort = 1;
      if (n_kk) mbar_drain(bar(kbKK), (uint32_t)((n_kk - 1) & 1));
      // no copy is in flight when the CTA ends (they have all been used unless a wait gave up)
      for (int i = n_kq > 3 ? n_kq - 3 : 0; i < n_kq; ++i) mbar_drain(bar(kbKQFull + i % 3), (uint32_t)((i / 3) & 1));
      for (int i = n_v > 2 ? n_v - 2 : 0; i < n_v; ++i) mbar_drain(bar(kbVFull + (i & 1)), (uint32_t)((i >> 1) & 1));
      __syncwarp();
    }
  }
  tc_before();
  __syncthreads();
  if (tid == 0 && *abort) *(a.status ? a.status : &g_delta_status) = 3;
  if (warp == kIssueWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <int DK, bool BF16>
cudaError_t launch(const DeltaArgs& a, cudaStream_t st) {
  constexpr int smem = Wide<DK, BF16>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(delta_wide_kernel<DK, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  alignas(64) DeltaMaps maps;
  const cuuint64_t qk[3] = {(cuuint64_t)DK, (cuuint64_t)(a.v_heads / a.group), (cuuint64_t)a.tokens};
  const cuuint64_t v[3] = {(cuuint64_t)a.d_v, (cuuint64_t)a.v_heads, (cuuint64_t)a.tokens};
  const cuuint32_t box[3] = {64, 1, kC}, v_box[3] = {kCols, 1, kC};
  const long long qs[2] = {a.q_head, a.q_token}, ks[2] = {a.k_head, a.k_token}, vs[2] = {a.v_head, a.v_token}, os[2] = {a.o_head, a.o_token};
  if (!tensor_map(&maps.q, BF16, a.q, 3, qk, qs, box) || !tensor_map(&maps.k, BF16, a.k, 3, qk, ks, box) ||
      !tensor_map(&maps.v, BF16, a.v, 3, v, vs, v_box, false) || !tensor_map(&maps.out, BF16, a.out, 3, v, os, v_box, false))
    return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((a.d_v + kCols - 1) / kCols), (unsigned)a.v_heads, (unsigned)a.requests);
  delta_wide_kernel<DK, BF16><<<grid, kWideThreads, smem, st>>>(a, maps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t delta_status(int* host, cudaStream_t st) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(host, g_delta_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *host) {
    static const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_delta_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

cudaError_t launch_delta_wide(const DeltaArgs& a, bool bf16, cudaStream_t st) {
  if (a.d_k == 64) return bf16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  return bf16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

}  // namespace vq3
