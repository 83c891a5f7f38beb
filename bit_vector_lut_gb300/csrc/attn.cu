// Attention of a few query rows per request over a long cache (single tokens, short verify
// steps), and the pass that combines the parts of a unit split between CTAs.
//
//   out[row] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - max),  j < seen(row)
//
// in one pass over the keys with a running maximum and sum (FP32). The keys and values of a
// request are read once for all rows of a key/value head: bound by the memory they are read
// from. Every warp walks its own groups of 16 tokens with its own maximum, sum and output
// and needs neither shared memory nor barriers until the end of a unit:
//   S^T[16 tokens][8 rows] = K Q^T: the A operand of m16n8k16 is taken straight from global
//     memory, 16 bytes a lane. Lane (g, t) of the MMA (g = lane / 4, t = lane % 4) reads
//     d = 32 c + 8 t .. + 7 of tokens g and g + 8; the order of d inside a 32-wide chunk is
//     permuted against the MMA's, the same way in Q.
//   O^T[16 d][8 rows] += V^T P^T: lane (g, t) reads d = 64 c + 8 g .. + 7 of tokens 2t, 2t + 1,
//     2t + 8, 2t + 9 (16 bytes each) and pairs neighbouring tokens with a byte permute; P^T is
//     S^T's accumulator packed to 16 bits and transposed by movmatrix.
// So the loads are whole 64- and 128-byte lines and the next group's keys and values load
// while this group's products run. 64 requests decoding at up to 16K keys of 8 x 128 (1.23 GB):
// 185-193 us, 6.4-6.6 TB/s, 94-98% of a plain copy's rate. A single request of 4,097 keys of
// 4 x 256 takes 14.5 us (2.5 us at that rate): finding the range, the first keys from
// memory, joining the 132 CTAs' parts.
#include "attn_common.cuh"

namespace vq3 {
VQ3_BOUNDS_RECORD(attn)
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = kWarps * 16;  // tokens of a tile: one group of 16 per warp
// Fewest tiles per CTA. (1 / 2 / 4: one token at some 1,000 keys of 8 x 128 7.9 / 8.6 / 10.1 us, four such
// 9.5 / 9.8 / 10.7, one at 4,097 of 4 x 256 14.8 / 14.7 / 15.6.)
constexpr int kMinTiles = 2;

// CTAs per SM: what registers allow (Q, O, and one group's K and V per thread).
template <int D, int NR>
constexpr int rows_occ() {
  return D == 256 ? 2 : (D == 128 ? (NR == 1 ? 3 : 2) : 4);
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (AttnType<T>::kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// 16 bytes, read once: not kept in L1.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

template <typename T, int D, int NR>
__global__ void __launch_bounds__(kThreads, rows_occ<D, NR>()) attn_rows_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int kRows = 8 * NR;
  constexpr int kC = D / 32;  // K chunks of 32
  constexpr int kV = D / 64;  // V chunks of 64
  constexpr float kOff = AttnType<T>::kOff;
  __shared__ unsigned s_sum[3 * kWarps];
  __shared__ AttnPos s_pos;
  __shared__ __align__(16) float s_o[kWarps][kRows][D + 4];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  const AttnPos pos = a.requests <= kWarpRequests ? attn_locate_warp(a, kTile, kMinTiles)
                                                  : attn_locate_block<kThreads>(a, kTile, kMinTiles, s_sum, &s_pos);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  AttnRec rec{};
  AttnWalk w;
  for (bool on = w.start(a, pos, kTile); on; on = w.next(a, kTile)) {
    const int rows = w.q.n_new * a.group, base = w.j * kRows;
    // Q: the B operand of S^T = K Q^T; row g of each block of 8
    uint4 qf[NR][kC];
    int lim[NR][2];  // keys that rows 2t and 2t + 1 of the block see
    int low = 0x7fffffff;
#pragma unroll
    for (int b = 0; b < NR; ++b) {
      const int p = base + b * 8 + g;
      const bool live = p < rows;
      const RowPlace rp = row_place(a, w.q.q0, w.h, live ? p : 0);
      const T* src = static_cast<const T*>(a.q) + rp.token * a.q_token + rp.head * a.q_head + 8 * t;
#pragma unroll
      for (int c = 0; c < kC; ++c)
        qf[b][c] = live && VQ3_IN(rp.token, a.tokens, 1) ? __ldg(reinterpret_cast<const uint4*>(src + 32 * c))
                                                          : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int pe = base + b * 8 + 2 * t + e;
        // rows beyond the last are computed on zeros and not written: nothing to mask
        lim[b][e] = pe < rows ? attn_seen(w.q, a.by_group(pe)) : 0x7fffffff;
      }
    }
    low = attn_seen(w.q, a.by_group(base));  // what the first row sees: no less than nothing is masked

    float m[NR][2], l[NR][2];
    float o[NR][D / 16][4];
#pragma unroll
    for (int b = 0; b < NR; ++b) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[b][e] = -INFINITY;
        l[b][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[b][i][e] = 0.f;
    }

    const int first = w.t0 * kTile + warp * 16;
    const int stop = w.t1 * kTile < w.end ? w.t1 * kTile : w.end;
    // page of the group that starts at token x (16 tokens never straddle pages of 16 and more)
    const auto page_of = [&](int x) -> int {
      if (!a.table) return 0;
      if (x >= stop) return -1;
      const size_t at = (size_t)w.r * a.max_pages + (x >> a.page_shift);
      return VQ3_IN(at, (size_t)a.requests * a.max_pages, 2) ? __ldg(a.table + at) : -1;
    };
    const T* const kh = static_cast<const T*>(a.k) + (long long)w.h * a.k_head;
    const T* const vh = static_cast<const T*>(a.v) + (long long)w.h * a.v_head;
    // A page number outside the cache reads as zeros; so do tokens the request does not have.
    const auto bad = [&](int page) { return a.table && (unsigned)page >= (unsigned)a.n_pages; };
    uint4 kf[kC][2], vf[kV][4];
    const auto load_k = [&](int x, int page) {
      const long long in = a.table ? (long long)(x & ((1 << a.page_shift) - 1)) : (long long)w.q.q0 + x;
      const T* p = kh + (long long)(a.table ? page : 0) * a.k_page + 8 * t;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = g + 8 * e;
        const bool ok = x + tok < stop && !bad(page);
#pragma unroll
        for (int c = 0; c < kC; ++c)
          kf[c][e] = ok ? ldg_stream(p + (in + tok) * a.k_token + 32 * c) : make_uint4(0, 0, 0, 0);
      }
    };
    const auto load_v = [&](int x, int page) {
      const long long in = a.table ? (long long)(x & ((1 << a.page_shift) - 1)) : (long long)w.q.q0 + x;
      const T* p = vh + (long long)(a.table ? page : 0) * a.v_page + 8 * g;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int tok = 2 * t + (e & 1) + 8 * (e >> 1);
        const bool ok = x + tok < stop && !bad(page);
#pragma unroll
        for (int c = 0; c < kV; ++c)
          vf[c][e] = ok ? ldg_stream(p + (in + tok) * a.v_token + 64 * c) : make_uint4(0, 0, 0, 0);
      }
    };

    int page = page_of(first), next_page = page_of(first + kTile);
    if (first < stop) {
      load_k(first, page);
      load_v(first, page);
    }
    for (int x = first; x < stop; x += kTile) {
      float s[NR][4];
#pragma unroll
      for (int b = 0; b < NR; ++b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[b][e] = 0.f;
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          mma16816<T>(s[b], kf[c][0].x, kf[c][1].x, kf[c][0].y, kf[c][1].y, qf[b][c].x, qf[b][c].y);
          mma16816<T>(s[b], kf[c][0].z, kf[c][1].z, kf[c][0].w, kf[c][1].w, qf[b][c].z, qf[b][c].w);
        }
      }
      const int xn = x + kTile;
      page = next_page;
      if (xn < stop) load_k(xn, page);
      next_page = page_of(xn + kTile);

      bool raise = false;
#pragma unroll
      for (int b = 0; b < NR; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[b][e] *= a.scale_log2;
          if (x + 16 > low || x + 16 > stop) {
            const int tok = x + g + 8 * (e >> 1);
            if (tok >= lim[b][e & 1] || tok >= stop) s[b][e] = -INFINITY;
          }
          raise |= s[b][e] > m[b][e & 1] + kLag;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int b = 0; b < NR; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[b][e], s[b][e + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            mx = fmaxf(mx, m[b][e]);
            const float f = m[b][e] == mx ? 1.f : ex2(m[b][e] - mx);  // equal infinities: nothing to rescale
            m[b][e] = mx;
            l[b][e] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[b][i][e] *= f;
              o[b][i][e + 2] *= f;
            }
          }
      }
      uint32_t pb[NR][2];
#pragma unroll
      for (int b = 0; b < NR; ++b) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mm = m[b][e & 1] == -INFINITY ? 0.f : m[b][e & 1];
          p[e] = ex2(s[b][e] - mm + kOff);
          l[b][e & 1] += p[e];
        }
        pb[b][0] = transpose8x8(pack2<T>(p[0], p[1]));
        pb[b][1] = transpose8x8(pack2<T>(p[2], p[3]));
      }
#pragma unroll
      for (int c = 0; c < kV; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x0 = word(vf[c][0], i), x1 = word(vf[c][1], i), x2 = word(vf[c][2], i), x3 = word(vf[c][3], i);
          const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
          const uint32_t a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
          for (int b = 0; b < NR; ++b) mma16816<T>(o[b][4 * c + i], a0, a1, a2, a3, pb[b][0], pb[b][1]);
        }
      if (xn < stop) load_v(xn, page);
    }

    // the warps' parts of this unit, side by side in shared memory
#pragma unroll
    for (int b = 0; b < NR; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
        const int row = b * 8 + 2 * t + e;
        if (g == 0) {
          s_m[warp][row] = m[b][e];
          s_l[warp][row] = l[b][e];
        }
#pragma unroll
        for (int c = 0; c < kV; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = 64 * c + 8 * g + 2 * i;
            *reinterpret_cast<float2*>(&s_o[warp][row][d]) = make_float2(o[b][4 * c + i][e], o[b][4 * c + i][e + 2]);
          }
      }
    __syncthreads();
    const bool whole = w.whole();
    const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
    if (!whole) {
      if (w.t0 > 0) {
        rec.flags |= kRecHead | (w.t1 == w.n ? kRecEnd : 0);
      } else {
        rec.flags |= kRecTail;
        rec.q0 = w.q.q0;
        rec.rows = rows;
        rec.base = base;
        rec.head = w.h;
        rec.used = w.q.used;
      }
    }
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
      // four columns of a row: neighbouring threads take a row's columns of the output, or the
      // rows of a part ([slot][D / 4][rows] of four columns)
      const int row = whole ? i / (D / 4) : i % kRows, d = (whole ? i % (D / 4) : i / kRows) * 4;
      if (base + row >= rows) continue;
      float mx = s_m[0][row];
#pragma unroll
      for (int v = 1; v < kWarps; ++v) mx = fmaxf(mx, s_m[v][row]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float f = s_m[v][row] == mx ? 1.f : ex2(s_m[v][row] - mx);
        const float4 x = *reinterpret_cast<const float4*>(&s_o[v][row][d]);
        sum += f * s_l[v][row];
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      if (whole) {
        const RowPlace rp = row_place(a, w.q.q0, w.h, base + row);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (VQ3_IN(rp.token, a.tokens, 3)) {
          uint2 y;
          y.x = pack2<T>(acc.x * inv, acc.y * inv);
          y.y = pack2<T>(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + rp.token * a.o_token + rp.head * a.o_head + d) = y;
          if (a.lse && d == 0)
            a.lse[rp.token * a.heads + rp.head] = sum == 0.f ? -INFINITY : (mx - kOff + log2f(sum)) * 0.6931471805599453f;
        }
      } else {
        const size_t at = (size_t)slot * kRows + row;
        if (VQ3_IN(at, (size_t)2 * gridDim.x * kRows, 4)) {
          __stcg(reinterpret_cast<float4*>(a.part) + ((size_t)slot * (D / 4) + d / 4) * kRows + row, acc);
          if (d == 0) __stcg(reinterpret_cast<float2*>(a.part_ml + 2 * at), make_float2(mx, sum));
        }
      }
    }
    __syncthreads();  // before the next unit's parts
  }
  if (tid == 0) a.rec[blockIdx.x] = rec;
}

// ---------------------------------------------------------------- combining pass
//
// The parts of a split unit are slot 2c + 1 of the CTA c that began it and then slot 2c' of the
// CTAs right behind, up to the one that ends it. Block (c, y) takes rows and columns y of the
// unit that CTA c began, if it did. A thread sums four columns of a row over the parts, in CTA
// order, a batch of parts at a time; the row kernel's units, of few rows and often very many
// parts, get 32 columns a block and four groups of threads, each a fixed quarter of the
// parts. Bound by latency, so there are two dependent reads in all: the records, then the
// parts. Only one warp of a block reads records: they are few lines of L2, and all warps of all
// blocks asking for them took longer than the sums.
constexpr int kCThreads = 256;
constexpr int kMaxGrid = 608;  // CTAs of an attention kernel

template <bool kWide, int D>
struct CombineCfg {
  static constexpr int kRows = kWide ? 16 : 8;      // rows of a block
  static constexpr int kQuads = kWide ? 16 : 8;     // its columns, in fours, of one pass
  static constexpr int kPasses = kWide ? D / 64 : 1;
  static constexpr int kGroups = kWide ? 1 : 4;     // groups of threads that share the parts
  static constexpr int kBatch = 4;                   // parts read at once
  static constexpr int kAcross = D / 4 / kQuads / kPasses;    // blocks over the columns
  static_assert(kRows * kQuads * kGroups == kCThreads, "a thread per row, four columns and group");
};

struct Merge {  // running maximum (log2 domain), sum and four columns
  float m, l;
  float4 o;
  __device__ __forceinline__ void scale(float up) {
    const float f = m == up ? 1.f : ex2(m - up);  // equal infinities: nothing to rescale
    m = up;
    l *= f;
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
  }
  __device__ __forceinline__ void add(float pm, float pl, const float4& po) {  // pm <= m
    const float f = pm == m ? 1.f : ex2(pm - m);
    l += f * pl;
    o.x += f * po.x;
    o.y += f * po.y;
    o.z += f * po.z;
    o.w += f * po.w;
  }
};

template <typename T, int D, bool kWide>
__global__ void __launch_bounds__(kCThreads) attn_combine_kernel(const __grid_constant__ AttnArgs a, int grid,
                                                                 int slot_rows) {
  using C = CombineCfg<kWide, D>;
  __shared__ Merge s_merge[C::kGroups > 1 ? C::kGroups - 1 : 1][64];
  __shared__ int4 s_rec;  // of the unit: parts (0: none), q0, rows, base
  __shared__ int2 s_more;  // key/value head, rows of a block that are used
  const int tid = threadIdx.x, c = blockIdx.x;
  const int row0 = (int)blockIdx.y / C::kAcross * C::kRows, q0 = (int)blockIdx.y % C::kAcross * C::kQuads;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel has ended
  if (tid < 32) {
    // from L2: this block may have started before the records were written
    int4 rec = __ldcg(reinterpret_cast<const int4*>(a.rec + c));  // flags, q0, rows, base
    const int2 more = make_int2(__ldcg(&a.rec[c].head), __ldcg(&a.rec[c].used));
    int flags = c + 1 + tid < grid ? __ldcg(&a.rec[c + 1 + tid].flags) : kRecEnd;
    int n = 0;
    if ((rec.x & kRecTail) && attn_packed_row(a, row0, rec.w, rec.z, more.y) >= 0) {
      // parts: up to the first CTA that ends the unit
      for (n = 1;;) {
        const unsigned ends = __ballot_sync(0xffffffffu, flags & kRecEnd);
        n += ends ? __ffs(ends) : 32;
        if (ends) break;
        flags = c + n + tid < grid ? __ldcg(&a.rec[c + n + tid].flags) : kRecEnd;
      }
      if (n > grid - c) n = grid - c;
    }
    rec.x = n;
    if (tid == 0) {
      s_rec = rec;
      s_more = more;
    }
  }
  if (c == 0 && blockIdx.y == 0) {
    // the workspace's status word: whether a wait of any CTA gave up
    int failed = 0;
    for (int i = tid; i < grid; i += kCThreads) failed |= __ldcg(&a.rec[i].flags) & kRecFailed;
    failed = __syncthreads_or(failed);
    if (tid == 0) *a.status = failed ? 3 : 0;
  }
  __syncthreads();
  const int4 rec = s_rec;
  const int n = rec.x;
  if (n == 0) return;
  const int row = row0 + tid % C::kRows, group = tid / (C::kRows * C::kQuads);
  const int p = attn_packed_row(a, row, rec.w, rec.z, s_more.y);
  const RowPlace rp = row_place(a, rec.y, s_more.x, p < 0 ? 0 : p);
  const bool ok = p >= 0 && VQ3_IN(rp.token, a.tokens, 6);
  const float2* const ml = reinterpret_cast<const float2*>(a.part_ml) + row;
#pragma unroll 1
  for (int pass = 0; pass < C::kPasses; ++pass) {
    const int quad = q0 + pass * C::kQuads + tid / C::kRows % C::kQuads;
    const float4* const src = reinterpret_cast<const float4*>(a.part) + (size_t)quad * slot_rows + row;
    Merge acc = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (ok) {
      for (int i0 = group; i0 < n; i0 += C::kGroups * C::kBatch) {
        float2 w[C::kBatch];
        float4 x[C::kBatch];
#pragma unroll
        for (int k = 0; k < C::kBatch; ++k) {
          const int i = i0 + k * C::kGroups;
          const size_t slot = 2 * (c + i) + (i == 0);
          const bool in = i < n && VQ3_IN(slot, 2 * grid, 5);
          w[k] = in ? __ldcg(ml + slot * slot_rows) : make_float2(-INFINITY, 0.f);
          x[k] = in ? __ldcg(src + slot * (D / 4) * slot_rows) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float up = acc.m;
#pragma unroll
        for (int k = 0; k < C::kBatch; ++k) up = fmaxf(up, w[k].x);
        acc.scale(up);
#pragma unroll
        for (int k = 0; k < C::kBatch; ++k) acc.add(w[k].x, w[k].y, x[k]);
      }
    }
    if constexpr (C::kGroups > 1) {
      if (group) s_merge[group - 1][tid & 63] = acc;
      __syncthreads();
      if (group) return;
#pragma unroll
      for (int v = 0; v < C::kGroups - 1; ++v) {
        const Merge x = s_merge[v][tid];
        acc.scale(fmaxf(acc.m, x.m));
        acc.add(x.m, x.l, x.o);
      }
    }
    if (!ok) return;
    const float inv = acc.l == 0.f ? 0.f : 1.f / acc.l;
    uint2 y;
    y.x = pack2<T>(acc.o.x * inv, acc.o.y * inv);
    y.y = pack2<T>(acc.o.z * inv, acc.o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + rp.token * a.o_token + rp.head * a.o_head + 4 * quad) = y;
    if (a.lse && quad == 0)
      a.lse[rp.token * a.heads + rp.head] =
          acc.l == 0.f ? -INFINITY : (acc.m - AttnType<T>::kOff + log2f(acc.l)) * 0.6931471805599453f;
  }
}

template <typename T, int D, int NR>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t st) {
  attn_rows_kernel<T, D, NR><<<attn_rows_grid(D, 8 * NR), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_rows_t(const AttnArgs& a, int d, int nr, cudaStream_t st) {
  if (d == 64) return nr == 1 ? launch_rows<T, 64, 1>(a, st) : launch_rows<T, 64, 2>(a, st);
  if (d == 128) return nr == 1 ? launch_rows<T, 128, 1>(a, st) : launch_rows<T, 128, 2>(a, st);
  return launch_rows<T, 256, 1>(a, st);
}

template <typename T, int D, bool kWide>
cudaError_t launch_combine(const AttnArgs& a, int grid, int slot_rows, cudaStream_t st) {
  using C = CombineCfg<kWide, D>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, slot_rows / C::kRows * C::kAcross);
  cfg.blockDim = dim3(kCThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its launch overlaps the attention kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_combine_kernel<T, D, kWide>, a, grid, slot_rows);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename T, bool kWide>
cudaError_t launch_combine_t(const AttnArgs& a, int d, int grid, int slot_rows, cudaStream_t st) {
  if (d == 64) return launch_combine<T, 64, kWide>(a, grid, slot_rows, st);
  if (d == 128) return launch_combine<T, 128, kWide>(a, grid, slot_rows, st);
  return launch_combine<T, 256, kWide>(a, grid, slot_rows, st);
}

}  // namespace

int attn_rows_limit(int head_dim) { return head_dim == 256 ? 8 : 16; }

int attn_rows_unit_cost() { return 1; }

int attn_rows_grid(int head_dim, int rows) {
  const bool one = rows <= 8;
  const int occ = head_dim == 256   ? rows_occ<256, 1>()
                  : head_dim == 128 ? (one ? rows_occ<128, 1>() : rows_occ<128, 2>())
                                    : (one ? rows_occ<64, 1>() : rows_occ<64, 2>());
  const int g = occ * device_sm_count();
  return g > kMaxGrid ? kMaxGrid : g;
}

cudaError_t launch_attn_rows(const AttnArgs& a, int head_dim, bool bf16, int nr, cudaStream_t st) {
  return bf16 ? launch_rows_t<__nv_bfloat16>(a, head_dim, nr, st) : launch_rows_t<__half>(a, head_dim, nr, st);
}

cudaError_t launch_attn_combine(const AttnArgs& a, int head_dim, bool bf16, int grid, int slot_rows,
                                cudaStream_t st) {
  if (slot_rows > 16)
    return bf16 ? launch_combine_t<__nv_bfloat16, true>(a, head_dim, grid, slot_rows, st)
                : launch_combine_t<__half, true>(a, head_dim, grid, slot_rows, st);
  return bf16 ? launch_combine_t<__nv_bfloat16, false>(a, head_dim, grid, slot_rows, st)
              : launch_combine_t<__half, false>(a, head_dim, grid, slot_rows, st);
}

}  // namespace vq3
