// What the two attention kernels and their combining pass share: arguments, the row
// packing of grouped heads, and the division of the work between CTAs.
//
// A unit is one request, one key/value head and up to `unit_rows` packed query rows; the
// rows of a key/value head are (new token, query head of its group), row p = token p / G,
// query head p % G, so the G heads of a group share every key and value that is read. A
// unit's keys [0, end) are walked in tiles of kv_tile; end is what its last row sees.
// All units, laid end to end (request, key/value head, row block), each as long as its tiles
// and unit_cost more for starting and ending it, are cut into equal contiguous ranges, one
// per CTA. (Without the unit_cost the launch ran 25% longer than the mean CTA of a 4,096-token
// prompt of 32 x 128.) A CTA that holds all of a unit writes its output; otherwise it leaves
// (max, sum, unnormalised output) in a slot of its own, at most two per CTA: slot 2c for a unit
// that an earlier CTA began, slot 2c + 1 for one that it begins and does not end. The combining
// pass sums a unit's slots in CTA order, so results do not depend on timing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vq3_internal.h"

namespace vq3 {

// Per-CTA record of what it left in its slots.
struct AttnRec {
  int flags;                 // kRec*
  int q0, rows, base, head, used;  // of the unit it begins in slot 2c + 1: first query row, packed
                                   // rows of the request, first packed row of the unit, key/value
                                   // head, rows of a block that are used
  int pad[2];
};
constexpr int kRecHead = 1;     // slot 2c holds a part of a unit that an earlier CTA began
constexpr int kRecEnd = 2;      // and the unit ends there
constexpr int kRecTail = 4;     // slot 2c + 1 holds the first part of a unit
constexpr int kRecFailed = 8;   // a bounded wait of this CTA gave up

// x / d for 0 <= x < 2^31 by a multiplication: with s = ceil(log2 d) and m = floor(2^(31 + s) /
// d) + 1, m d exceeds 2^(31 + s) by at most d <= 2^s, so x m / 2^(31 + s) lies in [x / d, x / d +
// 1 / d) and its floor is the quotient.
struct FastDiv {
  unsigned m = 0;
  int s = 0, d = 1;
  FastDiv() = default;
  explicit FastDiv(int div) : d(div) {
    while ((1LL << s) < div) ++s;
    m = (unsigned)((1ULL << (31 + s)) / (unsigned)div + 1);
    s += 31;
  }
  __device__ __forceinline__ int operator()(int x) const {
    return (int)(((unsigned long long)(unsigned)x * m) >> s);
  }
};

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;  // or null
  long long q_token, q_head, o_token, o_head;  // strides in elements
  long long k_page, k_token, k_head, v_page, v_token, v_head;
  const int* q_start;  // [requests + 1]
  const int* kv_len;   // [requests] (paged) or null: as many keys as new tokens, at row q_start
  const int* table;    // [requests][max_pages] or null
  int tokens, requests, heads, kv_heads, group;
  int page_shift, max_pages, n_pages;
  int max_kv;          // no request sees more keys than this (paged: max_pages pages)
  // A unit has unit_blocks blocks of block_rows rows, all of them used, or only token_rows of them
  // so that a block holds whole tokens (see attn_request).
  int unit_blocks, block_rows, token_rows;
  int unit_cost;       // what a unit costs beside its tiles, in tiles
  FastDiv by_group, by_unit, by_token_unit;  // group, unit_blocks * block_rows, unit_blocks * token_rows
  float scale_log2;    // scale * log2(e)
  float* part;         // [2 * grid][slot rows][D] unnormalised outputs
  float* part_ml;      // [2 * grid][slot rows][2] max (log2 domain), sum
  AttnRec* rec;        // [grid]
  int* status;         // workspace status word
};

// P is rounded to the type of V: exp2(s - max + kOff). FP16 keeps 2^-14 .. 65504 at full
// precision; the offset moves that window to where the probabilities are (2^-21 .. 2^8
// relative to the running maximum, which may lag by 2^kLag).
template <typename T>
struct AttnType;
template <>
struct AttnType<__half> {
  static constexpr float kOff = 7.f;
  static constexpr bool kBf16 = false;
};
template <>
struct AttnType<__nv_bfloat16> {
  static constexpr float kOff = 0.f;
  static constexpr bool kBf16 = true;
};
// The running maximum is only raised once a score exceeds it by 2^kLag: rescaling the
// output is then rare after the first tiles, and exp2 stays below 2^(kLag + kOff).
constexpr float kLag = 8.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (AttnType<T>::kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- units and ranges

struct AttnRequest {
  int q0, n_new, kv, units;  // first query row, new tokens, keys, units per key/value head
  int used;                  // rows of a block that are used
};

// Lengths from device memory, clamped so that no later index leaves its buffer. Starts that do not
// ascend make requests overlap; each still lies inside q and out, but the batch's cost, which the
// entry points bound for ascending ones, may then pass 2^32: a range is cut wrongly, its place is
// still one inside some request (an offset found in a request is below that request's own cost).
__device__ __forceinline__ AttnRequest attn_request(const AttnArgs& a, int r) {
  AttnRequest q;
  int s = a.q_start[r], e = a.q_start[r + 1];
  s = s < 0 ? 0 : (s > a.tokens ? a.tokens : s);
  e = e < s ? s : (e > a.tokens ? a.tokens : e);
  q.q0 = s;
  q.n_new = e - s;
  if (a.kv_len) {
    const int n = a.kv_len[r];
    q.kv = n < 0 ? 0 : (n > a.max_kv ? a.max_kv : n);
  } else {
    q.kv = q.n_new;
  }
  // A block of whole tokens is copied at once, one that cuts a token token by token and row by row:
  // worth it where it saves a tenth of the units (64 tokens of 6 heads: 3 blocks instead of 4, 173
  // -> 139 us behind 98,304 keys of 4 x 256; prompts of thousands of such tokens: 390 -> 441 us).
  const int rows = q.n_new * a.group;
  q.used = a.block_rows;
  q.units = a.by_unit(rows + a.unit_blocks * a.block_rows - 1);
  if (a.token_rows != a.block_rows) {
    const int aligned = a.by_token_unit(rows + a.unit_blocks * a.token_rows - 1);
    if (10 * aligned <= 11 * q.units) {
      q.used = a.token_rows;
      q.units = aligned;
    }
  }
  return q;
}

// Keys that new token t of the request sees: 0 .. kv - n_new + t.
__device__ __forceinline__ int attn_seen(const AttnRequest& q, int t) {
  const int n = q.kv - q.n_new + t + 1;
  return n < 0 ? 0 : n;
}
// Keys that the last row of unit j sees.
__device__ __forceinline__ int attn_unit_end(const AttnArgs& a, const AttnRequest& q, int j) {
  const int t = a.by_group((j + 1) * a.unit_blocks * q.used - 1);  // tokens * heads < 2^30
  return attn_seen(q, t < q.n_new - 1 ? t : q.n_new - 1);
}
// Tiles of unit j; a unit that sees nothing still counts as one, its rows are written too.
__device__ __forceinline__ int attn_unit_tiles(const AttnArgs& a, const AttnRequest& q, int j, int kv_tile) {
  const int n = (int)((unsigned)(attn_unit_end(a, q, j) + kv_tile - 1) / (unsigned)kv_tile);
  return n < 1 ? 1 : n;
}

struct AttnPos {
  int r, h, j, at;  // request, key/value head, unit of the head, offset in it: unit_cost, then its tiles
  unsigned cost;    // length of this CTA's range (0: none)
};

// How a batch is divided. Plain: all tiles in one line, cut into equal ranges. Where the
// units of a request share its keys (several row blocks) and units are few, every unit gets
// CTAs of its own instead, in proportion to its tiles, and its tiles are cut evenly among
// them: units of equal length are then walked in step and all but the first read find the
// keys in L2. Taken up to half as many units as CTAs. Behind 98,304 keys of 4 x 256, 24 heads, CTAs
// of their own / the plain cut: 12 units (64 tokens) 141 / 203 us, 24 units 244 / 268, 52 units 673
// / 738, 64 units 679 / 789. The shares are whole CTAs, rounded down, which costs most at the border:
// 76 units (384 tokens) get one or two each, 1,323 us against 721. Above it both are far from their
// operations, 100 units (512 tokens) 1,299 / 1,425 (666). 32 heads on 8 x 128: 8 units 103 to 134 /
// 141, 32 units 385 / 348.
struct AttnCut {
  unsigned cost;  // of the batch
  int units;      // of the batch; 0: the plain cut
  int ctas;
};
// What unit j counts: its cost, or the CTAs that are its own. (The batch's costs stay below
// 2^32: the entry points check a bound.)
__device__ __forceinline__ unsigned attn_unit_cost(const AttnArgs& a, const AttnRequest& q, int j, int kv_tile,
                                                   int min_tiles, const AttnCut& cut) {
  const unsigned n = attn_unit_tiles(a, q, j, kv_tile);
  if (cut.units == 0) return n + a.unit_cost;
  const unsigned spare = cut.ctas - cut.units, most = n / min_tiles;
  // at most the exact share, so that all shares fit the grid: the factor outweighs three roundings
  const unsigned c = 1 + (unsigned)((float)spare * (n + a.unit_cost) / cut.cost * 0.999999f);
  return c <= most ? c : (most < 1 ? 1 : most);
}

// Cost of each lane's request (0 beyond the last), found by the whole warp where a request
// has many units.
__device__ __forceinline__ unsigned attn_costs(const AttnArgs& a, int r, int kv_tile, int min_tiles,
                                               const AttnCut& cut, int lane, int* units) {
  AttnRequest q{};
  if (r < a.requests) q = attn_request(a, r);
  *units = q.units;
  unsigned c = 0;
  if (q.units <= 4)
    for (int j = 0; j < q.units; ++j) c += attn_unit_cost(a, q, j, kv_tile, min_tiles, cut);
  unsigned big = __ballot_sync(0xffffffffu, q.units > 4);
  while (big) {
    const int src = __ffs(big) - 1;
    big &= big - 1;
    AttnRequest o;
    o.q0 = 0;
    o.n_new = __shfl_sync(0xffffffffu, q.n_new, src);
    o.kv = __shfl_sync(0xffffffffu, q.kv, src);
    o.units = __shfl_sync(0xffffffffu, q.units, src);
    o.used = __shfl_sync(0xffffffffu, q.used, src);
    unsigned s = 0;
    for (int j = lane; j < o.units; j += 32) s += attn_unit_cost(a, o, j, kv_tile, min_tiles, cut);
    s = __reduce_add_sync(0xffffffffu, s);
    if (lane == src) c = s;
  }
  return c * a.kv_heads;
}

// This CTA's range of `total`, in tiles (plain cut) or as the number of a CTA.
__device__ __forceinline__ void attn_range(const AttnCut& cut, unsigned total, int min_tiles, unsigned* s0,
                                           unsigned* s1) {
  const unsigned c = blockIdx.x;
  if (cut.units) {
    *s0 = c;
    *s1 = c < total ? c + 1 : c;
    return;
  }
  unsigned live = total / min_tiles;
  live = live < 1 ? 1 : (live > (unsigned)cut.ctas ? cut.ctas : live);
  const unsigned each = total / live, more = total - each * live;  // the first `more` CTAs take one more
  *s0 = c < live ? each * c + (c < more ? c : more) : total;
  *s1 = c < live ? *s0 + each + (c < more ? 1 : 0) : total;
}

// The whole warp: where inside request r (whose cost is `cost`) offset `off` falls.
__device__ __forceinline__ void attn_inside(const AttnArgs& a, int r, unsigned cost, unsigned off, int kv_tile,
                                            int min_tiles, const AttnCut& cut, unsigned plain, int lane,
                                            AttnPos* pos) {
  const unsigned per_head = cost / a.kv_heads;
  const AttnRequest q = attn_request(a, r);
  const int h = (int)(off / per_head);
  unsigned left = off - h * per_head;
  int j = 0, at = 0, n = 0;
  for (int j0 = 0; j0 < q.units; j0 += 32) {
    const int mine = j0 + lane;
    const unsigned c = mine < q.units ? attn_unit_cost(a, q, mine, kv_tile, min_tiles, cut) : 0;
    unsigned in = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned o = __shfl_up_sync(0xffffffffu, in, d);
      if (lane >= d) in += o;
    }
    const unsigned here = __ballot_sync(0xffffffffu, left >= in - c && left < in);
    if (here) {
      const int src = __ffs(here) - 1;
      j = j0 + src;
      n = (int)__shfl_sync(0xffffffffu, c, src);
      at = (int)(left - __shfl_sync(0xffffffffu, in, src)) + n;
      break;
    }
    left -= __shfl_sync(0xffffffffu, in, 31);
  }
  pos->r = r;
  pos->h = h;
  pos->j = j;
  if (cut.units) {  // CTA `at` of the unit's n
    const unsigned long long tiles = attn_unit_tiles(a, q, j, kv_tile);
    const unsigned t0 = (unsigned)(tiles * at / n), t1 = (unsigned)(tiles * (at + 1) / n);
    pos->at = t0 ? (int)t0 + a.unit_cost : 0;
    pos->cost = t1 + a.unit_cost - pos->at;
  } else {
    pos->at = at;
    pos->cost = plain;
  }
}

// Few requests: every warp finds the CTA's range by itself, without a barrier. (Single tokens of 32
// heads on 8 x 128, up to 600 keys, each warp / the warps together: 48 requests 19.4 / 20.1 us, 100
// and 120 no difference, 200 49.5 / 48.3, 800 168.7 / 159.6.)
constexpr int kWarpRequests = 128;
__device__ __forceinline__ AttnPos attn_locate_warp(const AttnArgs& a, int kv_tile, int min_tiles) {
  const int lane = threadIdx.x & 31, per = (a.requests + 31) / 32;
  AttnCut cut{0, 0, (int)gridDim.x};
  AttnPos pos{};
  unsigned mine, total, before;
  for (int pass = 0;; ++pass) {
    int units = 0, most = 0;
    mine = 0;
    for (int i = 0; i < per; ++i) {
      int u;
      mine += attn_costs(a, lane * per + i, kv_tile, min_tiles, cut, lane, &u);
      units += u * a.kv_heads < cut.ctas ? u * a.kv_heads : cut.ctas;
      most = u > most ? u : most;
    }
    unsigned incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    before = incl - mine;
    if (pass || !__any_sync(0xffffffffu, most > 1)) break;
    const int all = __reduce_add_sync(0xffffffffu, units);
    if (2 * all > cut.ctas) break;
    cut.cost = total;
    cut.units = all;
  }
  unsigned s0, s1;
  attn_range(cut, total, min_tiles, &s0, &s1);
  if (s1 <= s0) return pos;
  for (int i = 0; i < per; ++i) {
    int u;
    const int r = lane * per + i;
    const unsigned cost = per == 1 ? mine : attn_costs(a, r, kv_tile, min_tiles, cut, lane, &u);
    const unsigned hit = __ballot_sync(0xffffffffu, before <= s0 && s0 < before + cost);
    if (hit) {
      const int src = __ffs(hit) - 1;
      attn_inside(a, __shfl_sync(0xffffffffu, r, src), __shfl_sync(0xffffffffu, cost, src),
                  s0 - __shfl_sync(0xffffffffu, before, src), kv_tile, min_tiles, cut, s1 - s0, lane, &pos);
      break;
    }
    before += cost;
  }
  return pos;
}

// Many requests: the CTA's warps share them. Thread i looks after requests [i * per, (i + 1) *
// per), so the order is the requests'. Every thread of the CTA calls it; `sm` is shared memory
// for 3 * kThreads / 32 sums and `result` the shared result.
template <int kThreads>
__device__ __noinline__ AttnPos attn_locate_block(const AttnArgs& a, int kv_tile, int min_tiles, unsigned* sm,
                                                  AttnPos* result) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (a.requests + kThreads - 1) / kThreads;
  AttnCut cut{0, 0, (int)gridDim.x};
  unsigned mine, total, before;
  for (int pass = 0;; ++pass) {
    int units = 0, most = 0;
    mine = 0;
    for (int i = 0; i < per; ++i) {
      int u;
      mine += attn_costs(a, tid * per + i, kv_tile, min_tiles, cut, lane, &u);
      units += u * a.kv_heads < cut.ctas ? u * a.kv_heads : cut.ctas;
      most = u > most ? u : most;
    }
    unsigned incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    units = __reduce_add_sync(0xffffffffu, units);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) {
      sm[warp] = incl;
      sm[kWarps + warp] = units;
      sm[2 * kWarps + warp] = most;
    }
    __syncthreads();
    unsigned all = 0, big = 0;
    total = 0;
    before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm[w];
      total += sm[w];
      all += sm[kWarps + w];
      big = sm[2 * kWarps + w] > big ? sm[2 * kWarps + w] : big;
    }
    __syncthreads();
    if (pass || big <= 1 || 2 * all > (unsigned)cut.ctas) break;
    cut.cost = total;
    cut.units = (int)all;
  }
  unsigned s0, s1;
  attn_range(cut, total, min_tiles, &s0, &s1);
  if (tid == 0) result->cost = 0;
  __syncthreads();
  const unsigned warp_end = __shfl_sync(0xffffffffu, before + mine, 31);
  if (s1 > s0 && __shfl_sync(0xffffffffu, before, 0) <= s0 && s0 < warp_end) {
    // this warp's requests hold the range's start
    for (int i = 0; i < per; ++i) {
      int u;
      const int r = tid * per + i;
      const unsigned cost = attn_costs(a, r, kv_tile, min_tiles, cut, lane, &u);
      const unsigned hit = __ballot_sync(0xffffffffu, before <= s0 && s0 < before + cost);
      if (hit) {
        const int src = __ffs(hit) - 1;
        AttnPos pos{};
        attn_inside(a, __shfl_sync(0xffffffffu, r, src), __shfl_sync(0xffffffffu, cost, src),
                    s0 - __shfl_sync(0xffffffffu, before, src), kv_tile, min_tiles, cut, s1 - s0, lane, &pos);
        // one writer, also where starts that do not ascend let the sums pass 2^32 and two warps find a
        // place: a mixture of two would be none (a found place has a cost of at least 1)
        if (lane == 0 && atomicCAS(&result->cost, 0u, pos.cost) == 0u) {
          result->r = pos.r;
          result->h = pos.h;
          result->j = pos.j;
          result->at = pos.at;
        }
        break;
      }
      before += cost;
    }
  }
  __syncthreads();
  return *result;
}

// Walks a CTA's range unit by unit.
struct AttnWalk {
  AttnRequest q;
  int r, h, j, t0, t1, n, end;  // tiles [t0, t1) of the unit's n; end: keys its last row sees
  unsigned left;                // cost of the range from this unit on

  // The range's share of unit j from offset `at` on. False: it ends before the unit's first tile.
  __device__ __forceinline__ bool unit(const AttnArgs& a, int kv_tile, int at) {
    end = attn_unit_end(a, q, j);
    n = (int)((unsigned)(end + kv_tile - 1) / (unsigned)kv_tile);
    if (n < 1) n = 1;
    const int whole = n + a.unit_cost, stop = left < (unsigned)(whole - at) ? at + (int)left : whole;
    t0 = at > a.unit_cost ? at - a.unit_cost : 0;
    t1 = stop > a.unit_cost ? stop - a.unit_cost : 0;
    left -= stop - at;
    return t1 > t0;
  }
  __device__ __forceinline__ bool start(const AttnArgs& a, const AttnPos& p, int kv_tile) {
    left = p.cost;
    if (left == 0) return false;
    r = p.r;
    h = p.h;
    j = p.j;
    q = attn_request(a, r);
    return unit(a, kv_tile, p.at);
  }
  __device__ __forceinline__ bool next(const AttnArgs& a, int kv_tile) {
    if (left == 0) return false;
    if (++j >= q.units) {
      j = 0;
      if (++h >= a.kv_heads) {
        h = 0;
        do {
          if (++r >= a.requests) return false;
          q = attn_request(a, r);
        } while (q.units == 0);
      }
    }
    return unit(a, kv_tile, 0);
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }
};

// Place of packed row p of a request in q, out and lse.
struct RowPlace {
  long long token;
  int head;
};
__device__ __forceinline__ RowPlace row_place(const AttnArgs& a, int q0, int kv_head, int p) {
  const int t = a.by_group(p);
  return {(long long)(q0 + t), kv_head * a.group + (p - t * a.group)};
}

// The packed row (of the request) at row i of a slot whose unit starts at packed row `base`, or -1.
__device__ __forceinline__ int attn_packed_row(const AttnArgs& a, int i, int base, int rows, int used) {
  const int b = i >= a.block_rows ? 1 : 0, o = i - b * a.block_rows;
  const int p = base + b * used + o;
  return o < used && p < rows ? p : -1;
}

// The two kernels and the combining pass.
int attn_rows_limit(int head_dim);          // most packed rows of a request that the row kernel takes
int attn_rows_grid(int head_dim, int rows); // CTAs of the row kernel
int attn_rows_unit_cost();                  // AttnArgs::unit_cost
int attn_wide_unit_cost(int head_dim);
int attn_wide_grid();
int attn_wide_blocks(int head_dim);  // row blocks of 128 of a unit of the tensor-core kernel
cudaError_t launch_attn_rows(const AttnArgs& a, int head_dim, bool bf16, int nr, cudaStream_t st);
cudaError_t launch_attn_wide(const AttnArgs& a, int head_dim, bool bf16, cudaStream_t st);
cudaError_t launch_attn_combine(const AttnArgs& a, int head_dim, bool bf16, int grid, int slot_rows, cudaStream_t st);

}  // namespace vq3
