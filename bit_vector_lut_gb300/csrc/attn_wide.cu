// Attention of many query rows on the 5th-generation tensor cores: prefill chunks over the
// paged cache, whole prompts, and verify steps whose rows fill more than the row kernel takes.
//
// One persistent CTA per SM walks its range of (request, key/value head, row block, 128-key
// tile). Per tile, in one pass with a running maximum and sum:
//   S[128 rows][128 keys] = Q K^T     tcgen05.mma, Q and K in shared memory (128-byte swizzle)
//   P = exp2(S scale - max)           read from and written back to tensor memory as 16 bits
//   O[128 rows][D] += P V             tcgen05.mma, P from tensor memory, V from shared memory
// The rows of a block are (token, query head of the group), so the heads of a group share
// every tile. head_dim 64 and 128: two blocks of 128 rows (A, B) share a tile, one warpgroup
// each, so that one block's softmax runs under the other's products. head_dim 256: O alone
// takes half of tensor memory, so there is one block, whose softmax the two warpgroups share
// by key columns (64 each, the row maxima exchanged through shared memory), and two S
// buffers, so that the next tile's Q K^T runs under it.
//   warps 0-3, 4-7  softmax, rescaling and output of block A / B (or keys 0-63 / 64-127)
//   warp 8          TMA: the lanes each copy a page's rows (page numbers prefetched a tile
//                   ahead) into a ring of stages, in the order in which the MMA warp uses them
//   warp 9          issues the MMAs, the blocks' in turn: that keeps one block's softmax under
//                   the other's products (two issuing warps let both softmaxes fall together,
//                   8% slower)
// O is rescaled only when a row's maximum rises by more than 2^8 (see kLag), by the softmax
// warps themselves.
// Keys behind the last that the block sees are masked in S; of V only the 16-row steps that
// hold keys are multiplied, the rest of the last such step zeroed first, so that what lies
// behind a request's keys is never used.
// All waits are bounded: one that runs out ends the CTA's work and marks its record.
#include <cuda.h>  // CUtensorMap; the encoder is fetched from the driver at run time

#include "attn_common.cuh"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(attn_wide)
namespace {

constexpr int kTile = 128;      // keys per tile
// Fewest tiles per CTA. (1 / 2 / 4: eight tokens behind 4,097 keys, 24 heads on 4 x 256, 32.1 / 24.3 / 23.2 us;
// batches that fill the GPU do not depend on it.)
constexpr int kMinTiles = 2;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 12 * 32;  // warps 10 and 11 fill up the third warpgroup
// Registers per thread: at launch 168; the softmax warpgroups take what the third gives up.
template <int D>
constexpr int kRegsSoftmax = D == 256 ? 200 : 208;  // a row's 64 or 128 scores and what goes with them
template <int D>
constexpr int kRegsOther = 3 * 168 - 2 * kRegsSoftmax<D>;
static_assert(kRegsOther<128> % 8 == 0 && kRegsOther<256> % 8 == 0, "register shares");
constexpr int kBlock = 128;  // rows of a block

// ---------------------------------------------------------------- kernel

template <int D>
struct WideCfg {
  static constexpr int kBlocks = D == 256 ? 1 : 2;          // row blocks of a unit
  static constexpr int kStageCols = D == 64 ? 64 : 128;     // head_dim columns of a stage
  static constexpr int kParts = D / kStageCols;             // stages per K or V tile
  static constexpr int kCb = kStageCols / 64;               // 64-column blocks of a stage
  static constexpr int kCbBytes = kTile * 128;              // 16 KB: 128 rows of 128 bytes
  static constexpr int kStageBytes = kCb * kCbBytes;
  static constexpr int kQBytes = kBlocks * (D / 64) * kCbBytes;
  static constexpr int kStages = D == 64 ? 10 : 5;
  static constexpr int kMisc = 3 * 1024;  // barriers, range, exchange of row maxima
  static constexpr int kSmem = kQBytes + kStages * kStageBytes + kMisc;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static_assert(2 * kSmem > 228 * 1024, "one CTA per SM: it takes all of tensor memory");
  // tensor memory columns: two S buffers of 128 (P over them), then O
  static constexpr uint32_t kO = 256;
};

// Column of P's step of 16 keys inside its S buffer: each half of P lies over the half of S
// that it was made from.
__device__ __forceinline__ uint32_t p_col(int step) { return (uint32_t)(step < 4 ? 8 * step : 64 + 8 * (step - 4)); }

// Place in a ring of N stages: the stage and the parity of its current use.
template <int N>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ Ring plus(int n) const {
    Ring r;
    r.s = s + n < N ? s + n : s + n - N;
    r.phase = s + n < N ? phase : phase ^ 1u;
    return r;
  }
};

struct WideMaps {
  CUtensorMap q, q_token, q_row, k, v;  // of q: a block of whole tokens, one token's group of heads, one row
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) attn_wide_kernel(const __grid_constant__ AttnArgs a,
                                                                const __grid_constant__ WideMaps maps) {
  using C = WideCfg<D>;
  constexpr int NB = C::kBlocks;
  constexpr bool kBf16 = AttnType<T>::kBf16;
  constexpr float kOff = AttnType<T>::kOff;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* const misc = smem + C::kQBytes + C::kStages * C::kStageBytes;
  float* const s_max = reinterpret_cast<float*>(misc);                 // [2][2][128]
  unsigned long long* const bars = reinterpret_cast<unsigned long long*>(misc + 2048);  // 40
  AttnPos* const s_pos = reinterpret_cast<AttnPos*>(misc + 2048 + 320);
  unsigned* const s_sum = reinterpret_cast<unsigned*>(misc + 2048 + 384);  // 3 * kThreads / 32
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(misc + 2048 + 704);
  volatile int* const abort = reinterpret_cast<volatile int*>(misc + 2048 + 708);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(smem), bar0 = smem_u32(bars);
  const auto q_at = [&](int block, int cb) { return base + (uint32_t)((block * (D / 64) + cb) * C::kCbBytes); };
  const auto stage_at = [&](int s) { return base + (uint32_t)(C::kQBytes + s * C::kStageBytes); };
  const auto full = [&](int s) { return bar0 + 8u * s; };                    // stage holds a tile part
  const auto empty = [&](int s) { return bar0 + 8u * (C::kStages + s); };    // its products are done
  constexpr int kB0 = 2 * C::kStages;
  const uint32_t q_full = bar0 + 8u * kB0, q_empty = bar0 + 8u * (kB0 + 1);
  const auto s_full = [&](int b) { return bar0 + 8u * (kB0 + 2 + b); };      // S buffer b holds scores
  const auto p_full = [&](int b) { return bar0 + 8u * (kB0 + 4 + b); };      // and now probabilities
  const auto pv_done = [&](int b) { return bar0 + 8u * (kB0 + 6 + b); };     // P V done: of block b's unit, or of buffer b's tile
  const auto o_empty = [&](int b) { return bar0 + 8u * (kB0 + 8 + b); };     // O of block b read out
  const auto p_half = [&](int b) { return bar0 + 8u * (kB0 + 10 + b); };     // two blocks: the first 64 keys' probabilities
  const uint32_t drain = bar0 + 8u * (kB0 + 12);                             // all products
  static_assert(kB0 + 13 <= 40, "barriers");

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(p_full(b), NB == 2 ? 4 : 8);
      mbar_init(pv_done(b), 1);
      mbar_init(o_empty(b), NB == 2 ? 4 : 8);
      mbar_init(p_half(b), 4);
    }
    mbar_init(drain, 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kTmaWarp && lane < 5) {  // the descriptors' first fetch, ahead of the copies
    const CUtensorMap* const m = &maps.q + lane;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  const AttnPos pos = a.requests <= kWarpRequests ? attn_locate_warp(a, kTile, kMinTiles)
                                                  : attn_locate_block<kThreads>(a, kTile, kMinTiles, s_sum, s_pos);
  __syncthreads();  // the set-up above
  tc_after();
  const uint32_t tmem = *s_tmem;
  // Once a wait gave up (`dead`, the same for the whole warp), the copy and MMA warps issue nothing
  // more; the softmax warps, which meet at barriers, walk on over what is there.
  bool dead = false;
  const auto wait = [&](uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
    dead = __any_sync(0xffffffffu, !mbar_wait(bar, parity, abort)) || dead;
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther<D>));
    if (warp == kTmaWarp) {
      // ------------------------------------------------------------ copies
      const int box = a.table ? (1 << a.page_shift < kTile ? 1 << a.page_shift : kTile) : kTile;  // rows per copy
      const int boxes = kTile / box;
      const int my_box = lane & (boxes - 1), my_cb = lane / boxes;  // this lane's copy of a stage
      Ring<C::kStages> at;
      int it = 0, units = 0;
      AttnWalk w;
      for (bool on = w.start(a, pos, kTile); on; on = w.next(a, kTile)) {
        if (w.end == 0) continue;
        const int rows = w.q.n_new * a.group, first = w.j * NB * w.q.used;
        // Q of the unit, once the last one's is used up
        const auto copy_q = [&] {
          if (units) wait(q_empty, (uint32_t)((units - 1) & 1));
          if (dead) return;
          const int blocks = NB == 2 && first + w.q.used < rows ? 2 : 1;
          if (w.q.used == a.token_rows) {
            if (lane == 0) {
              mbar_expect_tx(q_full, (uint32_t)(blocks * (D / 64) * a.token_rows * 128));
              for (int b = 0; b < blocks; ++b)
                for (int cb = 0; cb < D / 64; ++cb)
                  tma_3d(q_at(b, cb), &maps.q, cb * 64, w.h * a.group, w.q.q0 + a.by_group(first + b * a.token_rows),
                         q_full);
            }
          } else {
            // a lane per token: its heads in one copy, or row by row where the block cuts them
            const int last = first + blocks * kBlock < rows ? first + blocks * kBlock : rows;
            if (lane == 0) mbar_expect_tx(q_full, (uint32_t)((last - first) * (D / 64) * 128));
            __syncwarp();
            for (int b = 0; b < blocks; ++b) {
              const int p0 = first + b * kBlock, p1 = p0 + kBlock < last ? p0 + kBlock : last;
              for (int t = a.by_group(p0) + lane; t * a.group < p1; t += 32) {
                const int r0 = t * a.group > p0 ? t * a.group : p0, r1 = (t + 1) * a.group < p1 ? (t + 1) * a.group : p1;
                for (int cb = 0; cb < D / 64; ++cb) {
                  if (r1 - r0 == a.group) {
                    tma_3d(q_at(b, cb) + (uint32_t)(r0 - p0) * 128, &maps.q_token, cb * 64, w.h * a.group, w.q.q0 + t,
                           q_full);
                  } else {
                    for (int r = r0; r < r1; ++r)
                      tma_3d(q_at(b, cb) + (uint32_t)(r - p0) * 128, &maps.q_row, cb * 64,
                             w.h * a.group + r - t * a.group, w.q.q0 + t, q_full);
                  }
                }
              }
            }
          }
          __syncwarp();
          ++units;
        };
        // the page of this lane's rows of tile t
        const auto page_of = [&](int t) -> int {
          const int x = t * kTile + my_box * box;
          if (!a.table || t >= w.t1 || x >= w.end) return 0;
          const size_t at = (size_t)w.r * a.max_pages + (x >> a.page_shift);
          return VQ3_IN(at, (size_t)a.requests * a.max_pages, 1) ? __ldg(a.table + at) : -1;
        };
        const auto copy = [&](const CUtensorMap* map, int t, int page) {
          const int left = w.end - t * kTile;  // keys of the tile that count
          const int n = a.table ? ((left < kTile ? left : kTile) + box - 1) / box : 1;
          const int x = t * kTile + my_box * box;
          const int row = a.table ? x & ((1 << a.page_shift) - 1) : w.q.q0 + x;
#pragma unroll
          for (int part = 0; part < C::kParts; ++part, ++it, at = at.plus(1)) {
            const int s = at.s;
            if (it >= C::kStages) wait(empty(s), at.phase ^ 1u);
            if (dead) return;
            if (lane == 0) mbar_expect_tx(full(s), (uint32_t)(n * C::kCb * box * 128));
            __syncwarp();
            if (my_box < n && my_cb < C::kCb)
              tma_4d(stage_at(s) + (uint32_t)(my_cb * C::kCbBytes + my_box * box * 128), map,
                     part * C::kStageCols + my_cb * 64, row, w.h, a.table ? page : 0, full(s));
          }
        };
        // the first keys go ahead of Q: their stage is free sooner
        int page = page_of(w.t0);
        copy(&maps.k, w.t0, page);
        copy_q();
        if constexpr (NB == 2) {
          for (int t = w.t0; t < w.t1; ++t) {
            const int next = page_of(t + 1);
            if (t > w.t0) copy(&maps.k, t, page);
            copy(&maps.v, t, page);
            page = next;
          }
        } else {
          int ahead = page_of(w.t0 + 1);
          for (int t = w.t0; t < w.t1; ++t) {
            const int next = page_of(t + 2);
            if (t + 1 < w.t1) copy(&maps.k, t + 1, ahead);
            copy(&maps.v, t, page);
            page = ahead;
            ahead = next;
          }
        }
      }
      // no copy is in flight when the CTA ends (they have all been used unless a wait gave up)
      if (units) mbar_drain(q_full, (uint32_t)((units - 1) & 1));
      for (int j = it > C::kStages ? it - C::kStages : 0; j < it; ++j)
        mbar_drain(full(j % C::kStages), (uint32_t)((j / C::kStages) & 1));
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      constexpr uint32_t id_qk = idesc(kTile, kBf16, false), id_pv = idesc(C::kStageCols, kBf16, true);
      using Place = Ring<C::kStages>;
      Place it;                   // the next stage of the ring
      int units = 0;
      int tiles[2] = {0, 0};      // tiles of block b (one block: all, [0])
      int outs[2] = {0, 0};       // units of block b
      AttnWalk w;
      // A wait or a commit between two products leaves the tensor pipe idle once the few that are
      // queued have run, so the waits for stages (mostly long since filled) and the releases of
      // stages sit between the parts of a product, not between two products.
      // Part of S buffer `buf` = Q of block b times the stages at `at`
      const auto qk = [&](int b, int buf, Place at, int part) {
        if (dead) return;
#pragma unroll
        for (int c = 0; c < C::kCb; ++c)
          mma_ss4(tmem + (uint32_t)(buf * kTile), desc_sw128(q_at(b, part * C::kCb + c), 16),
                  desc_sw128(stage_at(at.plus(part).s) + (uint32_t)(c * C::kCbBytes), 16), id_qk, part + c > 0);
      };
      // Part of O of block b (+)= P in S buffer `buf`, steps [k0, k1) of 16 keys, times the stages at `at`
      const auto pv = [&](int b, int buf, Place at, int part, int k0, int k1, bool first) {
        if (dead) return;
        const uint32_t p = tmem + (uint32_t)(buf * kTile);
        const uint64_t v = desc_sw128(stage_at(at.plus(part).s), C::kCbBytes);
        const uint32_t o = tmem + C::kO + (uint32_t)(b * D + part * C::kStageCols);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (k0 <= 4 * h && k1 >= 4 * h + 4) {
            mma_ts4<128>(o, p + 64u * h, v + 512u * h, id_pv, !first || h > 0);
          } else {
            for (int k = k0 > 4 * h ? k0 : 4 * h; k < k1 && k < 4 * h + 4; ++k)
              mma_ts1(o, p + p_col(k), v + 128u * k, id_pv, !first || k > 0);
          }
        }
      };
      const auto release = [&](Place at) {
#pragma unroll
        for (int p = 0; p < C::kParts; ++p) mma_commit(empty(at.plus(p).s));
      };
      const auto wait_stages = [&](Place at) {
#pragma unroll
        for (int p = 0; p < C::kParts; ++p) wait(full(at.plus(p).s), at.plus(p).phase);
      };
      // V rows of the last step that lie behind the keys: zero (the probabilities there are zero,
      // but what the memory holds need not be finite)
      const auto clear_tail = [&](Place at, int keys) {
        if (keys % 16 == 0 || dead) return;
        const int r0 = keys, r1 = (keys + 15) & ~15;
        for (int i = lane; i < (r1 - r0) * C::kCb * C::kParts * 8; i += 32) {
          const int chunk = i & 7, cb = (i >> 3) % (C::kCb * C::kParts), r = r0 + (i >> 3) / (C::kCb * C::kParts);
          const uint32_t p = stage_at(at.plus(cb / C::kCb).s) +
                             (uint32_t)((cb % C::kCb) * C::kCbBytes + r * 128 + chunk * 16);
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(p), "r"(0) : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      };
      for (bool on = w.start(a, pos, kTile); on; on = w.next(a, kTile)) {
        if (w.end == 0) continue;
        const int rows = w.q.n_new * a.group, first = w.j * NB * w.q.used;
        const int blocks = NB == 2 && first + w.q.used < rows ? 2 : 1;
        wait(q_full, (uint32_t)(units & 1));
        ++units;
        wait_stages(it);
        tc_after();
        if constexpr (NB == 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (b >= blocks) continue;
            qk(b, b, it, 0);
            mma_commit(s_full(b));
          }
          release(it);
          it = it.plus(1);
          if (w.t1 - w.t0 == 1) mma_commit(q_empty);
          wait_stages(it);
          for (int t = w.t0; t < w.t1; ++t) {
            const int keys = w.end - t * kTile < kTile ? w.end - t * kTile : kTile, steps = (keys + 15) / 16;
            const Place vs = it, ks = it.plus(1), next = it.plus(2);
            const bool more = t + 1 < w.t1;
            clear_tail(vs, keys);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (b >= blocks) continue;
              const bool last = b + 1 == blocks;
              if (t == w.t0 && outs[b]) wait(o_empty(b), (uint32_t)((outs[b] - 1) & 1));
              wait(p_half(b), (uint32_t)(tiles[b] & 1));
              tc_after();
              pv(b, b, vs, 0, 0, steps < 4 ? steps : 4, t == w.t0);
              if (b == 0 && more) wait_stages(ks);
              wait(p_full(b), (uint32_t)(tiles[b] & 1));
              tc_after();
              pv(b, b, vs, 0, 4, steps, false);
              ++tiles[b];
              if (more) {
                if (last) wait_stages(next);  // the next tile's values
                qk(b, b, ks, 0);
                mma_commit(s_full(b));
              } else {
                mma_commit(pv_done(b));
              }
            }
            release(vs);
            if (more) release(ks);
            if (t + 2 == w.t1) mma_commit(q_empty);
            it = more ? next : ks;
          }
          ++outs[0];
          if (blocks == 2) ++outs[1];
        } else {
#pragma unroll
          for (int p = 0; p < C::kParts; ++p) qk(0, tiles[0] & 1, it, p);
          mma_commit(s_full(tiles[0] & 1));
          release(it);
          it = it.plus(C::kParts);
          if (w.t1 - w.t0 == 1) mma_commit(q_empty);
          for (int t = w.t0; t < w.t1; ++t, ++tiles[0]) {
            const int keys = w.end - t * kTile < kTile ? w.end - t * kTile : kTile, steps = (keys + 15) / 16;
            const int buf = tiles[0] & 1;
            const bool more = t + 1 < w.t1;
            const Place ks = it, vs = more ? it.plus(C::kParts) : it, next = vs.plus(C::kParts);
            if (more) {  // S of the next tile; its keys have been waited for
              wait_stages(ks);
              tc_after();
              qk(0, buf ^ 1, ks, 0);
              qk(0, buf ^ 1, ks, 1);
              mma_commit(s_full(buf ^ 1));
              release(ks);
              if (t + 2 == w.t1) mma_commit(q_empty);
            }
            wait_stages(vs);
            clear_tail(vs, keys);
            if (t == w.t0 && outs[0]) wait(o_empty(0), (uint32_t)((outs[0] - 1) & 1));
            wait(p_full(buf), (uint32_t)((tiles[0] >> 1) & 1));
            tc_after();
            pv(0, buf, vs, 0, 0, steps, t == w.t0);
            pv(0, buf, vs, 1, 0, steps, t == w.t0);
            mma_commit(pv_done(buf));
            release(vs);
            it = next;
          }
          ++outs[0];
        }
      }
      // every product has completed before tensor memory is freed
      mma_commit(drain);
      mbar_drain(drain, 0);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax<D>));
    constexpr int kCols = NB == 2 ? 128 : 64;  // key columns of a thread
    constexpr int kOut = NB == 2 ? D : 128;    // output columns of a thread
    const int wg = warp >> 2, sub = warp & 3, row = sub * 32 + lane;
    const int block = NB == 2 ? wg : 0, c0 = NB == 2 ? 0 : wg * 64;
    const uint32_t lanes = (uint32_t)(sub * 32) << 16;
    const uint32_t o_at = tmem + lanes + C::kO + (uint32_t)(NB == 2 ? block * D : wg * 128);
    int tiles = 0, outs = 0;  // tiles and units of this block
    int flags = 0;
    AttnRec rec{};
    AttnWalk w;
    const auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + sub) : "memory"); };
    for (bool on = w.start(a, pos, kTile); on; on = w.next(a, kTile)) {
      const int rows = w.q.n_new * a.group, first = w.j * NB * w.q.used;
      const bool whole = w.whole();
      if (!whole) {
        if (w.t0 > 0) {
          flags |= kRecHead | (w.t1 == w.n ? kRecEnd : 0);
        } else {
          flags |= kRecTail;
          rec.q0 = w.q.q0;
          rec.rows = rows;
          rec.base = first;
          rec.head = w.h;
          rec.used = w.q.used;
        }
      }
      if (NB == 2 && block == 1 && first + w.q.used >= rows) continue;  // no rows in block B
      const int p = row < w.q.used && first + block * w.q.used + row < rows ? first + block * w.q.used + row : -1;
      const bool live = __any_sync(0xffffffffu, p >= 0);  // dead warps only keep the barriers
      const int lim = p >= 0 ? attn_seen(w.q, a.by_group(p)) : 0;
      float m = -INFINITY, l = 0.f;
      if (w.end > 0) {
        for (int t = w.t0; t < w.t1; ++t, ++tiles) {
          const int buf = NB == 2 ? block : tiles & 1;
          const uint32_t s_at = tmem + lanes + (uint32_t)(buf * kTile + c0);
          mbar_wait(s_full(buf), (uint32_t)((NB == 2 ? tiles : tiles >> 1) & 1), abort);
          tc_after();
          if (live) {
            uint32_t s[kCols];
#pragma unroll
            for (int c = 0; c < kCols; c += 32) tmem_ld32(s_at + c, s + c);
            tc_wait_ld();
            const int seen = lim - t * kTile - c0;  // of this thread's columns
            if (seen < kCols) {
#pragma unroll
              for (int c = 0; c < kCols; ++c)
                if (c >= seen) s[c] = 0xff800000u;  // -infinity
            }
            float x0 = -INFINITY, x1 = -INFINITY, x2 = -INFINITY, x3 = -INFINITY;
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
              x0 = max3(x0, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
              x1 = max3(x1, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
              x2 = max3(x2, __uint_as_float(s[c + 4]), __uint_as_float(s[c + 5]));
              x3 = max3(x3, __uint_as_float(s[c + 6]), __uint_as_float(s[c + 7]));
            }
            float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * a.scale_log2;
            if constexpr (NB == 1) {
              // the other half's maximum of the row (buffers alternate: one barrier per tile)
              float* const ex = s_max + (tiles & 1) * 256;
              ex[wg * 128 + row] = mx;
              pair_sync();
              mx = fmaxf(mx, ex[(wg ^ 1) * 128 + row]);
            }
            if (__any_sync(0xffffffffu, mx > m + kLag)) {
              const float up = fmaxf(m, mx);
              const float f = m == up ? 1.f : ex2(m - up);  // equal infinities: nothing to rescale
              m = up;
              l *= f;
              if (t > w.t0) {
                // O = P V up to the last tile; with two S buffers that product may still run
                // (pv_done of tile t - 1. Not every phase of that barrier is waited for, and a parity tells a
                // phase from the next one only: its last one, P V of t - 3, has to be complete here. It is: S of
                // t is multiplied behind P V of t - 2, so s_full of t, waited for above, comes a whole product
                // after it. Waiting for every phase cost 1 to 2% of prompts of 24 x 256.)
                if (NB == 1) {
                  mbar_wait(pv_done((tiles - 1) & 1), (uint32_t)(((tiles - 1) >> 1) & 1), abort);
                  tc_after();
                }
#pragma unroll 1
                for (int c = 0; c < kOut; c += 32) {
                  uint32_t o[32];
                  tmem_ld32(o_at + c, o);
                  tc_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st32(o_at + c, o);
                }
              }
            }
            const float mm = m == -INFINITY ? 0.f : m;
            const uint64_t sc = f2(a.scale_log2, a.scale_log2), off = f2(kOff - mm, kOff - mm);
#pragma unroll
            for (int c = 0; c < kCols; c += 64) {
              uint32_t pk[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float e0, e1;
                un2(fma2(f2(__uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1])), sc, off), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                s[c + 2 * i] = __float_as_uint(e0);
                s[c + 2 * i + 1] = __float_as_uint(e1);
                pk[i] = pack2<T>(e0, e1);
              }
              tmem_st32(s_at + c, pk);
              tc_wait_st();
              tc_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(c + 64 < kCols ? p_half(buf) : p_full(buf));
            }
            // the row's sum, under the product
            uint64_t l0 = 0, l1 = 0, l2 = 0, l3 = 0;
#pragma unroll
            for (int c = 0; c < kCols; c += 8) {
              l0 = add2(l0, f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])));
              l1 = add2(l1, f2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])));
              l2 = add2(l2, f2(__uint_as_float(s[c + 4]), __uint_as_float(s[c + 5])));
              l3 = add2(l3, f2(__uint_as_float(s[c + 6]), __uint_as_float(s[c + 7])));
            }
            float y0, y1;
            un2(add2(add2(l0, l1), add2(l2, l3)), y0, y1);
            l += y0 + y1;
          } else {
            tc_before();
            __syncwarp();
            if (lane == 0) {
              if (NB == 2) mbar_arrive(p_half(buf));
              mbar_arrive(p_full(buf));
            }
          }
        }
      }
      // the unit's output, or its part of it
      float inv = 0.f;
      if (w.end > 0) {
        if (NB == 2)
          mbar_wait(pv_done(block), (uint32_t)(outs & 1), abort);
        else  // of the unit's last tile; s_full of that tile comes behind P V of the one two before it
          mbar_wait(pv_done((tiles - 1) & 1), (uint32_t)(((tiles - 1) >> 1) & 1), abort);
        ++outs;
        tc_after();
      }
      if (live) {
        if constexpr (NB == 1) {
          // the halves' sums
          float* const ex = s_max + (tiles & 1) * 256;
          ex[wg * 128 + row] = l;
          pair_sync();
          l += ex[(wg ^ 1) * 128 + row];
          pair_sync();
        }
        inv = l == 0.f ? 0.f : 1.f / l;
        const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
        const size_t at = (size_t)slot * (NB * 128) + block * 128 + row;
        const RowPlace rp = row_place(a, w.q.q0, w.h, p < 0 ? 0 : p);
        T* const dst = static_cast<T*>(a.out) + rp.token * a.o_token + rp.head * a.o_head + (NB == 2 ? 0 : wg * 128);
        // parts: [slot][D / 4][rows] of four columns, so that a warp's rows are written side by side
        float4* const part = reinterpret_cast<float4*>(a.part) +
                             ((size_t)slot * (D / 4) + (NB == 2 ? 0 : wg * 32)) * (NB * 128) + block * 128 + row;
        const bool ok = p >= 0 && VQ3_IN(rp.token, a.tokens, 2) && VQ3_IN(at, (size_t)2 * gridDim.x * NB * 128, 3);
#pragma unroll 1
        for (int c = 0; c < kOut; c += 32) {
          uint32_t o[32];
          if (w.end > 0) {
            tmem_ld32(o_at + c, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          }
          if (ok && whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                y[e] = pack2<T>(__uint_as_float(o[i + 2 * e]) * inv, __uint_as_float(o[i + 2 * e + 1]) * inv);
              store32(dst + c + i, y);
            }
          } else if (ok) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(part + (size_t)((c + i) / 4) * (NB * 128),
                     make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                 __uint_as_float(o[i + 3])));
          }
        }
        if (ok && (NB == 2 || wg == 0)) {
          if (!whole)
            __stcg(reinterpret_cast<float2*>(a.part_ml + 2 * at), make_float2(m, l));
          else if (a.lse)
            a.lse[rp.token * a.heads + rp.head] =
                l == 0.f ? -INFINITY : (m - kOff + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (w.end > 0) {
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty(block));
      }
    }
    if (tid == 0) {
      rec.flags = flags;
      a.rec[blockIdx.x] = rec;
    }
  }

  tc_before();
  __syncthreads();
  if (tid == 0 && *abort) a.rec[blockIdx.x].flags = kRecFailed;
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ---------------------------------------------------------------- launch

template <typename T, int D>
cudaError_t launch_wide(const AttnArgs& a, cudaStream_t st) {
  constexpr bool bf16 = AttnType<T>::kBf16;
  constexpr int smem = WideCfg<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(attn_wide_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  alignas(64) WideMaps maps;
  const int page = 1 << a.page_shift;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.heads, (cuuint64_t)a.tokens};
    const long long strides[2] = {a.q_head, a.q_token};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)(a.token_rows / a.group)};
    const cuuint32_t token[3] = {64, (cuuint32_t)a.group, 1}, row[3] = {64, 1, 1};
    if (!tensor_map(&maps.q, bf16, a.q, 3, dims, strides, box) ||
        !tensor_map(&maps.q_token, bf16, a.q, 3, dims, strides, token) ||
        !tensor_map(&maps.q_row, bf16, a.q, 3, dims, strides, row))
      return cudaErrorInvalidValue;
  }
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)(a.table ? page : a.tokens), (cuuint64_t)a.kv_heads,
                              (cuuint64_t)(a.table ? a.n_pages : 1)};
  const cuuint32_t box[4] = {64, (cuuint32_t)(a.table && page < kTile ? page : kTile), 1, 1};
  const long long ks[3] = {a.k_token, a.k_head, a.table ? a.k_page : D};
  const long long vs[3] = {a.v_token, a.v_head, a.table ? a.v_page : D};
  if (!tensor_map(&maps.k, bf16, a.k, 4, dims, ks, box) || !tensor_map(&maps.v, bf16, a.v, 4, dims, vs, box))
    return cudaErrorInvalidValue;
  attn_wide_kernel<T, D><<<attn_wide_grid(), kThreads, smem, st>>>(a, maps);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_wide_t(const AttnArgs& a, int d, cudaStream_t st) {
  if (d == 64) return launch_wide<T, 64>(a, st);
  if (d == 128) return launch_wide<T, 128>(a, st);
  return launch_wide<T, 256>(a, st);
}

}  // namespace

int attn_wide_grid() { return device_sm_count() < 608 ? device_sm_count() : 608; }
// Measured on an 8,192-token prompt of 32 x 128 (0 tiles: 506 us; 1 and 2: 459 to 466 us, which of the two
// leads changed with the build), packed prompts of 16 x 64 (0 / 1 / 2: 45.2 / 42.3 / 43.2 us) and ragged
// prompts of 24 x 256 (0 / 2 / 3 / 4: 391 / 337 / 327 / 333 us).
int attn_wide_unit_cost(int head_dim) { return head_dim == 256 ? 3 : 1; }
int attn_wide_blocks(int head_dim) { return head_dim == 256 ? 1 : 2; }

cudaError_t launch_attn_wide(const AttnArgs& a, int head_dim, bool bf16, cudaStream_t st) {
  return bf16 ? launch_wide_t<__nv_bfloat16>(a, head_dim, st) : launch_wide_t<__half>(a, head_dim, st);
}

}  // namespace vq3
