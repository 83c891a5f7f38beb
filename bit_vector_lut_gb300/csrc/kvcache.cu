// The paged key/value cache: the page plan of a serving step and the append of new rows.
#include "vq3_internal.h"

namespace vq3 {
VQ3_BOUNDS_RECORD(kvcache)
namespace {

// ---------------------------------------------------------------- page plan
//
// held = ceil(cached / P) pages, need = ceil((cached + new) / P); the need - held new pages of
// the requests are taken from the ring of free pages in request order. Every CTA finds the
// prefix sums of all requests itself (8 bytes a request, from L2: cheaper than handing them
// over between CTAs or launches) and then writes its share of the tokens, new pages and
// requests. Bound by latency: two dependent reads from memory and one scan (4 requests 3.2 us;
// 700 requests with 63K new tokens 6.3 us, 0.8 MB written).
constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 1024;  // tokens per CTA

// First index i in [0, n) with prefix[i + 1] > x (prefix ascending, prefix[n] > x).
__device__ __forceinline__ int find(const int* prefix, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid + 1] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int s_prefix[];  // tokens [requests + 1], then pages [requests + 1]
  __shared__ long long s_tok[kPlanThreads / 32], s_pag[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.requests, shift = a.page_shift, page = 1 << shift;
  int* const tokens = s_prefix;
  int* const pages = s_prefix + R + 1;
  const int head = __ldg(a.ring_state), count = __ldg(a.ring_state + 1);

  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  int bad = 0;
  if (head < 0 || head >= a.ring_size || count < 0 || count > a.ring_size) bad |= VQ3_PLAN_BAD_LENGTH;
  long long tok = 0, pag = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r >= R) break;
    const long long c = __ldg(a.cached + r), n = __ldg(a.fresh + r);
    if (c < 0 || n < 0 || c + n > 0x3fffffff) {
      bad |= VQ3_PLAN_BAD_LENGTH;
      continue;
    }
    const long long held = (c + page - 1) >> shift, need = (c + n + page - 1) >> shift;
    if (need > a.max_pages) bad |= VQ3_PLAN_NARROW_TABLE;
    tok += n;
    pag += need - held;
  }
  long long it = tok, ip = pag;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ot = __shfl_up_sync(0xffffffffu, it, d), op = __shfl_up_sync(0xffffffffu, ip, d);
    if (lane >= d) {
      it += ot;
      ip += op;
    }
  }
  if (lane == 31) {
    s_tok[warp] = it;
    s_pag[warp] = ip;
  }
  int status = __syncthreads_or(bad & VQ3_PLAN_BAD_LENGTH) ? VQ3_PLAN_BAD_LENGTH : 0;
  if (__syncthreads_or(bad & VQ3_PLAN_NARROW_TABLE)) status |= VQ3_PLAN_NARROW_TABLE;
  long long bt = 0, bp = 0, all_t = 0, all_p = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      bt += s_tok[w];
      bp += s_pag[w];
    }
    all_t += s_tok[w];
    all_p += s_pag[w];
  }
  if (all_p > count) status |= VQ3_PLAN_NO_PAGES;
  if (all_t > a.max_tokens) status |= VQ3_PLAN_TOO_MANY_TOKENS;
  const bool fail = status != 0;

  if (!fail) {
    long long t = bt + it - tok, p = bp + ip - pag;
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r >= R) break;
      tokens[r] = (int)t;
      pages[r] = (int)p;
      const int c = __ldg(a.cached + r), n = __ldg(a.fresh + r);
      t += n;
      p += ((c + n + page - 1) >> shift) - ((c + page - 1) >> shift);
    }
    if (tid == 0) {
      tokens[R] = (int)all_t;
      pages[R] = (int)all_p;
    }
  }
  __syncthreads();

  const int threads = gridDim.x * kPlanThreads, me = blockIdx.x * kPlanThreads + tid;
  // requests
  for (int r = me; r <= R; r += threads) {
    if (VQ3_IN(r, R + 1, 1)) a.q_start[r] = fail ? 0 : tokens[r];
    if (r < R && VQ3_IN(r, R, 2)) a.kv_len[r] = fail ? 0 : __ldg(a.cached + r) + __ldg(a.fresh + r);
  }
  // new pages
  if (!fail) {
    for (int p = me; p < (int)all_p; p += threads) {
      const int r = find(pages, R, p);
      const int at = ((__ldg(a.cached + r) + page - 1) >> shift) + p - pages[r];
      long long from = (long long)head + p;
      if (from >= a.ring_size) from -= a.ring_size;
      if (VQ3_IN((size_t)r * a.max_pages + at, (size_t)R * a.max_pages, 3) && VQ3_IN(from, a.ring_size, 4))
        a.table[(size_t)r * a.max_pages + at] = __ldg(a.ring + from);
    }
  }
  // tokens
  for (int t = me; t < a.max_tokens; t += threads) {
    long long slot = -1;
    int pos = -1;
    if (!fail && t < (int)all_t) {
      const int r = find(tokens, R, t);
      const int c = __ldg(a.cached + r);
      pos = c + t - tokens[r];
      const int at = pos >> shift, held = (c + page - 1) >> shift;
      int id;
      if (at < held) {
        id = VQ3_IN((size_t)r * a.max_pages + at, (size_t)R * a.max_pages, 5) ? a.table[(size_t)r * a.max_pages + at] : -1;
      } else {
        long long from = (long long)head + pages[r] + at - held;
        if (from >= a.ring_size) from -= a.ring_size;
        id = VQ3_IN(from, a.ring_size, 6) ? __ldg(a.ring + from) : -1;
      }
      if (id >= 0) slot = ((long long)id << shift) + (pos & (page - 1));
    }
    if (VQ3_IN(t, a.max_tokens, 7)) {
      a.slots[t] = slot;
      a.positions[t] = pos;
    }
  }
  if (me == 0) {
    a.ring_state_out[0] = fail ? head : (int)(((long long)head + all_p) % a.ring_size);
    a.ring_state_out[1] = fail ? count : count - (int)all_p;
    *a.status = status;
  }
}

// ---------------------------------------------------------------- append
//
// Copies row t of k and v to its slot's place, 16 bytes a thread and step, keys and values
// together. Bound by memory: rows are read once past L1, the cache lines written stay in L2
// for the attention that reads them next. 16,411 tokens of 8 x 128 (134 MB in and out): 23.5 us,
// 5.7 TB/s, 84% of a plain copy's rate; two or four chunks a thread in flight took 24.0 and
// 27.3 us.
constexpr int kAppThreads = 256;

__device__ __forceinline__ uint4 ldg_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
  const int per_row = a.kv_heads << a.chunk_shift;  // 16-byte chunks of a row
  const long long total = (long long)a.tokens * per_row;
  const long long limit = (long long)a.n_pages << a.page_shift;
  for (long long u = (long long)blockIdx.x * kAppThreads + threadIdx.x; u < total; u += (long long)gridDim.x * kAppThreads) {
    const int t = (int)(u / per_row), c = (int)(u - (long long)t * per_row);
    const int h = c >> a.chunk_shift, d = (c - (h << a.chunk_shift)) * 8;
    const long long slot = __ldg(a.slots + t);
    if (slot < 0 || slot >= limit) continue;
    const uint4 k = ldg_once(a.k_rows + t * a.k_row + h * a.k_row_head + d);
    const uint4 v = ldg_once(a.v_rows + t * a.v_row + h * a.v_row_head + d);
    const long long page = slot >> a.page_shift, in = slot & ((1 << a.page_shift) - 1);
    if (VQ3_IN(page, a.n_pages, 8)) {
      *reinterpret_cast<uint4*>(a.k_pages + page * a.k_page + in * a.k_token + h * a.k_head + d) = k;
      *reinterpret_cast<uint4*>(a.v_pages + page * a.v_page + in * a.v_token + h * a.v_head + d) = v;
    }
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  // Without opting in a launch gets 48 KB, static shared memory counted in. The opt-in is the same for every
  // call: one of a call's own size could be lowered by another host thread before the launch.
  const auto bytes = [](int requests) { return 2 * (requests + 1) * (int)sizeof(int); };
  const int smem = bytes(a.requests);
  if (smem > 32 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kMaxRequests));
    if (e != cudaSuccess) return e;
  }
  const int want = (a.max_tokens + kPlanTokens - 1) / kPlanTokens, cap = device_sm_count();
  paged_plan_kernel<<<want < 1 ? 1 : (want > cap ? cap : want), kPlanThreads, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t st) {
  const long long total = (long long)a.tokens * (a.kv_heads << a.chunk_shift);
  const long long want = (total + kAppThreads - 1) / kAppThreads, cap = 8LL * device_sm_count();
  kv_append_kernel<<<(int)(want > cap ? cap : want), kAppThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace vq3
