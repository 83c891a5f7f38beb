// C ABI of the attention token mixer and its paged cache: argument checks, workspace carving
// and the choice of kernel.
#include <cmath>

#include "api_checks.h"
#include "attn_common.cuh"

namespace vq3 {
namespace {

constexpr int kMaxKeys = 1 << 30;  // of one request
constexpr int kMaxKvHeads = 1 << 16;
constexpr float kLog2e = 1.4426950408889634f;

// The append counts a row's 16-byte chunks (up to 32 a head) in 32 bits.
int check_kv_heads(int n, const char* who) {
  if (n <= 0) return report_error(VQ3_EINVAL, "%s: kv_heads=%d", who, n);
  if (n > kMaxKvHeads) return report_error(VQ3_EUNSUPPORTED, "%s: kv_heads=%d above %d", who, n, kMaxKvHeads);
  return VQ3_OK;
}
int check_head_dim(int d, const char* who) {
  if (d != 64 && d != 128 && d != 256)
    return report_error(VQ3_EUNSUPPORTED, "%s: head_dim=%d must be 64, 128 or 256", who, d);
  return VQ3_OK;
}
int check_cache(vq3_kv_cache* c, const char* who) {
  if (int rc = check_kv_heads(c->kv_heads, who)) return rc;
  if (int rc = check_head_dim(c->head_dim, who)) return rc;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return report_error(VQ3_EUNSUPPORTED, "%s: page_size=%d must be a power of two in [16, 256]", who, c->page_size);
  if (c->n_pages <= 0) return report_error(VQ3_EINVAL, "%s: n_pages=%d", who, c->n_pages);
  if (!c->k || !c->v) return report_error(VQ3_EINVAL, "%s: null cache", who);
  if (!on(c->k, 16) || !on(c->v, 16)) return report_error(VQ3_EALIGN, "%s: cache not 16-byte aligned", who);
  struct {
    long long* s;
    long long extent;
    const char* what;
  } ax[] = {{&c->k_page, c->n_pages, "k page"},   {&c->v_page, c->n_pages, "v page"},
            {&c->k_token, c->page_size, "k token"}, {&c->v_token, c->page_size, "v token"},
            {&c->k_head, c->kv_heads, "k head"},  {&c->v_head, c->kv_heads, "v head"}};
  for (auto& x : ax)
    if (int rc = check_stride(x.s, x.extent, c->head_dim, who, x.what)) return rc;
  return VQ3_OK;
}

int check_rows(vq3_kv_rows* r, const char* who) {
  if (int rc = check_kv_heads(r->kv_heads, who)) return rc;
  if (int rc = check_head_dim(r->head_dim, who)) return rc;
  if (r->tokens < 0) return report_error(VQ3_EINVAL, "%s: tokens=%d", who, r->tokens);
  if (r->tokens == 0) return VQ3_OK;
  if (!r->k || !r->v) return report_error(VQ3_EINVAL, "%s: null k or v", who);
  if (!on(r->k, 16) || !on(r->v, 16)) return report_error(VQ3_EALIGN, "%s: k and v must be 16-byte aligned", who);
  struct {
    long long* s;
    long long extent;
    const char* what;
  } ax[] = {{&r->k_token, r->tokens, "k token"},
            {&r->v_token, r->tokens, "v token"},
            {&r->k_head, r->kv_heads, "k head"},
            {&r->v_head, r->kv_heads, "v head"}};
  for (auto& x : ax)
    if (int rc = check_stride(x.s, x.extent, r->head_dim, who, x.what)) return rc;
  return VQ3_OK;
}

AppendArgs append_args(const vq3_kv_rows& r, const vq3_kv_cache& c, const long long* slots) {
  return AppendArgs{static_cast<const uint16_t*>(r.k), static_cast<const uint16_t*>(r.v), static_cast<uint16_t*>(c.k),
                    static_cast<uint16_t*>(c.v), slots, r.k_token, r.k_head, r.v_token, r.v_head, c.k_page, c.k_token,
                    c.k_head, c.v_page, c.v_token, c.v_head, r.tokens, r.kv_heads, log2_of(r.head_dim / 8), c.n_pages,
                    log2_of(c.page_size)};
}

// Which kernel a call runs, how many CTAs and how many rows a partial slot has.
// Up to 8 (head_dim 256) or 16 packed rows a request the row kernel streams keys and values
// through registers; above, they are shared by 128 or 256 rows on the tensor cores.
struct Choice {
  bool wide;
  int nr, grid, slot_rows;
};
Choice choose(int head_dim, int group, int rows) {
  Choice c{};
  c.wide = group <= 128 && (rows == 0 || rows > attn_rows_limit(head_dim));
  if (c.wide) {
    c.grid = attn_wide_grid();
    c.slot_rows = 128 * attn_wide_blocks(head_dim);
    return c;
  }
  c.nr = (rows > 0 && rows <= 8) || head_dim == 256 ? 1 : 2;
  c.grid = attn_rows_grid(head_dim, 8 * c.nr);
  c.slot_rows = 8 * c.nr;
  return c;
}

// Rows of a block that are used where it holds whole tokens.
int token_rows(int head_dim, int group, const Choice& c) {
  if (!c.wide) return c.slot_rows;
  return c.slot_rows / attn_wide_blocks(head_dim) / group * group;
}
// Whether the kernel's 32-bit count of tiles (64 or 128 keys) holds the batch, every request at max_kv keys.
bool counts(const vq3_attn* at, int kv_heads, int head_dim, const Choice& c, int max_kv) {
  const int group = at->heads / kv_heads, blocks = c.wide ? attn_wide_blocks(head_dim) : 1;
  const double units = (double)at->tokens * group / (blocks * token_rows(head_dim, group, c)) + at->requests;
  return units * kv_heads * (max_kv / (c.wide ? 128.0 : 64.0) + 8) <= 4e9;
}

struct Ws {
  size_t rec, ml, part, total;
};
Ws carve(int head_dim, const Choice& c) {
  Ws w{};
  const size_t slots = (size_t)2 * c.grid * c.slot_rows;
  w.rec = 256;
  w.ml = up256(w.rec + (size_t)c.grid * sizeof(AttnRec));
  w.part = up256(w.ml + slots * 2 * sizeof(float));
  w.total = up256(w.part + slots * head_dim * sizeof(float));
  return w;
}

int run(const vq3_attn* at, int kv_heads, int head_dim, AttnArgs& a, void* workspace, size_t ws_bytes, void* stream,
        const char* who) {
  const int group = at->heads / kv_heads;
  const long long rows = (long long)at->max_new * group;
  Choice c = choose(head_dim, group, rows > (1 << 20) ? 1 << 20 : (int)rows);
  // max_new only picks the kernel: one that is too small for the batch must not get it refused
  const bool other = !c.wide && !counts(at, kv_heads, head_dim, c, a.max_kv);
  if (other) c = choose(head_dim, group, 0);
  if (!counts(at, kv_heads, head_dim, c, a.max_kv))
    return report_error(VQ3_EUNSUPPORTED, "%s: too many (row block, key tile) pairs: %d tokens, keys up to %d", who,
                        at->tokens, a.max_kv);
  const Ws w = carve(head_dim, c);
  if (!workspace) return report_error(VQ3_EINVAL, "%s: null workspace", who);
  if (!on(workspace, 256)) return report_error(VQ3_EALIGN, "%s: workspace must be 256-byte aligned", who);
  if (ws_bytes < w.total)
    return report_error(VQ3_ENOSPACE, "%s: workspace %zu < %zu bytes%s", who, ws_bytes, w.total,
                        other ? ", those of max_new 0, which this batch needs" : "");
  char* ws = static_cast<char*>(workspace);
  a.q = at->q;
  a.out = at->out;
  a.lse = at->lse;
  a.q_token = at->q_token;
  a.q_head = at->q_head;
  a.o_token = at->out_token;
  a.o_head = at->out_head;
  a.q_start = at->q_start;
  a.tokens = at->tokens;
  a.requests = at->requests;
  a.heads = at->heads;
  a.kv_heads = kv_heads;
  a.group = group;
  a.unit_cost = c.wide ? attn_wide_unit_cost(head_dim) : attn_rows_unit_cost();
  a.unit_blocks = c.wide ? attn_wide_blocks(head_dim) : 1;
  a.block_rows = c.slot_rows / a.unit_blocks;
  a.token_rows = token_rows(head_dim, group, c);
  a.by_group = FastDiv(group);
  a.by_unit = FastDiv(c.slot_rows);
  a.by_token_unit = FastDiv(a.unit_blocks * a.token_rows);
  a.scale_log2 = at->scale * kLog2e;
  a.status = reinterpret_cast<int*>(ws);
  a.rec = reinterpret_cast<AttnRec*>(ws + w.rec);
  a.part_ml = reinterpret_cast<float*>(ws + w.ml);
  a.part = reinterpret_cast<float*>(ws + w.part);
  const bool bf16 = at->type == VQ3_TYPE_BF16;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = c.wide ? launch_attn_wide(a, head_dim, bf16, st) : launch_attn_rows(a, head_dim, bf16, c.nr, st);
  if (e == cudaSuccess) e = launch_attn_combine(a, head_dim, bf16, c.grid, c.slot_rows, st);
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return report_ok();
}

// A call without rows or requests: only the status word of its workspace, if it has one.
int nothing(void* workspace, size_t ws_bytes, void* stream, const char* who) {
  if (!workspace || ws_bytes < sizeof(int)) return report_ok();
  if (!on(workspace, 256)) return report_error(VQ3_EALIGN, "%s: workspace must be 256-byte aligned", who);
  const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(int), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "%s: status word: %s", who, cudaGetErrorString(e));
  return report_ok();
}

// Checks of the query side that both forms share. *done: a valid call with nothing to do.
int check_attn(vq3_attn* at, int kv_heads, int head_dim, const char* who, bool* done) {
  *done = false;
  if (at->type != VQ3_TYPE_F16 && at->type != VQ3_TYPE_BF16)
    return report_error(VQ3_EUNSUPPORTED, "%s: unknown type %d", who, at->type);
  if (at->heads <= 0 || at->heads % kv_heads)
    return report_error(VQ3_EINVAL, "%s: heads=%d must be a positive multiple of kv_heads=%d", who, at->heads, kv_heads);
  if (at->tokens < 0 || at->requests < 0 || at->max_new < 0)
    return report_error(VQ3_EINVAL, "%s: tokens=%d requests=%d max_new=%d", who, at->tokens, at->requests, at->max_new);
  if (at->requests > kMaxRequests)
    return report_error(VQ3_EUNSUPPORTED, "%s: requests=%d above %d", who, at->requests, kMaxRequests);
  if ((long long)at->tokens * at->heads > 0x3fffffffLL)
    return report_error(VQ3_EUNSUPPORTED, "%s: tokens * heads above 2^30", who);
  // the kernels use scale * log2(e): that has to be finite, too
  if (!(at->scale > 0.f) || !std::isfinite(at->scale * kLog2e))
    return report_error(VQ3_EINVAL, "%s: scale=%g must be positive and at most 2e38", who, (double)at->scale);
  if (at->tokens == 0 || at->requests == 0) {
    *done = true;
    return VQ3_OK;
  }
  if (!at->q || !at->out || !at->q_start) return report_error(VQ3_EINVAL, "%s: null q, out or q_start", who);
  if (!on(at->q, 16) || !on(at->out, 16)) return report_error(VQ3_EALIGN, "%s: q and out must be 16-byte aligned", who);
  if (!on(at->q_start, 4) || (at->lse && !on(at->lse, 4)))
    return report_error(VQ3_EALIGN, "%s: q_start and lse must be 4-byte aligned", who);
  if (int rc = check_stride(&at->q_token, at->tokens, head_dim, who, "q token")) return rc;
  if (int rc = check_stride(&at->q_head, at->heads, head_dim, who, "q head")) return rc;
  if (int rc = check_stride(&at->out_token, at->tokens, head_dim, who, "out token")) return rc;
  if (int rc = check_stride(&at->out_head, at->heads, head_dim, who, "out head")) return rc;
  if (rows_overlap(at->tokens, at->out_token, at->heads, at->out_head, head_dim))
    return report_error(VQ3_EINVAL, "%s: the rows of out overlap", who);
  if (at->out == at->q) return report_error(VQ3_EINVAL, "%s: out must not alias q", who);
  return VQ3_OK;
}

}  // namespace
}  // namespace vq3

using namespace vq3;

extern "C" {

int vq3_paged_plan(const int* cached, const int* fresh, int requests, int page_size, const int* ring, int ring_size,
                   const int* ring_state, int* table, int max_pages, int max_tokens, int* q_start, int* kv_len,
                   long long* slots, int* positions, int* ring_state_out, int* status, void* stream) {
  if (requests < 0 || max_tokens < 0 || max_pages <= 0 || ring_size <= 0)
    return report_error(VQ3_EINVAL, "paged_plan: requests=%d max_tokens=%d max_pages=%d ring_size=%d", requests,
                        max_tokens, max_pages, ring_size);
  if (requests > kMaxRequests)
    return report_error(VQ3_EUNSUPPORTED, "paged_plan: requests=%d above %d", requests, kMaxRequests);
  if (max_tokens > (1 << 30))
    return report_error(VQ3_EUNSUPPORTED, "paged_plan: max_tokens=%d above 2^30", max_tokens);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return report_error(VQ3_EUNSUPPORTED, "paged_plan: page_size=%d must be a power of two in [16, 256]", page_size);
  if (!ring || !ring_state || !q_start || !ring_state_out || !status ||
      (requests && (!cached || !fresh || !table || !kv_len)) || (max_tokens && (!slots || !positions)))
    return report_error(VQ3_EINVAL, "paged_plan: null pointer");
  if (!on(cached, 4) || !on(fresh, 4) || !on(ring, 4) || !on(ring_state, 4) || !on(table, 4) || !on(q_start, 4) ||
      !on(kv_len, 4) || !on(slots, 8) || !on(positions, 4) || !on(ring_state_out, 4) || !on(status, 4))
    return report_error(VQ3_EALIGN, "paged_plan: pointers must be 4-byte (slots 8-byte) aligned");
  if (ring_state == ring_state_out || (requests && (table == ring || kv_len == cached || kv_len == fresh)))
    return report_error(VQ3_EINVAL, "paged_plan: outputs must not alias inputs");
  PlanArgs a{cached, fresh,     ring,           ring_state, table,    q_start,           kv_len,    slots,
             positions, ring_state_out, status,     requests, log2_of(page_size), ring_size, max_pages, max_tokens};
  const cudaError_t e = launch_paged_plan(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "paged_plan: launch: %s", cudaGetErrorString(e));
  return report_ok();
}

int vq3_kv_append(const vq3_kv_rows* rows, const long long* slots, const vq3_kv_cache* cache, void* stream) {
  if (!rows || !cache) return report_error(VQ3_EINVAL, "kv_append: null descriptor");
  vq3_kv_rows r = *rows;
  vq3_kv_cache c = *cache;
  if (int rc = check_cache(&c, "kv_append")) return rc;
  if (r.kv_heads != c.kv_heads || r.head_dim != c.head_dim)
    return report_error(VQ3_EINVAL, "kv_append: rows of %d x %d into a cache of %d x %d", r.kv_heads, r.head_dim,
                        c.kv_heads, c.head_dim);
  if (int rc = check_rows(&r, "kv_append")) return rc;
  if (r.tokens == 0) return report_ok();
  if (!slots) return report_error(VQ3_EINVAL, "kv_append: null slots");
  if (!on(slots, 8)) return report_error(VQ3_EALIGN, "kv_append: slots must be 8-byte aligned");
  const AppendArgs a = append_args(r, c, slots);
  const cudaError_t e = launch_kv_append(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "kv_append: launch: %s", cudaGetErrorString(e));
  return report_ok();
}

int vq3_kv_append_rotary(const vq3_rotary* rotary, const vq3_kv_rows* rows, const long long* slots,
                         const vq3_kv_cache* cache, void* stream) {
  const char* who = "kv_append_rotary";
  if (!rotary || !rows || !cache) return report_error(VQ3_EINVAL, "%s: null descriptor", who);
  vq3_rotary t = *rotary;
  vq3_kv_rows r = *rows;
  vq3_kv_cache c = *cache;
  if (t.type != VQ3_TYPE_F16 && t.type != VQ3_TYPE_BF16)
    return report_error(VQ3_EUNSUPPORTED, "%s: unknown type %d", who, t.type);
  if (int rc = check_cache(&c, who)) return rc;
  if (r.kv_heads != c.kv_heads || r.head_dim != c.head_dim)
    return report_error(VQ3_EINVAL, "%s: rows of %d x %d into a cache of %d x %d", who, r.kv_heads, r.head_dim,
                        c.kv_heads, c.head_dim);
  if (int rc = check_rows(&r, who)) return rc;
  if (t.heads < 0) return report_error(VQ3_EINVAL, "%s: heads=%d", who, t.heads);
  if (t.heads > kMaxKvHeads) return report_error(VQ3_EUNSUPPORTED, "%s: heads=%d above %d", who, t.heads, kMaxKvHeads);
  if (t.rotated <= 0 || t.rotated > r.head_dim || t.rotated % 16)
    return report_error(VQ3_EUNSUPPORTED, "%s: rotated=%d must be a multiple of 16 in [16, head_dim=%d]", who, t.rotated,
                        r.head_dim);
  if (r.tokens == 0) return report_ok();
  if (!slots || !t.positions || !t.freq) return report_error(VQ3_EINVAL, "%s: null slots, positions or freq", who);
  if (!on(slots, 8)) return report_error(VQ3_EALIGN, "%s: slots must be 8-byte aligned", who);
  if (!on(t.positions, 4) || !on(t.freq, 4))
    return report_error(VQ3_EALIGN, "%s: positions and freq must be 4-byte aligned", who);
  if (t.heads) {
    if (!t.q || !t.q_out) return report_error(VQ3_EINVAL, "%s: null q or q_out", who);
    if (!on(t.q, 16) || !on(t.q_out, 16)) return report_error(VQ3_EALIGN, "%s: q and q_out must be 16-byte aligned", who);
    if (int rc = check_stride(&t.q_token, r.tokens, r.head_dim, who, "q token")) return rc;
    if (int rc = check_stride(&t.q_head, t.heads, r.head_dim, who, "q head")) return rc;
    if (int rc = check_stride(&t.out_token, r.tokens, r.head_dim, who, "q_out token")) return rc;
    if (int rc = check_stride(&t.out_head, t.heads, r.head_dim, who, "q_out head")) return rc;
    if (rows_overlap(r.tokens, t.out_token, t.heads, t.out_head, r.head_dim))
      return report_error(VQ3_EINVAL, "%s: the rows of q_out overlap", who);
    if (t.q == t.q_out && (t.q_token != t.out_token || t.q_head != t.out_head))
      return report_error(VQ3_EINVAL, "%s: in place q and q_out have the same strides", who);
  }
  RotaryArgs a{};
  a.kv = append_args(r, c, slots);
  a.q = static_cast<const uint16_t*>(t.q);
  a.q_out = static_cast<uint16_t*>(t.q_out);
  a.positions = t.positions;
  a.freq = t.freq;
  a.q_token = t.q_token;
  a.q_head = t.q_head;
  a.o_token = t.out_token;
  a.o_head = t.out_head;
  a.heads = t.heads;
  a.half = t.rotated / 2;
  a.interleaved = t.interleaved != 0;
  const cudaError_t e = launch_kv_append_rotary(a, t.type == VQ3_TYPE_BF16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return report_ok();
}

size_t vq3_attention_workspace_bytes(int heads, int kv_heads, int head_dim, int max_new) {
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || kv_heads <= 0 || kv_heads > kMaxKvHeads ||
      heads <= 0 || heads % kv_heads || max_new < 0)
    return 0;
  const int group = heads / kv_heads;
  const long long rows = (long long)max_new * group;
  return carve(head_dim, choose(head_dim, group, rows > (1 << 20) ? 1 << 20 : (int)rows)).total;
}

int vq3_paged_attention(const vq3_attn* attn, const vq3_kv_cache* cache, const int* table, int max_pages,
                        const int* kv_len, void* workspace, size_t ws_bytes, void* stream) {
  if (!attn || !cache) return report_error(VQ3_EINVAL, "paged_attention: null descriptor");
  vq3_attn at = *attn;
  vq3_kv_cache c = *cache;
  if (int rc = check_cache(&c, "paged_attention")) return rc;
  bool done;
  if (int rc = check_attn(&at, c.kv_heads, c.head_dim, "paged_attention", &done)) return rc;
  if (max_pages <= 0) return report_error(VQ3_EINVAL, "paged_attention: max_pages=%d", max_pages);
  if ((long long)max_pages * c.page_size > kMaxKeys)
    return report_error(VQ3_EUNSUPPORTED, "paged_attention: max_pages * page_size above 2^30");
  if (done) return nothing(workspace, ws_bytes, stream, "paged_attention");
  if (!table || !kv_len) return report_error(VQ3_EINVAL, "paged_attention: null table or kv_len");
  if (!on(table, 4) || !on(kv_len, 4))
    return report_error(VQ3_EALIGN, "paged_attention: table and kv_len must be 4-byte aligned");
  AttnArgs a{};
  a.k = c.k;
  a.v = c.v;
  a.k_page = c.k_page;
  a.k_token = c.k_token;
  a.k_head = c.k_head;
  a.v_page = c.v_page;
  a.v_token = c.v_token;
  a.v_head = c.v_head;
  a.kv_len = kv_len;
  a.table = table;
  a.page_shift = log2_of(c.page_size);
  a.max_pages = max_pages;
  a.n_pages = c.n_pages;
  a.max_kv = max_pages * c.page_size;
  return run(&at, c.kv_heads, c.head_dim, a, workspace, ws_bytes, stream, "paged_attention");
}

int vq3_prompt_attention(const vq3_attn* attn, const vq3_kv_rows* rows, void* workspace, size_t ws_bytes,
                         void* stream) {
  if (!attn || !rows) return report_error(VQ3_EINVAL, "prompt_attention: null descriptor");
  vq3_attn at = *attn;
  vq3_kv_rows r = *rows;
  if (int rc = check_rows(&r, "prompt_attention")) return rc;
  bool done;
  if (int rc = check_attn(&at, r.kv_heads, r.head_dim, "prompt_attention", &done)) return rc;
  if (r.tokens != at.tokens)
    return report_error(VQ3_EINVAL, "prompt_attention: %d rows of k and v for %d of q", r.tokens, at.tokens);
  if (done) return nothing(workspace, ws_bytes, stream, "prompt_attention");
  AttnArgs a{};
  a.k = r.k;
  a.v = r.v;
  a.k_token = r.k_token;
  a.k_head = r.k_head;
  a.v_token = r.v_token;
  a.v_head = r.v_head;
  a.max_kv = at.tokens;
  return run(&at, r.kv_heads, r.head_dim, a, workspace, ws_bytes, stream, "prompt_attention");
}

}  // extern "C"
