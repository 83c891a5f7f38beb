// C ABI of the delta-rule token mixer for packed requests: the rule itself and the short convolution in front of it.
#include <cmath>

#include "api_checks.h"

namespace vq3 {
namespace {

// The batch; *done: a valid call without requests.
int check_batch(const vq3_batch& b, const char* who, bool* done) {
  *done = false;
  if (b.tokens < 0 || b.requests < 0 || b.slots < 0)
    return report_error(VQ3_EINVAL, "%s: tokens=%d requests=%d slots=%d", who, b.tokens, b.requests, b.slots);
  if (b.requests > kMaxRequests)
    return report_error(VQ3_EUNSUPPORTED, "%s: requests=%d above %d", who, b.requests, kMaxRequests);
  if (b.tokens > (1 << 30)) return report_error(VQ3_EUNSUPPORTED, "%s: tokens=%d above 2^30", who, b.tokens);
  if (b.requests == 0) {
    *done = true;
    return VQ3_OK;
  }
  if (!b.q_start) return report_error(VQ3_EINVAL, "%s: null q_start", who);
  if (!on(b.q_start, 4) || !on(b.slot_in, 4) || !on(b.slot_out, 4))
    return report_error(VQ3_EALIGN, "%s: q_start and slots must be 4-byte aligned", who);
  return VQ3_OK;
}
int check_type(int type, const char* who) {
  if (type != VQ3_TYPE_F16 && type != VQ3_TYPE_BF16) return report_error(VQ3_EUNSUPPORTED, "%s: unknown type %d", who, type);
  return VQ3_OK;
}

}  // namespace
}  // namespace vq3

using namespace vq3;

extern "C" {

int vq3_delta_rule_batch(const vq3_batch* batch, const vq3_delta* delta, void* stream) {
  const char* who = "delta_rule_batch";
  if (!batch || !delta) return report_error(VQ3_EINVAL, "%s: null descriptor", who);
  const vq3_batch& b = *batch;
  vq3_delta d = *delta;
  bool done;
  if (int rc = check_type(d.type, who)) return rc;
  if (int rc = check_batch(b, who, &done)) return rc;
  if (d.qk_heads <= 0 || d.v_heads <= 0 || d.v_heads % d.qk_heads)
    return report_error(VQ3_EINVAL, "%s: v_heads=%d must be a positive multiple of qk_heads=%d", who, d.v_heads, d.qk_heads);
  if (d.v_heads > 65535) return report_error(VQ3_EUNSUPPORTED, "%s: v_heads=%d above 65535", who, d.v_heads);
  if (d.d_k != 64 && d.d_k != 128 && d.d_k != 256)
    return report_error(VQ3_EUNSUPPORTED, "%s: d_k=%d must be 64, 128 or 256", who, d.d_k);
  if (d.d_v <= 0 || d.d_v % 16 || d.d_v > 4096)
    return report_error(VQ3_EUNSUPPORTED, "%s: d_v=%d must be a multiple of 16 up to 4096", who, d.d_v);
  if (d.max_new < 0) return report_error(VQ3_EINVAL, "%s: max_new=%d", who, d.max_new);
  if (!std::isfinite(d.scale)) return report_error(VQ3_EINVAL, "%s: scale=%g", who, (double)d.scale);
  if (!on(d.status, 4)) return report_error(VQ3_EALIGN, "%s: status must be 4-byte aligned", who);
  if (done) return report_ok();
  const long long state = (long long)d.v_heads * d.d_k * d.d_v;
  if (b.slots) {
    if (!d.states) return report_error(VQ3_EINVAL, "%s: null states", who);
    if (!on(d.states, 16)) return report_error(VQ3_EALIGN, "%s: states must be 16-byte aligned", who);
    if (b.slots == 1) d.state_slot = state;
    if (d.state_slot < state || d.state_slot >= (1LL << 38))
      return report_error(VQ3_EINVAL, "%s: slot stride %lld must be at least %lld (and below 2^38)", who, d.state_slot, state);
    if (d.state_slot % 4) return report_error(VQ3_EALIGN, "%s: slot stride %lld is not a multiple of 4", who, d.state_slot);
  }
  if (b.tokens) {
    if (!d.q || !d.k || !d.v || !d.out || !d.alpha || !d.beta)
      return report_error(VQ3_EINVAL, "%s: null q, k, v, out, alpha or beta", who);
    if (!on(d.q, 16) || !on(d.k, 16) || !on(d.v, 16) || !on(d.out, 16))
      return report_error(VQ3_EALIGN, "%s: q, k, v and out must be 16-byte aligned", who);
    if (!on(d.alpha, 4) || !on(d.beta, 4)) return report_error(VQ3_EALIGN, "%s: alpha and beta must be 4-byte aligned", who);
    if (int rc = check_stride(&d.q_token, b.tokens, d.d_k, who, "q token")) return rc;
    if (int rc = check_stride(&d.q_head, d.qk_heads, d.d_k, who, "q head")) return rc;
    if (int rc = check_stride(&d.k_token, b.tokens, d.d_k, who, "k token")) return rc;
    if (int rc = check_stride(&d.k_head, d.qk_heads, d.d_k, who, "k head")) return rc;
    if (int rc = check_stride(&d.v_token, b.tokens, d.d_v, who, "v token")) return rc;
    if (int rc = check_stride(&d.v_head, d.v_heads, d.d_v, who, "v head")) return rc;
    if (int rc = check_stride(&d.out_token, b.tokens, d.d_v, who, "out token")) return rc;
    if (int rc = check_stride(&d.out_head, d.v_heads, d.d_v, who, "out head")) return rc;
    if (rows_overlap(b.tokens, d.out_token, d.v_heads, d.out_head, d.d_v))
      return report_error(VQ3_EINVAL, "%s: the rows of out overlap", who);
    if (d.out == d.q || d.out == d.k || d.out == d.v || d.out == d.states)
      return report_error(VQ3_EINVAL, "%s: out must not alias an input", who);
    for (long long* s : {&d.alpha_token, &d.beta_token}) {
      if (b.tokens == 1) *s = d.v_heads;
      if (*s < d.v_heads || *s >= (1LL << 38))
        return report_error(VQ3_EINVAL, "%s: alpha or beta token stride %lld must be at least v_heads=%d (and below 2^38)",
                            who, *s, d.v_heads);
    }
  }
  DeltaArgs a{};
  a.q = d.q;
  a.k = d.k;
  a.v = d.v;
  a.out = d.out;
  a.alpha = d.alpha;
  a.beta = d.beta;
  a.states = d.states;
  a.status = d.status;
  a.q_start = b.q_start;
  a.slot_in = b.slot_in;
  a.slot_out = b.slot_out;
  a.q_token = d.q_token;
  a.q_head = d.q_head;
  a.k_token = d.k_token;
  a.k_head = d.k_head;
  a.v_token = d.v_token;
  a.v_head = d.v_head;
  a.o_token = d.out_token;
  a.o_head = d.out_head;
  a.alpha_token = d.alpha_token;
  a.beta_token = d.beta_token;
  a.state_slot = d.state_slot;
  a.tokens = b.tokens;
  a.requests = b.requests;
  a.slots = b.slots;
  a.v_heads = d.v_heads;
  a.group = d.v_heads / d.qk_heads;
  a.d_k = d.d_k;
  a.d_v = d.d_v;
  a.max_new = d.max_new;
  a.scale = d.scale;
  const cudaError_t e = launch_delta_batch(a, d.type == VQ3_TYPE_BF16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return report_ok();
}

int vq3_delta_status(int* status_host, void* stream) {
  if (!status_host) return report_error(VQ3_EINVAL, "delta_status: null pointer");
  const cudaError_t e = delta_status(status_host, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "delta_status: %s", cudaGetErrorString(e));
  return report_ok();
}

int vq3_short_conv(const vq3_batch* batch, const vq3_conv* conv, void* stream) {
  const char* who = "short_conv";
  if (!batch || !conv) return report_error(VQ3_EINVAL, "%s: null descriptor", who);
  const vq3_batch& b = *batch;
  vq3_conv c = *conv;
  bool done;
  if (int rc = check_type(c.type, who)) return rc;
  if (int rc = check_batch(b, who, &done)) return rc;
  if (c.width < 2 || c.width > 4) return report_error(VQ3_EUNSUPPORTED, "%s: width=%d must be 2, 3 or 4", who, c.width);
  if (c.channels <= 0 || c.channels % 8 || c.channels > (1 << 20))
    return report_error(VQ3_EUNSUPPORTED, "%s: channels=%d must be a multiple of 8 up to 2^20", who, c.channels);
  if (c.unit_heads < 0) return report_error(VQ3_EINVAL, "%s: unit_heads=%d", who, c.unit_heads);
  if (c.unit_heads) {
    if (c.head_dim < 8 || c.head_dim > 256 || (c.head_dim & (c.head_dim - 1)))
      return report_error(VQ3_EUNSUPPORTED, "%s: head_dim=%d must be a power of two in [8, 256]", who, c.head_dim);
    if ((long long)c.unit_heads * c.head_dim > c.channels)
      return report_error(VQ3_EINVAL, "%s: %d heads of %d in %d channels", who, c.unit_heads, c.head_dim, c.channels);
    if (!(c.eps >= 0.f) || !std::isfinite(c.eps)) return report_error(VQ3_EINVAL, "%s: eps=%g", who, (double)c.eps);
  }
  if (done) return report_ok();
  if (b.slots) {
    if (!c.states) return report_error(VQ3_EINVAL, "%s: null states", who);
    if (!on(c.states, 16)) return report_error(VQ3_EALIGN, "%s: states must be 16-byte aligned", who);
    if (int rc = check_stride(&c.state_row, c.width - 1, c.channels, who, "state row")) return rc;
    if (int rc = check_stride(&c.state_slot, b.slots, (c.width - 2) * c.state_row + c.channels, who, "slot")) return rc;
  }
  if (b.tokens) {
    if (!c.x || !c.weight || !c.out) return report_error(VQ3_EINVAL, "%s: null x, weight or out", who);
    if (!on(c.x, 16) || !on(c.weight, 16) || !on(c.out, 16) || !on(c.bias, 16))
      return report_error(VQ3_EALIGN, "%s: x, weight, bias and out must be 16-byte aligned", who);
    if (int rc = check_stride(&c.x_token, b.tokens, c.channels, who, "x token")) return rc;
    if (int rc = check_stride(&c.out_token, b.tokens, c.channels, who, "out token")) return rc;
    if (c.out == c.x || c.out == c.states) return report_error(VQ3_EINVAL, "%s: out must not alias an input", who);
  }
  ConvArgs a{};
  a.x = static_cast<const uint16_t*>(c.x);
  a.weight = static_cast<const uint16_t*>(c.weight);
  a.bias = static_cast<const uint16_t*>(c.bias);
  a.states = static_cast<uint16_t*>(c.states);
  a.out = static_cast<uint16_t*>(c.out);
  a.q_start = b.q_start;
  a.slot_in = b.slot_in;
  a.slot_out = b.slot_out;
  a.x_token = c.x_token;
  a.o_token = c.out_token;
  a.state_slot = c.state_slot;
  a.state_row = c.state_row;
  a.tokens = b.tokens;
  a.requests = b.requests;
  a.slots = b.slots;
  a.channels = c.channels;
  a.unit_channels = c.unit_heads * c.head_dim;
  a.head_chunks = c.unit_heads ? c.head_dim / 8 : 1;
  a.silu = c.silu != 0;
  a.eps = c.eps;
  const cudaError_t e = launch_short_conv(a, c.width, c.type == VQ3_TYPE_BF16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(VQ3_ECUDA, "%s: launch: %s", who, cudaGetErrorString(e));
  return report_ok();
}

}  // extern "C"
