"""Argument checks of the delta rule for packed requests, the short convolution and the rotated append (no GPU):
every refusal comes before a launch, with the documented status; and the oracle's own pins."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")
vq3 = pytest.importorskip("bit_vector_lut_gb300.vq3", reason="libvq3.so not built")

from oracle import delta_rule as D  # noqa: E402
from oracle import mixers as O  # noqa: E402
from tests.test_attention_cpu import ALIGN, INVALID, P, UNSUPPORTED, cache, rows  # noqa: E402


def batch(**kw):
    b = dict(tokens=7, requests=2, slots=3, q_start=P, slot_in=P, slot_out=P)
    b.update(kw)
    return vq3.vq3_batch(**b)


def delta(b=None, **kw):
    d = dict(type=0, qk_heads=2, v_heads=4, d_k=64, d_v=32, max_new=4, scale=1.0, q=P, k=P, v=P, out=2 * P, beta=P, alpha=P,
             states=3 * P, q_token=128, q_head=64, k_token=128, k_head=64, v_token=128, v_head=32, out_token=128, out_head=32,
             beta_token=4, alpha_token=4, state_slot=4 * 64 * 32)
    d.update(kw)
    return vq3.lib.vq3_delta_rule_batch(ctypes.byref(b or batch()), ctypes.byref(vq3.vq3_delta(**d)), None)


def conv(b=None, **kw):
    c = dict(type=0, channels=64, width=4, silu=1, unit_heads=2, head_dim=16, eps=1e-6, x=P, weight=P, bias=None, states=3 * P,
             out=2 * P, x_token=64, out_token=64, state_slot=192, state_row=64)
    c.update(kw)
    return vq3.lib.vq3_short_conv(ctypes.byref(b or batch()), ctypes.byref(vq3.vq3_conv(**c)), None)


def rotary(r=None, c=None, slots=P, **kw):
    t = dict(type=0, heads=8, rotated=64, interleaved=0, freq=P, positions=P, q=P, q_out=2 * P, q_token=1024, q_head=128,
             out_token=1024, out_head=128)
    t.update(kw)
    return vq3.lib.vq3_kv_append_rotary(ctypes.byref(vq3.vq3_rotary(**t)), ctypes.byref(r or rows()), slots,
                                        ctypes.byref(c or cache()), None)


@pytest.mark.parametrize("bad,code", [
    (dict(tokens=-1), INVALID), (dict(requests=-1), INVALID), (dict(slots=-1), INVALID), (dict(requests=8193), UNSUPPORTED),
    (dict(tokens=(1 << 30) + 1), UNSUPPORTED), (dict(q_start=None), INVALID), (dict(q_start=P + 2), ALIGN),
    (dict(slot_in=P + 1), ALIGN), (dict(slot_out=P + 3), ALIGN)])
def test_batch_is_checked(bad, code):
    assert delta(batch(**bad)) == code and conv(batch(**bad)) == code, vq3.lib.vq3_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(type=2), UNSUPPORTED), (dict(qk_heads=0), INVALID), (dict(v_heads=0), INVALID), (dict(v_heads=3), INVALID),
    (dict(v_heads=65536), UNSUPPORTED), (dict(d_k=32), UNSUPPORTED), (dict(d_k=96), UNSUPPORTED), (dict(d_v=24), UNSUPPORTED),
    (dict(d_v=0), UNSUPPORTED), (dict(d_v=4112), UNSUPPORTED), (dict(max_new=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(alpha=None), INVALID), (dict(beta=None), INVALID), (dict(states=None), INVALID),
    (dict(q=P + 8), ALIGN), (dict(v=P + 2), ALIGN), (dict(out=P + 4), ALIGN), (dict(states=P + 8), ALIGN), (dict(alpha=P + 2), ALIGN),
    (dict(q_token=32), INVALID), (dict(k_head=68), ALIGN), (dict(v_head=0), INVALID), (dict(out_token=-128), INVALID),
    (dict(out_token=40), INVALID), (dict(out=P), INVALID), (dict(out=3 * P), INVALID), (dict(alpha_token=3), INVALID),
    (dict(beta_token=0), INVALID), (dict(state_slot=4 * 64 * 32 - 4), INVALID), (dict(state_slot=4 * 64 * 32 + 2), ALIGN),
    (dict(status=P + 2), ALIGN)])
def test_delta_refuses(bad, code):
    assert delta(**bad) == code, vq3.lib.vq3_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(type=-1), UNSUPPORTED), (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED), (dict(channels=0), UNSUPPORTED),
    (dict(channels=60), UNSUPPORTED), (dict(channels=(1 << 20) + 8), UNSUPPORTED), (dict(unit_heads=-1), INVALID),
    (dict(unit_heads=5), INVALID), (dict(head_dim=24), UNSUPPORTED), (dict(head_dim=4), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(weight=None), INVALID), (dict(out=None), INVALID), (dict(states=None), INVALID), (dict(x=P + 8), ALIGN),
    (dict(weight=P + 2), ALIGN), (dict(bias=P + 4), ALIGN), (dict(states=P + 8), ALIGN), (dict(x_token=56), INVALID),
    (dict(x_token=68), ALIGN), (dict(out_token=0), INVALID), (dict(out=P), INVALID), (dict(out=3 * P), INVALID),
    (dict(state_row=8), INVALID), (dict(state_row=68), ALIGN), (dict(state_slot=184), INVALID), (dict(state_slot=196), ALIGN)])
def test_conv_refuses(bad, code):
    assert conv(**bad) == code, vq3.lib.vq3_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(type=5), UNSUPPORTED), (dict(heads=-1), INVALID), (dict(heads=65537), UNSUPPORTED), (dict(rotated=0), UNSUPPORTED),
    (dict(rotated=24), UNSUPPORTED), (dict(rotated=144), UNSUPPORTED), (dict(freq=None), INVALID), (dict(positions=None), INVALID),
    (dict(freq=P + 2), ALIGN), (dict(positions=P + 1), ALIGN), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(q=P + 8), ALIGN), (dict(q_out=P + 2), ALIGN), (dict(q_token=100), INVALID), (dict(q_head=132), ALIGN),
    (dict(out_head=0), INVALID), (dict(out_token=136), INVALID), (dict(q_out=P, out_token=2048), INVALID),
    (dict(slots=None), INVALID), (dict(slots=P + 4), ALIGN)])
def test_rotary_refuses(bad, code):
    assert rotary(**bad) == code, vq3.lib.vq3_last_error()


def test_rotary_checks_rows_and_cache():
    assert rotary(c=cache(page_size=24)) == UNSUPPORTED and rotary(r=rows(head_dim=64)) == INVALID
    assert rotary(r=rows(kv_heads=2)) == INVALID and rotary(r=rows(k=None)) == INVALID and rotary(r=rows(v=P + 8)) == ALIGN
    f = vq3.lib.vq3_kv_append_rotary
    assert f(None, ctypes.byref(rows()), P, ctypes.byref(cache()), None) == INVALID
    assert vq3.lib.vq3_delta_rule_batch(None, None, None) == INVALID and vq3.lib.vq3_short_conv(None, None, None) == INVALID


def test_nothing_to_do():
    assert delta(batch(requests=0, q_start=None)) == 0 and conv(batch(requests=0, q_start=None)) == 0
    assert rotary(rows(tokens=0, k=None, v=None), slots=None) == 0


def test_binding_refuses_before_the_library():
    h, f, i = torch.float16, torch.float32, torch.int32
    q, v, g = torch.zeros(3, 2, 64, dtype=h), torch.zeros(3, 4, 32, dtype=h), torch.zeros(3, 4)
    s, st, sl = torch.zeros(5, 4, 64, 32), torch.zeros(3, dtype=i), torch.zeros(2, dtype=i)
    x, w, cs = torch.zeros(3, 64, dtype=h), torch.zeros(64, 4, dtype=h), torch.zeros(5, 3, 64, dtype=h)
    k, pages = torch.zeros(3, 2, 64, dtype=h), torch.zeros(2, 16, 2, 64, dtype=h)
    pos, slots, fr = torch.zeros(3, dtype=i), torch.zeros(3, dtype=torch.int64), torch.zeros(32)
    bad = [
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s, st),                       # CPU tensors
        lambda: vq3.delta_rule_batch(q, q.bfloat16(), v, g, g, s, st),
        lambda: vq3.delta_rule_batch(q, q[:, :1], v, g, g, s, st),
        lambda: vq3.delta_rule_batch(q[:2], q[:2], v, g, g, s, st),
        lambda: vq3.delta_rule_batch(q.float(), q.float(), v.float(), g, g, s, st),
        lambda: vq3.delta_rule_batch(q, q, v, g.half(), g, s, st),
        lambda: vq3.delta_rule_batch(q, q, v, g, g[:, :2], s, st),
        lambda: vq3.delta_rule_batch(q, q, v, g, g.t().contiguous().t(), s, st),  # heads not side by side
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s.half(), st),
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s.transpose(2, 3), st),
        lambda: vq3.delta_rule_batch(q, q, v, g, g, torch.zeros(5, 4, 32, 64), st),
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s, st.long()),
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s, st, slot_in=st),           # slots of another batch
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s, st, slot_out=sl.long()),
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s, st, out=v[:2]),
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s, st, status=sl),
        lambda: vq3.delta_rule_batch(q, q, v, g, g, s, st, status=st[:1].long()),
        lambda: vq3.delta_rule_batch(q.transpose(0, 2), q.transpose(0, 2), v, g, g, s, st),
        lambda: vq3.short_conv(x, w, cs, st),
        lambda: vq3.short_conv(x, w[:32], cs, st),
        lambda: vq3.short_conv(x, w.float(), cs, st),
        lambda: vq3.short_conv(x, w.t().contiguous().t(), cs, st),
        lambda: vq3.short_conv(x, w, cs[:, :2], st),
        lambda: vq3.short_conv(x, w, cs.float(), st),
        lambda: vq3.short_conv(x, w, cs, st, bias=torch.zeros(64)),
        lambda: vq3.short_conv(x, w, cs, st, slot_in=st),
        lambda: vq3.short_conv(x, w, cs, st, out=x[:, :32]),
        lambda: vq3.kv_append_rotary(k, k, k, pos, slots, fr, pages, pages),
        lambda: vq3.kv_append_rotary(k.bfloat16(), k, k, pos, slots, fr, pages, pages),
        lambda: vq3.kv_append_rotary(k[:2], k, k, pos, slots, fr, pages, pages),
        lambda: vq3.kv_append_rotary(k, k, k, pos[:2], slots, fr, pages, pages),
        lambda: vq3.kv_append_rotary(k, k, k, slots, slots, fr, pages, pages),
        lambda: vq3.kv_append_rotary(k, k, k, pos, pos, fr, pages, pages),
        lambda: vq3.kv_append_rotary(k, k, k, pos, slots, fr.double(), pages, pages),
        lambda: vq3.kv_append_rotary(None, k, k, pos, slots, fr, pages, pages, q_out=k),
        lambda: vq3.kv_append_rotary(k, k, k, pos, slots, fr, pages.bfloat16(), pages.bfloat16()),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(vq3.Vq3Error):
            call()
            pytest.fail(f"call {n} went through")
    assert f is torch.float32


def test_packed_structures_are_the_structures():
    for cls, pack in ((vq3.vq3_batch, vq3._pack_batch), (vq3.vq3_delta, vq3._pack_delta), (vq3.vq3_conv, vq3._pack_conv),
                      (vq3.vq3_rotary, vq3._pack_rotary)):
        values = [1.5 if t is ctypes.c_float else 3 + i for i, (_, t) in enumerate(cls._fields_)]
        assert pack(*values) == bytes(cls(*values))
        with pytest.raises(vq3.Vq3Error):
            pack(1 << 40, *values[1:])


@pytest.mark.parametrize("src", ["delta_batch.cu", "delta_wide.cu", "conv.cu", "rotary.cu"])
def test_bounds_check_variant_compiles(tmp_path, src):
    from bit_vector_lut_gb300 import build as B
    r = subprocess.run([B.nvcc(), *B.ARCH, *B.NVCC_FLAGS, "-DVQ3_BOUNDS_CHECK", "-c", os.path.join(B.CSRC, src), "-o",
                        str(tmp_path / "x.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


# ---------------------------------------------------------------- the oracle's pins

def test_oracle_delta_is_the_recurrence():
    rng = np.random.default_rng(0)
    q, k, v, s = rng.normal(size=(5, 8)), rng.normal(size=(5, 8)), rng.normal(size=(5, 4)), rng.normal(size=(8, 4))
    b, a = rng.uniform(size=5), rng.uniform(size=5)
    out, S, info = O.delta(q, k, v, b, a, s, 0.5)
    ref, ref_S = D.recurrent(q, k, v, b, a, s)
    assert np.allclose(out, 0.5 * ref) and np.allclose(S, ref_S)
    assert (np.abs(out) <= 0.5 * info["reach"] + 1e-12).all() and (info["top"] >= np.linalg.norm(S, axis=0) - 1e-12).all()


def test_oracle_conv_pins():
    x, old, w = np.array([[1.0], [2.0], [4.0]]), np.array([[8.0], [16.0], [32.0]]), np.array([[1.0, 10.0, 100.0, 1000.0]])
    y, kept, _ = O.conv(x, old, w, None, False, 0, 0, 0.0)
    assert y[:, 0].tolist() == [8 + 160 + 3200 + 1000, 16 + 320 + 100 + 2000, 32 + 10 + 200 + 4000] and kept[:, 0].tolist() == [1, 2, 4]
    y, kept, _ = O.conv(x[:1], old, w, np.array([0.5]), True, 0, 0, 0.0)
    assert np.isclose(y[0, 0], 4368.5) and kept[:, 0].tolist() == [16, 32, 1]
    y, _, _ = O.conv(np.ones((1, 4)), np.zeros((1, 4)), np.array([[0, 3.0], [0, 4.0], [0, 5.0], [0, 12.0]]), None, False, 1, 2, 0.0)
    assert np.allclose(y, [[0.6, 0.8, 5, 12]])


def test_oracle_rotation_pins():
    x = np.arange(8.0)[None, None]
    y, _ = O.rotate(x, np.array([1]), [np.pi / 2, np.pi], False)
    assert np.allclose(y[0, 0], [-2, -1, 0, -3, 4, 5, 6, 7])
    y, _ = O.rotate(x, np.array([1]), [np.pi / 2, np.pi], True)
    assert np.allclose(y[0, 0], [-1, 0, -2, -3, 4, 5, 6, 7])
