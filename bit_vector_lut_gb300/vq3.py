"""Python binding of libvq3.so (argument marshalling only).

Every step of the VQ3 MLP path runs in the library's CUDA kernels; this module
only turns torch tensors into raw pointers and streams, and raises on a
non-zero status. PyTorch supplies device memory and streams. Importing this
module fails loudly when the library has not been built: there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import struct
from ctypes import POINTER, c_float, c_int, c_longlong, c_size_t, c_uint8, c_void_p
from typing import NamedTuple

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# VQ3_LIB may name another build of the same library (the bounds-check build, libvq3_bc.so)
LIB_PATH = os.environ.get("VQ3_LIB") or os.path.join(_PKG, "libvq3.so")

VQ3_OK, VQ3_ENOSPACE = 0, -5
ERRORS = {-1: "VQ3_EINVAL", -2: "VQ3_EALIGN", -3: "VQ3_EUNSUPPORTED", -4: "VQ3_ECUDA", -5: "VQ3_ENOSPACE"}


class Vq3Error(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


class vq3_linear(ctypes.Structure):
    _fields_ = [("d_in", c_int), ("d_out", c_int), ("block", c_int), ("packed", c_void_p),
                ("codebook", c_void_p), ("scales", c_void_p), ("signs", c_void_p), ("format", c_int),
                ("lr_rank", c_int), ("lr_u", c_void_p), ("lr_v", c_void_p)]


# index formats (VQ3_FORMAT_* in vq3.h): name -> (code, index bits, output channels per index)
FORMATS = {"2x64": (0, 6, 2), "2x16": (1, 4, 2), "lut4": (2, 4, 1)}


class vq3_mlp_layer(ctypes.Structure):
    _fields_ = [("gate", vq3_linear), ("up", vq3_linear), ("down", vq3_linear)]


class vq3_blob_view(ctypes.Structure):
    _fields_ = [("d_in", c_int), ("d_out", c_int), ("block", c_int), ("format", c_int), ("lr_rank", c_int),
                ("has_signs", c_int), ("canonical", c_void_p), ("packed", c_void_p), ("scales", c_void_p),
                ("codebook", c_void_p), ("codebook_bytes", c_size_t), ("signs", c_void_p), ("lr_u", c_void_p),
                ("lr_v", c_void_p)]


class vq3_kv_cache(ctypes.Structure):
    _fields_ = [("kv_heads", c_int), ("head_dim", c_int), ("page_size", c_int), ("n_pages", c_int), ("k", c_void_p),
                ("v", c_void_p), ("k_page", c_longlong), ("k_token", c_longlong), ("k_head", c_longlong),
                ("v_page", c_longlong), ("v_token", c_longlong), ("v_head", c_longlong)]


class vq3_kv_rows(ctypes.Structure):
    _fields_ = [("kv_heads", c_int), ("head_dim", c_int), ("tokens", c_int), ("k", c_void_p), ("v", c_void_p),
                ("k_token", c_longlong), ("k_head", c_longlong), ("v_token", c_longlong), ("v_head", c_longlong)]


class vq3_attn(ctypes.Structure):
    _fields_ = [("type", c_int), ("heads", c_int), ("tokens", c_int), ("requests", c_int), ("max_new", c_int),
                ("scale", c_float), ("q", c_void_p), ("out", c_void_p), ("lse", c_void_p), ("q_start", c_void_p),
                ("q_token", c_longlong), ("q_head", c_longlong), ("out_token", c_longlong), ("out_head", c_longlong)]


class vq3_rotary(ctypes.Structure):
    _fields_ = [("type", c_int), ("heads", c_int), ("rotated", c_int), ("interleaved", c_int), ("freq", c_void_p),
                ("positions", c_void_p), ("q", c_void_p), ("q_out", c_void_p), ("q_token", c_longlong),
                ("q_head", c_longlong), ("out_token", c_longlong), ("out_head", c_longlong)]


class vq3_batch(ctypes.Structure):
    _fields_ = [("tokens", c_int), ("requests", c_int), ("slots", c_int), ("q_start", c_void_p), ("slot_in", c_void_p),
                ("slot_out", c_void_p)]


class vq3_delta(ctypes.Structure):
    _fields_ = [("type", c_int), ("qk_heads", c_int), ("v_heads", c_int), ("d_k", c_int), ("d_v", c_int),
                ("max_new", c_int), ("scale", c_float), ("q", c_void_p), ("k", c_void_p), ("v", c_void_p),
                ("out", c_void_p), ("beta", c_void_p), ("alpha", c_void_p), ("states", c_void_p),
                ("q_token", c_longlong), ("q_head", c_longlong), ("k_token", c_longlong), ("k_head", c_longlong),
                ("v_token", c_longlong), ("v_head", c_longlong), ("out_token", c_longlong), ("out_head", c_longlong),
                ("beta_token", c_longlong), ("alpha_token", c_longlong), ("state_slot", c_longlong), ("status", c_void_p)]


class vq3_conv(ctypes.Structure):
    _fields_ = [("type", c_int), ("channels", c_int), ("width", c_int), ("silu", c_int), ("unit_heads", c_int),
                ("head_dim", c_int), ("eps", c_float), ("x", c_void_p), ("weight", c_void_p), ("bias", c_void_p),
                ("states", c_void_p), ("out", c_void_p), ("x_token", c_longlong), ("out_token", c_longlong),
                ("state_slot", c_longlong), ("state_row", c_longlong)]


def _packer(cls):
    """Makes the bytes of a structure, in half the time of the structure itself."""
    letters = {c_int: "i", c_float: "f", c_void_p: "P", c_longlong: "q"}
    form = struct.Struct("@" + "".join(letters[t] for _, t in cls._fields_))
    assert form.size == ctypes.sizeof(cls)

    def pack(*values):
        try:
            return form.pack(*values)
        except struct.error as e:  # a number that its field does not hold
            raise Vq3Error(-1, f"{cls.__name__}: {e}") from None

    return pack


_pack_batch, _pack_delta, _pack_conv, _pack_rotary = (_packer(c) for c in (vq3_batch, vq3_delta, vq3_conv, vq3_rotary))

# VQ3_TYPE_* in vq3.h
TYPES = {torch.float16: 0, torch.bfloat16: 1}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "vq3_packed_bytes": (c_size_t, [c_int, c_int]),
        "vq3_pack_layout": (c_int, [POINTER(c_uint8), c_int, c_int, c_void_p]),
        "vq3_unpack_layout": (c_int, [c_void_p, c_int, c_int, POINTER(c_uint8)]),
        "vq3_packed_bytes_fmt": (c_size_t, [c_int, c_int, c_int]),
        "vq3_pack_layout_fmt": (c_int, [c_int, POINTER(c_uint8), c_int, c_int, c_void_p]),
        "vq3_unpack_layout_fmt": (c_int, [c_int, c_void_p, c_int, c_int, POINTER(c_uint8)]),
        "vq3_blob_bytes": (c_size_t, [c_int, c_int, c_int, c_int, c_int]),
        "vq3_blob_write": (c_int, [c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int,
                                   c_void_p, c_void_p, c_void_p, c_size_t]),
        "vq3_blob_read": (c_int, [c_void_p, c_size_t, POINTER(vq3_blob_view)]),
        "fwht_rotate": (c_int, [c_void_p, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p]),
        "vq3_linear_workspace_bytes": (c_size_t, [c_int, POINTER(vq3_linear)]),
        "vq3_mlp_workspace_bytes": (c_size_t, [c_int, POINTER(vq3_mlp_layer)]),
        "vq3_workspace_init": (c_int, [c_void_p, c_size_t, c_void_p]),
        "vq3_workspace_status": (c_int, [c_void_p, POINTER(c_int), c_void_p]),
        "vq3_linear_forward": (c_int, [c_void_p, c_int, POINTER(vq3_linear), c_void_p, c_void_p, c_size_t, c_void_p]),
        "vq3_mlp_forward": (c_int, [c_void_p, c_int, POINTER(vq3_mlp_layer), c_void_p, c_void_p, c_size_t, c_void_p]),
        "vq3_mlp_kernel_launches": (c_int, [c_int, POINTER(vq3_mlp_layer)]),
        "vq3_linear_kernel_launches": (c_int, [c_int, POINTER(vq3_linear)]),
        "vq3_mlp_host_workspace_bytes": (c_size_t, [c_int, POINTER(vq3_mlp_layer)]),
        "vq3_mlp_forward_host": (c_int, [c_void_p, c_int, POINTER(vq3_mlp_layer), c_void_p, c_void_p, c_size_t,
                                         c_void_p]),
        "vq3_residual_rmsnorm": (c_int, [c_void_p, c_void_p, c_int, c_int, c_float, c_void_p, c_void_p]),
        "vq3_dequant_dense": (c_int, [POINTER(vq3_linear), c_int, c_void_p, c_void_p]),
        "vq3_delta_rule_forward": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                           c_int, c_void_p, c_void_p, c_void_p]),
        "vq3_mlp_forward_residual": (c_int, [c_void_p, c_void_p, c_int, POINTER(vq3_mlp_layer), c_float, c_void_p,
                                             c_void_p, c_void_p, c_size_t, c_void_p]),
        "vq3_mlp_prenorm_step": (c_int, [c_void_p, c_void_p, c_int, POINTER(vq3_mlp_layer), c_float, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
        "vq3_mlp_forward_noalloc": (c_int, [c_void_p, c_int, POINTER(vq3_mlp_layer), c_void_p, c_void_p]),
        "vq3_noalloc_status": (c_int, [POINTER(c_int), c_void_p]),
        "vq3_paged_plan": (c_int, [c_void_p, c_void_p, c_int, c_int, c_void_p, c_int, c_void_p, c_void_p, c_int, c_int,
                                   c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
        "vq3_kv_append": (c_int, [POINTER(vq3_kv_rows), c_void_p, POINTER(vq3_kv_cache), c_void_p]),
        "vq3_attention_workspace_bytes": (c_size_t, [c_int, c_int, c_int, c_int]),
        "vq3_paged_attention": (c_int, [POINTER(vq3_attn), POINTER(vq3_kv_cache), c_void_p, c_int, c_void_p, c_void_p,
                                        c_size_t, c_void_p]),
        "vq3_prompt_attention": (c_int, [POINTER(vq3_attn), POINTER(vq3_kv_rows), c_void_p, c_size_t, c_void_p]),
        # vq3_rotary, vq3_batch, vq3_delta and vq3_conv come as their bytes or by reference
        "vq3_kv_append_rotary": (c_int, [c_void_p, POINTER(vq3_kv_rows), c_void_p, POINTER(vq3_kv_cache), c_void_p]),
        "vq3_delta_rule_batch": (c_int, [c_void_p, c_void_p, c_void_p]),
        "vq3_delta_status": (c_int, [POINTER(c_int), c_void_p]),
        "vq3_short_conv": (c_int, [c_void_p, c_void_p, c_void_p]),
        "vq3_last_error": (ctypes.c_char_p, []),
        "vq3_version": (ctypes.c_char_p, []),
        "vq3_bounds_check": (c_int, [POINTER(ctypes.c_uint), c_int, c_int]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def _check(rc: int) -> None:
    if rc != VQ3_OK:
        raise Vq3Error(rc, lib.vq3_last_error().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def version() -> str:
    return lib.vq3_version().decode()


BOUNDS_FILES = ("decode", "lowrank", "delta", "rotate", "prefill", "prefill_wide", "attn", "attn_wide", "kvcache",
                "delta_batch", "delta_wide", "conv", "rotary")


def bounds_check(reset: bool = True) -> dict[str, tuple[int, int]]:
    """Bounds-check build only: {kernel file: (accesses skipped, site of the first)}.
    Raises Vq3Error (VQ3_EUNSUPPORTED) in the normal build."""
    buf = (ctypes.c_uint * (2 * len(BOUNDS_FILES)))()
    _check(lib.vq3_bounds_check(buf, len(buf), 1 if reset else 0))
    return {name: (int(buf[2 * f]), int(buf[2 * f + 1])) for f, name in enumerate(BOUNDS_FILES)}


# ---------------------------------------------------------------- layout (host)

def packed_bytes(d_in: int, d_out: int, fmt: str = "2x64") -> int:
    return int(lib.vq3_packed_bytes_fmt(FORMATS[fmt][0], d_in, d_out))


def pack_layout(canonical: np.ndarray, d_in: int, d_out: int, fmt: str = "2x64") -> np.ndarray:
    """Canonical little-endian index stream -> GPU layout (host bytes)."""
    src = np.ascontiguousarray(canonical, dtype=np.uint8)
    dst = np.empty(max(packed_bytes(d_in, d_out, fmt), 1), dtype=np.uint8)
    _check(lib.vq3_pack_layout_fmt(FORMATS[fmt][0], src.ctypes.data_as(POINTER(c_uint8)), d_in, d_out,
                                   dst.ctypes.data_as(c_void_p)))
    return dst


def unpack_layout(packed: np.ndarray, d_in: int, d_out: int, fmt: str = "2x64") -> np.ndarray:
    code, nb, vec = FORMATS[fmt]
    src = np.ascontiguousarray(packed, dtype=np.uint8)
    n = (nb * (d_out // vec) * d_in + 7) // 8
    dst = np.empty(n, dtype=np.uint8)
    _check(lib.vq3_unpack_layout_fmt(code, src.ctypes.data_as(c_void_p), d_in, d_out,
                                     dst.ctypes.data_as(POINTER(c_uint8))))
    return dst


# ---------------------------------------------------------------- weights on the device

_FORMAT_NAMES = {v[0]: k for k, v in FORMATS.items()}


def blob_bytes(d_in: int, d_out: int, fmt: str = "2x64", lr_rank: int = 0, has_signs: bool = False) -> int:
    """Size of the packed-weight blob of one matrix (0 if the descriptor is unsupported)."""
    return int(lib.vq3_blob_bytes(d_in, d_out, FORMATS[fmt][0], lr_rank, int(bool(has_signs))))


def _np_ptr(a):
    return None if a is None else a.ctypes.data_as(c_void_p)


def save_blob(m) -> bytes:
    """The packed-weight blob of one matrix (any object with d_in, d_out, block, stream, codebook,
    scales, signs and optionally fmt, lr_u, lr_v), built by vq3_blob_write."""
    fmt = getattr(m, "fmt", "2x64") or "2x64"
    stream = np.ascontiguousarray(m.stream, dtype=np.uint8)
    scales = np.ascontiguousarray(m.scales, dtype=np.float16)
    codebook = np.ascontiguousarray(m.codebook, dtype=np.float16).reshape(-1)
    signs = None if m.signs is None else np.ascontiguousarray(m.signs, dtype=np.uint32)
    lr_u, lr_v = getattr(m, "lr_u", None), getattr(m, "lr_v", None)
    rank = 0
    if lr_u is not None:
        lr_u = np.ascontiguousarray(lr_u, dtype=np.float16)
        lr_v = np.ascontiguousarray(lr_v, dtype=np.float16)
        rank = int(lr_u.shape[1])
    n = blob_bytes(m.d_in, m.d_out, fmt, rank, signs is not None)
    if n == 0:
        raise Vq3Error(-3, f"blob: unsupported matrix {m.d_in} x {m.d_out} ({fmt}, rank {rank})")
    out = np.empty(n, dtype=np.uint8)
    _check(lib.vq3_blob_write(m.d_in, m.d_out, m.block, FORMATS[fmt][0], _np_ptr(stream), _np_ptr(scales),
                              _np_ptr(codebook), _np_ptr(signs), rank, _np_ptr(lr_u), _np_ptr(lr_v),
                              _np_ptr(out), n))
    return out.tobytes()


def load_blob(data: bytes) -> dict:
    """Checks a packed-weight blob (vq3_blob_read) and returns copies of its parts as numpy arrays."""
    buf = np.frombuffer(data, dtype=np.uint8)
    view = vq3_blob_view()
    _check(lib.vq3_blob_read(_np_ptr(buf), buf.size, ctypes.byref(view)))
    base = buf.ctypes.data

    def part(ptr, count, dtype):
        off = ptr - base
        return buf[off:off + count * np.dtype(dtype).itemsize].view(dtype).copy()

    fmt = _FORMAT_NAMES[view.format]
    nbytes = packed_bytes(view.d_in, view.d_out, fmt)
    out = {"d_in": view.d_in, "d_out": view.d_out, "block": view.block, "fmt": fmt,
           "stream": part(view.canonical, nbytes, np.uint8), "packed": part(view.packed, nbytes, np.uint8),
           "scales": part(view.scales, view.d_out, np.float16),
           "codebook": part(view.codebook, view.codebook_bytes // 2, np.float16),
           "signs": part(view.signs, view.d_in // 32, np.uint32) if view.has_signs else None,
           "lr_u": None, "lr_v": None}
    if view.lr_rank:
        out["lr_u"] = part(view.lr_u, view.d_out * view.lr_rank, np.float16).reshape(view.d_out, view.lr_rank)
        out["lr_v"] = part(view.lr_v, view.lr_rank * view.d_in, np.float16).reshape(view.lr_rank, view.d_in)
    return out


class Linear:
    """One VQ3 matrix resident on the GPU (packed indices, codebook, scales, signs)."""

    def __init__(self, d_in, d_out, block, packed: torch.Tensor, codebook: torch.Tensor, scales: torch.Tensor,
                 signs: torch.Tensor | None = None, fmt: str = "2x64", lr_u: torch.Tensor | None = None,
                 lr_v: torch.Tensor | None = None):
        self.d_in, self.d_out, self.block, self.fmt = int(d_in), int(d_out), int(block), fmt
        self.packed, self.codebook, self.scales, self.signs = packed, codebook, scales, signs
        self.lr_u, self.lr_v = lr_u, lr_v
        rank = 0 if lr_u is None else int(lr_u.shape[1])
        self.struct = vq3_linear(self.d_in, self.d_out, self.block, _ptr(packed), _ptr(codebook), _ptr(scales),
                                 _ptr(signs), FORMATS[fmt][0], rank, _ptr(lr_u), _ptr(lr_v))

    @classmethod
    def from_canonical(cls, d_in, d_out, block, stream, codebook, scales, signs=None, device="cuda",
                       fmt: str = "2x64", lr_u=None, lr_v=None):
        packed = torch.from_numpy(pack_layout(stream, d_in, d_out, fmt)).to(device)
        cb = torch.from_numpy(np.ascontiguousarray(codebook, dtype=np.float16).reshape(-1)).to(device)
        sc = torch.from_numpy(np.ascontiguousarray(scales, dtype=np.float16)).to(device)
        sg = None
        if signs is not None:
            sg = torch.from_numpy(np.ascontiguousarray(signs, dtype=np.uint32).view(np.int32)).to(device)
        lu = lv = None
        if lr_u is not None:
            lu = torch.from_numpy(np.ascontiguousarray(lr_u, dtype=np.float16)).to(device)
            lv = torch.from_numpy(np.ascontiguousarray(lr_v, dtype=np.float16)).to(device)
        return cls(d_in, d_out, block, packed, cb, sc, sg, fmt, lu, lv)

    @classmethod
    def from_blob(cls, data: bytes, device="cuda"):
        """From a packed-weight blob (save_blob): its GPU-layout section is copied as it is."""
        b = load_blob(data)
        packed = torch.from_numpy(b["packed"]).to(device)
        cb = torch.from_numpy(b["codebook"]).to(device)
        sc = torch.from_numpy(b["scales"]).to(device)
        sg = None if b["signs"] is None else torch.from_numpy(b["signs"].view(np.int32)).to(device)
        lu = lv = None
        if b["lr_u"] is not None:
            lu = torch.from_numpy(b["lr_u"]).to(device)
            lv = torch.from_numpy(b["lr_v"]).to(device)
        return cls(b["d_in"], b["d_out"], b["block"], packed, cb, sc, sg, b["fmt"], lu, lv)

    @classmethod
    def from_matrix(cls, m, device="cuda"):
        """From any object with d_in, d_out, block, stream, codebook, scales, signs (and fmt) fields."""
        return cls.from_canonical(m.d_in, m.d_out, m.block, m.stream, m.codebook, m.scales, m.signs, device,
                                  getattr(m, "fmt", "2x64") or "2x64", getattr(m, "lr_u", None),
                                  getattr(m, "lr_v", None))


class MLP:
    """One SwiGLU block: gate and up share the input rotation; down has its own."""

    def __init__(self, gate: Linear, up: Linear, down: Linear):
        self.gate, self.up, self.down = gate, up, down
        self.struct = vq3_mlp_layer(gate.struct, up.struct, down.struct)

    @classmethod
    def from_block(cls, blk, device="cuda"):
        gate = Linear.from_matrix(blk.gate, device)
        if blk.up.signs is not None and blk.gate.signs is not None and np.array_equal(blk.up.signs, blk.gate.signs):
            up = Linear.from_canonical(blk.up.d_in, blk.up.d_out, blk.up.block, blk.up.stream, blk.up.codebook,
                                       blk.up.scales, None, device, getattr(blk.up, "fmt", "2x64") or "2x64")
            up.signs = gate.signs
            up.struct.signs = gate.struct.signs
        else:
            up = Linear.from_matrix(blk.up, device)
        down = Linear.from_matrix(blk.down, device)
        return cls(gate, up, down)

    @property
    def hidden(self) -> int:
        return self.gate.d_in


# ---------------------------------------------------------------- workspaces

def linear_workspace_bytes(rows: int, lin: Linear) -> int:
    return int(lib.vq3_linear_workspace_bytes(rows, ctypes.byref(lin.struct)))


def mlp_workspace_bytes(rows: int, layer: MLP) -> int:
    return int(lib.vq3_mlp_workspace_bytes(rows, ctypes.byref(layer.struct)))


def mlp_host_workspace_bytes(rows: int, layer: MLP) -> int:
    return int(lib.vq3_mlp_host_workspace_bytes(rows, ctypes.byref(layer.struct)))


def workspace(nbytes: int, device="cuda", stream=None) -> torch.Tensor:
    """A device buffer of nbytes, zero-filled by the library (counters start at zero)."""
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    _check(lib.vq3_workspace_init(ws.data_ptr(), ws.numel(), _stream(stream)))
    return ws


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    """0 unless a kernel's bounded wait ran out while using this workspace."""
    v = c_int(0)
    _check(lib.vq3_workspace_status(ws.data_ptr(), ctypes.byref(v), _stream(stream)))
    return int(v.value)


# ---------------------------------------------------------------- operations

def fwht_rotate(x: torch.Tensor, block: int, signs: torch.Tensor | None = None, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    rows, n = x.shape
    if out is None:
        out = torch.empty_like(x)
    _check(lib.fwht_rotate(x.data_ptr(), rows, n, block, _ptr(signs), out.data_ptr(), _stream(stream)))
    return out


def linear_forward(x: torch.Tensor, lin: Linear, out=None, ws=None, stream=None) -> torch.Tensor:
    rows = x.shape[0]
    if out is None:
        out = torch.empty((rows, lin.d_out), dtype=torch.float16, device=x.device)
    if ws is None:
        ws = workspace(linear_workspace_bytes(rows, lin), x.device, stream)
    _check(lib.vq3_linear_forward(x.data_ptr(), rows, ctypes.byref(lin.struct), out.data_ptr(), ws.data_ptr(),
                                  ws.numel(), _stream(stream)))
    return out


def mlp_forward(x: torch.Tensor, layer: MLP, out=None, ws=None, stream=None) -> torch.Tensor:
    rows = x.shape[0]
    if out is None:
        out = torch.empty((rows, layer.down.d_out), dtype=torch.float16, device=x.device)
    if ws is None:
        ws = workspace(mlp_workspace_bytes(rows, layer), x.device, stream)
    _check(lib.vq3_mlp_forward(x.data_ptr(), rows, ctypes.byref(layer.struct), out.data_ptr(), ws.data_ptr(),
                               ws.numel(), _stream(stream)))
    return out


def mlp_forward_noalloc(x: torch.Tensor, layer: MLP, out=None, stream=None) -> torch.Tensor:
    """The MLP block with its scratch in the library's fixed device array (no workspace)."""
    rows = x.shape[0]
    if out is None:
        out = torch.empty((rows, layer.down.d_out), dtype=torch.float16, device=x.device)
    _check(lib.vq3_mlp_forward_noalloc(x.data_ptr(), rows, ctypes.byref(layer.struct), out.data_ptr(),
                                       _stream(stream)))
    return out


def noalloc_status(stream=None) -> int:
    """Status word of the fixed array: 0, or 3 when a wait in the last no-alloc call gave up."""
    v = c_int(0)
    _check(lib.vq3_noalloc_status(ctypes.byref(v), _stream(stream)))
    return int(v.value)


def mlp_kernel_launches(rows: int, layer: MLP) -> int:
    return int(lib.vq3_mlp_kernel_launches(rows, ctypes.byref(layer.struct)))


def linear_kernel_launches(rows: int, lin: Linear) -> int:
    return int(lib.vq3_linear_kernel_launches(rows, ctypes.byref(lin.struct)))


def mlp_forward_host(x: np.ndarray, layer: MLP, ws: torch.Tensor, out: np.ndarray | None = None,
                     stream=None) -> np.ndarray:
    """Host buffers in and out (the library copies through the workspace and waits)."""
    x = np.ascontiguousarray(x, dtype=np.float16)
    rows = x.shape[0]
    if out is None:
        out = np.empty((rows, layer.down.d_out), dtype=np.float16)
    _check(lib.vq3_mlp_forward_host(x.ctypes.data_as(c_void_p), rows, ctypes.byref(layer.struct),
                                    out.ctypes.data_as(c_void_p), ws.data_ptr(), ws.numel(), _stream(stream)))
    return out


def residual_rmsnorm(resid: torch.Tensor, delta: torch.Tensor | None, eps: float = 1e-6, normed=None,
                     stream=None) -> torch.Tensor:
    rows, n = resid.shape
    if normed is None:
        normed = torch.empty_like(resid)
    _check(lib.vq3_residual_rmsnorm(resid.data_ptr(), _ptr(delta), rows, n, eps, normed.data_ptr(), _stream(stream)))
    return normed


def dequant_dense(lin: Linear, apply_scale: bool, stream=None) -> torch.Tensor:
    w = torch.empty((lin.d_out, lin.d_in), dtype=torch.float16, device=lin.packed.device)
    _check(lib.vq3_dequant_dense(ctypes.byref(lin.struct), 1 if apply_scale else 0, w.data_ptr(), _stream(stream)))
    return w


# ---------------------------------------------------------------- gated delta rule

def delta_rule_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, alpha: torch.Tensor,
                       state: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """Gated delta-rule token mixer over blocks of 8 tokens; `state` [H, d_k, d_v] FP32 is updated in place."""
    tokens, heads, d_k = q.shape
    d_v = v.shape[2]
    if out is None:
        out = torch.empty((tokens, heads, d_v), dtype=torch.float16, device=q.device)
    _check(lib.vq3_delta_rule_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), alpha.data_ptr(),
                                      tokens, heads, d_k, d_v, state.data_ptr(), out.data_ptr(), _stream(stream)))
    return out


def mlp_forward_residual(r_in: torch.Tensor, delta: torch.Tensor | None, layer: MLP, r_out: torch.Tensor,
                         out: torch.Tensor, eps: float = 1e-6, ws=None, stream=None) -> torch.Tensor:
    """One pre-norm residual layer: r_out = fp16(r_in + delta); out = MLP(RMSNorm(r_out))."""
    rows = r_in.shape[0]
    if ws is None:
        ws = workspace(mlp_workspace_bytes(rows, layer), r_in.device, stream)
    _check(lib.vq3_mlp_forward_residual(r_in.data_ptr(), _ptr(delta), rows, ctypes.byref(layer.struct), eps,
                                        r_out.data_ptr(), out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
    return out


def mlp_prenorm_step(r: torch.Tensor, layer: MLP, out: torch.Tensor, r_next: torch.Tensor,
                     ss: torch.Tensor | None = None, ss_next: torch.Tensor | None = None, eps: float = 1e-6,
                     ws=None, stream=None) -> torch.Tensor:
    """One pre-norm MLP sublayer: out = MLP(RMSNorm(r)), r_next = fp16(r + out); ss / ss_next are the
    rows' FP32 sums of squares per 16 columns ([rows][d / 16]) of r and r_next."""
    rows = r.shape[0]
    if ws is None:
        ws = workspace(mlp_workspace_bytes(rows, layer), r.device, stream)
    _check(lib.vq3_mlp_prenorm_step(r.data_ptr(), _ptr(ss), rows, ctypes.byref(layer.struct), eps, out.data_ptr(),
                                    r_next.data_ptr(), _ptr(ss_next), ws.data_ptr(), ws.numel(), _stream(stream)))
    return r_next


# ---------------------------------------------------------------- attention and its paged cache

class PagedPlan(NamedTuple):
    """What paged_plan writes beside the table (device tensors); `status` is 0 or a sum of VQ3_PLAN_* bits."""
    q_start: torch.Tensor     # int32 [requests + 1]
    kv_len: torch.Tensor      # int32 [requests]
    slots: torch.Tensor       # int64 [max_tokens]
    positions: torch.Tensor   # int32 [max_tokens]
    ring_state: torch.Tensor  # int32 {head, count} after the step
    status: torch.Tensor      # int32 [1]


def _want(ok: bool, msg: str) -> None:
    if not ok:
        raise Vq3Error(-1, msg)


# The calls below take a few microseconds on the GPU in a decode step: what Python does per call is kept short.
# `stream`: where a call runs, the current stream by default. The caller orders it behind the inputs' writers and the
# outputs' readers behind it. Making it current costs some microseconds: done only where a call makes buffers.
_INT, _LONG, _FLOAT = torch.int32, torch.int64, torch.float32
_empty = torch.empty


def _ints_ok(index: int, t: torch.Tensor) -> bool:
    return t.dtype is _INT and t.is_contiguous() and t.get_device() == index


def _elsewhere(index: int, stream) -> bool:
    """Whether a call that makes buffers has to run in _at, with another device or stream current."""
    return index < 0 or stream is not None or index != torch._C._cuda_getDevice()


def _at(index: int, stream):
    """Context in which such a call runs: CUDA device `index`, the tensors', is current (what the library answers about
    sizes is about it), and so is the caller's stream, if there is one: the buffers come from the pool of the stream
    that writes them. (A block that was just freed on another stream may still be read or written by what is queued
    there.)"""
    if index < 0:
        raise Vq3Error(-1, "tensors must be on a CUDA device")
    if stream is None:
        return torch.cuda.device(index)
    if stream.device_index != index:
        raise Vq3Error(-1, f"stream of CUDA device {stream.device_index}, tensors on {index}")
    return torch.cuda.stream(stream)


def _launch(index: int, stream, call, *args) -> None:
    """call(*args, stream) with CUDA device `index` current; the stream is the caller's or the device's current one."""
    if index >= 0 and index == torch._C._cuda_getDevice() and (stream is None or stream.device_index == index):
        rc = call(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    else:
        with _at(index, stream):
            rc = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != VQ3_OK:
        raise Vq3Error(rc, lib.vq3_last_error().decode())


def _handed_out(index: int, stream, *tensors) -> None:
    """Tensors made on a stream of the caller's and returned: their memory is not given out again on that stream
    before what the current one, on which the caller goes on, does with them."""
    if stream is not None:
        here = torch.cuda.current_stream(index)
        if here != stream:
            for t in tensors:
                t.record_stream(here)


def paged_plan(cached: torch.Tensor, fresh: torch.Tensor, table: torch.Tensor, ring: torch.Tensor,
               ring_state: torch.Tensor, page_size: int, max_tokens: int, out: PagedPlan | None = None,
               stream=None) -> PagedPlan:
    """Block tables and slot maps of a serving step (vq3_paged_plan): `cached` and `fresh` [requests] int32 lengths,
    `table` [requests, max_pages] int32 gets the new pages in place, taken from the ring of free pages. `out`: a
    plan of the same sizes to write into (its ring_state must not be the one passed in)."""
    index = table.get_device()
    _want(table.dim() == 2, "table must be [requests, max_pages]")
    requests, max_pages = table.shape
    if not (_ints_ok(index, table) and _ints_ok(index, cached) and _ints_ok(index, fresh) and _ints_ok(index, ring)
            and _ints_ok(index, ring_state) and cached.numel() == requests and fresh.numel() == requests
            and ring_state.numel() == 2):
        raise Vq3Error(-1, "table, cached, fresh, ring and ring_state must be contiguous int32 tensors on one device, "
                           "cached and fresh with one entry per table row, ring_state with two")
    if out is None:
        if _elsewhere(index, stream):
            with _at(index, stream):
                out = paged_plan(cached, fresh, table, ring, ring_state, page_size, max_tokens)
            _handed_out(index, stream, *out)
            return out
        device, size = table.device, max(int(max_tokens), 0)
        out = PagedPlan(_empty(requests + 1, dtype=_INT, device=device), _empty(requests, dtype=_INT, device=device),
                        _empty(size, dtype=_LONG, device=device), _empty(size, dtype=_INT, device=device),
                        _empty(2, dtype=_INT, device=device), _empty(1, dtype=_INT, device=device))
    else:
        _want(_ints_ok(index, out.q_start) and _ints_ok(index, out.kv_len) and _ints_ok(index, out.positions) and
              _ints_ok(index, out.ring_state) and _ints_ok(index, out.status) and out.slots.dtype is _LONG and
              out.slots.is_contiguous() and out.slots.get_device() == index and
              out.q_start.numel() == requests + 1 and out.kv_len.numel() == requests and
              out.positions.numel() == max_tokens and out.slots.numel() == max_tokens and
              out.ring_state.numel() == 2 and out.status.numel() == 1, "out is a plan of other sizes")
    _launch(index, stream, lib.vq3_paged_plan, cached.data_ptr(), fresh.data_ptr(), requests, page_size,
            ring.data_ptr(), ring.numel(), ring_state.data_ptr(), table.data_ptr(), max_pages, max_tokens,
            out.q_start.data_ptr(), out.kv_len.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(),
            out.ring_state.data_ptr(), out.status.data_ptr())
    return out


def _kv_cache(k_pages: torch.Tensor, v_pages: torch.Tensor) -> vq3_kv_cache:
    shape, (kp, kt, kh, kd), (vp, vt, vh, vd) = _pair(k_pages, v_pages, 4)
    if kd != 1 or vd != 1:
        raise Vq3Error(-1, "the head_dim axis of the cache must be contiguous")
    return vq3_kv_cache(shape[2], shape[3], shape[1], shape[0], k_pages.data_ptr(), v_pages.data_ptr(), kp, kt, kh, vp,
                        vt, vh)


def _kv_rows(k: torch.Tensor, v: torch.Tensor) -> vq3_kv_rows:
    shape, (kt, kh, kd), (vt, vh, vd) = _pair(k, v, 3)
    if kd != 1 or vd != 1:
        raise Vq3Error(-1, "the head_dim axis of k and v must be contiguous")
    return vq3_kv_rows(shape[1], shape[2], shape[0], k.data_ptr(), v.data_ptr(), kt, kh, vt, vh)


def _pair(k: torch.Tensor, v: torch.Tensor, dim: int):
    """Shape and strides of keys and values, which are alike."""
    shape = k.shape
    if len(shape) != dim or v.shape != shape or k.dtype is not v.dtype or k.dtype not in TYPES or \
            k.get_device() != v.get_device():
        raise Vq3Error(-1, "keys and values must be FP16 or BF16 tensors alike: rows [tokens, kv_heads, head_dim], "
                           "pages [n_pages, page_size, kv_heads, head_dim]")
    return shape, k.stride(), v.stride()


def kv_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
              stream=None) -> None:
    """Writes rows k, v [tokens, kv_heads, head_dim] into the paged cache [n_pages, page_size, kv_heads, head_dim] (any
    strides) at `slots` [>= tokens] int64 (vq3_kv_append); negative slots are skipped."""
    cache, rows = _kv_cache(k_pages, v_pages), _kv_rows(k, v)
    index = k.get_device()
    if k.dtype is not k_pages.dtype or k_pages.get_device() != index:
        raise Vq3Error(-1, "rows and cache must have one type and device")
    if slots.dtype is not _LONG or not slots.is_contiguous() or slots.numel() < rows.tokens or \
            slots.get_device() != index:
        raise Vq3Error(-1, "slots must be a contiguous int64 tensor with an entry per row")
    _launch(index, stream, lib.vq3_kv_append, ctypes.byref(rows), slots.data_ptr(), ctypes.byref(cache))


def kv_append_rotary(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                     slots: torch.Tensor, freq: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                     interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """kv_append with the position rotation on the way (vq3_kv_append_rotary): the first 2 * freq.numel() entries of
    every head of q [tokens, heads, head_dim] and k are turned by `positions` [>= tokens] int32 times `freq` FP32
    (radians a position), entries i and i + freq.numel() as a pair, or 2 i and 2 i + 1 if interleaved. Turned queries
    go to `q_out` (q itself: in place) and are returned, keys and values to `slots` of the cache. Rows with a negative
    position (plan.positions behind the last) are left as they were. q None: keys and values only."""
    cache, rows = _kv_cache(k_pages, v_pages), _kv_rows(k, v)
    index, dtype = k.get_device(), k.dtype
    if dtype is not k_pages.dtype or k_pages.get_device() != index:
        raise Vq3Error(-1, "rows and cache must have one type and device")
    if slots.dtype is not _LONG or not slots.is_contiguous() or slots.numel() < rows.tokens or \
            slots.get_device() != index or not _ints_ok(index, positions) or positions.numel() < rows.tokens:
        raise Vq3Error(-1, "slots (int64) and positions (int32) must be contiguous with an entry per row")
    if freq.dtype is not _FLOAT or not freq.is_contiguous() or freq.get_device() != index:
        raise Vq3Error(-1, "freq must be a contiguous float32 tensor on the rows' device")
    heads = qp = op = q_token = q_head = out_token = out_head = 0
    if q is None:
        if q_out is not None:
            raise Vq3Error(-1, "q_out without q")
    else:
        shape = q.shape
        if len(shape) != 3 or shape[0] != rows.tokens or shape[2] != rows.head_dim or q.dtype is not dtype or \
                q.get_device() != index:
            raise Vq3Error(-1, f"q must be [{rows.tokens}, heads, {rows.head_dim}] of the keys' type and device")
        if q_out is None:
            if _elsewhere(index, stream):
                with _at(index, stream):
                    q_out = kv_append_rotary(q, k, v, positions, slots, freq, k_pages, v_pages, interleaved)
                _handed_out(index, stream, q_out)
                return q_out
            q_out = _empty(shape, dtype=dtype, device=q.device)
        elif q_out.shape != shape or q_out.dtype is not dtype or q_out.get_device() != index:
            raise Vq3Error(-1, "q_out must be like q")
        heads, qp, op = shape[1], q.data_ptr(), q_out.data_ptr()
        q_token, q_head, qd = q.stride()
        out_token, out_head, od = q_out.stride()
        if qd != 1 or od != 1:
            raise Vq3Error(-1, "the head_dim axis of q and q_out must be contiguous")
    rot = _pack_rotary(TYPES[dtype], heads, 2 * freq.numel(), bool(interleaved), freq.data_ptr(), positions.data_ptr(), qp,
                       op, q_token, q_head, out_token, out_head)
    _launch(index, stream, lib.vq3_kv_append_rotary, rot, ctypes.byref(rows), slots.data_ptr(), ctypes.byref(cache))
    return q_out


def attention_workspace_bytes(heads: int, kv_heads: int, head_dim: int, max_new: int = 0) -> int:
    """Workspace of paged_attention and prompt_attention on the current device; it needs no initialisation."""
    return int(lib.vq3_attention_workspace_bytes(heads, kv_heads, head_dim, max_new))


def _attention(call, q, kv, dtype, index, q_start, max_new, scale, out, lse, ws, stream, *more) -> torch.Tensor:
    shape = q.shape
    if len(shape) != 3 or q.dtype is not dtype or shape[2] != kv.head_dim or q.get_device() != index:
        raise Vq3Error(-1, f"q must be [tokens, heads, {kv.head_dim}] of the keys' type and device")
    tokens, heads, head_dim = shape
    if not _ints_ok(index, q_start) or q_start.numel() < 1:
        raise Vq3Error(-1, "q_start must be a contiguous int32 tensor [requests + 1] on q's device")
    made = out is None
    if not made and (out.shape != shape or out.dtype is not dtype or out.get_device() != index):
        raise Vq3Error(-1, "out must be like q")
    if lse is not None and (lse.shape != shape[:2] or lse.dtype is not _FLOAT or not lse.is_contiguous()
                            or lse.get_device() != index):
        raise Vq3Error(-1, "lse must be a contiguous float32 tensor [tokens, heads]")
    if (made or ws is None) and _elsewhere(index, stream):
        with _at(index, stream):
            out = _attention(call, q, kv, dtype, index, q_start, max_new, scale, out, lse, ws, None, *more)
        if made:
            _handed_out(index, stream, out)
        return out
    if made:
        out = _empty(shape, dtype=dtype, device=q.device)
    qt, qh, qd = q.stride()
    ot, oh, od = out.stride()
    if qd != 1 or od != 1:
        raise Vq3Error(-1, "the head_dim axis of q and out must be contiguous")
    own = ws is None
    if own:
        # 256 bytes at least, for the status word
        ws = _empty(max(lib.vq3_attention_workspace_bytes(heads, kv.kv_heads, head_dim, max_new), 256),
                    dtype=torch.uint8, device=q.device)
    elif ws.get_device() != index or not ws.is_contiguous():
        raise Vq3Error(-1, "ws must be a contiguous tensor on q's device")
    a = vq3_attn(TYPES[dtype], heads, tokens, q_start.numel() - 1, max_new,
                 head_dim ** -0.5 if scale is None else scale, q.data_ptr(), out.data_ptr(),
                 None if lse is None else lse.data_ptr(), q_start.data_ptr(), qt, qh, ot, oh)
    try:
        _launch(index, stream, call, ctypes.byref(a), ctypes.byref(kv), *more, ws.data_ptr(), ws.nbytes)
    except Vq3Error as e:
        if not own or e.code != VQ3_ENOSPACE:
            raise
        # max_new is too small for so large a batch: what the kernel for any batch needs
        ws = _empty(lib.vq3_attention_workspace_bytes(heads, kv.kv_heads, head_dim, 0), dtype=torch.uint8,
                    device=q.device)
        _launch(index, stream, call, ctypes.byref(a), ctypes.byref(kv), *more, ws.data_ptr(), ws.nbytes)
    return out


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                    q_start: torch.Tensor, kv_len: torch.Tensor, max_new: int = 0, scale: float | None = None,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Causal attention of packed new tokens q [tokens, heads, head_dim] over the paged cache (vq3_paged_attention):
    `table` [requests, max_pages], `q_start` [requests + 1], `kv_len` [requests] int32 on the device, kv_len with the
    new tokens counted in. max_new: most new tokens of a request, 0 if unknown. It only picks the kernel, but say it
    where it is known: single tokens take up to twice as long with 0. scale: 1 / sqrt(head_dim) by default. `lse`
    [tokens, heads] FP32 is filled if given."""
    cache = _kv_cache(k_pages, v_pages)
    index = k_pages.get_device()
    if not (_ints_ok(index, table) and _ints_ok(index, kv_len) and table.dim() == 2
            and table.shape[0] == kv_len.numel() == q_start.numel() - 1):
        raise Vq3Error(-1, "table [requests, max_pages] and kv_len [requests] must be contiguous int32 tensors on the "
                           "cache's device, q_start [requests + 1]")
    return _attention(lib.vq3_paged_attention, q, cache, k_pages.dtype, index, q_start, max_new, scale, out, lse, ws,
                      stream, table.data_ptr(), table.shape[1], kv_len.data_ptr())


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, max_new: int = 0,
                     scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention over whole packed prompts (vq3_prompt_attention): q [tokens, heads, head_dim], k and v [tokens,
    kv_heads, head_dim], request r at rows q_start[r] .. q_start[r + 1] - 1 of all three."""
    return _attention(lib.vq3_prompt_attention, q, _kv_rows(k, v), k.dtype, k.get_device(), q_start, max_new, scale, out,
                      lse, ws, stream)


# ---------------------------------------------------------------- the delta rule for packed requests

def _batch(index: int, tokens: int, slots: int, q_start, slot_in, slot_out) -> bytes:
    if not _ints_ok(index, q_start) or q_start.numel() < 1:
        raise Vq3Error(-1, "q_start must be a contiguous int32 tensor [requests + 1] on the inputs' device")
    requests = q_start.numel() - 1
    for s in (slot_in,) if slot_in is slot_out else (slot_in, slot_out):
        if s is not None and not (_ints_ok(index, s) and s.numel() == requests):
            raise Vq3Error(-1, "slot_in and slot_out must be contiguous int32 tensors [requests] on the inputs' device")
    return _pack_batch(tokens, requests, slots, q_start.data_ptr(), 0 if slot_in is None else slot_in.data_ptr(),
                       0 if slot_out is None else slot_out.data_ptr())


def delta_rule_batch(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor, alpha: torch.Tensor,
                     states: torch.Tensor, q_start: torch.Tensor, slot_in: torch.Tensor | None = None,
                     slot_out: torch.Tensor | None = None, max_new: int = 0, scale: float = 1.0,
                     out: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gated delta rule over packed requests (vq3_delta_rule_batch): q, k [tokens, qk_heads, d_k], v [tokens,
    v_heads, d_v] FP16 or BF16 (slices of one buffer, for instance), beta, alpha [tokens, v_heads] FP32, `states`
    [slots, v_heads, d_k, d_v] FP32. Request r has rows q_start[r] .. q_start[r + 1] - 1, goes on from slot
    slot_in[r] (negative, or slot_in None: from zeros) and leaves its state in slot_out[r] (negative, or None: nowhere).
    max_new: most new tokens of a request, 0 if unknown. It only picks the kernel, but say it where it is known.
    status: an int32 tensor [1] that becomes 3 if a wait inside the call gave up (its results are invalid then);
    without one delta_status tells."""
    index, dtype = v.get_device(), v.dtype
    qs, vs = q.shape, v.shape
    if dtype not in TYPES or len(qs) != 3 or k.shape != qs or len(vs) != 3 or vs[0] != qs[0] or q.dtype is not dtype or \
            k.dtype is not dtype or q.get_device() != index or k.get_device() != index:
        raise Vq3Error(-1, "q and k [tokens, qk_heads, d_k] and v [tokens, v_heads, d_v] must be FP16 or BF16 tensors of "
                           "one type and device")
    tokens, heads, d_v = vs
    qk_heads, d_k = qs[1], qs[2]
    for g in (beta, alpha):
        if g.shape != (tokens, heads) or g.dtype is not _FLOAT or g.get_device() != index or (heads > 1 and g.stride(1) != 1):
            raise Vq3Error(-1, "beta and alpha must be float32 [tokens, v_heads], the heads side by side")
    ss, st = states.shape, states.stride()
    if states.dtype is not _FLOAT or len(ss) != 4 or ss[1] != heads or ss[2] != d_k or ss[3] != d_v or \
            states.get_device() != index or (heads > 1 and st[1] != d_k * d_v) or st[2] != d_v or st[3] != 1:
        raise Vq3Error(-1, "states must be float32 [slots, v_heads, d_k, d_v], contiguous within a slot")
    if status is not None and not (_ints_ok(index, status) and status.numel() == 1):
        raise Vq3Error(-1, "status must be an int32 tensor [1] on the inputs' device")
    batch = _batch(index, tokens, ss[0], q_start, slot_in, slot_out)
    if out is None:
        if _elsewhere(index, stream):
            with _at(index, stream):
                out = delta_rule_batch(q, k, v, beta, alpha, states, q_start, slot_in, slot_out, max_new, scale, status=status)
            _handed_out(index, stream, out)
            return out
        out = _empty(vs, dtype=dtype, device=v.device)
    elif out.shape != vs or out.dtype is not dtype or out.get_device() != index:
        raise Vq3Error(-1, "out must be like v")
    (qt, qh, qd), (kt, kh, kd), (vt, vh, vd), (ot, oh, od) = q.stride(), k.stride(), v.stride(), out.stride()
    if qd != 1 or kd != 1 or vd != 1 or od != 1:
        raise Vq3Error(-1, "the last axis of q, k, v and out must be contiguous")
    d = _pack_delta(TYPES[dtype], qk_heads, heads, d_k, d_v, max_new, scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                    out.data_ptr(), beta.data_ptr(), alpha.data_ptr(), states.data_ptr(), qt, qh, kt, kh, vt, vh, ot, oh,
                    beta.stride(0), alpha.stride(0), st[0], 0 if status is None else status.data_ptr())
    _launch(index, stream, lib.vq3_delta_rule_batch, batch, d)
    return out


def delta_status(device=None, stream=None) -> int:
    """0, or 3 when a wait gave up in a delta_rule_batch call on `device` (the current one) that was given no `status`,
    since the last answer other than 0 (vq3_delta_status). Waits for the stream; ask before results are handed on."""
    device = torch.device("cuda" if device is None else device)
    v = c_int(0)
    _launch(torch.cuda.current_device() if device.index is None else device.index, stream, lib.vq3_delta_status,
            ctypes.byref(v))
    return int(v.value)


def short_conv(x: torch.Tensor, weight: torch.Tensor, states: torch.Tensor, q_start: torch.Tensor,
               slot_in: torch.Tensor | None = None, slot_out: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, silu: bool = True, unit_heads: int = 0, head_dim: int = 0,
               eps: float = 1e-6, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The short causal convolution over packed requests (vq3_short_conv): x [tokens, channels], weight [channels,
    width], bias [channels] or None, `states` [slots, width - 1, channels] (the last inputs), all of one type; slots as
    in delta_rule_batch. The first unit_heads heads of head_dim channels come out with unit length."""
    index, dtype, xs = x.get_device(), x.dtype, x.shape
    ws, ss = weight.shape, states.shape
    if dtype not in TYPES or len(xs) != 2 or len(ws) != 2 or ws[0] != xs[1] or weight.dtype is not dtype \
            or not weight.is_contiguous() or weight.get_device() != index:
        raise Vq3Error(-1, "x [tokens, channels] and weight [channels, width] must be FP16 or BF16 tensors of one type and "
                           "device, weight contiguous")
    tokens, channels = xs
    width = ws[1]
    if bias is not None and (bias.shape != (channels,) or bias.dtype is not dtype or not bias.is_contiguous()
                             or bias.get_device() != index):
        raise Vq3Error(-1, "bias must be a contiguous tensor [channels] of x's type and device")
    st = states.stride()
    if len(ss) != 3 or ss[1] != width - 1 or ss[2] != channels or states.dtype is not dtype or \
            states.get_device() != index or st[2] != 1:
        raise Vq3Error(-1, "states must be [slots, width - 1, channels] of x's type and device")
    batch = _batch(index, tokens, ss[0], q_start, slot_in, slot_out)
    if out is None:
        if _elsewhere(index, stream):
            with _at(index, stream):
                out = short_conv(x, weight, states, q_start, slot_in, slot_out, bias, silu, unit_heads, head_dim, eps)
            _handed_out(index, stream, out)
            return out
        out = _empty(xs, dtype=dtype, device=x.device)
    elif out.shape != xs or out.dtype is not dtype or out.get_device() != index:
        raise Vq3Error(-1, "out must be like x")
    xt, xc = x.stride()
    ot, oc = out.stride()
    if xc != 1 or oc != 1:
        raise Vq3Error(-1, "the channels of x and out must be contiguous")
    c = _pack_conv(TYPES[dtype], channels, width, bool(silu), unit_heads, head_dim, eps, x.data_ptr(), weight.data_ptr(),
                   0 if bias is None else bias.data_ptr(), states.data_ptr(), out.data_ptr(), xt, ot, st[0], st[1])
    _launch(index, stream, lib.vq3_short_conv, batch, c)
    return out
