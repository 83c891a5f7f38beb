"""One call of every kernel of the delta rule for packed requests, the short convolution and the rotated append on
fixed seeded inputs, outputs saved (npz), with the library that VQ3_LIB selects; run twice by the bounds-check test, as
tests/attention_workloads.py.

    VQ3_LIB=.../libvq3_bc.so python -m tests.mixers_workloads out.npz
"""

import sys

import numpy as np
import torch

NEW = [70, 0, 1, 3, 200, 64, 9]
ODD_IN, ODD_OUT = [0, -5, 1 << 20], [1 << 30, -1, 1]


def odd_starts(hint):
    """Starts outside the batch: requests of 4, 0 and 51 tokens. Slots 0 and 1 are used, the others do not exist."""
    from tests.test_gpu_delta_batch import Case
    c = Case(42, [4, 0, 51], 1, 2, 128, 64, "f16", behind=0, spare=0)
    c.slot_in, c.slot_out = ODD_IN, ODD_OUT
    c.states[0] = 0.5
    c.q_start = torch.tensor([-9, 4, 4, 1 << 30], dtype=torch.int32, device="cuda")
    return c


def run(vq3) -> dict[str, np.ndarray]:
    from tests.test_gpu_conv_rotary import Conv, Rotary
    from tests.test_gpu_delta_batch import Case
    out: dict[str, np.ndarray] = {}

    def keep(name, t):
        out[name] = t.detach().float().cpu().numpy().copy()

    for dk in (64, 128, 256):
        for dv in (32, 144):
            for dtype in ("f16", "bf16"):
                c = Case(41, NEW, 1, 2, dk, dv, dtype, before=3)
                for hint in (0, 1, 8):
                    o, s = c.run(vq3, hint)
                    keep(f"delta_{dk}_{dv}_{dtype}_{hint}", o)
                    keep(f"states_{dk}_{dv}_{dtype}_{hint}", s)
    for hint in (0, 1, 8):
        o, t = odd_starts(hint).run(vq3, hint, ODD_IN, ODD_OUT)
        keep(f"odd_{hint}", o)
        keep(f"odd_states_{hint}", t)
    for width in (2, 3, 4):
        for dtype in ("f16", "bf16"):
            c = Conv(43, NEW, 192, width, dtype, bias=True, before=3)
            o, s = c.run(vq3, unit_heads=2, head_dim=64)
            keep(f"conv_{width}_{dtype}", o)
            keep(f"conv_states_{width}_{dtype}", s)
    for dtype in ("f16", "bf16"):
        for T in (5, 4000):
            r = Rotary(44, [i * 3 if i % 7 else -1 for i in range(T)], 6, 2, 128, 64, 16, dtype)
            for i, t in enumerate((r.run(vq3), *r.pages)):
                keep(f"rotary_{dtype}_{T}_{i}", t)
    return out


def main(path: str) -> None:
    from bit_vector_lut_gb300 import vq3
    out = run(vq3)
    try:
        for name, (count, site) in vq3.bounds_check(reset=True).items():
            out[f"bounds_{name}"] = np.array([count, site], dtype=np.int64)
    except vq3.Vq3Error:
        pass  # the normal build records nothing
    out["version"] = np.array(vq3.version())
    np.savez(path, **out)


if __name__ == "__main__":
    main(sys.argv[1])
