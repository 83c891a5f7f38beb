"""Convolution and rotated append with starts, slots and positions outside their buffers, on fixed seeded inputs whose
buffers lie between guard rows; outputs saved (npz) with the library that VQ3_LIB selects, as tests/mixers_workloads.py.

    VQ3_LIB=.../libvq3_bc.so python -m tests.mixers_guard_workloads out.npz
"""

import sys

import numpy as np
import torch

GUARD = 6  # rows and slots on either side
FAR = 1 << 30
# starts of a batch of 90 rows, and the ascending ones that mean the same once they are brought into it; None: which of
# the requests are done is not said
STARTS = [
    ([0, 40, 41, 90], [0, 40, 41, 90]),
    ([-9, 4, 4, FAR], [0, 4, 4, 90]),
    ([-FAR, -1, 50, 91], [0, 0, 50, 90]),
    ([FAR, FAR, FAR, FAR], [90, 90, 90, 90]),
    ([60, 10, 80, 30], None),
    ([90, 0, 90, 0], None),
    ([FAR, 3, -FAR, 70], None),
]
SLOTS = [([1, 0, 3], [4, 2, 5]), ([-1, 6, FAR], [0, -FAR, 1])]  # of a pool of 6


class Conv:
    """90 rows of 72 channels and 6 slots between guards; the inputs' guards are NaN."""

    def __init__(self, width=4, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.full((90 + 2 * GUARD, 72), float("nan"), dtype=torch.float16, device="cuda")
        self.x[GUARD:-GUARD] = torch.randn(90, 72, generator=g).half().cuda()
        self.w = torch.randn(72, width, generator=g).half().cuda()
        self.pool = torch.randn(6 + 2 * GUARD, width - 1, 72, generator=g).half().cuda()

    def run(self, vq3, starts, slot_in, slot_out):
        """(out, pool) with their guards; out starts at 7."""
        ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        out, pool = torch.full_like(self.x, 7.0), self.pool.clone()
        vq3.short_conv(self.x[GUARD:-GUARD], self.w, pool[GUARD:-GUARD], ints(starts), ints(slot_in), ints(slot_out),
                       out=out[GUARD:-GUARD], unit_heads=2, head_dim=16)
        torch.cuda.synchronize()
        return out, pool


class Rotary:
    """Rows whose slots and positions leave the cache: kept where both are inside."""

    positions = [0, 5, -1, 2**31 - 1, -(2**31), 7, 8, 9]
    slots = [0, -1, 3, 31, 5, 32, 1 << 62, -(1 << 62)]  # of 2 pages of 16

    def __init__(self, seed=2):
        g = torch.Generator().manual_seed(seed)
        self.q, self.k, self.v = (torch.randn(8, h, 64, generator=g).half().cuda() for h in (3, 2, 2))
        self.freq = torch.tensor([1e4 ** (-i / 16) for i in range(16)], dtype=torch.float32, device="cuda")

    def run(self, vq3):
        """(queries, key pages, value pages), the pages between guard pages; everything starts at 5."""
        q = torch.full_like(self.q, 5.0)
        pools = [torch.full((2 + 2 * GUARD, 16, 2, 64), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)]
        vq3.kv_append_rotary(self.q, self.k, self.v, torch.tensor(self.positions, dtype=torch.int32, device="cuda"),
                             torch.tensor(self.slots, device="cuda"), self.freq, *(p[GUARD:-GUARD] for p in pools), q_out=q)
        torch.cuda.synchronize()
        return q, *pools


def run(vq3) -> dict[str, np.ndarray]:
    out = {}
    for i, (starts, _) in enumerate(STARTS):
        for j, slots in enumerate(SLOTS):
            for width in (2, 4):
                for name, t in zip(("out", "pool"), Conv(width).run(vq3, starts, *slots)):
                    out[f"conv_{i}_{j}_{width}_{name}"] = t.cpu().numpy()
    for name, t in zip("qkv", Rotary().run(vq3)):
        out[f"rotary_{name}"] = t.cpu().numpy()
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
