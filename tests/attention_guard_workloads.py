"""Attention calls whose starts in device memory are none that the header allows: every one has to stay inside its
buffers. Run in a process of its own by the guard test, with the library that VQ3_LIB selects, as
tests/attention_workloads.py.

    VQ3_LIB=.../libvq3_bc.so python -m tests.attention_guard_workloads out.npz
"""

import sys

import numpy as np
import torch

DEV = "cuda"
GUARD = 64  # rows in front of out and lse and behind them
FILL = 7.0


def guarded(T, heads, dim, dtype):
    """out and lse with guard rows on both sides, and a check that those are as they were."""
    out = torch.full((T + 2 * GUARD, heads, dim), FILL, dtype=dtype, device=DEV)
    lse = torch.full((T + 2 * GUARD, heads), FILL, device=DEV)

    def check():
        for t in (out, lse):
            assert (t[:GUARD] == FILL).all() and (t[GUARD + T :] == FILL).all(), "rows outside were written"

    return out[GUARD : GUARD + T], lse[GUARD : GUARD + T], check


# starts and the ascending ones that mean the same once they are cut to the rows of the batch (8); None: overlapping
STARTS = [([0, 100, 8], [0, 8, 8]), ([-5, 4, 8], [0, 4, 8]), ([0, 8, 4], [0, 8, 8]), ([8, 8, 8], [8, 8, 8]),
          ([9, 20, 30], [8, 8, 8]), ([-9, -3, 0], [0, 0, 0]), ([5, -1, 8], None), ([2**31 - 1, -(2**31), 3], [0, 0, 3]),
          ([-(2**31), 2**31 - 1, 4], [0, 8, 8])]


def overlapping(unit, tile, unit_cost, requests=8192, kv=1 << 20):
    """Starts 0, T, 0, T, ... whose requests' costs add up to a little more than 2^32, nothing behind them but one more
    such request at the very end. Returns T, the starts and kv."""
    def cost(T):
        return sum(-(-(kv - T + min((j + 1) * unit, T)) // tile) + unit_cost for j in range(-(-T // unit)))

    T = unit
    while cost(T) * 3000 <= 1 << 32:
        T += unit
    m = (1 << 32) // cost(T) + 1
    starts = np.zeros(requests + 1, dtype=np.int64)
    starts[1 : 2 * m : 2] = T
    starts[requests] = T
    return T, starts, kv


def run(vq3) -> dict[str, np.ndarray]:
    from tests.test_gpu_attention import Batch, ints, normal
    got: dict[str, np.ndarray] = {}
    for dim in (64, 128, 256):
        b = Batch(60, [(64, 4), (64, 4)], 4, 1, dim, 16, "f16", behind=0)
        g = torch.Generator().manual_seed(61)
        k, v = normal(g, (8, 1, dim), "f16"), normal(g, (8, 1, dim), "f16")
        for max_new in (1, 0):
            def call(starts, paged):
                out, lse, check = guarded(8, 4, dim, b.q.dtype)
                ws = torch.empty(vq3.attention_workspace_bytes(4, 1, dim, max_new), dtype=torch.uint8, device=DEV)
                if paged:
                    vq3.paged_attention(b.q, b.k, b.v, b.table, ints(starts), b.kv_len, max_new=max_new, out=out,
                                        lse=lse, ws=ws)
                else:
                    vq3.prompt_attention(b.q, k, v, ints(starts), max_new=max_new, out=out, lse=lse, ws=ws)
                assert vq3.workspace_status(ws) == 0
                check()
                return out, lse

            for i, (starts, same) in enumerate(STARTS):
                for paged in (True, False):
                    out, lse = call(starts, paged)
                    assert torch.isfinite(out).all()
                    if same is not None:
                        ref, ref_lse = call(same, paged)
                        assert torch.equal(out, ref) and torch.equal(lse, ref_lse), (starts, dim, max_new, paged)
                        got[f"starts_{dim}_{max_new}_{i}_{paged}"] = out.float().cpu().numpy()
    # sums past 2^32: no answer is defined (every page is outside the cache and reads as zeros)
    for dim, max_new, unit, tile, cost in ((128, 1, 8, 64, 1), (128, 0, 256, 128, 1), (256, 0, 128, 128, 3)):
        T, starts, kv = overlapping(unit, tile, cost)
        R = len(starts) - 1
        q = torch.ones(T, 1, dim, dtype=torch.float16, device=DEV)
        pages = torch.ones(2, 256, 1, dim, dtype=torch.float16, device=DEV)
        table = torch.full((R, kv // 256), -1, dtype=torch.int32, device=DEV)
        out, lse, check = guarded(T, 1, dim, q.dtype)
        ws = torch.empty(vq3.attention_workspace_bytes(1, 1, dim, max_new), dtype=torch.uint8, device=DEV)
        vq3.paged_attention(q, pages, pages, table, ints(starts), torch.full((R,), kv, dtype=torch.int32, device=DEV),
                            max_new=max_new, out=out, lse=lse, ws=ws)
        assert vq3.workspace_status(ws) == 0
        check()
    return got


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
