"""One call of every kernel path of the attention token mixer on fixed seeded inputs, outputs saved (npz), with
the library that VQ3_LIB selects; run twice by the bounds-check test, as tests/bounds_workloads.py.

    VQ3_LIB=.../libvq3_bc.so python -m tests.attention_workloads out.npz
"""

import sys

import numpy as np
import torch

DEV = "cuda"


def run(vq3) -> dict[str, np.ndarray]:
    from tests.test_gpu_attention import Batch, ints, normal
    out: dict[str, np.ndarray] = {}

    def keep(name, t):
        torch.cuda.synchronize()
        out[name] = t.detach().float().cpu().numpy().copy()

    # row kernel and tensor-core kernels, whole units and split ones, few and many requests
    for dim, heads, kv in ((64, 8, 2), (128, 6, 2), (256, 6, 1)):
        for new in (1, 3, 70):
            reqs = [(3000 + 7 * dim, new), (5, min(new, 5)), (0, 1), (130, new)]
            b = Batch(31, reqs, heads, kv, dim, 16 if new == 3 else 64, "f16")
            o, lse = b.run(vq3)
            keep(f"paged_{dim}_{new}", o[: b.starts[-1]])
            keep(f"paged_{dim}_{new}_lse", lse[: b.starts[-1]])
        b = Batch(32, [(40 + i % 50, 1 + i % 3) for i in range(150)], heads, kv, dim, 16, "bf16")
        keep(f"many_{dim}", b.run(vq3)[0][: b.starts[-1]])
        g = torch.Generator().manual_seed(33)
        lens = [1, 300, 0, 65]
        starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
        q, k, v = (normal(g, (sum(lens), h, dim), "f16") for h in (heads, kv, kv))
        keep(f"prompt_{dim}", vq3.prompt_attention(q, k, v, ints(starts), max_new=300))
    # plan and append
    table = ints([[3, 9, -1, -1], [-1] * 4, [5, -1, -1, -1]])
    p = vq3.paged_plan(ints([20, 0, 16]), ints([30, 40, 1]), table, ints([1, 2, 4, 6, 7, 8, 0]), ints([5, 7]), 16, 80)
    for name, t in p._asdict().items():
        keep("plan_" + name, t)
    keep("plan_table", table)
    g = torch.Generator().manual_seed(34)
    pages = [torch.zeros(10, 16, 2, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    vq3.kv_append(normal(g, (80, 2, 128), "f16"), normal(g, (80, 2, 128), "f16"), p.slots, *pages)
    keep("append_k", pages[0])
    keep("append_v", pages[1])
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
