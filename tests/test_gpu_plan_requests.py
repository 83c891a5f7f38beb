"""The page plan at the numbers of requests around which its shared memory passes what a launch gets without
opting in: in a process of its own, so that no larger plan has opted in before, and from two host threads."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention as A  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# 8 bytes a request and one more, beside 128 bytes: 48 KB are full at 6,127 requests
BORDER = (6126, 6127, 6128, 6143, 6144)


def batch(R, seed=5):
    rng = np.random.default_rng(seed + R)
    cached, fresh = rng.integers(0, 64, R), rng.integers(0, 3, R)
    held = -(-cached // 16)
    ids = rng.permutation(int(held.sum()) + 3 * R)
    table, at = np.full((R, 5), -1), 0
    for r in range(R):
        table[r, : held[r]] = ids[at : at + held[r]]
        at += held[r]
    return cached, fresh, table, ids[at:], int(fresh.sum()) + 3


def plan(vq3, b):
    cached, fresh, table, ring, T = b
    i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    t = i(table)
    return t, vq3.paged_plan(i(cached), i(fresh), t, i(ring), i([7, len(ring)]), 16, T)


def check(b, t, p):
    cached, fresh, table, ring, T = b
    want = A.plan(cached.tolist(), fresh.tolist(), table, ring.tolist(), 7, len(ring), 16, T)
    assert want[0] == 0 and p.status.item() == 0
    assert np.array_equal(t.cpu().numpy(), want[1])
    for got, ref in zip((p.q_start, p.kv_len, p.slots, p.positions), want[2:6]):
        assert got.tolist() == list(ref)


@pytest.mark.parametrize("requests", BORDER)
def test_plan_without_a_larger_one_before(requests):
    r = subprocess.run([sys.executable, "-m", "tests.test_gpu_plan_requests", str(requests)], cwd=ROOT,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]


def test_plans_of_two_threads():
    from bit_vector_lut_gb300 import vq3
    sizes = (6500, 8192)
    batches = [batch(R) for R in sizes]
    failed = []

    def work(b):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(150):
                    t, p = plan(vq3, b)
                check(b, t, p)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(b,)) for b in batches]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


if __name__ == "__main__":
    from bit_vector_lut_gb300 import vq3 as lib
    b = batch(int(sys.argv[1]))
    check(b, *plan(lib, b))
