"""A batch too large for the kernel that a small max_new picks."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_attention import check, ints, normal, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_small_max_new_and_a_long_prompt(vq3):  # noqa: F811
    # one request of 65,536 new tokens, a table of 2^20 keys: blocks of 8 rows are too many for the row kernel's count
    T, H, Hkv, D, page = 1 << 16, 32, 8, 64, 256
    g = torch.Generator().manual_seed(50)
    q, k, v = (normal(g, (T, h, D), "f16") for h in (H, Hkv, Hkv))
    k_pages, v_pages = (x.view(T // page, page, Hkv, D) for x in (k, v))
    table = torch.full((1, 4096), -1, dtype=torch.int32, device=DEV)
    table[0, : T // page] = torch.arange(T // page, device=DEV)
    args = (q, k_pages, v_pages, table, ints([0, T]), ints([T]))
    want = vq3.paged_attention(*args, max_new=T)
    assert torch.equal(vq3.paged_attention(*args, max_new=1), want)
    need = vq3.attention_workspace_bytes(H, Hkv, D, 0)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert torch.equal(vq3.paged_attention(*args, max_new=1, ws=ws), want) and vq3.workspace_status(ws) == 0
    with pytest.raises(vq3.Vq3Error, match="VQ3_ENOSPACE"):
        vq3.paged_attention(*args, max_new=1, ws=ws[: vq3.attention_workspace_bytes(H, Hkv, D, 1)])
    pick = [0, 1, 777, 40000, T - 1]
    check(want[pick], None, q[pick], [k], [v], [0, len(pick)], [[i + 1 for i in pick]], D**-0.5, "f16")
