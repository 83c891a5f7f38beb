"""SiLU of the convolution where exp(-y) comes near the end of FP32's range and the result is still a BF16 number."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_conv_rotary import HALF, TINY, Conv, f64  # noqa: E402
from tests.test_gpu_delta_batch import vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [[24], [1] * 24])  # several tokens a request, single ones
def test_silu_to_the_end_of_exp(vq3, new):  # noqa: F811
    # y = x; exp(88.5) is the last below 2^128
    c = Conv(1, new, 64, 4, "bf16", behind=0)
    c.w[:] = torch.tensor([0.0, 0.0, 0.0, 1.0])
    c.x[:] = torch.linspace(-88.5, -60.0, 24 * 64).view(24, 64).to(c.x.dtype)
    c.x[3, :8] = torch.tensor([0.0, -0.0, 88.5, 1e30, 3e38, 1e-30, -1e-30, 1.0]).to(c.x.dtype)
    c.states[:] = 0
    out, _ = c.run(vq3)
    # y is exact here; the exponential, the sum and the quotient leave 2^-23 (5 + 1.2 |y|) as in oracle/mixers.py
    y = f64(c.x)
    with np.errstate(over="ignore"):
        ref = y / (1 + np.exp(-y))
    assert (np.abs(ref[4:]) > 2.0**-126).all()
    made = np.abs(ref) * 2.0**-23 * (5 + 1.2 * np.minimum(np.abs(y), 100))
    e = np.abs(f64(out) - ref)
    bad = np.argwhere(~(e <= HALF["bf16"] * np.abs(ref) + (1 + HALF["bf16"]) * made + TINY["bf16"]))
    assert len(bad) == 0, f"{len(bad)} outputs, first {y[tuple(bad[0])]}: {f64(out)[tuple(bad[0])]} for {ref[tuple(bad[0])]}"
