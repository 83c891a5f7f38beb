"""The device's status word of delta_rule_batch calls that bring none (a wait is not run out on purpose: the word
stays 0), eager and captured."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_delta_batch import DEV, DT, Case, ints, vq3  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hint", [0, 1, 8])
def test_status_without_a_word(vq3, hint):  # noqa: F811
    c = Case(60, [130, 2, 70], 1, 2, 128, 32)
    out, states = c.run(vq3, hint)
    assert vq3.delta_status() == 0 and vq3.delta_status(DEV) == 0 and vq3.delta_status(0, torch.cuda.Stream()) == 0
    c.check(out, states)


def test_status_of_a_captured_call(vq3):  # noqa: F811
    c = Case(61, [130], 1, 2, 128, 32, behind=0)
    dev = [x.to(DEV) for x in (c.q, c.k, c.v, c.beta, c.alpha)] + [c.states.to(DEV).clone(), c.q_start, ints(c.slot_in), ints(c.slot_out)]
    out = torch.empty(c.v.shape, dtype=DT["f16"], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq3.delta_rule_batch(*dev, scale=c.scale, out=out)
    graph.replay()
    assert vq3.delta_status() == 0
    c.check(out, dev[5])
