"""Calls of the delta rule's, the convolution's and the append's binding that the documentation allows or refuses, on
the CPU (no GPU: none gets as far as a launch)."""

import pytest

torch = pytest.importorskip("torch")
vq3 = pytest.importorskip("bit_vector_lut_gb300.vq3", reason="libvq3.so not built")


def test_delta_status_refuses_a_null_pointer():
    assert vq3.lib.vq3_delta_status(None, None) == -1 and b"null" in vq3.lib.vq3_last_error()


def delta_call(states=None, **kw):
    h = torch.float16
    q, v, g = torch.zeros(3, 2, 64, dtype=h), torch.zeros(3, 4, 32, dtype=h), torch.zeros(3, 4)
    states = torch.zeros(5, 4, 64, 32) if states is None else states
    v, g = v[:, : states.shape[1]], g[:, : states.shape[1]]
    return vq3.delta_rule_batch(q[:, :1], q[:, :1], v, g, g, states, torch.zeros(3, dtype=torch.int32), out=v.clone(), **kw)



@pytest.mark.parametrize("states", [torch.zeros(1, 5, 64, 32).transpose(0, 1),                            # heads in front
                                    torch.zeros(5, 3, 64, 32)[:, :1],                                      # one of several
                                    torch.zeros(5, 64, 32).as_strided((5, 1, 64, 32), (2048, 7, 32, 1))])
def test_a_pool_of_one_head_has_no_stride_of_heads(states):
    # past the checks of shapes and strides (the tensors are on the CPU, which is what is refused)
    with pytest.raises(vq3.Vq3Error, match="CUDA device"):
        delta_call(states)


def test_pools_whose_slots_are_not_contiguous_are_refused():
    for states in (torch.zeros(5, 4, 64, 64)[..., :32], torch.zeros(5, 4, 128, 32)[:, :, :64], torch.zeros(5, 1, 32, 64).transpose(2, 3),
                   torch.zeros(4, 5, 64, 32).transpose(0, 1)):
        with pytest.raises(vq3.Vq3Error, match="states must be"):
            delta_call(states)
