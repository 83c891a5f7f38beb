"""Calls of the delta rule's, the convolution's and the append's binding that the documentation allows or refuses, on
the CPU (no GPU: none gets as far as a launch)."""

import pytest

torch = pytest.importorskip("torch")
vq3 = pytest.importorskip("bit_vector_lut_gb300.vq3", reason="libvq3.so not built")


def test_delta_status_refuses_a_null_pointer():
    assert vq3.lib.vq3_delta_status(None, None) == -1 and b"null" in vq3.lib.vq3_last_error()
