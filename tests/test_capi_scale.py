"""The log probabilities' scale on the host (no GPU needed): the kernels take it times log2(e), in 32 bits."""

import numpy as np
import pytest

import unstructured_sparse_transformer_amd as tw

AT = 1 << 30  # a never dereferenced fake device address
NULL, SHAPE = -1, -3
MOST = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("scale", [MOST, 3e38, 2.4e38])
def test_a_scale_past_32_bits_is_refused(scale):
    """A product with log2(e) that is infinite would make (z - m) of the largest logit times it no number, and L -inf."""
    lib = tw.load()
    assert lib.twell_logprob_forward(AT, 100, 8, 100, 1, scale, None, 64, None, None, None, None, None, 0, None, 0, None) == SHAPE
    assert lib.twell_logprob_backward(AT, 100, 8, 100, 1, scale, AT, 64, AT, AT, AT, AT, 2 * AT, 100, None) == SHAPE


@pytest.mark.parametrize("scale", [2.3e38, 1.0, 1e-30])
def test_others_are_served(scale):
    """(Without any result, or without a norm, the calls that pass the scale's check end at the next one.)"""
    lib = tw.load()
    assert lib.twell_logprob_forward(AT, 100, 8, 100, 1, scale, None, 64, None, None, None, None, None, 0, None, 0, None) == NULL
    assert lib.twell_logprob_backward(AT, 100, 8, 100, 1, scale, AT, 64, None, AT, AT, AT, 2 * AT, 100, None) == NULL
