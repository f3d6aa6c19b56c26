"""Temperatures at the end of their range (no GPU is needed)."""

import numpy as np
import pytest

from test_kv4_refusals import ARG, _logprobs, lib  # noqa: F401


@pytest.mark.parametrize("temperature", [3.4e-39, 3.5e-39, 4.2e-39])
def test_temperatures_whose_factor_is_infinite_are_refused(lib, temperature):
    """The factor of the exponentials, log2(e) / temperature, leaves fp32's range before 1 / temperature does."""
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(1) / np.float32(temperature) * np.float32(1.4426950408889634))
    assert _logprobs(lib, temp=temperature, batch=0) == ARG      # (batch 0: the call ends behind the check of the temperature)


@pytest.mark.parametrize("temperature", [4.25e-39, 1e-30, 1.0, 2.9e38])
def test_temperatures_within_it_are_taken(lib, temperature):
    assert _logprobs(lib, temp=temperature, batch=0) == 0
