"""The ends of the temperatures that are taken, on the host."""
import math

import pytest

from test_logprobs_abi import ARG, CALLS, SV_OK, lib, rows, workspace_bytes  # noqa: F401


@pytest.mark.parametrize("T", [math.nextafter(2.0 ** 117, math.inf) * 1.0000001, 2.0 ** 118, 1e36, 3e38, math.inf])
def test_temperatures_past_which_differences_of_logits_would_be_lost(lib, T):  # noqa: F811
    for call in CALLS:
        assert call(lib, rows(T=T)) == ARG, call.__name__
    assert workspace_bytes(lib, rows(T=T)) == ARG


def test_temperatures_at_the_ends(lib):  # noqa: F811
    for T in (2.0 ** 117, 1e35, 1e-38, 5e-39):
        assert workspace_bytes(lib, rows(T=T)) > 0
        for call in CALLS:
            assert call(lib, rows(T=T, outer=0)) == SV_OK, call.__name__
