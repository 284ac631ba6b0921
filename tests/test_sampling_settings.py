"""What the sampling calls of the wrapper hand to the library as settings; no GPU call is made."""
import math

import numpy as np
import pytest

import speculative_decoding_verification_14_gb300 as sv


def settings(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    return sv.Verifier._settings(None, temperature, top_k, top_p, min_p, 4)


def test_a_temperature_below_any_float_is_not_greedy():
    """The library refuses temperatures that are no normal numbers; rounded to 0 it would not see one."""
    for t in (1e-46, 1e-60, 5e-324, -1e-46):
        assert math.isnan(settings(temperature=t).temperature), t
    for t in (0, 0.0, -0.0, 1e-40, 1.2e-38, 0.7, 1, np.float32(0.3)):
        assert settings(temperature=t).temperature == np.float32(t), t


def test_top_k_is_a_whole_number():
    """0.5 rounded down would turn the filter off."""
    for k in (0.5, 1.5, -0.5, float("nan")):
        with pytest.raises(ValueError):
            settings(top_k=k)
    for k, want in ((0, 0), (-3, 0), (50, 50), (50.0, 50), (np.int64(7), 7), (1 << 40, 0x7fffffff)):
        assert settings(top_k=k).top_k == want
