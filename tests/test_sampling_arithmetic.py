"""The sampling kernels' arithmetic on weights, compiled for the host from the header the kernels
use (sampling_arithmetic.cpp), against wider arithmetic."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def figures(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("arithmetic") / "run")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-o", exe,
                    os.path.join(HERE, "sampling_arithmetic.cpp")], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    return {k: float(v) for k, v in (line.split() for line in out.splitlines())}


def test_shares_of_a_mass_are_exact(figures):
    """floor(u x) and ceil(p x) have no rounding before the last step; a uniform of -0 is 0."""
    assert figures["zero_share"] == 0
    assert figures["shares_off"] == 0


def test_weights_keep_their_bound(figures):
    """A weight is off by 2^-39 of itself and half a unit of 2^-43, which is not in `weight_off`."""
    assert figures["weight_off"] <= 2.0 ** -39
    assert 0.997 <= figures["least_parts"] and figures["most_parts"] < 2


def test_sums_of_weights_keep_their_bound(figures):
    """2^-30 of themselves, where a table's part and three roundings of 2^-33 all agree."""
    assert figures["sum_off"] <= 2.0 ** -30


def test_splitting_keys_ends(figures):
    """After three parts of 2048, also where a search finds no part: of a row that changes under it."""
    assert figures["key_ranges_outside"] == 0
    assert figures["key_range_rounds"] <= 3
