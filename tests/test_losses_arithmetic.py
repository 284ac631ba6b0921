"""The losses' arithmetic in two floats, compiled for the host from the header the kernels use
(two_floats_arithmetic.cpp), against doubles."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def figures(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("arithmetic") / "run")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-o", exe,
                    os.path.join(HERE, "two_floats_arithmetic.cpp")], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    return {k: float(v) for k, v in (line.split() for line in out.splitlines())}


def test_series_keep_their_bounds(figures):
    assert figures["exp_off"] <= 2.0 ** -28 and figures["log_off"] <= 2.0 ** -29
    assert figures["ends"] == 1


def test_sums_products_and_quotients(figures):
    """Sums are off by less than 2^-46 of their terms (Dekker's bound for them is 2^-46 of the larger), products and
    quotients by a few units of 2^-47."""
    assert figures["sum_off"] <= 2.0 ** -46
    assert figures["product_off"] <= 2.0 ** -44 and figures["quotient_off"] <= 2.0 ** -44
