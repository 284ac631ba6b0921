"""The committed ncu summaries of the sampling and log-probability kernels match the sources: each entry of
profiles/sampling.json names one and carries the sha256 of the sources it was captured on."""
import json
import os

import bench

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")


def test_summaries_are_of_the_present_sources():
    entries = {k: v for k, v in json.load(open(os.path.join(PROFILES, "sampling.json"))).items() if isinstance(v, dict)}
    assert {e["summary"] for e in entries.values()} == {
        f for f in os.listdir(PROFILES) if f.startswith(("sv_sample_", "sv_filter_", "sv_logprobs_"))}
    for key, e in entries.items():
        assert e["kernel_source_sha256"] == bench.kernel_source_hash(e["sources"]), (
            f"{key}: captured on other sources of the {e['sources']} kernel; re-capture it")
        text = open(os.path.join(PROFILES, e["summary"])).read()
        assert "ncu " in text and "--clock-control none" in text
        assert f"DRAM traffic: {e['dram_bytes_per_launch'] / 1e6:.1f} MB" in text


def test_every_source_of_a_kernel_is_in_its_hash():
    """What a kernel's file includes, and what those include."""
    import re
    from speculative_decoding_verification_14_gb300 import build
    for mode, files in bench.KERNEL_SOURCES.items():
        for f in files:
            text = open(os.path.join(build.CSRC, f)).read()
            for inc in re.findall(r'#include "([^"/]+)"', text):
                assert inc in files or inc == "sv_internal.h" and mode in ("sampling", "logprobs"), (mode, f, inc)
