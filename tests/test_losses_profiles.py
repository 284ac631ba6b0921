"""The committed ncu summaries of the losses' kernels match the sources: each entry of profiles/losses.json names one
and carries the sha256 of the sources it was captured on."""
import json
import os

import bench

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")


def test_summaries_are_of_the_present_sources():
    entries = {k: v for k, v in json.load(open(os.path.join(PROFILES, "losses.json"))).items() if isinstance(v, dict)}
    assert {e["summary"] for e in entries.values()} == {
        f for f in os.listdir(PROFILES) if f.startswith(("sv_distill_", "sv_ce_"))}
    for key, e in entries.items():
        assert e["kernel_source_sha256"] == bench.kernel_source_hash(e["sources"]), (
            f"{key}: captured on other sources of the {e['sources']} kernel; re-capture it")
        text = open(os.path.join(PROFILES, e["summary"])).read()
        assert "ncu " in text and "--clock-control none" in text
        assert f"DRAM traffic: {e['dram_bytes_per_launch'] / 1e6:.1f} MB" in text
