"""The committed kernel statistics of the FP4-weight products and the routing
were taken on the present kernels (their sources, comments aside)."""
import json
import os
import re

from test_bench_summary import load_bench


def test_operator_profile_is_of_the_present_sources():
    bench = load_bench()
    path = os.path.join(bench.PROFILES, "kernel_stats_operators")
    prof = json.load(open(path + ".json"))
    assert prof["source_digest"] == bench.operator_digest(), \
        "the kernels changed: take profiles/kernel_stats_operators again (rocprofv3, every listed case)"
    assert f"`{prof['source_digest']}`" in open(path + ".md").read()


def test_operator_digest_reads_every_source_and_no_comments(tmp_path, monkeypatch):
    bench = load_bench()
    csrc = bench.CSRC
    for f in os.listdir(csrc):
        (tmp_path / f).write_text(open(os.path.join(csrc, f)).read())
    base = bench.operator_digest()
    monkeypatch.setattr(bench, "CSRC", str(tmp_path))
    assert bench.operator_digest() == base
    one = tmp_path / "linear_tile.hpp"
    text = one.read_text()
    one.write_text(re.sub(r"//[^\n]*", "", text) + "\n// 1.0 us\n")
    assert bench.operator_digest() == base
    for f in bench.OPERATOR_SOURCES + ("fp4q_device.hpp",):
        src = tmp_path / f
        keep = src.read_text()
        src.write_text(keep + "\nint changed;\n")
        assert bench.operator_digest() != base, f
        src.write_text(keep)
    quantize = set(f for f in os.listdir(csrc) if f.endswith((".hip", ".hpp"))) - set(bench.OPERATOR_SOURCES)
    included = re.findall(r'#include "([^"]+\.hpp)"', "".join(open(os.path.join(csrc, f)).read()
                                                              for f in bench.OPERATOR_SOURCES))
    assert set(included) & quantize <= {"fp4q_device.hpp"}          # nothing else of the others is built in
