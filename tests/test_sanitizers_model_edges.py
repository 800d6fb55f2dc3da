"""Edges of what the host layer of the gated recurrence, the norm and the
vocabulary loss (csrc/host_model.cpp) accepts, built on the CPU under the
address and undefined-behaviour sanitizers."""
import os

from test_sanitizers import CSRC, HERE, ROOT, build_and_run


def test_model_host_edges_under_sanitizers(tmp_path):
    out = build_and_run(tmp_path, "g++",
                        [os.path.join(HERE, "host_model_edges.cpp"), os.path.join(CSRC, "host_model.cpp"), os.path.join(CSRC, "host.cpp")],
                        ["-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC], "host_model_edges")
    assert "host model edges ok" in out
