"""The host-side layer of the causal mixer and beam search
(csrc/host_causal.cpp: validation, overflow guards, workspace sizes, the choice
of a cut) built on the CPU under the address and undefined-behaviour
sanitizers."""
import os

from test_sanitizers import CSRC, HERE, ROOT, build_and_run


def test_causal_host_layer_under_sanitizers(tmp_path):
    out = build_and_run(tmp_path, "g++",
                        [os.path.join(HERE, "host_causal_checks.cpp"), os.path.join(CSRC, "host_causal.cpp"),
                         os.path.join(CSRC, "host.cpp")],
                        ["-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC], "host_causal_checks")
    assert "host causal checks ok" in out
