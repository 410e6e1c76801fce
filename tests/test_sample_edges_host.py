"""Sampled decoding where it can go wrong, without a GPU."""
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "speculative_decode_gated_gdn_gb300", "csrc")


def read(name):
    return open(os.path.join(CSRC, name)).read()


def test_a_warp_writes_each_shared_result_at_one_place():
    """What every warp leaves for the whole CTA, which reads all of it behind the next barrier: an array written at a second
    place before another barrier can be read half old, half new.  (The largest logit of a slice's first granules and that of
    the whole slice are such results.)"""
    body = read("sample.cu").split("sample_kernel(const SampleParams p) {")[1].split("cudaError_t launch(")[0]
    written = [n for line in re.findall(r"if \(lane == 0\) (s\.\w+\[warp\] = [^;]*;)", body) for n in re.findall(r"s\.(\w+)\[warp\] =", line)]
    assert {"warp_top", "warp_low", "warp_bound"} <= set(written)
    assert len(written) == len(set(written)), written
