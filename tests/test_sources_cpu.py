"""What the compiled sources may not hold.

One library serves every rank of a job, so each of its tensor loads goes to one
CTA: a load that is multicast over a cluster belongs in code that runs on one GPU
only."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "muon_newton_schulz_step_gb300", "csrc")


def sources(pattern):
    return [(os.path.basename(f), open(f).read()) for f in sorted(glob.glob(os.path.join(CSRC, pattern)))]


def test_products_of_8_bits_load_without_multicast():
    for name, text in sources("fp8_*.cu"):
        assert not re.search(r"tma_load\w*_mc\b", text), name


def test_no_tensor_load_is_multicast():
    for name, text in sources("*.cu") + sources("*.cuh"):
        for asm in re.findall(r"asm volatile\((.*?)\);", text, re.S):
            assert not ("cp.async.bulk" in asm and "multicast" in asm), name


def test_traffic_record_is_of_these_sources():
    """The bench leaves the traffic out where the committed capture is of other sources."""
    import bench

    assert bench._traffic_record() is not None
