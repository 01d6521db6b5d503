"""The recorded counters belong to the present kernels: every digest in
profiles/traffic.txt is that of the code that its key names."""
import os

import bench

PROFILES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")


def test_recorded_traffic_is_of_the_present_code():
    lines = open(os.path.join(PROFILES, "traffic.txt")).read().splitlines()
    entries = [ln.split() for ln in lines if ln and not ln.startswith("#")]
    assert entries
    for key, nbytes, digest in entries:
        assert digest == bench.kernel_source_digest(key), key
        assert bench.committed_traffic(key) == float(nbytes)
