"""Rings of shared-memory stages: every stage that threads read and the next copy
overwrites is given back and taken through the fenced helpers."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_115_gb300", "csrc")


def test_stages_are_given_back_and_taken_behind_fences():
    rings = 0
    for path in glob.glob(os.path.join(CSRC, "*.cuh")):
        text = open(path).read()
        if path.endswith("pkv_device.cuh"):
            release = text[text.index("void ring_release"):][:300]
            acquire = text[text.index("bool ring_acquire"):][:300]
            assert release.index("__threadfence_block") < release.index("__syncwarp") < release.index("mbar_arrive")
            assert acquire.index("mbar_wait_bounded") < acquire.index("fence_proxy_async_smem")
            continue
        # an arrival by a thread on an empty barrier goes through ring_release; the
        # tensor core's own commits (its reads are the async proxy's) do not
        assert not re.search(r"mbar_arrive\([^;]*empty", text), path
        if "ring_release(" in text:
            rings += 1
            assert "ring_acquire(" in text, path
    assert rings == 3
