"""Clusters of CTAs (CPU: the sources are read): a CTA writes or reads another
one's shared memory only behind a barrier of the whole cluster, since nothing
else says that the other one has started."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mamba_selective_state_gb300", "csrc")


def sources_with_clusters():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        if "map_shared_rank" in text:
            yield os.path.basename(path), text


@pytest.mark.parametrize("name,text", list(sources_with_clusters()), ids=lambda x: x if x.endswith(".cu") else "")
def test_first_remote_access_waits_for_the_cluster(name, text):
    for kernel in re.split(r"__global__", text)[1:]:
        first = kernel.find("map_shared_rank")
        if first < 0:
            continue
        before = kernel[:first]
        split = "barrier_arrive()" in before and "barrier_wait()" in before
        assert split or "cluster.sync()" in before, name
