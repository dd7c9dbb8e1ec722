"""Shared memory of another CTA of a cluster may be touched only while that CTA is known to
run: every remote store in the kernels' sources has a completed barrier.cluster before
it, and another behind it before the first CTA to end may do so."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_plane_select_gb300", "csrc")


def kernels():
    """(file, text of a __global__ function) for each."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"^__global__.*?^}\n", text, re.S | re.M):
            yield os.path.basename(path), m.group(0)


def test_the_sources_have_remote_stores():
    assert any("st.shared::cluster" in k for _, k in kernels())


@pytest.mark.parametrize("name,text", [k for k in kernels() if re.search(r"\bst\.(async\.)?shared::cluster", k[1])],
                         ids=lambda x: x[:20] if x.endswith(".cu") else "kernel")
def test_remote_stores_lie_between_cluster_barriers(name, text):
    stores = [m.start() for m in re.finditer(r"\bst\.(async\.)?shared::cluster", text)]
    # an arrive and, later, its wait: each completed barrier is one pair
    arrives = [m.start() for m in re.finditer(r"barrier\.cluster\.arrive", text)]
    waits = [m.start() for m in re.finditer(r"barrier\.cluster\.wait", text)]
    assert len(arrives) == len(waits) >= 2
    assert arrives[0] < waits[0] < min(stores) and max(stores) < arrives[-1] < waits[-1]
