"""A CTA of a cluster may be stored to only once it runs, which a cluster barrier says and
being scheduled together does not. Checked in the sources: a store to a CTA that has not
started is no case to provoke on a GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bounded_expert_cache_gb300", "csrc")
BARRIER = r"cluster\.(sync|barrier_wait)\(\)"


def before_remote_accesses(source):
    """kernel -> its text up to the first access to another CTA's shared memory, by itself or by a helper."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    head, *kernels = text.split("__global__")
    helpers = [m.group(1) for m in re.finditer(r"__device__ [^{;]*?(\w+)\([^{;]*\) \{\n((?:  .*\n)+)\}", text)
               if "map_shared_rank" in m.group(2)]
    found = {}
    for body in kernels:
        body = body.split("\n}\n")[0]
        at = [m.start() for name in ["map_shared_rank"] + helpers for m in re.finditer(rf"\b{name}\(", body)]
        if at:
            found[re.search(r"\b(\w+_kernel)\(", body).group(1)] = body[:min(at)]
    return found


@pytest.mark.parametrize("source,kernels", [("sample.cu", {"sample_kernel"}), ("kv_pages.cu", {"reserve_kernel", "compact_kernel"})])
def test_a_cluster_has_started_before_its_shared_memory_is_accessed(source, kernels):
    found = before_remote_accesses(source)
    assert set(found) == kernels
    for name, before in found.items():
        assert re.search(BARRIER, before), name


def test_sources_with_remote_accesses_are_known():
    used = {os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu*")) if "map_shared_rank" in open(f).read()}
    assert used == {"sample.cu", "kv_pages.cu"}


@pytest.mark.gpu
@pytest.mark.parametrize("V", [32769, 33000, 65537])
def test_rows_whose_last_slices_are_empty(V):
    """CTAs without a token reach the first exchange before the others have loaded theirs."""
    import bounded_expert_cache_gb300 as bec
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    for rows in (1, 2, 4):
        z = torch.randn((rows, V), device="cuda", generator=g) * 3
        u = torch.rand((rows,), device="cuda", generator=g)
        top = z.argmax(1).int()
        one = bec.sample(z, u, 0.0)[0]
        want = bec.sample(z, u, 0.9, 50, 0.9)
        for _ in range(50):
            got = bec.sample(z, u, 0.9, 50, 0.9)
            assert torch.equal(bec.sample(z, u, 0.0)[0], top)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(one, top)
