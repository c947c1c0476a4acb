"""Order of a paged kernel's steps that no result shows, read out of its source."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "causal_sliding_window_rope_b200", "csrc")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "paged*.cuh"))):
        text = open(path).read()
        at = [m.start() for m in re.finditer(r"__global__", text)] + [len(text)]
        for a, b in zip(at, at[1:]):
            yield re.search(r"(\w+_kernel)\(", text[a:b]).group(1), text[a:b]


OWNERS = {name: body for name, body in kernels() if "tmem_alloc(" in body}


def test_the_owners_of_tensor_memory_are_found():
    assert set(OWNERS) == {"tile_kernel", "weigh_tile_kernel"}


@pytest.mark.parametrize("name", sorted(OWNERS))
def test_the_next_kernel_may_start_only_once_tensor_memory_is_held(name):
    """A successor may take tensor memory before it waits for its predecessor's end (the dense kernels do): one that
    ran beside a CTA that has still to take its own could hold what that CTA waits for, each waiting for the other."""
    body = OWNERS[name]
    assert body.count("pdl_launch_dependents()") == 1
    assert body.index("pdl_wait()") < body.index("tmem_alloc(") < body.index("pdl_launch_dependents()")
