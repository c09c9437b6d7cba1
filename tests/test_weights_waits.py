"""What the sources say about waiting in the kernel that adds weights up over many rows,
without a GPU: its roles leave at different places after a bounded wait ran out."""

import os
import re

import pytest

from test_bounded_waits import CSRC, functions


def roles():
    with open(os.path.join(CSRC, "fa_weights.cu")) as f:
        found = functions(f.read())
    return {n: b for n, b in found.items() if n.endswith("_role")}


def test_all_roles_are_looked_at():
    assert set(roles()) == {"unit_role", "load_role", "lse_role", "widen_role", "mma_role", "sum_role"}


@pytest.mark.parametrize("name", sorted(roles()))
def test_roles_wait_with_a_bound(name):
    body = roles()[name]
    assert "sh.wait" in body
    assert not re.search(r"named_barrier|bar\.sync|barrier\.sync|__syncthreads", body)
    # nor a wait whose answer nobody looks at
    assert not re.search(r"^\s*(sh\.wait\w*|paged::wait_warp|in\.next)\(", body, flags=re.M)
