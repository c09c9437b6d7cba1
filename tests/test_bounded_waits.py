"""What the sources say about waiting, without a GPU: a role that leaves after a
bounded wait ran out must not be waited for at a barrier without a bound."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_78_gb300", "csrc")


def functions(text):
    """{name: body} of the functions of a CUDA source, comments taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    out = {}
    for m in re.finditer(r"\b(\w+)\([^;{}]*\)\s*(?:const\s*)?\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out.setdefault(m.group(1), "")
        out[m.group(1)] += text[m.end():i]
    return out


def roles():
    with open(os.path.join(CSRC, "fa_paged_chunk.cu")) as f:
        found = functions(f.read())
    return {n: b for n, b in found.items() if n.endswith("_role")}


def test_all_roles_are_looked_at():
    assert set(roles()) == {"scheduler_role", "load_role", "clean_role", "widen_role", "softmax_role",
                            "correction_role", "mma_role"}


@pytest.mark.parametrize("name", sorted(roles()))
def test_chunk_roles_wait_with_a_bound(name):
    """A chunk kernel's role returns when a wait gives up, at different places in
    different warps: a barrier of the hardware's between them would hold those
    that come to it later, and the block would never end."""
    body = roles()[name]
    assert "sh.wait" in body or "in.next" in body
    assert not re.search(r"named_barrier|bar\.sync|barrier\.sync|__syncthreads", body)
    # nor a wait whose answer nobody looks at
    assert not re.search(r"^\s*(sh\.wait\w*|paged::wait_warp|in\.next)\(", body, flags=re.M)
