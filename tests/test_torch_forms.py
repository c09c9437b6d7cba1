"""The binding's allocation and streams without torch's private short forms."""

import types

import pytest
import torch

import exact_attention_78_gb300 as fa


class Missing:
    """A torch without the private forms."""


def test_public_forms_stand_in(monkeypatch):
    calls = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=70 + device))
    monkeypatch.setattr(torch.cuda, "caching_allocator_alloc", lambda size, stream: calls.append((size, stream)) or 4096)
    monkeypatch.setattr(torch.cuda, "caching_allocator_delete", lambda adr: calls.append(adr))
    stream, alloc, free = fa.binding._torch_forms(Missing)
    assert stream(1) == 71
    assert alloc(512, 71) == 4096
    free(4096)
    assert calls == [(512, 71), 4096]


def test_no_other_private_names():
    """torch._C is looked at in one place alone, with a public form beside each name."""
    with open(fa.binding.__file__) as f:
        text = f.read()
    assert text.count("torch._C") == 1 and "_torch_forms(torch._C)" in text


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 60])
def test_same_results(monkeypatch, new):
    fa.load_library(build_if_missing=True)
    from paged_case import Cache, randn
    c = Cache([300, 100], 2, 64, 16, False, seed=1)
    q = randn((2, new, 4, 64), 2).cuda()
    args = (q, c.k_pages, c.v_pages, c.block_table, c.seq_lens)
    o, lse = fa.fwd_paged(*args)
    for name, form in zip(("_current_stream", "_alloc", "_free"), fa.binding._torch_forms(Missing)):
        monkeypatch.setattr(fa.binding, name, form)
    before = torch.cuda.memory_allocated()
    o2, lse2 = fa.fwd_paged(*args)
    kept = torch.cuda.memory_allocated() - before
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and fa.get_device_error() == 0
    assert kept <= 2 * (o.numel() * 2 + lse.numel() * 4) + 1024          # the workspace is back
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, lse3 = fa.fwd_paged(*args, stream=side)
    side.synchronize()
    assert torch.equal(o, o3) and torch.equal(lse, lse3)
