"""The paged-cache calls refuse bad arguments on the host, before they touch
the device; workspace sizes; the binding's own checks."""

import ctypes

import pytest
import torch

A = ctypes.c_void_p(1 << 20)          # never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    import exact_attention_78_gb300 as fa
    return fa.load_library(build_if_missing=True)


def _attn(lib, q=A, kp=A, vp=A, ks=None, vs=None, o=A, lse=A, B=2, Hq=4, Hkv=2, Sn=1, D=128, num_pages=8, page=16,
          max_pages=4, causal=1, scale=0.1, bt=A, lens=A, cu=None, max_q=0, ws=A, nbytes=1 << 40):
    return lib.fa_fwd_paged(q, kp, vp, ks, vs, o, lse, B, Hq, Hkv, Sn, D, num_pages, page, max_pages, causal, scale,
                            bt, lens, cu, max_q, ws, nbytes, None)


CACHE_BAD = [
    (dict(kp=None), 1), (dict(vp=MIS), 1), (dict(ks=A), 1), (dict(vs=A), 1), (dict(ks=MIS, vs=A), 1),
    (dict(bt=None), 1), (dict(bt=MIS), 1), (dict(lens=MIS), 1), (dict(cu=MIS, Sn=4, max_q=1), 1),
    (dict(B=0), 1), (dict(Hkv=0), 1), (dict(Sn=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1),
    (dict(page=0), 1), (dict(page=48), 1), (dict(page=8), 2), (dict(page=2048), 2), (dict(D=96), 2),
    (dict(B=1025), 2), (dict(max_pages=1 << 27, page=16), 2), (dict(num_pages=1 << 30, Hkv=4, Hq=4), 2),
    (dict(B=1024, Sn=1 << 22), 2),
]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(q=None), 1), (dict(q=MIS), 1), (dict(o=None), 1), (dict(lse=MIS), 1), (dict(lens=None), 1),
    (dict(Hq=3), 1), (dict(causal=2), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(cu=A, Sn=4, max_q=0), 1), (dict(cu=A, Sn=4, max_q=5), 1), (dict(Hq=129 * 2), 2),
    (dict(ws=None), 5), (dict(ws=ctypes.c_void_p((1 << 20) + 16)), 5), (dict(nbytes=100), 5),
])
def test_attention_refusals(lib, kw, status):
    assert _attn(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [c for c in CACHE_BAD if "Hq" not in c[0]] + [
    (dict(k=None), 1), (dict(v=MIS), 1), (dict(lens=None), 1)])
def test_write_refusals(lib, kw, status):
    a = dict(k=A, v=A, kp=A, vp=A, ks=None, vs=None, B=2, Hkv=2, Sn=1, D=128, num_pages=8, page=16, max_pages=4, bt=A,
             lens=A, cu=None)
    a.update({k: v for k, v in kw.items() if k != "max_q"})
    assert lib.fa_cache_write(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [c for c in CACHE_BAD if not {"Hq", "lens"} & set(c[0]) and c[0].get("B") != 1024] + [
    (dict(k=None), 1), (dict(v=MIS), 1), (dict(cu=None), 1)])
def test_read_refusals(lib, kw, status):
    a = dict(kp=A, vp=A, ks=None, vs=None, k=A, v=A, B=2, Hkv=2, Sn=10, D=128, num_pages=8, page=16, max_pages=4, bt=A,
             cu=A)
    a.update({k: v for k, v in kw.items() if k != "max_q"})
    assert lib.fa_cache_read(*a.values(), None) == status


def _rope(lib, q=A, k=A, qo=A, ko=A, tokens=4, Hq=2, Hkv=1, D=128, pos=A, axes=1, sections=(64,), base=1e4, restart=0,
          interleaved=0, inverse=0):
    s = (ctypes.c_int * len(sections))(*sections) if sections is not None else None
    return lib.fa_rope(q, k, qo, ko, tokens, Hq, Hkv, D, pos, axes, s, base, restart, interleaved, inverse, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(k=None), 1), (dict(q=MIS), 1), (dict(ko=MIS), 1),
    (dict(pos=None), 1), (dict(pos=MIS), 1), (dict(sections=None), 1), (dict(tokens=0), 1), (dict(Hq=0), 1),
    (dict(Hkv=0), 1), (dict(axes=0), 1), (dict(axes=5, sections=(1,) * 5), 1), (dict(sections=(65,)), 1),
    (dict(axes=2, sections=(64, 0)), 1), (dict(axes=2, sections=(40, 30)), 1), (dict(D=64, sections=(33,)), 1),
    (dict(base=0.5), 1), (dict(base=float("nan")), 1), (dict(base=float("inf")), 1), (dict(restart=2), 1),
    (dict(interleaved=-1), 1), (dict(inverse=3), 1), (dict(D=96, sections=(8,)), 2), (dict(Hq=1 << 21), 2)])
def test_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status


def test_workspace_size_does_not_depend_on_lengths(lib):
    import exact_attention_78_gb300 as fa
    n = fa.fwd_paged_workspace_size(4, 8, 2, 1, 128)
    assert n > 0 and n % 256 == 0
    assert fa.fwd_paged_workspace_size(4, 8, 2, 100, 128, packed=True, max_q=101) == 0
    assert fa.fwd_paged_workspace_size(4, 8, 3, 1, 128) == 0
    assert fa.fwd_paged_workspace_size(4, 8, 2, 1, 96) == 0
    assert fa.fwd_paged_workspace_size(1025, 8, 2, 1, 64) == 0


def test_binding_refuses_host_tensors(lib):
    import exact_attention_78_gb300 as fa
    x = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cache_write(x, x, pages, pages, table, lens)
    with pytest.raises(ValueError):
        fa.fwd_paged(x, pages, pages, table, lens)
    with pytest.raises(ValueError):
        fa.cache_read(pages, pages, table, lens, 2)
    with pytest.raises(ValueError):
        fa.rope(x, x, torch.zeros(2, 1, dtype=torch.int32))
