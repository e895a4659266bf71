"""Refusals of the dense attention entry points and of the cache (no GPU needed): bad arguments
are rejected before any device work is queued."""
import ctypes

import pytest
import torch

from block_sparse_online_b200 import solattn

placeholder = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers are used only without a GPU")
EINVAL, EUNS, EWS = solattn.SOLATTN_EINVAL, solattn.SOLATTN_EUNSUPPORTED, solattn.SOLATTN_EWORKSPACE
NO_GPU = (solattn.SOLATTN_ECUDA, solattn.SOLATTN_EUNSUPPORTED)


def view(ptr=4096, b=1 << 20, h=1 << 14, n=128):
    return solattn._View(ptr, b, h, n)


def cross(q=None, k=None, v=None, out=None, key_len=4096, B=2, H=4, Hkv=2, Nq=10, Nk=20, d=128, dtype=0, ws=4096,
          ws_bytes=1 << 40):
    return solattn._lib.solattn_cross(q or view(), k or view(), v or view(), out or view(), key_len, B, H, Hkv, Nq, Nk, d,
                                      dtype, ws, ws_bytes, None)


@placeholder
@pytest.mark.parametrize("kw,want", [
    (dict(B=0), EINVAL), (dict(H=3), EINVAL), (dict(Hkv=0), EINVAL), (dict(H=0), EINVAL), (dict(Nq=-1), EINVAL),
    (dict(Nk=-1), EINVAL), (dict(d=96), EUNS), (dict(dtype=2), EINVAL), (dict(dtype=-1), EINVAL),
    (dict(q=view(None)), EINVAL), (dict(q=view(4104)), EINVAL), (dict(k=view(n=132)), EINVAL), (dict(v=view(h=-128)), EINVAL),
    (dict(out=view(n=0)), EINVAL), (dict(out=view(b=0)), EINVAL), (dict(key_len=4098), EINVAL),
    (dict(Nq=1 << 30, H=4, Hkv=1), EUNS), (dict(ws=None), EWS), (dict(ws=4096 + 64), EWS), (dict(ws_bytes=1000), EWS),
])
def test_cross_rejects_bad_arguments(kw, want):
    assert cross(**kw) == want


@placeholder
def test_cross_accepts_what_it_documents():
    for kw in (dict(), dict(key_len=None), dict(k=view(b=0), v=view(b=0)), dict(Nk=0, k=view(None), v=view(None)),
               dict(dtype=1, d=64), dict(B=1, out=view(b=0)), dict(Nk=1, k=view(n=3))):
        assert cross(**kw) in NO_GPU, kw
    assert cross(Nq=0, q=view(None), out=view(None)) == 0  # nothing to do


def cache(k=None, v=None, ks=4096, vs=4096, pages=10, Hkv=2, page=16, d=128, kind=1):
    return solattn._Cache(k or view(b=1 << 13, h=1 << 12), v or view(b=1 << 13, h=1 << 12), ks, vs, pages, Hkv, page, d, kind)


def seqs(table=4096, cu=4096, length=4096, B=2, width=4, total=10):
    return solattn._Seqs(table, cu, length, B, width, total)


def paged(q=None, out=None, c=None, s=None, H=4, max_new=1, causal=1, dtype=0, ws=4096, ws_bytes=1 << 40):
    return solattn._lib.solattn_paged_forward(q or view(), out or view(), c or cache(), s or seqs(), H, max_new, causal,
                                              dtype, ws, ws_bytes, None)


BAD_CACHE = [
    (dict(pages=0), EINVAL), (dict(Hkv=0), EINVAL), (dict(kind=3), EINVAL), (dict(kind=-1), EINVAL), (dict(d=32), EUNS),
    (dict(page=8), EUNS), (dict(page=48), EUNS), (dict(page=256), EUNS), (dict(ks=None), EINVAL), (dict(vs=4097), EINVAL),
    (dict(k=view(None)), EINVAL), (dict(v=view(4100)), EINVAL), (dict(k=view(n=136)), EINVAL), (dict(v=view(b=0)), EINVAL),
]
BAD_SEQS = [(dict(B=0), EINVAL), (dict(total=-1), EINVAL), (dict(width=0), EINVAL), (dict(table=None), EINVAL),
            (dict(cu=None), EINVAL), (dict(length=None), EINVAL), (dict(cu=4097), EINVAL), (dict(width=1 << 28), EUNS)]


@placeholder
@pytest.mark.parametrize("kw,want", [(dict(c=cache(**a)), w) for a, w in BAD_CACHE] + [(dict(s=seqs(**a)), w) for a, w in BAD_SEQS] + [
    (dict(H=3), EINVAL), (dict(max_new=-1), EINVAL), (dict(causal=2), EINVAL), (dict(dtype=5), EINVAL), (dict(q=view(None)), EINVAL),
    (dict(out=view(h=0)), EINVAL), (dict(q=view(n=100)), EINVAL), (dict(ws=None), EWS), (dict(ws_bytes=1 << 10), EWS)])
def test_paged_rejects_bad_arguments(kw, want):
    assert paged(**kw) == want


@placeholder
def test_paged_accepts_what_it_documents():
    for kw in (dict(), dict(c=cache(kind=0, ks=None, vs=None)), dict(c=cache(kind=2)), dict(max_new=0), dict(causal=0)):
        assert paged(**kw) in NO_GPU, kw
    assert paged(s=seqs(total=0), q=view(None), out=view(None)) == 0


@placeholder
@pytest.mark.parametrize("write", [True, False])
def test_cache_calls_reject_bad_arguments(write):
    def call(c=None, k=None, v=None, s=None, dtype=0, status=4096):
        c, k, v, s = c or cache(), k or view(), v or view(), s or seqs()
        if write:
            return solattn._lib.solattn_cache_append(c, k, v, s, dtype, status, None)
        return solattn._lib.solattn_cache_read(c, s, k, v, dtype, status, None)

    for a, want in BAD_CACHE:
        assert call(c=cache(**a)) == want, a
    for a, want in BAD_SEQS:
        assert call(s=seqs(**a)) == want, a
    assert call(dtype=2) == EINVAL and call(status=None) == EWS and call(status=4100) == EWS
    assert call(k=view(None)) == EINVAL and call(v=view(n=4)) == EINVAL
    assert call(k=view(n=0)) in (NO_GPU if write else (EINVAL,))  # inputs may repeat, outputs may not
    assert call(s=seqs(total=0)) == 0
    assert call() in NO_GPU


def test_workspace_sizes():
    f, g = solattn.solattn_cross_workspace_size, solattn.solattn_paged_workspace_size
    assert f(1, 12, 12, 32760, 512, 128) > 256 and g(1, 12, 12, 1560, 128) > 256
    assert f(0, 1, 1, 1, 1, 64) == f(1, 3, 2, 1, 1, 64) == f(1, 1, 1, 1, 1, 80) == f(1, 1, 1, -1, 1, 64) == 0
    assert g(0, 1, 1, 1, 64) == g(1, 3, 2, 1, 64) == g(1, 1, 1, -1, 64) == g(1, 1, 1, 1, 32) == 0


def test_strerror_names_the_table():
    assert "page" in solattn.strerror(solattn.SOLATTN_ETABLE)


def test_binding_refuses_wrong_tensors():
    bf = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        solattn.solattn_cross(bf, bf, bf)  # not on a GPU
    with pytest.raises(ValueError):
        solattn.solattn_cross(bf.float(), bf, bf)
    with pytest.raises(ValueError):
        solattn.PagedCache(bf.float(), bf)
    with pytest.raises(ValueError):
        solattn.PagedCache(bf, bf)  # not on a GPU
    with pytest.raises(ValueError):
        solattn.solattn_paged_forward(bf, None, None, None, None, 1)


def test_structures_match_the_header():
    assert ctypes.sizeof(solattn._View) == 32
    assert ctypes.sizeof(solattn._Cache) == 2 * 32 + 2 * 8 + 5 * 4 + 4
    assert ctypes.sizeof(solattn._Seqs) == 3 * 8 + 3 * 4 + 4
