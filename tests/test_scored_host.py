"""Host-side checks of attn_scored, attn_tree and tree_accept: what the library
refuses before it launches anything (no GPU needed)."""
import ctypes
import os

import pytest

from compressed_kv_attention_gb300 import _binding as B

FAKE = 0x7f0000000000  # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from compressed_kv_attention_gb300 import build
        build.build()
    return B.load()


def cache(D=128, Hkv=2, batch=3, cap=256, data=0x10000, signs=0x20000, v_bits=0, signs2=0):
    return B.CkvCacheStruct(D, Hkv, batch, v_bits, cap, data, signs, signs2)


def score(softcap=0.0, window=0, slopes=None, prefix=None, doc=None):
    return B.CkvScoreStruct(softcap, window, slopes, prefix, doc)


def attend(lib, tree, c=None, **kw):
    c = c or cache()
    a = dict(seq=FAKE, maxs=256, mask=FAKE, q=FAKE, qt=1, nq=4, hq=8, ql=None, scale=0.1, sc=score(), ns=2, out=FAKE,
             ot=0, lse=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    head = (ctypes.byref(c), a["seq"], a["maxs"])
    tail = (a["q"], a["qt"], a["nq"], a["hq"], a["ql"], a["scale"], ctypes.byref(a["sc"]) if a["sc"] else None, a["ns"],
            a["out"], a["ot"], a["lse"], a["ws"], a["wsb"], None)
    return lib.ckv_attn_tree(*head, a["mask"], *tail) if tree else lib.ckv_attn_scored(*head, *tail)


@pytest.mark.parametrize("tree", [False, True])
def test_attention_refusals(lib, tree):
    for status, kw in [
        (-1, dict(seq=None)), (-1, dict(q=None)), (-1, dict(out=None)), (-1, dict(lse=None)),
        (-1, dict(q=FAKE + 8)), (-1, dict(out=FAKE + 2)), (-1, dict(seq=FAKE + 2)), (-1, dict(ql=FAKE + 1)),
        (-1, dict(qt=0)), (-1, dict(qt=3)), (-1, dict(ot=3)), (-1, dict(ot=-1)),
        (-1, dict(scale=float("inf"))), (-1, dict(scale=float("nan"))),
        (-1, dict(sc=score(softcap=-1.0))), (-1, dict(sc=score(softcap=float("nan")))),
        (-1, dict(sc=score(softcap=float("inf")))), (-1, dict(sc=score(window=-1))),
        (-1, dict(sc=score(slopes=FAKE + 2))), (-1, dict(maxs=-1)), (-2, dict(maxs=1 << 31)),
        (-1, dict(ns=-1)), (-1, dict(ns=1025)), (-2, dict(hq=7)), (-1, dict(hq=0)),
        (-3, dict(ws=None)), (-3, dict(ws=FAKE + 16)), (-3, dict(wsb=255)),
        (-2, dict(c=cache(D=96))), (-1, dict(c=cache(cap=250))), (-1, dict(c=cache(v_bits=5))),
        (-2, dict(c=cache(Hkv=2, batch=32768))), (-2, dict(c=cache(Hkv=1, batch=60000), nq=64, hq=600)),
    ]:
        assert attend(lib, tree, **kw) == status, kw
        assert lib.ckv_last_error()
    assert attend(lib, tree, nq=0) == (-2 if tree else -1)


def test_tree_refusals(lib):
    assert attend(lib, True, mask=None) == -1
    assert attend(lib, True, mask=FAKE + 4) == -1
    assert attend(lib, True, nq=65) == -2
    assert attend(lib, True, sc=score(prefix=FAKE)) == -1
    assert attend(lib, True, sc=score(doc=FAKE)) == -1
    c = cache()
    assert lib.ckv_attn_tree_workspace(ctypes.byref(c), 256, 65, 8, 0) == 0
    assert lib.ckv_attn_tree_workspace(ctypes.byref(c), 256, 64, 8, 2) > 0


def test_workspace_covers_every_split_count(lib):
    c = cache(D=256, cap=8192)
    for n_q in (1, 3, 200):
        sizes = [lib.ckv_attn_scored_workspace(ctypes.byref(c), 8192, n_q, 8, s) for s in (1, 2, 7, 40)]
        assert all(s > 0 for s in sizes) and sizes == sorted(sizes)
    assert lib.ckv_attn_scored_workspace(ctypes.byref(c), 8192, 1, 7, 0) == 0


def test_accept_refusals(lib):
    def call(c=None, **kw):
        a = dict(seq=FAKE, nq=8, ql=None, path=FAKE + 4096, mp=4, pl=FAKE + 8192, new=FAKE + 12288, flag=None)
        a.update(kw)
        return lib.ckv_tree_accept(ctypes.byref(c or cache()), a["seq"], a["nq"], a["ql"], a["path"], a["mp"], a["pl"],
                                   a["new"], a["flag"], None)
    for status, kw in [
        (-1, dict(seq=None)), (-1, dict(path=None)), (-1, dict(pl=None)), (-1, dict(new=None)),
        (-1, dict(new=FAKE)), (-1, dict(new=FAKE + 8)), (-1, dict(new=FAKE + 8192)),  # the outputs over an input
        (-1, dict(new=FAKE + 4096 + 44)), (-1, dict(ql=FAKE + 12288)), (-1, dict(path=FAKE + 2)),
        (-1, dict(flag=FAKE + 1)), (-2, dict(nq=0)), (-2, dict(nq=65)), (-2, dict(mp=0)), (-2, dict(mp=65)),
        (-2, dict(c=cache(D=80))), (-2, dict(c=cache(batch=65536))),
    ]:
        assert call(**kw) == status, kw


@pytest.mark.parametrize("tree", [False, True])
def test_scales_beyond_float32_are_refused(lib, tree):
    for kw in (dict(scale=1e32), dict(sc=score(softcap=1e-40)), dict(sc=score(softcap=3e38))):
        assert attend(lib, tree, **kw) == -1, kw
