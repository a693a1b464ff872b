"""Host-side refusals of the speculative step's calls: nothing is launched (no
GPU needed)."""

import ctypes

import pytest
import torch

from mla_latent_kv_03_gb300 import libmla as L

P4, P8, P16 = ctypes.c_void_p(4100), ctypes.c_void_p(4104), ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)
WS = ctypes.c_void_p(1 << 20)
BIG = 1 << 50
NONE = None


@pytest.fixture(scope="module")
def lib():
    return L.load(build_if_missing=True)


def _cfg(heads=16, bs=64, dtype="bf16"):
    return L.make_config(heads, bs, dtype, num_ctas=8)


def _plan(lib, cfg, **kw):
    a = dict(par=P4, sl=P4, qsl=P4, bt=P4, mb=4, nb=8, batch=1, nq=4, words=1, mask=P8, pos=P4, slots=P8, status=P4)
    a.update(kw)
    return lib.mla_tree_plan(cfg and ctypes.byref(cfg), a["par"], a["sl"], a["qsl"], a["bt"], a["mb"], a["nb"],
                             a["batch"], a["nq"], a["words"], a["mask"], a["pos"], a["slots"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(par=NONE), 1), (dict(sl=NONE), 1), (dict(qsl=NONE), 1), (dict(bt=NONE), 1), (dict(mask=NONE), 1),
    (dict(pos=NONE), 1), (dict(slots=NONE), 1), (dict(batch=0), 1), (dict(batch=-1), 1), (dict(nq=-1), 1),
    (dict(nb=-1), 1), (dict(mb=-1), 1), (dict(words=0), 1), (dict(words=17), 2), (dict(mask=P4), 1),
    (dict(slots=P4), 1), (dict(par=ODD), 1), (dict(status=ODD), 1), (dict(pos=ODD), 1),
    (dict(nb=(1 << 31) // 64 + 1), 2), (dict(mb=(1 << 30) // 64 + 1), 2), (dict(nq=(1 << 30) + 1), 2),
])
def test_plan_refuses(lib, kw, want):
    assert _plan(lib, _cfg(), **kw) == want


def _decode(lib, cfg, **kw):
    a = dict(q=P16, cache=P16, nb=8, bt=P4, mb=4, sl=P4, qsl=P4, batch=1, nq=1, mask=P8, words=1, w=P16, ws=WS,
             wsb=BIG, out=P16)
    a.update(kw)
    return lib.mla_tree_decode(cfg and ctypes.byref(cfg), a["q"], a["cache"], a["nb"], a["bt"], a["mb"], a["sl"],
                               a["qsl"], a["batch"], a["nq"], a["mask"], a["words"], a["w"], a["ws"], a["wsb"],
                               a["out"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=NONE), 1), (dict(cache=NONE), 1), (dict(bt=NONE), 1), (dict(sl=NONE), 1), (dict(qsl=NONE), 1),
    (dict(mask=NONE), 1), (dict(w=NONE), 1), (dict(ws=NONE), 1), (dict(out=NONE), 1), (dict(q=P8), 1),
    (dict(cache=P8), 1), (dict(w=P8), 1), (dict(out=P8), 1), (dict(mask=P4), 1), (dict(bt=ODD), 1),
    (dict(sl=ODD), 1), (dict(qsl=ODD), 1), (dict(ws=ctypes.c_void_p((1 << 20) + 128)), 1), (dict(batch=0), 1),
    (dict(batch=-1), 1), (dict(nq=-1), 1), (dict(nb=-1), 1), (dict(mb=-1), 1), (dict(words=0), 1),
    (dict(words=17), 2), (dict(nq=48 * 1024 + 1), 2), (dict(nb=(1 << 31) // 64 + 1), 2), (dict(wsb=4096), 3),
    (dict(mb=(1 << 30) // 64 + 1), 2), (dict(nq=48 * 1024, mb=(1 << 29) // (48 * 1024) + 1), 2),
])
def test_decode_refuses(lib, kw, want):
    assert _decode(lib, _cfg(), **kw) == want


def _verify(lib, **kw):
    a = dict(p=P16, q=P16, v=100, tok=P4, par=P4, qsl=P4, batch=1, nq=4, u=P4, f=P4, path=P4, mp=4, lens=P4, nxt=P4,
             status=P4)
    a.update(kw)
    return lib.mla_tree_verify(a["p"], a["q"], a["v"], a["tok"], a["par"], a["qsl"], a["batch"], a["nq"], a["u"],
                               a["f"], a["path"], a["lens"], a["mp"], a["nxt"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(p=NONE), 1), (dict(tok=NONE), 1), (dict(par=NONE), 1), (dict(qsl=NONE), 1), (dict(u=NONE), 1),
    (dict(f=NONE), 1), (dict(path=NONE), 1), (dict(lens=NONE), 1), (dict(nxt=NONE), 1), (dict(v=0), 1),
    (dict(v=(1 << 20) + 1), 2), (dict(batch=-1), 1), (dict(nq=-1), 1), (dict(mp=0), 1), (dict(p=P8), 1),
    (dict(q=P8), 1), (dict(tok=ODD), 1), (dict(status=ODD), 1), (dict(f=ODD), 1), (dict(nq=(1 << 30) + 1), 2),
])
def test_verify_refuses(lib, kw, want):
    assert _verify(lib, **kw) == want


def _commit(lib, cfg, **kw):
    a = dict(cache=P16, layers=2, nb=8, rb=1152, bt=P4, mb=4, sl=P4, qsl=P4, batch=1, path=P4, lens=P4, mp=4, new=P4,
             status=P4)
    a.update(kw)
    return lib.mla_tree_commit(cfg and ctypes.byref(cfg), a["cache"], a["layers"], a["nb"], a["rb"], a["bt"],
                               a["mb"], a["sl"], a["qsl"], a["batch"], a["path"], a["lens"], a["mp"], a["new"],
                               a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(cache=NONE), 1), (dict(bt=NONE), 1), (dict(sl=NONE), 1), (dict(qsl=NONE), 1), (dict(path=NONE), 1),
    (dict(lens=NONE), 1), (dict(new=NONE), 1), (dict(cache=P8), 1), (dict(layers=-1), 1), (dict(nb=-1), 1),
    (dict(mb=-1), 1), (dict(batch=-1), 1), (dict(mp=0), 1), (dict(rb=2304), 2), (dict(rb=1024), 2),
    (dict(nb=(1 << 31) // 64 + 1), 2), (dict(mb=(1 << 30) // 64 + 1), 2), (dict(layers=65536), 2),
    (dict(status=ODD), 1), (dict(new=ODD), 1),
])
def test_commit_refuses(lib, kw, want):
    assert _commit(lib, _cfg(), **kw) == want


def test_configs_and_empty_calls(lib):
    assert _plan(lib, None) == _decode(lib, None) == _commit(lib, None) == 1
    assert _decode(lib, _cfg(dtype="f32")) == 2
    assert _commit(lib, _cfg(dtype="f32"), rb=1152) == _commit(lib, _cfg(dtype="f32"), rb=640) == 2
    bad = _cfg()
    bad.block_size = 48
    assert _plan(lib, bad) == _decode(lib, bad) == _commit(lib, bad) == 2
    assert _plan(lib, _cfg(), nq=0, par=NONE, batch=0) == 0
    assert _decode(lib, _cfg(), nq=0, batch=0, q=NONE, out=NONE) == 0
    assert _verify(lib, batch=0, nq=0, p=NONE) == 0
    assert _commit(lib, _cfg(), batch=0, cache=NONE) == 0
    size = lib.mla_tree_decode_workspace_size
    c, f = _cfg(), _cfg(dtype="f32")
    assert size(ctypes.byref(c), 8, 2) > 8 * 16 * 512 * 4
    assert size(ctypes.byref(c), 9, 2) >= size(ctypes.byref(c), 8, 2) >= size(ctypes.byref(c), 8, 1)
    assert size(None, 8, 2) == size(ctypes.byref(f), 8, 2) == size(ctypes.byref(c), -1, 2) == 0
    assert size(ctypes.byref(c), 8, -1) == size(ctypes.byref(c), 48 * 1024 + 1, 2) == 0


def test_binding_refuses_shapes():
    c = _cfg()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="positions must have shape"):
        L.mla_tree_plan(c, i32(4), i32(1), i32(2), i32(1, 4), 8, torch.zeros(4, 1, dtype=torch.int64), i32(3),
                        torch.zeros(4, dtype=torch.int64))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="tree_mask must have shape"):
        L.mla_tree_decode(c, bf(4, 16, 576), bf(8, 64, 576), i32(1, 4), i32(1), i32(2),
                          torch.zeros(3, 1, dtype=torch.int64), bf(16, 512, 128), torch.zeros(8), bf(4, 16, 128))
    with pytest.raises(ValueError, match="draft_probs must have shape"):
        L.mla_tree_verify(torch.zeros(4, 10), torch.zeros(4, 9), i32(4), i32(4), i32(2), torch.zeros(4),
                          torch.zeros(1), i32(1, 4), i32(1), i32(1))
    with pytest.raises(ValueError, match="cache must have shape"):
        L.mla_tree_commit(c, bf(2, 8, 32, 576), i32(1, 4), i32(1), i32(2), i32(1, 4), i32(1), i32(1))
