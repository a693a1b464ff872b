"""Host-side refusals of the page-scaled cache's and eviction's calls: nothing
is launched (no GPU needed)."""

import ctypes

import pytest
import torch

from mla_latent_kv_03_gb300 import libmla as L


@pytest.fixture(scope="module")
def lib():
    return L.load(build_if_missing=True)


P4, P8, P16 = ctypes.c_void_p(4100), ctypes.c_void_p(4104), ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)
WS = ctypes.c_void_p(1 << 20)
BIG = 1 << 50
NONE = None


def _cfg(heads=16, bs=64, dtype="bf16"):
    return L.make_config(heads, bs, dtype, num_ctas=8)


def _write(lib, cfg, **kw):
    a = dict(c_kv=P16, k_pe=P16, pos=P4, slots=P8, n=4, w=P16, cache=P16, scales=P4, nb=8, mass=P4,
             ws=WS, wsb=BIG, status=P4)
    a.update(kw)
    return lib.mla_page8_cache_write(
        cfg and ctypes.byref(cfg), a["c_kv"], a["k_pe"], a["pos"], a["slots"], a["n"], a["w"],
        a["cache"], a["scales"], a["nb"], a["mass"], a["ws"], a["wsb"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(c_kv=NONE), 1), (dict(k_pe=NONE), 1), (dict(pos=NONE), 1), (dict(slots=NONE), 1),
    (dict(w=NONE), 1), (dict(cache=NONE), 1), (dict(scales=NONE), 1), (dict(ws=NONE), 1),
    (dict(c_kv=P8), 1), (dict(k_pe=P8), 1), (dict(slots=P4), 1), (dict(w=P8), 1),
    (dict(cache=P8), 1), (dict(scales=ODD), 1), (dict(mass=ODD), 1), (dict(status=ODD), 1),
    (dict(pos=ODD), 1), (dict(ws=ctypes.c_void_p((1 << 20) + 64)), 1), (dict(n=-1), 1),
    (dict(n=(1 << 30) + 1), 1), (dict(nb=-1), 1), (dict(nb=(1 << 31) // 64 + 1), 2),
    (dict(wsb=0), 3), (dict(n=5000, wsb=1024), 3),
])
def test_write_refuses(lib, kw, want):
    assert _write(lib, _cfg(), **kw) == want


def test_write_configs_and_empty_calls(lib):
    assert _write(lib, None) == 1
    assert _write(lib, _cfg(dtype="f32")) == 2
    bad = _cfg()
    bad.block_size = 48
    assert _write(lib, bad) == 2
    assert _write(lib, _cfg(), n=0, c_kv=NONE, ws=NONE, wsb=0) == 0
    size = lib.mla_page8_write_workspace_size
    c = _cfg()
    assert size(ctypes.byref(c), 0, 0) > 0
    # pages touched by many tokens: an entry for each page and each of their rows
    assert size(ctypes.byref(c), 100000, 5000) >= 5000 * 4 + 5000 * 64 * 4
    assert size(ctypes.byref(c), -1, 8) == size(ctypes.byref(c), 4, -1) == 0
    assert size(None, 4, 8) == 0
    f = _cfg(dtype="f32")
    assert size(ctypes.byref(f), 4, 8) == 0


def _decode(lib, cfg, with_mass, **kw):
    a = dict(q=P16, cache=P16, scales=P4, nb=8, bt=P4, mb=4, sl=P4, qsl=P4, batch=1, nq=1, w=P16,
             mass=P4, decay=0.5, ws=WS, wsb=BIG, out=P16)
    a.update(kw)
    head = [cfg and ctypes.byref(cfg), a["q"], a["cache"], a["scales"], a["nb"], a["bt"], a["mb"],
            a["sl"], a["qsl"], a["batch"], a["nq"], a["w"]]
    if with_mass:
        return lib.mla_page8_decode_mass(*head, a["mass"], ctypes.c_float(a["decay"]), a["ws"],
                                         a["wsb"], a["out"], None)
    return lib.mla_page8_decode(*head, a["ws"], a["wsb"], a["out"], None)


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(q=NONE), 1), (dict(cache=NONE), 1), (dict(scales=NONE), 1), (dict(bt=NONE), 1),
    (dict(sl=NONE), 1), (dict(qsl=NONE), 1), (dict(w=NONE), 1), (dict(ws=NONE), 1),
    (dict(out=NONE), 1), (dict(q=P8), 1), (dict(cache=P8), 1), (dict(w=P8), 1), (dict(out=P8), 1),
    (dict(scales=ODD), 1), (dict(bt=ODD), 1), (dict(sl=ODD), 1), (dict(qsl=ODD), 1),
    (dict(ws=ctypes.c_void_p((1 << 20) + 128)), 1), (dict(batch=0), 1), (dict(batch=-1), 1),
    (dict(nq=-1), 1), (dict(nb=-1), 1), (dict(mb=-1), 1), (dict(nq=48 * 1024 + 1), 2),
    (dict(nb=(1 << 31) // 64 + 1), 2), (dict(wsb=4096), 3),
    (dict(mb=(1 << 30) // 64 + 1), 2), (dict(nq=48 * 1024, mb=(1 << 30) // (48 * 1024) + 1), 2),
])
def test_decode_refuses(lib, with_mass, kw, want):
    assert _decode(lib, _cfg(), with_mass, **kw) == want


def test_decode_configs_mass_and_empty_calls(lib):
    for wm in (False, True):
        assert _decode(lib, None, wm) == 1
        assert _decode(lib, _cfg(dtype="f32"), wm) == 2
        assert _decode(lib, _cfg(), wm, nq=0, batch=0, q=NONE, out=NONE) == 0
    for decay in (-0.1, 1.5, float("nan"), float("inf")):
        assert _decode(lib, _cfg(), True, decay=decay) == 1
    assert _decode(lib, _cfg(), True, mass=NONE) == 1
    assert _decode(lib, _cfg(), True, batch=65536) == 2
    assert _decode(lib, _cfg(), True, mass=ODD) == 1
    size = lib.mla_page8_decode_workspace_size
    c = _cfg()
    plain, mass = size(ctypes.byref(c), 4, 4, 10, 0), size(ctypes.byref(c), 4, 4, 10, 1)
    assert mass >= plain + 4 * 16 * 10 * 64 * 4       # the scores
    # a workspace sized without mass is refused with it
    assert _decode(lib, _cfg(), True, nq=4, batch=4, mb=10, wsb=plain) == 3
    assert size(None, 4, 4, 10, 0) == size(ctypes.byref(c), -1, 4, 10, 0) == 0
    f = _cfg(dtype="f32")
    assert size(ctypes.byref(f), 4, 4, 10, 0) == 0


def _select(lib, cfg, **kw):
    a = dict(mass=P4, nb=8, bt=P4, mb=4, sl=P4, batch=2, sinks=1, recent=2, budget=8, keep=P4,
             new=P4, status=P4)
    a.update(kw)
    return lib.mla_evict_select(
        cfg and ctypes.byref(cfg), a["mass"], a["nb"], a["bt"], a["mb"], a["sl"], a["batch"],
        a["sinks"], a["recent"], a["budget"], a["keep"], a["new"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(mass=NONE), 1), (dict(bt=NONE), 1), (dict(sl=NONE), 1), (dict(keep=NONE), 1),
    (dict(new=NONE), 1), (dict(mass=ODD), 1), (dict(bt=ODD), 1), (dict(sl=ODD), 1),
    (dict(keep=ODD), 1), (dict(new=ODD), 1), (dict(status=ODD), 1), (dict(sinks=-1), 1),
    (dict(recent=-1), 1), (dict(budget=0), 1), (dict(sinks=5, recent=4), 1),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1, budget=2 ** 31 - 1), 1), (dict(batch=-1), 1),
    (dict(nb=-1), 1), (dict(mb=-1), 1), (dict(nb=(1 << 31) // 64 + 1), 2),
    (dict(mb=(1 << 30) // 64 + 1), 2), (dict(batch=(1 << 27) + 1), 2), (dict(batch=0, mass=NONE), 0),
])
def test_select_refuses(lib, kw, want):
    assert _select(lib, _cfg(), **kw) == want
    assert _select(lib, None, **kw) == 1


def _compact(lib, cfg, **kw):
    a = dict(cache=P16, scales=P4, mass=P4, nb=8, bt=P4, mb=4, keep=P4, new=P4, batch=2, budget=8,
             dst=P4, dmb=2, status=P4)
    a.update(kw)
    return lib.mla_page8_compact(
        cfg and ctypes.byref(cfg), a["cache"], a["scales"], a["mass"], a["nb"], a["bt"], a["mb"],
        a["keep"], a["new"], a["batch"], a["budget"], a["dst"], a["dmb"], a["status"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(cache=NONE), 1), (dict(scales=NONE), 1), (dict(bt=NONE), 1), (dict(keep=NONE), 1),
    (dict(new=NONE), 1), (dict(dst=NONE), 1), (dict(cache=P8), 1), (dict(scales=ODD), 1),
    (dict(mass=ODD), 1), (dict(bt=ODD), 1), (dict(keep=ODD), 1), (dict(new=ODD), 1),
    (dict(dst=ODD), 1), (dict(status=ODD), 1), (dict(budget=0), 1), (dict(batch=-1), 1),
    (dict(nb=-1), 1), (dict(mb=-1), 1), (dict(dmb=-1), 1), (dict(nb=(1 << 31) // 64 + 1), 2),
    (dict(dmb=(1 << 30) // 64 + 1), 2), (dict(batch=65536), 2), (dict(batch=0, cache=NONE), 0),
])
def test_compact_refuses(lib, kw, want):
    assert _compact(lib, _cfg(), **kw) == want
    assert _compact(lib, _cfg(dtype="f32")) == 2


def test_binding_refuses_shapes_before_any_pointer_is_read():
    cfg = _cfg()
    z = torch.zeros
    with pytest.raises(ValueError, match="page_scales"):
        L.mla_page8_cache_write(cfg, z(1, 512), z(1, 64), z(1), z(1), z(512), z(4, 64, 640), z(3), z(8))
    with pytest.raises(ValueError, match="cache8"):
        L.mla_page8_decode(cfg, z(1, 16, 576), z(4, 32, 640), z(4), z(1, 2), z(1), z(2),
                           z(16, 512, 128), z(8), z(1, 16, 128))
    with pytest.raises(ValueError, match="mass"):
        L.mla_page8_decode_mass(cfg, z(1, 16, 576), z(4, 64, 640), z(4), z(1, 2), z(1), z(2),
                                z(16, 512, 128), z(4, 32), 1.0, z(8), z(1, 16, 128))
    with pytest.raises(ValueError, match="new_lens"):
        L.mla_evict_select(cfg, z(4, 64), z(2, 2), z(2), 0, 0, z(2, 5), z(3))
    with pytest.raises(ValueError, match="keep"):
        L.mla_page8_compact(cfg, z(4, 64, 640), z(4), None, z(2, 2), z(3, 5), z(2), z(2, 1))


@pytest.mark.parametrize("heads", [16, 32, 128])
@pytest.mark.parametrize("with_mass", [0, 1])
def test_decode_workspaces_of_fewer_rows_sequences_and_blocks_are_no_larger(lib, heads, with_mass):
    """A program sizes once for its most of each."""
    c = _cfg(heads=heads)
    size = lambda n, b, mb: lib.mla_page8_decode_workspace_size(ctypes.byref(c), n, b, mb, with_mass)  # noqa: E731
    steps = [1, 2, 7, 16, 38, 39, 63, 64, 300, 2048]
    for n in steps:
        for b in steps:
            for mb in (1, 64, 2048):
                most = size(n, b, mb)
                assert most > 0
                assert all(size(n2, b, mb) <= most for n2 in steps if n2 <= n)
                assert all(size(n, b2, mb) <= most for b2 in steps if b2 <= b)
                assert mb == 1 or size(n, b, mb // 2) <= most


@pytest.mark.parametrize("bs", [16, 64])
def test_write_workspaces_of_fewer_tokens_are_no_larger(lib, bs):
    c = _cfg(bs=bs)
    size = lambda n, nb: lib.mla_page8_write_workspace_size(ctypes.byref(c), n, nb)  # noqa: E731
    for nb in (1, 100, 4000, 50000):
        last = 0
        for n in sorted((0, 1, 2048, 2049, 3000, max(nb * bs // 8 - 1, 0), nb * bs // 8, nb, nb + 1, 1 << 20)):
            assert size(n, nb) >= max(last, 256)
            last = size(n, nb)


def test_compact_refuses_a_missing_table_unless_it_has_no_columns(lib):
    assert _compact(lib, _cfg(), dst=NONE, dmb=1) == 1
    assert _compact(lib, _cfg(), dst=NONE, dmb=0, keep=NONE) == 1
