"""Softmax scales of 0 and below: every form of the attention against the fp64 oracle, at
the bars of the other parity tests (_helpers.py)."""

import pytest
import torch

from _helpers import assert_close, ref_o_lat_from, to_f64
from test_gpu_naive import _expanded_ref
from mla_latent_kv_03_gb300 import libmla as L
from mla_latent_kv_03_gb300 import workloads as W
from mla_latent_kv_03_gb300.step import MlaDecodeStep

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SCALES = [-0.072, -0.01, 0.0]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L.load()


CASES = {
    "f32": lambda: W.make("f32", [7, 100, 33], [1, 3, 2], 16, 16, "f32", seed=81),
    "rows": lambda: W.make("rows", [1, 63, 65, 400], [1] * 4, 16, 64, "bf16", seed=82),
    "chunks": lambda: W.make("chunks", [150, 64, 20, 90], [40, 1, 20, 5], 16, 64, "bf16", seed=83),
    "h64": lambda: W.make("h64", [70, 2, 300], [1, 1, 3], 64, 32, "bf16", seed=84),
    "h128": lambda: W.make("h128", [17, 333, 1], [2, 1, 1], 128, 16, "bf16", seed=85),
}


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("name", sorted(CASES))
def test_decode(name, scale):
    w = CASES[name]()
    w.softmax_scale = scale
    s = MlaDecodeStep(w, device=DEV, cache_fill=float("nan"))
    s.populate()
    s.absorb()
    s.decode()
    s.combine()
    assert s.device_status()[0][0] == 0
    ref = ref_o_lat_from(w, to_f64(s.cache), to_f64(s.q_abs))
    assert_close(to_f64(s.o_lat), ref, w.dtype, f"o_lat {name}")
    s.o_lat.fill_(float("nan"))
    s.decode_paged_combine()
    assert s.device_status()[0][0] == 0
    assert_close(to_f64(s.o_lat), ref, w.dtype, f"o_lat, merged in the decode, {name}")


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("name", ["rows", "chunks", "h64"])
def test_expanded_prefill_and_decode(name, scale):
    w = CASES[name]()
    w.softmax_scale = scale
    s = MlaDecodeStep(w, device=DEV)
    s.naive_setup()
    s.naive_populate()
    ref = _expanded_ref(w, s)
    for call in (s.naive_prefill, s.naive_decode):
        s.out_naive.fill_(float("nan"))
        call()
        assert L.mla_get_device_status(s.naive_ws)[0] == 0
        assert_close(to_f64(s.out_naive), ref, "bf16", f"{call.__name__} {name}")
