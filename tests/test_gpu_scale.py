"""Softmax scales of 0 and below: every form of the attention against the fp64 oracle, at
the bars of the other parity tests (_helpers.py)."""

import numpy as np
import pytest
import torch

import test_gpu_page8 as page8
from _helpers import assert_close, ref_o_lat_from, to_f64
from mla_latent_kv_03_gb300 import libmla as L
from mla_latent_kv_03_gb300 import workloads as W
from mla_latent_kv_03_gb300.step import MlaDecodeStep
from oracle import mla_oracle as O
from oracle import page8_oracle as P
from test_gpu_naive import _expanded_ref

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


@pytest.mark.parametrize("scale", SCALES)
def test_fp8_rows(scale):
    w = W.make("f8", [300, 64, 1, 129], [1] * 4, 16, 64, "bf16", seed=86)
    w.softmax_scale = scale
    s = MlaDecodeStep(w, device=DEV)
    s.fp8_setup(0.02)
    s.fp8_populate()
    s.absorb()
    s.decode_paged_combine_fp8()
    s.out_proj()
    assert s.device_status()[0][0] == 0
    codes, k_rot = O.fp8_latent_rows(w.c_kv_raw, w.k_pe_raw, w.kv_positions, w.rms_weight, w.rms_eps, w.rope_base, 0.02)
    rows = np.concatenate([O.e4m3_decode(codes) * 0.02, k_rot], -1)
    q_abs = O.absorb_q(w.q_nope, w.q_pe, w.q_positions, w.W_uk, w.rope_base)
    ref = np.zeros((w.num_q, w.num_heads, 128))
    for b in range(w.batch):
        tr, qr = w.token_range(b), w.q_range(b)
        o, _ = O.latent_attention(q_abs[qr], rows[tr], w.q_positions[qr], scale)
        ref[qr] = O.out_proj(o, w.W_uv)
    assert_close(to_f64(s.out), ref, "bf16", "fp8")


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("name", ["tails_bs64", "bs16_h32", "h128", "empty_rows", "chunks"])
def test_page_scaled_rows(name, scale):
    w, s = page8._step(name, with_mass=True)
    w.softmax_scale = s.cfg.softmax_scale = scale
    m0 = s.p8_mass.cpu().double().numpy()
    s.page8_decode(0.75)
    assert page8.status_bits(s.p8_ws) == 0
    rows = page8.oracle_rows(s)
    page8.check_out(w, s, s.out, rows)
    q = to_f64(s.q_abs)
    _, want = P.decode(q, np.nan_to_num(rows), w.block_table, w.seq_lens, w.query_start_loc, scale,
                       to_f64(s.W_uv), m0, 0.75)
    size = abs(scale) * max(float(np.einsum("nhk,tk->nht", np.abs(q[w.q_range(b)]),
                                            np.abs(O.gather_paged(rows, w.block_table[b], int(w.seq_lens[b]), w.block_size))).max())
                            for b in range(w.batch) if w.q_range(b).stop > w.q_range(b).start)
    tol = (2.0 ** -18 * size + 2.0 ** -20) * np.abs(want)    # (the mass tests' own)
    assert np.all(np.abs(s.p8_mass.cpu().double().numpy() - want) <= tol)
