"""GPU: the page-scaled 8-bit cache and eviction at the ends of their range:
the output's precision in every form, positions up to 2^31, NaN and infinities
beside what they must not reach, and the calls that follow an eviction."""

import numpy as np
import pytest
import torch

from _helpers import to_f64
from mla_latent_kv_03_gb300 import libmla as L
from mla_latent_kv_03_gb300 import workloads as W
from mla_latent_kv_03_gb300.step import MlaDecodeStep
from test_gpu_page8 import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L.load()


# -------------------------------------------------------------- precision
@pytest.mark.parametrize("heads,rows", [(16, 1), (16, 2), (32, 1), (128, 1)])
def test_weights_are_held_to_eleven_bits(heads, rows):
    """Every latent is 1, so an output is its column's sum of W_uv times the sum
    of the weights as held over the sum as they are: off by half a step of f16,
    2^-11, at most. The 128 columns' sums lie 2^-14 apart over one step of bf16
    (2^-7), where the mean of their roundings is 2^-15 at most."""
    lens = [rows + k % 9 for k in range(48)]
    w = W.make("p8_weights", lens, [rows] * 48, heads, 16, "bf16", 40 + heads)
    w.c_kv_raw[:] = 1.0
    column = 1.25 + (np.arange(128) + 0.5) * 2.0 ** -14
    w.W_uv[:] = 0.0
    w.W_uv[:, 0] = 1.25
    w.W_uv[:, 1] = column - 1.25
    s = MlaDecodeStep(w, device=DEV)
    s.page8_setup()
    s.page8_populate()
    s.absorb()
    s.page8_decode()
    torch.cuda.synchronize()
    off = to_f64(s.out).mean(-1) / column.mean() - 1
    assert np.abs(off).max() <= 2.0 ** -11 + 2.0 ** -14, np.abs(off).max()
