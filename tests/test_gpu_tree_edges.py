"""The speculative step's operators where they could go wrong: what no listed use
reaches every day. Helpers and tolerances are those of test_gpu_tree.py."""

import pytest
import torch

from mla_latent_kv_03_gb300 import libmla as L
from test_gpu_tree import Batch, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L.load()


# ---------------------------------------------------------------------- decode
@pytest.mark.parametrize("heads,seqs,num_ctas", [
    (16, [(0, 1), (3, 2), (60, 4), (40, 8)] * 60, 4),    # 120 segments of a tile in a share
    (16, [(5, 1)] * 300 + [(500, 2)] * 3 + [(9, 8)] * 50, 6),
    (128, [(10, 3), (1, 1), (0, 5)] * 8, 2),             # one share of all
    (64, [(20, 40)] * 3 + [(64, 1)] * 20, 0),
])
def test_decode_of_segments_of_one_tile(heads, seqs, num_ctas):
    """A segment of a tile takes three stages of the ring of four."""
    b = Batch(seqs, heads=heads, seed=heads + len(seqs), num_ctas=num_ctas).fill()
    b.decode()
    assert bits(b.ws) == 0
    b.check()
