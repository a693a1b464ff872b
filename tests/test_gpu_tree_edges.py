"""The speculative step's operators where they could go wrong: what no listed use
reaches every day. Helpers and tolerances are those of test_gpu_tree.py."""

import numpy as np
import pytest
import torch

from mla_latent_kv_03_gb300 import libmla as L
from test_gpu_tree import Batch, Verify, bits, random_tree

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


# ---------------------------------------------------------------------- verify
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V,sizes", [
    (33000, [1, 400, 2, 0, 1, 150, 5, 0, 7]),            # clusters of 16
    (9000, [1, 100, 0, 3] * 15),                         # of 4
    (20000, [20] * 20 + [0] * 17),                       # of 8
])
def test_verify_clusters_of_uneven_sequences(drawn, V, sizes):
    """Sequences without rows, of one row and of many next to one another, call after
    call: CTAs of a cluster start and gather at different times."""
    rng = np.random.default_rng(V)
    v = Verify([random_tree(rng, n, 3) for n in sizes], V, drawn, seed=V, near=0.3)
    v.run().check()
    first = [t.clone() for t in (v.path, v.lens, v.nxt)]
    for _ in range(5):
        v.run()
        assert bits(v.status) == 0
        assert all(torch.equal(a, b) for a, b in zip((v.path, v.lens, v.nxt), first))
    # entries that do not ascend: that cluster leaves at once, the others do not
    keep, v.qsl = v.qsl, v.qsl.copy()
    v.qsl[2] = -1
    v.run()
    assert bits(v.status) == L.DEV_BAD_SEQ
    assert v.lens[1:3].tolist() == [0, 0] and v.nxt[1:3].tolist() == [-1, -1]
    assert all(torch.equal(a[3:], b[3:]) for a, b in zip((v.path, v.lens, v.nxt), first))
    v.qsl = keep
