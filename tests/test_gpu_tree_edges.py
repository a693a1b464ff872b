"""The speculative step's operators where they could go wrong: what no listed use
reaches every day. Helpers and tolerances are those of test_gpu_tree.py."""

import numpy as np
import pytest
import torch

import test_gpu_tree
from mla_latent_kv_03_gb300 import libmla as L
from mla_latent_kv_03_gb300 import workloads as W
from mla_latent_kv_03_gb300.step import MlaDecodeStep
from oracle import tree_oracle as T
from test_gpu_tree import DEV, SCALE, Batch, Verify, bits, dev, random_tree

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


def test_decode_of_a_share_whose_q_blocks_pass_32_bits():
    """One cluster for 1,024 rows of 128 heads over 131,200 tokens (of 70 pages, again and
    again): a share of 2,099,200 units, times 1,024 q-blocks."""
    H, T_, n, bs = 128, 1024, 131200, 64
    cfg = L.make_config(H, bs, "bf16", num_ctas=2)
    g = torch.Generator(DEV).manual_seed(5)
    cache = torch.randn(70, bs, 576, device=DEV, generator=g).bfloat16()
    q = (torch.randn(T_, H, 576, device=DEV, generator=g) * 0.4).bfloat16()
    W_uv = (torch.randn(H, 512, 128, device=DEV, generator=g) * 512 ** -0.5).bfloat16()
    table = (torch.arange(n // bs, device=DEV, dtype=torch.int32) * 3 % 70)[None]
    mask = dev(T.words(np.tril(np.ones((T_, T_), bool)), 16), torch.int64)
    ws = torch.empty(L.mla_tree_decode_workspace_size(cfg, T_, 1), dtype=torch.uint8, device=DEV)
    L.mla_workspace_init(ws)
    out = torch.full((T_, H, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    L.mla_tree_decode(cfg, q, cache, table, dev([n], torch.int32), dev([0, T_], torch.int32), mask, W_uv, ws, out)
    assert bits(ws) == 0 and bool(out.isfinite().all())
    kv = cache[table[0].long()].reshape(n, 576).double()
    for r, h in ((0, 0), (1, 127), (500, 64), (1022, 3), (1023, 127)):
        rows = kv[:n - T_ + r + 1]
        s, part = (SCALE * (x @ q[r, h].double()[:c]) for x, c in ((rows, 576), (rows[:, :256], 256)))
        half = float(torch.maximum(part.abs(), (s - part).abs()).max())
        p = torch.softmax(s, 0)
        w = W_uv[h].double()
        want, size = p @ rows[:, :512] @ w, p @ rows[:, :512].abs() @ w.abs()
        bound = 2.0 ** -8 * want.abs() + (2 * 2.0 ** -8 + 2 * 2.0 ** -11 * half + 2.0 ** -11) * size
        assert bool(((out[r, h].double() - want).abs() <= bound).all()), (r, h)
        # (the output is far below that bound, which takes every rounding one way)
        assert float((out[r, h].double() - want).norm() / want.norm()) <= 5e-3


@pytest.mark.parametrize("scale", [-0.072, -0.5, 0.0, 1e-38, 0.9])
def test_decode_of_any_scale(scale, monkeypatch):
    """Tokens that are masked, not there or in a page out of range weigh nothing whatever
    the scale; a row that sees nothing is zero."""
    monkeypatch.setattr(test_gpu_tree, "SCALE", scale)
    b = Batch([(70, 9), (0, 3), (300, 65), (0, 12), (1, 1)], bs=32, seed=51)
    rng = np.random.default_rng(3)
    b.masks = [rng.random(m.shape) < 0.4 for m in b.masks]
    b.masks[1][1] = b.masks[3][:, 4:] = False
    b.cfg.softmax_scale = scale
    b.fill().decode()
    assert bits(b.ws) == 0
    b.check()
    assert not b.out[b.qsl[1] + 1].any()


# Columns of the latents and of the rope key, in either CTA's half.
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("col", [3, 300, 515, 560])
@pytest.mark.parametrize("place", [2, 64 * 5 + 7, 64 * 7 - 2, 64 * 7 + 4])
def test_decode_makes_rows_that_see_a_token_that_is_not_finite_nan(value, col, place):
    """In the first tile, in one that every row sees whole, and in the tree's own tiles:
    every output of a row that sees the token is NaN, the others are what they were. With
    one part a row and with several, merged in a kernel of their own and in the projection."""
    past, trees = 64 * 7 - 1, [[-1, 0, 0, 1, 2, 4, 3, 5]]
    for more, num_ctas in ((0, 2), (0, 0), (5, 6), (60, 0)):
        b = Batch([(past, 8)] + [(90, 1)] * more, trees=trees + [[-1]] * more, seed=71, num_ctas=num_ctas).fill()
        want = b.decode().clone()
        b.cache[int(b.table[0, place // 64]), place % 64, col] = value
        got = b.decode()
        seen = b.masks[0][:, place - past] if place >= past else np.ones(8, bool)
        for r in range(b.nq):
            if r < 8 and seen[r]:
                assert got[r].isnan().all(), r
            else:
                assert torch.equal(got[r], want[r]), r


@pytest.mark.parametrize("heads,seqs,behind", [
    (16, [(100, 5), (37, 6)], 21),                       # 512 (row, head)s: merged by themselves
    (16, [(100, 5), (37, 6)], 37),                       # where they are projected: 8 rows a CTA
    (128, [(700, 2), (5, 1), (0, 2)], 15),               # 16
    (16, [(300, 7)] * 40, 11), (16, [(1500, 3), (70, 30)], 380), (128, [(700, 2), (0, 3)], 35),   # 32
])
def test_decode_of_rows_behind_the_last_sequence(heads, seqs, behind):
    """Queries and masks of rows that no sequence has may hold anything: zeros there, and
    the others are what they are without them (bit by bit below 768 (row, head)s, from
    where on the parts are added in another order)."""
    b = Batch(seqs, heads=heads, seed=73).fill()
    want = b.decode().clone()
    b.check()
    n = b.nq + behind
    q = torch.full((n, heads, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    q[:b.nq] = b.t_q
    mask = torch.full((n, 1), -1, dtype=torch.int64, device=DEV)
    mask[:b.nq] = b.t_mask
    out = torch.full((n, heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((L.mla_tree_decode_workspace_size(b.cfg, n, len(seqs)),), 255, dtype=torch.uint8, device=DEV)
    L.mla_workspace_init(ws)
    L.mla_tree_decode(b.cfg, q, b.cache, b.t_table, b.t_lens, b.t_qsl, mask, b.t_W, ws, out)
    assert bits(ws) == 0 and not out[b.nq:].any()
    b.check(out[:b.nq])
    if n * heads < 768:
        assert torch.equal(out[:b.nq], want)


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


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [600, 9001])
def test_verify_of_values_that_are_no_probabilities(drawn, V):
    """NaN and what lies outside of [0, 1] in the target's rows, NaN and infinities in the
    draft's: the walk and the next token of every sequence are the definition's."""
    v = Verify([[-1, 0, 0, 0, 1, 1]] * 8, V, drawn, seed=9, near=1.0)
    v.u[:] = np.linspace(0.05, 0.999, len(v.u), dtype=np.float32)[::-1]
    n, rng = len(v.u), np.random.default_rng(3)
    for value in (np.nan, -1.0, np.inf, -np.inf):
        v.p[rng.integers(0, n, 60), rng.integers(0, V, 60)] = value if value != np.inf else 0.5
    for value in (np.nan, np.inf):
        v.q[rng.integers(0, n, 200), rng.integers(0, V, 200)] = value
    v.p[6:12, ::2] = np.nan
    v.q[12:18, 1::3] = np.nan
    v.p[18:24], v.p[18:24, 77] = 0, 2.0    # one token has all, which is more than 1
    v.q[24:30] = np.inf                    # a first rejection leaves nothing
    v.u[[31, 37]] = 0                      # accepted, if the target has any weight there
    lens = v.run().check()
    assert (lens > 1).any() and (lens == 1).any()
    assert bits(v.status) == 0


# --------------------------------------------------------- the step as a whole
def tree_step_of(seqs, t, seed):
    """A MlaDecodeStep whose sequences have `past` tokens and trees of t rows, with pages for
    three steps."""
    w = W.make("trees", [p + 3 * t for p in seqs], [t] * len(seqs), 16, 16, "bf16", seed)
    s = MlaDecodeStep(w, cache_fill=3.0)
    rng = np.random.default_rng(seed)
    trees = [random_tree(rng, t, 3) for _ in seqs]
    s.tree_setup(sum(trees, []))
    s.tr_lens.copy_(dev([p + t for p in seqs], torch.int32))
    return w, s, trees


@pytest.mark.parametrize("side", [False, True])
def test_step_of_fewer_rows_than_it_has_room_for(side):
    """Rows behind the last sequence write nothing, neither in a first step nor behind one
    in which they belonged to a sequence."""
    past, t = [40, 7, 20], 8
    for first in (True, False):
        w, s, trees = tree_step_of(past, t, 61)
        stream = torch.cuda.Stream() if side else None
        if not first:
            s.tree_step(stream)
            torch.cuda.synchronize()
        s.cache.fill_(3.0)
        # (trees of 8 and 5 rows; the last sequence has none, and 11 rows are nobody's)
        s.query_start_loc.copy_(dev([0, 8, 13, 13], torch.int32))
        s.tr_lens.copy_(dev([48, 12, 20], torch.int32))
        torch.cuda.synchronize()
        s.tree_step(stream)
        torch.cuda.synchronize()
        assert s.device_status() == ((0, 0), (0, 0)) and bits(s.tr_ws) == 0
        written = (s.cache != 3.0).any(-1).view(-1).nonzero()[:, 0].tolist()
        want = [int(w.block_table[b][j // 16]) * 16 + j % 16 for b, k in ((0, 8), (1, 5)) for j in range(past[b], past[b] + k)]
        assert written == sorted(want)
        assert not s.out[13:].any()


def test_step_of_a_sequence_that_outgrew_its_table():
    """It is flagged, and neither its cache nor its length is lost; the others go on."""
    past, t = [40, 7, 20], 8
    w, s, trees = tree_step_of(past, t, 62)
    room = w.block_table.shape[1] * 16
    full = room - 3                       # (sequence 0's table is full, of the longest)
    s.tr_lens.copy_(dev([full + t, 7 + t, 20 + t], torch.int32))
    before = s.cache.clone()
    V = 50
    v = Verify(trees, V, True, seed=1, near=0.1)
    args = [dev(x, k) for x, k in ((v.p, torch.float32), (v.q, torch.float32), (v.tok, torch.int32),
                                   (v.u, torch.float32), (v.f, torch.float32))]
    at = np.array([7, 20])
    for step in range(2):
        s.tree_step()
        s.tree_accept(*args, t)
        assert bits(s.status) == L.DEV_BAD_SEQ and bits(s.tr_ws) == L.DEV_BAD_SEQ
        kept = np.array([len(T.verify(v.p[r], v.q[r], v.tok[r], trees[b], v.u[r], v.f[b])[0])
                         for b, r in ((1, slice(8, 16)), (2, slice(16, 24)))])
        at = at + kept
        assert s.tr_lens.tolist() == [full + t, at[0] + t, at[1] + t]
    own = torch.from_numpy(w.block_table[0][w.block_table[0] >= 0].astype(np.int64)).to(DEV)
    assert torch.equal(s.cache[own], before[own])


def test_step_with_trees_of_other_sizes_than_the_first():
    """The lengths follow the rows that the sequences have now."""
    past, t = [40, 7, 20], 8
    w, s, trees = tree_step_of(past, t, 63)
    s.query_start_loc.copy_(dev([0, 8, 13, 13], torch.int32))
    s.tr_lens.copy_(dev([48, 12, 20], torch.int32))
    v = Verify([trees[0], trees[1][:5], []], 50, True, seed=2, near=0.1)
    pad = lambda x: np.concatenate([x, np.zeros((w.num_q - 13,) + x.shape[1:], x.dtype)])  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    s.tree_step()
    path, n, nxt = s.tree_accept(dev(pad(v.p), f32), dev(pad(v.q), f32), dev(pad(v.tok), i32), dev(pad(v.u), f32),
                                 dev(v.f, f32), t)
    assert s.device_status() == ((0, 0), (0, 0))
    want = [T.verify(v.p[r], v.q[r], v.tok[r], v.trees[b], v.u[r], v.f[b]) for b, r in ((0, slice(0, 8)), (1, slice(8, 13)))]
    assert n.tolist() == [len(want[0][0]), len(want[1][0]), 0] and nxt.tolist() == [want[0][1], want[1][1], -1]
    assert s.tr_lens.tolist() == [40 + int(n[0]) + 8, 7 + int(n[1]) + 5, 20]
