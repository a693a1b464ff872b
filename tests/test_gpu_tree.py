"""GPU parity of the speculative step (plan, attention, verification, commit)
against the fp64 oracle.

Tolerances, fixed before the first run:
  plan, verify, commit   equal;
  out       bf16. Half a step of the result, 2^-8 |out|. A weight is rounded to
            bf16, 2^-8 of it, and the sum of the weights by as much at most: twice
            2^-8 of g = sum_t p_t |v_t| |W| in the worst case. Half of a score's sum
            is rounded to f16, 2^-11 of it: with s the largest half score of a row
            (in units of the exponent), a weight and the weights' sum are off by
            2^-11 s each. fp32 sums of 576 products (2^-18 of sum |q||k| at most,
            below 2^-12 of s for these inputs), latents held to 16 bits, exp2:
            2^-11 of g together. Beyond that bound for each element, rel-L2 <= 5e-3.
"""

import numpy as np
import pytest
import torch

from _helpers import to_f64
from mla_latent_kv_03_gb300 import libmla as L
from mla_latent_kv_03_gb300 import workloads as W
from mla_latent_kv_03_gb300.step import MlaDecodeStep
from oracle import tree_oracle as T

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L.load()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


def bits(word):
    return L.mla_get_device_status(word)[1]


def random_tree(rng, n, spread):
    return [-1] + [int(rng.integers(max(0, i - 1 - spread), i)) for i in range(1, n)] if n else []


class Batch:
    """Sequences of (past, rows), their trees and a paged cache whose unwritten
    places hold NaN."""

    def __init__(self, seqs, heads=16, bs=64, seed=0, spread=3, words=None, num_ctas=0, trees=None, spare=1):
        self.rng = rng = np.random.default_rng(seed)
        self.seqs, self.H, self.bs = seqs, heads, bs
        self.trees = trees or [random_tree(rng, t, spread) for _, t in seqs]
        self.lens = np.array([p + t for p, t in seqs], np.int64)
        self.q_lens = np.array([t for _, t in seqs], np.int64)
        self.qsl = np.concatenate([[0], np.cumsum(self.q_lens)])
        self.nq = int(self.qsl[-1])
        most = max(1, int(max(-(-n // bs) for n in self.lens)))
        need = [-(-int(n) // bs) for n in self.lens]
        self.nb = sum(need) + spare
        perm, at = rng.permutation(self.nb), 0
        self.table = np.full((len(seqs), most), -1, np.int64)
        for b, k in enumerate(need):
            self.table[b, :k] = perm[at:at + k]
            at += k
        self.words = words or max(1, -(-int(self.q_lens.max()) // 64))
        self.masks = [T.ancestors(t) for t in self.trees]
        self.cfg = L.make_config(heads, bs, "bf16", num_ctas=num_ctas)
        self.t_lens, self.t_qsl = dev(self.lens, torch.int32), dev(self.qsl, torch.int32)
        self.t_table = dev(self.table, torch.int32)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def fill(self, sharp=1.0):
        rng = self.rng
        self.rows = [W.round_to_dtype(rng.standard_normal((int(n), 576)), "bf16") for n in self.lens]
        cache = np.full((self.nb, self.bs, 576), np.nan, np.float32)
        for b, r in enumerate(self.rows):
            for t in range(len(r)):
                cache[self.table[b, t // self.bs], t % self.bs] = r[t]
        self.cache = dev(cache, torch.bfloat16)
        size = np.concatenate([np.full(512, 0.4), np.ones(64)]) * sharp
        self.q = W.round_to_dtype(rng.standard_normal((self.nq, self.H, 576)) * size, "bf16")
        self.W_uv = W.round_to_dtype(rng.standard_normal((self.H, 512, 128)) * 512 ** -0.5, "bf16")
        self.t_q, self.t_W = dev(self.q, torch.bfloat16), dev(self.W_uv, torch.bfloat16)
        self.out = torch.full((self.nq, self.H, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        n = L.mla_tree_decode_workspace_size(self.cfg, self.nq, len(self.seqs))
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        L.mla_workspace_init(self.ws)
        return self

    def mask_words(self):
        out = np.zeros((self.nq, self.words), np.int64)
        for b, m in enumerate(self.masks):
            if len(m):
                out[self.qsl[b]:self.qsl[b + 1]] = T.words(m, self.words)
        return out

    def decode(self, stream=None):
        self.t_mask = dev(self.mask_words(), torch.int64)
        L.mla_tree_decode(self.cfg, self.t_q, self.cache, self.t_table, self.t_lens, self.t_qsl, self.t_mask,
                          self.t_W, self.ws, self.out, stream=stream)
        return self.out

    def check(self, got=None, seqs=None, heads=None):
        got = to_f64(self.out if got is None else got)
        num = den = 0.0
        hs = np.arange(self.H) if heads is None else np.asarray(heads)
        for b in range(len(self.seqs)) if seqs is None else seqs:
            q = slice(self.qsl[b], self.qsl[b + 1])
            if q.stop == q.start:
                continue
            ref, g, half = T.attend(self.q[q][:, hs], self.rows[b], self.masks[b], SCALE, self.W_uv[hs])
            bound = 2.0 ** -8 * np.abs(ref) + (2 * 2.0 ** -8 + (2 * 2.0 ** -11) * half[..., None] + 2.0 ** -11) * g
            d = np.abs(got[q][:, hs] - ref)
            assert np.all(d <= bound + 1e-30), (b, float((d - bound).max()))
            num, den = num + float((d ** 2).sum()), den + float((ref ** 2).sum())
        assert den == 0 or (num / den) ** 0.5 <= 5e-3, (num / den) ** 0.5
        return (num / den) ** 0.5 if den else 0.0


# ------------------------------------------------------------------------ plan
@pytest.mark.parametrize("seqs,bs,words,spread", [
    ([(5, 1)], 16, 1, 0), ([(0, 3), (100, 8), (63, 1), (15, 2)], 16, 1, 2),
    ([(1000, 64), (0, 64), (7, 63)], 64, 1, 40), ([(50, 65), (0, 128), (64, 1)], 32, 2, 0),
    ([(9, 1024), (0, 700), (5, 0), (3, 1)], 64, 16, 0), ([(9, 1000), (128, 333)], 16, 16, 999),
    ([(31, 10)] * 70, 32, 3, 4),
])
def test_plan(seqs, bs, words, spread):
    b = Batch(seqs, bs=bs, words=words, spread=spread, seed=len(seqs))
    n = b.nq + 3   # (rows that no sequence has are left as they were)
    mask = torch.full((n, words), 77, dtype=torch.int64, device=DEV)
    pos = torch.full((n,), 77, dtype=torch.int32, device=DEV)
    slots = torch.full((n,), 77, dtype=torch.int64, device=DEV)
    parents = dev([p for t in b.trees for p in t] + [5] * 3, torch.int32)
    L.mla_tree_plan(b.cfg, parents, b.t_lens, b.t_qsl, b.t_table, b.nb, mask, pos, slots, dev_status=b.status)
    assert bits(b.status) == 0
    assert np.array_equal(mask.cpu().numpy()[:-3], b.mask_words())
    want = np.concatenate([p + T.depths(t) for (p, _), t in zip(seqs, b.trees)])
    assert np.array_equal(pos.cpu().numpy()[:-3], want)
    at = [b.table[i, j // bs] * bs + j % bs for i, (p, t) in enumerate(seqs) for j in range(p, p + t)]
    assert np.array_equal(slots.cpu().numpy()[:-3], at)
    assert (mask[-3:] == 77).all() and (pos[-3:] == 77).all() and (slots[-3:] == 77).all()


def test_plan_flags_bad_sequences():
    b = Batch([(10, 4), (0, 4), (20, 4), (3, 4), (60, 70), (5, 3)], bs=16, words=1, spread=1)
    parents = [list(t) for t in b.trees]
    parents[0][2] = 2                    # not before its child
    parents[1][1] = -2
    table, lens = b.table.copy(), b.lens.copy()
    lens[2] = 3                          # more rows than tokens
    table[3, 0] = b.nb                   # a page out of range
    n = b.nq
    mask = torch.full((n, 1), 77, dtype=torch.int64, device=DEV)
    pos = torch.full((n,), 77, dtype=torch.int32, device=DEV)
    slots = torch.full((n,), 77, dtype=torch.int64, device=DEV)
    L.mla_tree_plan(b.cfg, dev(sum(parents, []), torch.int32), dev(lens, torch.int32), b.t_qsl,
                    dev(table, torch.int32), b.nb, mask, pos, slots, dev_status=b.status)
    assert bits(b.status) == L.DEV_BAD_SEQ | L.DEV_BAD_BLOCK
    m, p, s = mask.cpu().numpy()[:, 0], pos.cpu().numpy(), slots.cpu().numpy()
    for i in (0, 1, 2, 4):               # (4: more rows than the mask has bits)
        r = slice(b.qsl[i], b.qsl[i + 1])
        assert not m[r].any() and not p[r].any() and (s[r] == -1).all()
    r = slice(b.qsl[3], b.qsl[4])
    assert (s[r] == -1).all() and m[r].all() and p[r][0] == 3
    r = slice(b.qsl[5], b.qsl[6])
    assert (s[r] >= 0).all() and p[r][0] == 5


# ---------------------------------------------------------------------- decode
@pytest.mark.parametrize("heads,bs,seqs,num_ctas", [
    (16, 64, [(40, 1)], 0),
    (16, 16, [(327, 6)], 0),
    (16, 64, [(0, 1), (0, 8), (63, 1), (64, 1), (60, 8), (128, 5)], 0),
    (16, 32, [(1, 2), (127, 3), (5, 0), (129, 17), (1000, 4)], 0),
    (16, 64, [(300, 65), (10, 130), (0, 64)], 0),
    (32, 16, [(200, 9), (77, 33), (0, 12)], 0),
    (64, 64, [(500, 3), (64, 2), (191, 1)], 0),
    (128, 32, [(700, 4), (30, 1), (0, 5)], 0),
    (16, 64, [(900, 8)] * 5, 2),
    (16, 16, [(900, 21), (3, 40), (444, 1)], 6),
    (128, 64, [(640, 5), (800, 3)], 10),
])
def test_decode_matches_oracle(heads, bs, seqs, num_ctas):
    b = Batch(seqs, heads=heads, bs=bs, seed=heads + bs, num_ctas=num_ctas).fill()
    b.decode()
    assert bits(b.ws) == 0
    b.check()


@pytest.mark.parametrize("sharp", [0.05, 4.0, 30.0])
def test_decode_flat_and_sharp_scores(sharp):
    b = Batch([(500, 9), (70, 12)], seed=7).fill(sharp)
    b.decode()
    b.check()


def test_decode_maxima_that_grow():
    """Later tokens outgrow the earlier ones again and again: O is rescaled."""
    b = Batch([(800, 8)], seed=3, num_ctas=2).fill()
    for t in range(len(b.rows[0])):
        b.rows[0][t] *= 0.05 + t / 400
    b.rows[0] = W.round_to_dtype(b.rows[0], "bf16")
    cache = b.cache.cpu().float().numpy()
    for t in range(len(b.rows[0])):
        cache[b.table[0, t // 64], t % 64] = b.rows[0][t]
    b.cache = dev(cache, torch.bfloat16)
    b.decode()
    b.check()


def test_decode_any_mask_and_rows_that_see_nothing():
    b = Batch([(0, 12), (100, 70), (0, 3)], bs=32, seed=5)
    rng = np.random.default_rng(1)
    b.masks = [rng.random((t, t)) < 0.3 for _, t in b.seqs]
    b.masks[0][4] = b.masks[2][:] = False
    b.masks[1][:, 64] = True
    b.fill().decode()
    b.check()
    assert not b.out[4].any() and not b.out[b.qsl[2]:].any()


def test_decode_ignores_bits_behind_the_rows():
    b = Batch([(33, 5), (50, 9)], seed=2, words=2).fill()
    want = b.decode().clone()
    m = b.mask_words()
    for i, t in enumerate(b.q_lens):
        m[b.qsl[i]:b.qsl[i + 1], 0] |= -1 << int(t)
        m[b.qsl[i]:b.qsl[i + 1], 1] = -1
    L.mla_tree_decode(b.cfg, b.t_q, b.cache, b.t_table, b.t_lens, b.t_qsl, dev(m, torch.int64), b.t_W, b.ws, b.out)
    assert torch.equal(b.out, want)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("col", [3, 300, 560])
def test_decode_a_token_that_is_not_finite_touches_its_rows_only(value, col):
    trees = [[-1, 0, 0, 1, 2, 4]]
    b = Batch([(70, 6)], trees=trees, seed=9).fill()
    want = b.decode().clone()
    place = 70 + 2                                        # row 2: seen by rows 2, 4 and 5
    b.cache[int(b.table[0, place // 64]), place % 64, col] = value
    got = b.decode().clone()
    for r in (0, 1, 3):
        assert torch.equal(got[r], want[r])
    for r in (2, 4, 5):
        if value != value:
            assert got[r].isnan().all()
        else:
            assert not got[r].isfinite().all(1).any() or col == 560


def test_decode_flags_and_skips():
    b = Batch([(40, 4), (200, 8), (10, 3), (90, 70), (20, 5)], bs=64, seed=11, words=1).fill()
    table, lens = b.table.copy(), b.lens.copy()
    lens[0] = 3                                           # more rows than tokens
    table[1, 1] = b.nb                                    # a page out of range: its tokens are not there
    lens[2] = table.shape[1] * 64 + 1                     # longer than its table
    b.masks[3] = b.masks[3][:, :64]                       # (4: more rows than bits)
    m = np.zeros((b.nq, 1), np.int64)
    for i in (0, 1, 2, 4):
        m[b.qsl[i]:b.qsl[i + 1]] = T.words(b.masks[i], 1)
    b.out.fill_(7.0)
    L.mla_tree_decode(b.cfg, b.t_q, b.cache, dev(table, torch.int32), dev(lens, torch.int32), b.t_qsl,
                      dev(m, torch.int64), b.t_W, b.ws, b.out)
    assert bits(b.ws) == L.DEV_BAD_SEQ | L.DEV_BAD_BLOCK
    for i in (0, 2, 3):
        assert not b.out[b.qsl[i]:b.qsl[i + 1]].any()
    rows = b.rows[1]
    b.rows[1] = np.concatenate([rows[:64], rows[128:]])
    b.check(seqs=[1, 4])
    # query_start_loc that does not ascend: zeros, and nothing else is touched
    qsl = b.qsl.copy()
    qsl[2] = 1
    L.mla_tree_decode(b.cfg, b.t_q, b.cache, b.t_table, b.t_lens, dev(qsl, torch.int32), dev(m, torch.int64), b.t_W,
                      b.ws, b.out)
    assert bits(b.ws) == L.DEV_BAD_SEQ and not b.out.any()


def test_decode_split_does_not_matter():
    outs = []
    for c in (0, 2, 4, 14, 40):
        b = Batch([(1500, 12), (300, 33), (64, 1), (0, 9)], heads=32, seed=21, num_ctas=c).fill()
        outs.append(to_f64(b.decode()))
    for o in outs[1:]:
        # two roundings of out, and of the weights, apart
        assert np.abs(o - outs[0]).max() <= 2 ** -6 * np.abs(outs[0]).max()


def test_decode_workspace_of_more_rows_streams_and_replay():
    b = Batch([(700, 8), (50, 3)], seed=13).fill()
    want = b.decode().clone()
    n = L.mla_tree_decode_workspace_size(b.cfg, 100, 9)
    assert n >= b.ws.numel()
    b.ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    L.mla_workspace_init(b.ws)
    side = torch.cuda.Stream()
    b.out.fill_(7.0)
    torch.cuda.synchronize()
    b.decode(stream=side)
    side.synchronize()
    assert torch.equal(b.out, want)
    # captured, then replayed with another step's lengths and masks
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.mla_tree_decode(b.cfg, b.t_q, b.cache, b.t_table, b.t_lens, b.t_qsl, b.t_mask, b.t_W, b.ws, b.out)
    b.out.fill_(7.0)
    g.replay()
    assert torch.equal(b.out, want)
    b.t_lens.copy_(torch.tensor([300, 20]))
    b.rows, b.lens = [b.rows[0][:300], b.rows[1][:20]], np.array([300, 20])
    b.masks = [np.tril(np.ones((8, 8), bool)), np.eye(3, dtype=bool)]
    b.t_mask.copy_(dev(b.mask_words(), torch.int64))
    g.replay()
    torch.cuda.synchronize()
    b.check()


@pytest.mark.parametrize("heads,seqs,num_ctas", [
    (16, [(5, 64)] * 5 + [(900, 40)], 0),                # many rows: some with all their tokens in one share
    (128, [(30, 9)] * 3 + [(700, 4)], 0),
    (16, [(3, 1), (200, 2), (0, 1), (64, 1)] * 120, 0),  # more sequences than a CTA's threads
    (16, [(7, 1024), (0, 900)], 0),                      # the widest masks
    (16, [(5200, 8)], 0),                                # more than 32 parts a row: few rows
    (16, [(0, 1)] * 15 + [(5200, 2)] + [(1, 1)] * 16, 0),  # and many
    (16, [(2500, 3), (0, 1), (90, 40)], 300),            # shares of a tile
])
def test_decode_of_many_rows_sequences_and_parts(heads, seqs, num_ctas):
    b = Batch(seqs, heads=heads, seed=len(seqs), num_ctas=num_ctas).fill()
    b.decode()
    assert bits(b.ws) == 0
    # (of the largest, the heads at the ends)
    b.check(heads=None if b.nq * heads * max(b.lens) < 2e7 else [0, heads - 1])


@pytest.mark.parametrize("heads,seqs", [
    (16, [(100, 8)] * 8), (16, [(5200, 2)] + [(0, 1)] * 50),          # 8 rows a CTA; more parts than lanes
    (128, [(90, 7)] * 3 + [(5, 1)]), (128, [(5200, 1)] + [(0, 1)] * 20),   # 16 rows
    (16, [(5200, 2)] + [(0, 1)] * 400), (16, [(70, 3), (0, 0), (3, 12)] * 40),   # 32 rows
    (64, [(200, 5), (0, 2)] * 9),
])
def test_decode_merged_where_it_is_projected(heads, seqs):
    b = Batch(seqs, heads=heads, seed=heads + len(seqs)).fill()
    b.masks = [m.copy() for m in b.masks]
    b.masks[-1][:] = False                     # rows that see nothing but the past
    b.decode()
    assert bits(b.ws) == 0
    b.check()


def test_decode_rows_behind_the_last_sequence():
    b = Batch([(100, 5), (37, 6)], seed=31).fill()
    b.decode()
    q = torch.full((b.nq + 21, 16, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    q[:b.nq] = b.t_q
    mask = torch.full((b.nq + 21, 1), -1, dtype=torch.int64, device=DEV)
    mask[:b.nq] = b.t_mask
    out = torch.full((b.nq + 21, 16, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((L.mla_tree_decode_workspace_size(b.cfg, b.nq + 21, 2),), 255, dtype=torch.uint8, device=DEV)
    L.mla_workspace_init(ws)
    L.mla_tree_decode(b.cfg, q, b.cache, b.t_table, b.t_lens, b.t_qsl, mask, b.t_W, ws, out)
    # (Not bit for bit what 11 rows alone give: with 512 (row, head)s or more the parts
    # are added one behind another, with fewer in four groups. Both are within the bound,
    # whose fp32 term counts any order.)
    b.check(out[:b.nq])
    assert not out[b.nq:].any() and bits(ws) == 0


def test_decode_of_pages_that_sequences_share():
    """Two sequences over the same pages, with trees of their own."""
    b = Batch([(150, 7), (150, 7)], seed=17, trees=[[-1, 0, 0, 1, 2, 2, 5], [-1, 0, 1, 2, 3, 4, 5]]).fill()
    b.rows[1] = b.rows[0]
    b.t_table[1] = b.t_table[0]
    b.decode()
    b.check()


def test_decode_on_two_streams_at_once():
    bs = [Batch([(1200, 8)] * 6, seed=41).fill(), Batch([(40, 60), (2000, 3)], heads=32, bs=16, seed=42).fill()]
    want = [b.decode().clone() for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    for b in bs:
        b.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s in zip(bs, streams):
            L.mla_tree_decode(b.cfg, b.t_q, b.cache, b.t_table, b.t_lens, b.t_qsl, b.t_mask, b.t_W, b.ws, b.out, stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bs, want):
        assert torch.equal(b.out, w) and bits(b.ws) == 0


def test_decode_and_commit_behind_four_gigabytes():
    b = Batch([(130, 8), (3, 5)], seed=19).fill()
    far = (1 << 32) // (64 * 1152) + 5                   # pages whose bytes begin past 2^32
    cache = torch.zeros((far + b.nb, 64, 576), dtype=torch.bfloat16, device=DEV)
    cache[far:] = b.cache
    want = b.decode().clone()
    table = torch.where(b.t_table >= 0, b.t_table + far, b.t_table)
    b.out.fill_(7.0)
    L.mla_tree_decode(b.cfg, b.t_q, cache, table, b.t_lens, b.t_qsl, b.t_mask, b.t_W, b.ws, b.out)
    assert torch.equal(b.out, want) and bits(b.ws) == 0
    path, n = dev([[0, 3, 5, 7], [1, 4, -1, -1]], torch.int32), dev([4, 2], torch.int32)
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    b.cache.nan_to_num_(0.0)
    cache.nan_to_num_(0.0)
    L.mla_tree_commit(b.cfg, b.cache[None], b.t_table, b.t_lens, b.t_qsl, path, n, new, dev_status=b.status)
    L.mla_tree_commit(b.cfg, cache[None], table, b.t_lens, b.t_qsl, path, n, new, dev_status=b.status)
    assert torch.equal(cache[far:], b.cache) and not cache[:far].any()
    assert new.tolist() == [134, 5] and bits(b.status) == 0


# ---------------------------------------------------------------------- verify
class Verify:
    def __init__(self, trees, V, drawn, seed=0, near=0.4, temp=1.5):
        self.rng = rng = np.random.default_rng(seed)
        self.trees, self.V = trees, V
        self.qsl = np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int64)
        n = int(self.qsl[-1])
        x = rng.standard_normal((n, V)) * temp
        soft = lambda a: (np.exp(a - a.max(1, keepdims=True)) / np.exp(a - a.max(1, keepdims=True)).sum(1, keepdims=True)).astype(np.float32)  # noqa: E731,E501
        self.p, self.q = soft(x), soft(x + near * rng.standard_normal((n, V)))
        self.tok = np.zeros(n, np.int64)
        for b, t in enumerate(trees):
            rank = {}
            for i, up in enumerate(t):
                if up < 0:
                    continue
                row = self.q[self.qsl[b] + up].astype(np.float64)
                if drawn:
                    self.tok[self.qsl[b] + i] = rng.choice(V, p=row / row.sum())
                else:
                    k = rank.get(up, 0)
                    rank[up] = k + 1
                    self.tok[self.qsl[b] + i] = np.argsort(-row, kind="stable")[k % V]
        self.drawn = drawn
        self.u, self.f = rng.random(n, dtype=np.float32), rng.random(len(trees), dtype=np.float32)
        self.max_path = max([1] + [int(T.depths(t).max()) + 1 for t in trees if t])

    def run(self, max_path=None):
        mp, B = max_path or self.max_path, len(self.trees)
        self.path = torch.full((B, mp), 77, dtype=torch.int32, device=DEV)
        self.lens = torch.full((B,), 77, dtype=torch.int32, device=DEV)
        self.nxt = torch.full((B,), 77, dtype=torch.int32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        f32, i32 = torch.float32, torch.int32
        L.mla_tree_verify(dev(self.p, f32), dev(self.q, f32) if self.drawn else None, dev(self.tok, i32),
                          dev([p for t in self.trees for p in t], i32), dev(self.qsl, i32), dev(self.u, f32),
                          dev(self.f, f32), self.path, self.lens, self.nxt, dev_status=self.status)
        return self

    def check(self, max_path=None):
        path, lens, nxt = (t.cpu().numpy() for t in (self.path, self.lens, self.nxt))
        for b, t in enumerate(self.trees):
            if not t:
                assert lens[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
                continue
            r = slice(self.qsl[b], self.qsl[b + 1])
            want, after = T.verify(self.p[r], self.q[r] if self.drawn else None, self.tok[r], t, self.u[r], self.f[b],
                                   max_path)
            assert path[b][:lens[b]].tolist() == want and (path[b][lens[b]:] == -1).all(), b
            assert nxt[b] == after, (b, nxt[b], after)
        return lens


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V,batch,nodes,spread", [
    (1, 3, 2, 0), (2, 5, 4, 3), (3, 40, 6, 5), (127, 9, 12, 4), (128, 2, 1, 0), (1001, 33, 16, 15),
    (4099, 4, 60, 8), (32000, 1, 26, 8), (50001, 3, 9, 3), (102400, 2, 6, 0),
])
def test_verify(drawn, V, batch, nodes, spread):
    rng = np.random.default_rng(V)
    v = Verify([random_tree(rng, nodes, spread) for _ in range(batch)], V, drawn, seed=V + nodes).run()
    v.check()
    assert bits(v.status) == 0


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_many_siblings_a_long_chain_and_ragged_trees(drawn):
    # every child of the root is asked before one is kept
    v = Verify([[-1] + [0] * 40, [-1] + list(range(300)), [], [-1], [-1, 0, -1, 2]], 300, drawn, seed=4, near=1.5).run()
    v.check()
    # a draft that is the target: the whole chain
    v = Verify([[-1] + list(range(700))], 64, True, seed=5, near=0.0).run()
    assert v.check()[0] == 701


def test_verify_most_rows_kept():
    v = Verify([[-1] + list(range(12))] * 6, 500, True, seed=8, near=0.1)
    for mp in (1, 2, 5):
        v.run(mp).check(mp)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_odd_values(drawn):
    v = Verify([[-1, 0, 0, 1]] * 5, 600, drawn, seed=6)
    v.p[0] = 0                           # no weight at all
    v.u[1:4] = 0.5
    v.p[4, 5:50], v.p[5, ::2] = np.nan, -1.0
    v.q[4, 100:200] = np.nan if drawn else 0
    v.p[8] = 0
    v.p[8, 599] = 1.0                    # the last token
    v.f[:] = [0.3, 0.0, np.float32(1 - 2 ** -24), 0.999, 0.5]
    v.q = np.where(np.isnan(v.q), np.float32(0), v.q) if not drawn else v.q
    v.run()
    path, lens, nxt = (t.cpu().numpy() for t in (v.path, v.lens, v.nxt))
    assert nxt[0] == -1 and lens[0] == 1 and bits(v.status) == L.DEV_BAD_TOKEN
    for b in range(2, 5):
        r = slice(4 * b, 4 * b + 4)
        want, after = T.verify(v.p[r], v.q[r] if drawn else None, v.tok[r], v.trees[b], v.u[r], v.f[b])
        assert path[b][:lens[b]].tolist() == want and nxt[b] == after
    assert 0 <= nxt[1] < 600 and not np.isnan(v.p[4][nxt[1]]) or lens[1] > 1


def test_verify_flags_bad_rows():
    v = Verify([[-1, 0, 0], [-1, 0, 1], [-1, 0]], 100, False, seed=3)
    v.u[:] = 0                            # every child that can be is kept
    v.tok[1], v.tok[2] = 100, 5
    v.run()
    assert bits(v.status) == L.DEV_BAD_TOKEN
    v.check()
    v.tok[1], v.trees[1][2] = 4, 2
    v.run()
    assert bits(v.status) == L.DEV_BAD_SEQ
    assert v.path.cpu().numpy()[1][:2].tolist() == [0, 1] and int(v.lens[1]) == 2
    v.trees[1][2], v.qsl = 1, np.array([0, 3, 6, 9])     # past the rows
    v.run()
    assert bits(v.status) == L.DEV_BAD_SEQ and int(v.lens[2]) == 0 and int(v.nxt[2]) == -1


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_pieces_of_several_rounds(drawn):
    """One CTA a sequence, whose warps' pieces the draw looks through in rounds."""
    v = Verify([[-1, 0]] * 160, 40000, drawn, seed=12).run()
    v.check()
    assert bits(v.status) == 0


def test_plan_verify_and_commit_captured_and_replayed():
    trees = [[-1, 0, 0, 1, 2, 2, 4], [-1, 0, 1, 2, 3, 4, 5], [-1, 0, 0, 0, 0, 0, 0]]
    past = [70, 0, 33]
    b = Batch([(p, 7) for p in past], trees=trees, seed=23)
    rng = np.random.default_rng(23)
    V = 777
    first = Verify(trees, V, True, seed=1, near=0.2)
    i32, f32 = torch.int32, torch.float32
    par = dev(sum(trees, []), i32)
    p, q, tok, u, f = dev(first.p, f32), dev(first.q, f32), dev(first.tok, i32), dev(first.u, f32), dev(first.f, f32)
    mask = torch.zeros((21, 1), dtype=torch.int64, device=DEV)
    pos = torch.zeros(21, dtype=i32, device=DEV)
    slots = torch.zeros(21, dtype=torch.int64, device=DEV)
    path = torch.zeros((3, 7), dtype=i32, device=DEV)
    n, nxt, new = (torch.zeros(3, dtype=i32, device=DEV) for _ in range(3))
    cache = torch.zeros((2, b.nb, 64, 576), dtype=torch.bfloat16, device=DEV)

    def calls():
        L.mla_tree_plan(b.cfg, par, b.t_lens, b.t_qsl, b.t_table, b.nb, mask, pos, slots, dev_status=b.status)
        L.mla_tree_verify(p, q, tok, par, b.t_qsl, u, f, path, n, nxt, dev_status=b.status)
        L.mla_tree_commit(b.cfg, cache, b.t_table, b.t_lens, b.t_qsl, path, n, new, dev_status=b.status)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for seed in (2, 3, 4):
        v = Verify(trees, V, True, seed=seed, near=0.2)
        for t, x in ((p, v.p), (q, v.q), (tok, v.tok), (u, v.u), (f, v.f)):
            t.copy_(dev(x, t.dtype))
        rows = rng.standard_normal((2, b.nb, 64, 576)).astype(np.float32)
        cache.copy_(dev(rows, torch.bfloat16))
        want = to_f64(cache).reshape(2, -1, 576)
        g.replay()
        torch.cuda.synchronize()
        assert bits(b.status) == 0 and np.array_equal(mask.cpu().numpy(), b.mask_words())
        for i, t in enumerate(trees):
            r = slice(7 * i, 7 * i + 7)
            kept, after = T.verify(v.p[r], v.q[r], v.tok[r], t, v.u[r], v.f[i])
            assert path[i].tolist() == kept + [-1] * (7 - len(kept)) and int(nxt[i]) == after
            assert int(n[i]) == len(kept) and int(new[i]) == past[i] + len(kept)
            at = np.array([b.table[i, j // 64] * 64 + j % 64 for j in range(past[i] + 7)])
            for layer in range(2):
                want[layer, at] = T.commit(want[layer, at], past[i], kept)
        assert np.array_equal(to_f64(cache).reshape(2, -1, 576), want)


# ---------------------------------------------------------------------- commit
@pytest.mark.parametrize("dtype,layers,bs,seqs", [
    ("bf16", 1, 16, [(333, 26)]), ("bf16", 27, 64, [(60, 8), (0, 8), (128, 5), (63, 1), (7, 0)]),
    ("f32", 3, 32, [(31, 40), (0, 2)]), ("fp8", 5, 16, [(15, 33), (2, 3)] * 4), ("bf16", 2, 64, [(10, 700)]),
])
def test_commit(dtype, layers, bs, seqs):
    b = Batch(seqs, bs=bs, seed=layers)
    cfg = L.make_config(16, bs, "f32" if dtype == "f32" else "bf16")
    cols = 640 if dtype == "fp8" else 576
    cache = b.rng.integers(0, 256, (layers, b.nb, bs, cols)).astype(np.float32)
    t_cache = dev(cache, {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8}[dtype])
    paths = []
    for _, t in b.seqs:
        paths.append(sorted(b.rng.choice(t, int(b.rng.integers(0, t + 1)), replace=False)) if t else [])
    paths[0] = list(range(1, b.seqs[0][1]))[:40] if b.seqs[0][1] > 1 else paths[0]   # every row by one
    mp = max(1, max(len(p) for p in paths))
    path = np.array([list(p) + [-1] * (mp - len(p)) for p in paths])
    new = torch.full((len(seqs),), 77, dtype=torch.int32, device=DEV)
    L.mla_tree_commit(cfg, t_cache, b.t_table, b.t_lens, b.t_qsl, dev(path, torch.int32),
                      dev([len(p) for p in paths], torch.int32), new, dev_status=b.status)
    assert bits(b.status) == 0
    want = cache.copy()
    for i, (past, t) in enumerate(seqs):
        at = np.array([b.table[i, j // bs] * bs + j % bs for j in range(past + t)], np.int64)
        flat = want.reshape(layers, -1, cols)
        for layer in range(layers):
            flat[layer, at] = T.commit(flat[layer, at], past, paths[i])
    assert np.array_equal(t_cache.float().cpu().numpy(), want)
    assert new.tolist() == [p + len(x) for (p, _), x in zip(seqs, paths)]


def test_commit_flags_and_leaves_alone():
    b = Batch([(20, 4), (20, 4), (20, 4), (20, 4), (14, 4)], bs=16, seed=1)
    cache = torch.randn(2, b.nb, 16, 576, device=DEV).bfloat16()
    want = cache.clone()
    path = np.array([[0, 2, 2], [0, 4, -1], [0, 2, -1], [1, 2, 3], [1, 2, 3]])
    lens, table = b.lens.copy(), b.table.copy()
    lens[2] = 2
    table[3, 1] = -1                     # places 16 and on of sequence 3
    table[4, 0] = b.nb                   # places 14 and 15 of sequence 4
    new = torch.zeros(5, dtype=torch.int32, device=DEV)
    L.mla_tree_commit(b.cfg, cache, dev(table, torch.int32), dev(lens, torch.int32), b.t_qsl, dev(path, torch.int32),
                      dev([3, 2, 2, 3, 3], torch.int32), new, dev_status=b.status)
    assert bits(b.status) == L.DEV_BAD_SLOT | L.DEV_BAD_SEQ | L.DEV_BAD_BLOCK
    assert new.tolist() == [20, 20, 0, 23, 17]
    page = int(table[4, 1])              # only place 16 <- 17 of sequence 4 can move
    want[:, page, 0] = want[:, page, 1]
    assert torch.equal(cache, want)


# --------------------------------------------------------- the step as a whole
def test_step_then_the_kept_path_is_a_plain_cache():
    """Two steps of a program: plan, write, absorb, attention, verification and
    commit; then plain decoding over the cache that is left equals decoding over
    a cache in which only the kept tokens were ever written."""
    seqs, t = [(100, 8), (30, 8), (0, 8)], 8
    w = W.make("trees", [p + 3 * t for p, _ in seqs], [t] * 3, 16, 64, "bf16", 5)
    rng = np.random.default_rng(2)
    trees = [random_tree(rng, t, 3) for _ in seqs]
    s = MlaDecodeStep(w, cache_fill=float("nan"))
    s.populate(include_new=False)
    past = np.array([p for p, _ in seqs])
    s.tree_setup(sum(trees, []))
    s.tr_lens.copy_(dev(past + t, torch.int32))
    V, kept = 300, [[] for _ in seqs]
    c_kv, k_pe = s.c_kv_new.clone(), s.k_pe_new.clone()
    for step in range(2):
        s.c_kv_new.copy_(torch.roll(c_kv, step, 0))
        s.k_pe_new.copy_(torch.roll(k_pe, step, 0))
        out = s.tree_step().clone()
        assert s.device_status() == ((0, 0), (0, 0)) and bits(s.tr_ws) == 0
        lens = past + t
        # the attention against the oracle, on the GPU's own cache and queries
        cache, q = to_f64(s.cache), to_f64(s.q_abs)
        for b in range(3):
            at = np.arange(lens[b])
            rows = cache[w.block_table[b][at // 64], at % 64]
            ref, g, half = T.attend(q[t * b:t * b + t], rows, T.ancestors(trees[b]), w.softmax_scale, to_f64(s.W_uv))
            bound = 2.0 ** -8 * np.abs(ref) + (2 * 2.0 ** -8 + 2 * 2.0 ** -11 * half[..., None] + 2.0 ** -11) * g
            assert np.all(np.abs(to_f64(out[t * b:t * b + t]) - ref) <= bound)
        v = Verify(trees, V, True, seed=step, near=0.2)
        path, n, nxt = s.tree_accept(dev(v.p, torch.float32), dev(v.q, torch.float32), dev(v.tok, torch.int32),
                                     dev(v.u, torch.float32), dev(v.f, torch.float32), t)
        path, n = path.cpu().numpy(), n.cpu().numpy()
        for b in range(3):
            r = slice(t * b, t * b + t)
            want, after = T.verify(v.p[r], v.q[r], v.tok[r], trees[b], v.u[r], v.f[b])
            assert path[b][:n[b]].tolist() == want and int(nxt[b]) == after
            kept[b] += [(step, t * b + j) for j in want]
        past = past + n
        assert s.tr_lens.tolist() == (past + t).tolist()
    # the same tokens written one behind another
    assert max(len(k) for k in kept) > 2
    plain = torch.full_like(s.cache, float("nan"))
    s2 = MlaDecodeStep(w)
    s2.cache = plain
    s2.populate(include_new=False)
    for b, rows in enumerate(kept):
        for j, (step, r) in enumerate(rows):
            at = seqs[b][0] + j
            slot = torch.tensor([int(w.block_table[b][at // 64]) * 64 + at % 64], device=DEV)
            L.mla_cache_write(s.cfg, torch.roll(c_kv, step, 0)[r:r + 1].contiguous(),
                              torch.roll(k_pe, step, 0)[r:r + 1].contiguous(),
                              torch.tensor([at], dtype=torch.int32, device=DEV), slot, s.rms_weight, plain)
    for b in range(3):
        at = np.arange(past[b])
        pages, places = torch.from_numpy(w.block_table[b][at // 64].astype(np.int64)), torch.from_numpy(at % 64)
        assert torch.equal(s.cache[pages, places], plain[pages, places])
