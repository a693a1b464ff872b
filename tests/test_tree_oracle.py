"""The oracle of the speculative step pinned by brute force and closed forms."""

import itertools

import numpy as np
import pytest

from oracle import mla_oracle as O
from oracle import tree_oracle as T


def test_masks_depths_and_words():
    parents = [-1, 0, 0, 1, 2, 3, -1]
    m = T.ancestors(parents)
    assert m[5].nonzero()[0].tolist() == [0, 1, 3, 5] and m[4].nonzero()[0].tolist() == [0, 2, 4]
    assert m[6].nonzero()[0].tolist() == [6]
    assert T.depths(parents).tolist() == [0, 1, 1, 2, 2, 3, 0] == (m.sum(1) - 1).tolist()
    chain = T.ancestors([-1] + list(range(69)))
    assert np.array_equal(chain, np.tril(np.ones((70, 70), bool)))
    w = T.words(chain, 2)
    assert w[69].tolist() == [-1, 63] and w[63].tolist() == [-1, 0] and w[5].tolist() == [63, 0]


def test_a_chain_is_causal_attention_and_branches_do_not_mix():
    rng = np.random.default_rng(3)
    q, rows, W = rng.standard_normal((4, 2, 576)), rng.standard_normal((9, 576)), rng.standard_normal((2, 512, 128))
    out, _, _ = T.attend(q, rows, T.ancestors([-1, 0, 1, 2]), 0.1, W)
    o, _ = O.latent_attention(q, rows, np.arange(5, 9), 0.1)
    assert np.allclose(out, O.out_proj(o, W), atol=1e-12)
    # a row of a tree has what it has alone behind its ancestors
    parents = [-1, 0, 0, 2]
    out, _, _ = T.attend(q, rows, T.ancestors(parents), 0.1, W)
    o, _ = O.latent_attention(q[3:], rows[[0, 1, 2, 3, 4, 5, 7, 8]], np.array([7]), 0.1)
    assert np.allclose(out[3], O.out_proj(o, W)[0], atol=1e-12)
    # nothing seen: zeros
    out, _, _ = T.attend(q, rows[:4], np.zeros((4, 4), bool), 0.1, W)
    assert not out.any()


@pytest.mark.parametrize("drawn", [True, False])
def test_kept_tokens_are_distributed_as_the_targets(drawn):
    """One root with two children over three tokens: over the drafted tokens and
    a grid of the uniforms, the first emitted token (an accepted child's or the
    drawn one) has the target's probabilities, to the grid's step."""
    p0 = np.array([0.5, 0.2, 0.3], np.float32)
    q0 = np.array([0.25, 0.6, 0.15], np.float32)
    n = 16
    grid = (np.arange(n) + 0.5) / n
    got = np.zeros(3)
    cases = itertools.product(range(3), range(3)) if drawn else [(1, 0)]
    for x1, x2 in cases:
        weight = float(q0[x1]) * float(q0[x2]) if drawn else 1.0
        for u1, u2, u3 in itertools.product(grid, grid, grid):
            target = np.stack([p0, p0, p0])
            draft = np.stack([q0, q0, q0]) if drawn else None
            path, nxt = T.verify(target, draft, [0, x1, x2], [-1, 0, 0], [0, u1, u2], u3)
            first = (x1, x2)[path[1] - 1] if len(path) > 1 else nxt
            got[first] += weight / n ** 3
    assert np.abs(got - p0).max() < 2.0 / n


def test_walks_by_hand():
    eye = np.eye(4, dtype=np.float32)
    tok, par = [0, 1, 2, 3], [-1, 0, 1, 2]
    # the target wants the chain: all kept, the next token is the leaf's
    target = np.stack([eye[1], eye[2], eye[3], eye[0]])
    assert T.verify(target, None, tok, par, [0.9] * 4, 0.5) == ([0, 1, 2, 3], 0)
    assert T.verify(target, None, tok, par, [0.9] * 4, 0.5, max_path=2) == ([0, 1], 2)
    # it wants something else at row 1: cut there
    target[1] = eye[0]
    assert T.verify(target, None, tok, par, [0.9] * 4, 0.5) == ([0, 1], 0)
    # siblings: the first is rejected and its weight is gone
    half = np.array([0, 0.5, 0.5, 0], np.float32)
    assert T.verify(np.stack([half] * 3), None, [0, 1, 2], [-1, 0, 0], [0, 0.6, 0.99], 0.0) == ([0, 2], 1)
    # a draft equal to the target is always kept
    p = np.array([0.1, 0.2, 0.3, 0.4], np.float32)
    assert T.verify(np.stack([p] * 4), np.stack([p] * 4), tok, par, [0.999] * 4, 0.0)[0] == [0, 1, 2, 3]
    # nothing left behind a rejection: the target itself; no weight at all: none
    assert T.verify(np.stack([eye[2]] * 2), np.stack([eye[2]] * 2), [0, 1], [-1, 0], [0, 0.5], 0.3) == ([0], 2)
    assert T.verify(np.zeros((2, 4), np.float32), None, [0, 1], [-1, 0], [0, 0.5], 0.3) == ([0], -1)


def test_draw_borders():
    p = np.array([[0.25, 0.25, 0.0, 0.5]], np.float32)
    draw = lambda u: T.verify(p, None, [0], [-1], [0], u)[1]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.24999, 0.25, 0.49999, 0.5, 0.99999)] == [0, 0, 1, 1, 3, 3]


def test_commit_moves_up():
    rows = np.arange(10)
    assert T.commit(rows, 4, [0, 2, 3, 5]).tolist() == [0, 1, 2, 3, 4, 6, 7, 9, 8, 9]
