"""GPU: the page-scaled 8-bit cache and eviction at the ends of their range:
the output's precision in every form, positions up to 2^31, NaN and infinities
beside what they must not reach, and the calls that follow an eviction."""

import numpy as np
import pytest
import torch

from _helpers import bf16_ulp, to_f64
from mla_latent_kv_03_gb300 import libmla as L
from mla_latent_kv_03_gb300 import workloads as W
from mla_latent_kv_03_gb300.step import MlaDecodeStep
from oracle import mla_oracle as O
from oracle import page8_oracle as P
from test_gpu_page8 import (CASES, DEV, Writer, _step, _together, check_out, dev, oracle_rows, split_cache,
                            status_bits)

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


@pytest.mark.parametrize("name", sorted(CASES))
def test_the_output_is_rounded_once_in_every_form(name):
    """A bf16 output rounded once is off by 2^-7 / m of itself at the most on a
    mantissa m in [1, 2), half of it either way, uniformly: over mantissas with
    uniform logarithms a mean square of 2^-14 / 12 * (3/8) / ln 2, its root
    1.66e-3. Weights of 11 bits (2^-11, a root of 0.28e-3) make it 1.68e-3 at
    the most, latents of two bf16 terms (2^-16) no more, and 2,048 outputs or more
    settle the mean to a few percent. A second rounding to bf16 on the way would
    make it 2.3e-3."""
    w, s = _step(name)
    s.page8_decode()
    torch.cuda.synchronize()
    rows, q, W_uv, got = oracle_rows(s), to_f64(s.q_abs), to_f64(s.W_uv), to_f64(s.out)
    num = den = 0.0
    for b in range(w.batch):
        qr, n = w.q_range(b), int(w.seq_lens[b])
        if qr.stop == qr.start:
            continue
        kv = O.gather_paged(rows, w.block_table[b], n, w.block_size)
        o, _ = O.latent_attention(q[qr], kv, np.arange(n - (qr.stop - qr.start), n), w.softmax_scale)
        want = O.out_proj(o, W_uv)
        num += float(((got[qr] - want) ** 2).sum())
        den += float((want ** 2).sum())
    assert num <= (1.8e-3) ** 2 * den, (num / den) ** 0.5


# -------------------------------------------------------------- positions
@pytest.mark.parametrize("n", [40, 2100])            # either form of the write
@pytest.mark.parametrize("base", [10000.0, 1e6])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("around", [1 << 15, 1 << 17, 1 << 20, 1 << 22, 1 << 24, 1 << 26, 1 << 28, (1 << 31) - 2500])
def test_keys_of_far_positions(around, interleaved, base, n):
    """The angle is off by 2^-21 at 2^31 (53 bits of a frequency, here and in the
    oracle), its sine and cosine by 2^-23 more, two products and their sum by
    2^-24 each: in all below 2^-20 (|x1| + |x2|), and the bf16 rounding."""
    rng = np.random.default_rng(around % 1000 + n)
    nb = n // 16 + 1
    cfg = L.make_config(16, 16, "bf16", rope_base=base, rope_interleaved=interleaved)
    k = W.round_to_dtype(rng.standard_normal((n, 64)), "bf16")
    pos = around + rng.integers(-2500, 2500, n)
    cache = torch.zeros((nb, 16, 640), dtype=torch.uint8, device=DEV)
    ws = torch.empty(L.mla_page8_write_workspace_size(cfg, n, nb), dtype=torch.uint8, device=DEV)
    L.mla_page8_cache_write(cfg, dev(rng.standard_normal((n, 512)), torch.bfloat16), dev(k, torch.bfloat16),
                            dev(pos, torch.int32), dev(np.arange(n), torch.int64),
                            dev(np.ones(512), torch.bfloat16), cache, torch.zeros(nb, device=DEV), ws)
    torch.cuda.synchronize()
    got = split_cache(cache)[1].reshape(-1, 64)[:n]
    want = O.rope(k, pos, base, interleaved)
    i = np.arange(32)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
    size = np.abs(np.asarray(k, np.float64))
    pair = np.zeros_like(size)
    pair[:, a] = pair[:, b] = size[:, a] + size[:, b]
    off = np.abs(got - want)
    assert np.all(off <= bf16_ulp(want) + 2.0 ** -20 * pair), float(off.max())


# ----------------------------------------------------------- page scales
@pytest.mark.parametrize("nb", [200, 2000])          # last tokens by slot and by page
@pytest.mark.parametrize("n", [100, 2100])           # either form of the write
def test_a_token_whose_slot_is_taken_again_leaves_the_scale_alone(n, nb):
    w = Writer(nb=nb, bs=16, seed=n + nb)
    x, k = w.tokens(n)
    slots = np.arange(n) + 3
    x[:n - 1:7, 11] = 3000.0                             # outliers in every page,
    late = np.arange(0, n - 1, 7)                        # each followed by another token for its slot
    x = np.concatenate([x, x[late + 1]])
    k = np.concatenate([k, k[late + 1]])
    slots = np.concatenate([slots, slots[late]])
    pos = np.arange(len(slots)).astype(np.int32)
    before = split_cache(w.cache), to_f64(w.scales), w.mass.cpu().clone()
    ws = torch.empty(L.mla_page8_write_workspace_size(w.cfg, len(slots), nb), dtype=torch.uint8, device=DEV)
    L.mla_page8_cache_write(w.cfg, dev(x, torch.bfloat16), dev(k, torch.bfloat16), dev(pos, torch.int32),
                            dev(slots, torch.int64), dev(w.weight, torch.bfloat16), w.cache, w.scales, ws,
                            mass=w.mass, dev_status=w.status)
    torch.cuda.synchronize()
    w.check(before, x, k, pos, slots, True)
    assert to_f64(w.scales).max() <= 2.0 ** -5           # (c_hat of an outlier: 22, a scale of 2^-4)


# --------------------------------------------------------------- eviction
def test_an_eviction_reads_lengths_and_table_of_another_streams_memory():
    """The lengths and the table of one eviction are of its stream's memory. The
    next one reads them on a stream that is late; what the first stream allocates
    meanwhile must not take their place."""
    def run(first, second):
        w, s, dst, budget = _together()
        s.absorb()
        s.page8_decode(0.9)
        torch.cuda.synchronize()
        with torch.cuda.stream(first):
            dst = dst.clone()
        first.synchronize()
        s.page8_evict(budget, 4, 20, dst, stream=first)
        torch.cuda.synchronize()
        del dst                                          # the step alone has them now
        back = dev(w.block_table[:, :2], torch.int32)    # two of each sequence's old pages
        if second is not first:
            with torch.cuda.stream(second):
                torch.cuda._sleep(100_000_000)
        got = s.page8_evict(60, 4, 20, back, stream=second)
        with torch.cuda.stream(first):
            _ = [torch.ones((4, n), dtype=torch.int32, device=DEV) for n in (1, 5) * 8]
        torch.cuda.synchronize()
        return [*got, s.p8_cache[back.long()], s.p8_mass[back.long()]]

    one = torch.cuda.Stream()
    for want, got in zip(run(one, one), run(torch.cuda.Stream(), torch.cuda.Stream())):
        assert torch.equal(want, got)


def test_steps_after_an_eviction_go_behind_the_kept_tokens():
    """Three steps, of one, three and no new tokens a sequence, into pages that the
    eviction filled in part and beyond them: larger values grow the moved scales."""
    lens, qs, bs, budget = [400, 130, 64, 900], [1, 3, 0, 3], 16, 125
    w = W.make("p8_after", lens, qs, 16, bs, "bf16", 33)
    s = MlaDecodeStep(w, device=DEV)
    columns = (budget + 9 + bs - 1) // bs + 1
    s.page8_setup(with_mass=True, spare_blocks=4 * columns)
    s.p8_cache.fill_(0x33)
    s.page8_populate()
    s.absorb()
    s.page8_decode(0.9)
    table = np.arange(4 * columns).reshape(4, columns)[:, ::-1] + w.num_blocks
    _, cut = s.page8_evict(budget, 4, 20, dev(table, torch.int32))
    n = np.minimum(lens, budget)
    writer = Writer.__new__(Writer)
    writer.nb, writer.bs, writer.inter, writer.weight = s.p8_blocks, bs, False, w.rms_weight
    writer.cache, writer.scales, writer.mass = s.p8_cache, s.p8_scales, s.p8_mass
    seq = w.token_seq[w.is_new]
    nth = np.concatenate([np.arange(q) for q in qs])
    grown = 0
    for step in range(3):
        s.c_kv_new[:, 5] *= 50
        x, k = to_f64(s.c_kv_new), to_f64(s.k_pe_new)
        before = split_cache(s.p8_cache), to_f64(s.p8_scales), s.p8_mass.cpu().clone()
        s.page8_write_new()
        at = n[seq] + nth
        n = n + qs
        pos = w.kv_positions[w.is_new] + (step + 1) * np.asarray(qs)[seq]
        torch.cuda.synchronize()
        assert s.p8_lens.tolist() == n.tolist() and cut.tolist() == np.minimum(lens, budget).tolist()
        assert s.q_positions.tolist() == pos.tolist()
        writer.check(before, x, k, pos, table[seq, at // bs] * bs + at % bs, True)
        old = before[1]
        grown += int(((old > 0) & (to_f64(s.p8_scales) > old)).sum())
        m0 = to_f64(s.p8_mass)
        s.absorb()
        s.page8_decode(0.9)
        torch.cuda.synchronize()
        rows = oracle_rows(s)
        check_out(w, s, s.out, rows, table, n)
        _, mass = P.decode(to_f64(s.q_abs), rows, table, n, w.query_start_loc, w.softmax_scale,
                           to_f64(s.W_uv), m0, 0.9)
        # (a score is off by 2^-18 of sum |q||k|, exp2 and the sums by 2^-20)
        size = max(float(np.abs(O.gather_paged(rows, table[b], int(n[b]), bs)).max(0) @
                         np.abs(to_f64(s.q_abs[w.q_range(b)])).max((0, 1))) for b in (0, 1, 3))
        tol = 2.0 ** -18 * w.softmax_scale * size + 2.0 ** -20
        assert np.all(np.abs(to_f64(s.p8_mass) - mass) <= tol * np.abs(mass))
    assert grown > 0 and status_bits(s.status) == 0 and status_bits(s.p8_ws) == 0
    with pytest.raises(ValueError, match="page8_setup"):
        s.page8_populate()
    s.page8_setup(with_mass=True)
    s.page8_populate()
    assert s.q_positions.tolist() == w.q_positions.tolist()


def test_steps_after_an_eviction_captured_and_by_a_streams_handle():
    """The eviction and two steps: on the current stream, on a stream given by its
    handle, and captured and replayed twice from the same state."""
    def start():
        w, s, dst, budget = _together()
        s.p8_cache.zero_()                               # (compared whole)
        s.p8_scales.zero_()
        s.page8_populate()
        s.absorb()
        s.page8_decode(0.9)
        torch.cuda.synchronize()
        return s, dst

    def calls(s, dst, stream=None):
        s.page8_evict(140, 4, 20, dst, stream=stream)
        for _ in range(2):
            s.page8_write_new(stream=stream)
            s.absorb(stream=stream)
            s.page8_decode(0.9, stream=stream)

    def state(s):
        torch.cuda.synchronize()
        return [t.clone() for t in (s.out, s.p8_cache, s.p8_scales, s.p8_mass, s.p8_lens, s.q_positions)]

    s, dst = start()
    calls(s, dst)
    want = state(s)
    assert s.p8_lens.tolist() == [142, 132, 66, 142]
    s, dst = start()
    side = torch.cuda.Stream()
    calls(s, dst, side.cuda_stream)
    assert all(torch.equal(a, b) for a, b in zip(state(s), want))
    s, dst = start()
    keep = [s.p8_cache, s.p8_scales, s.p8_mass, s.q_positions]
    first = [t.clone() for t in keep]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(s, dst)
    for _ in range(2):
        for t, v in zip(keep, first):
            t.copy_(v)
        s.out.fill_(float("nan"))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(state(s), want))
    assert status_bits(s.status) == 0 and status_bits(s.p8_ws) == 0


def test_a_step_without_a_page_for_it_is_flagged():
    w, s, dst, budget = _together()
    s.p8_cache[w.num_blocks:] = 0x33                      # the free pages
    s.absorb()
    s.page8_decode(0.9)
    table = dst[:, :4].contiguous()                       # 128 tokens
    table[1, 3] = -1                                      # 96, of which 96 are kept
    keep, lens = s.page8_evict(96, 4, 20, table)
    assert lens.tolist() == [96, 96, 64, 96]
    cache = s.p8_cache.clone()
    s.page8_write_new()
    assert status_bits(s.status) == L.DEV_BAD_SLOT
    assert torch.equal(s.p8_cache[w.block_table[1][w.block_table[1] >= 0]], cache[w.block_table[1][w.block_table[1] >= 0]])
    changed = (s.p8_cache != cache).any(-1).any(-1).nonzero().view(-1).tolist()
    assert changed == sorted(int(table[b, i]) for b, i in ((0, 3), (2, 2), (3, 3)))


def test_eviction_refuses_tables_it_has_no_workspace_for():
    w, s, dst, budget = _together()
    with pytest.raises(ValueError, match="columns"):
        s.page8_evict(budget, 4, 20, dst.repeat(1, 40))
    with pytest.raises(ValueError, match="column"):
        s.page8_evict(budget, 4, 20, dst[:, :0])
    assert s.p8_table is s.block_table


def test_compaction_without_destination_pages_is_flagged():
    cfg = L.make_config(16, 16, "bf16")
    cache = torch.full((3, 16, 640), 5, dtype=torch.uint8, device=DEV)
    scales = torch.ones(3, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    table, none = dev([[0], [1]], torch.int32), torch.empty((2, 0), dtype=torch.int32, device=DEV)
    keep = dev([[3, 4], [1, -1]], torch.int32)
    for lens, want in (([0, 0], 0), ([0, 1], L.DEV_BAD_SEQ)):
        L.mla_page8_compact(cfg, cache, scales, None, table, keep, dev(lens, torch.int32), none, dev_status=status)
        torch.cuda.synchronize()
        assert status_bits(status) == want
    assert torch.all(cache == 5) and torch.all(scales == 1)


# ---------------------------------------------------- NaN and infinities
@pytest.mark.parametrize("num_ctas", [0, 1, 7])
@pytest.mark.parametrize("name", ["tails_bs64", "bs16_h32", "chunks", "speculative", "h128", "merged_pairs", "merged_h128"])
def test_a_nan_key_makes_the_weights_of_its_sequence_nan(name, num_ctas):
    """However its rows are cut into parts, and wherever the parts are merged; no
    other sequence's weights change."""
    w, s = _step(name, num_ctas, with_mass=True)
    m0 = s.p8_mass.clone()
    s.page8_decode(0.5)
    clean = s.p8_mass.clone()
    b = int(np.argmax(w.seq_lens))
    s.p8_mass.copy_(m0)
    s.p8_cache[int(w.block_table[b, 0]), 0, 30] = 0x7F
    s.page8_decode(0.5)
    torch.cuda.synchronize()
    t = np.arange(int(w.seq_lens[b]))
    at = torch.from_numpy(w.block_table[b][t // w.block_size].astype(np.int64) * w.block_size + t % w.block_size)
    its = torch.zeros(clean.numel(), dtype=torch.bool)
    its[at] = True
    got = s.p8_mass.cpu().view(-1)
    assert torch.isnan(got[its]).all()
    assert torch.equal(got[~its], clean.cpu().view(-1)[~its])
    assert torch.isnan(s.out[w.q_range(b)].float()).all()


@pytest.mark.parametrize("heads", [range(8), range(8, 16), [0, 15], range(1, 16)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_in_some_heads_leaves_the_others(heads, value):
    """First and second rows of pairs, and single ones: the other heads, and the
    rows beside them, keep every bit."""
    w, s = _step("chunks")
    s.page8_decode()
    clean = s.out.clone()
    bad = torch.zeros(w.num_q, 16, dtype=torch.bool)
    for n in (0, 1, 7, 38, 39, 40, 42, 44, 173):
        for h in heads:
            s.q_abs[n, h, 17] = value
            bad[n, h] = True
    s.page8_decode()
    torch.cuda.synchronize()
    assert torch.isnan(s.out.cpu()[bad].float()).all()
    assert torch.equal(s.out.cpu()[~bad], clean.cpu()[~bad])


# -------------------------------------------------------------- workspaces
@pytest.mark.parametrize("heads", [16, 32])
def test_one_workspace_for_the_most_rows_and_sequences(heads):
    """Sized once, then used by batches that shrink: the same rows over fewer
    sequences, fewer rows, narrower tables."""
    cfg = L.make_config(heads, 16, "bf16")
    ws = torch.empty(L.mla_page8_decode_workspace_size(cfg, 64, 64, 20), dtype=torch.uint8, device=DEV)
    L.mla_workspace_init(ws)
    for batch, rows in ((64, 1), (32, 2), (20, 3), (1, 64), (7, 1)):
        w = W.make("p8_fewer", [200 + b for b in range(batch)], [rows] * batch, heads, 16, "bf16", batch)
        s = MlaDecodeStep(w, device=DEV)
        s.page8_setup()
        s.p8_ws = ws
        s.page8_populate()
        s.absorb()
        s.page8_decode()
        torch.cuda.synchronize()
        assert status_bits(ws) == 0
        check_out(w, s, s.out, oracle_rows(s))
