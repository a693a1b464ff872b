"""GPU parity of the page-scaled 8-bit cache (write, attention, accumulated
weights) and of eviction (select, compact) against the fp64 oracle.

Tolerances, fixed before the first run:
  codes     equal to the oracle's, but where the exact value lies within fp32
            error (1e-5 relative) of a rounding midpoint;
  out       bf16. Half a step of the result (2^-8 |out|), half a step of the
            latent that enters the projection (2^-8 sum |o| |W|), and for the
            probabilities 9 significant bits, 2^-10 each, in the worst case all
            of one sign: 2^-10 sum_c (sum_t p |v|) |W|; taken 2^-9 for the fp32
            sums beside it. Beyond that bound for each element, rel-L2 <= 5e-3;
  mass      fp32. A score is off by at most 2^-18 of sum |q||k| (an fp32 sum of
            576 products, at most 64 of its roundings one after another), which
            is the relative error of its weight; 2^-20 for exp2 and the sums.
"""

import numpy as np
import pytest
import torch

from _helpers import bf16_ulp, to_f64
from mla_latent_kv_03_gb300 import libmla as L
from mla_latent_kv_03_gb300 import workloads as W
from mla_latent_kv_03_gb300.step import MlaDecodeStep
from oracle import mla_oracle as O
from oracle import page8_oracle as P

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    L.load()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=dtype)


def split_cache(c8):
    c8 = c8.cpu()
    rope = c8[..., 512:].contiguous().view(torch.bfloat16).double().numpy()
    return c8[..., :512].numpy().copy(), rope


def status_bits(word):
    return L.mla_get_device_status(word)[1]


# ------------------------------------------------------------------ write
class Writer:
    def __init__(self, nb, bs, seed, interleaved=False):
        self.nb, self.bs, self.inter = nb, bs, interleaved
        self.rng = np.random.default_rng(seed)
        self.cfg = L.make_config(16, bs, "bf16", rope_interleaved=interleaved)
        self.weight = W.round_to_dtype(1 + 0.2 * self.rng.standard_normal(512), "bf16")
        self.cache = torch.full((nb, bs, 640), 0x55, dtype=torch.uint8, device=DEV)
        self.cache[..., 512:] = 0
        self.scales = torch.zeros(nb, dtype=torch.float32, device=DEV)
        self.mass = torch.full((nb, bs), 7.0, dtype=torch.float32, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def tokens(self, n, outliers=0.0):
        x = self.rng.standard_normal((n, 512)).astype(np.float32)
        if outliers:
            x[self.rng.random(n) < outliers, 11] *= 60
        return (W.round_to_dtype(x, "bf16"),
                W.round_to_dtype(self.rng.standard_normal((n, 64)), "bf16"))

    def write(self, slots, outliers=0.0, check=True, with_mass=True):
        slots = np.asarray(slots, np.int64)
        n = len(slots)
        x, k = self.tokens(n, outliers)
        pos = self.rng.integers(0, 5000, n).astype(np.int32)
        ws = torch.empty(L.mla_page8_write_workspace_size(self.cfg, n, self.nb), dtype=torch.uint8, device=DEV)
        ws.fill_(0xA5)                                    # it needs no initialisation
        before = split_cache(self.cache), self.scales.cpu().double().numpy(), self.mass.cpu().clone()
        L.mla_page8_cache_write(self.cfg, dev(x, torch.bfloat16), dev(k, torch.bfloat16),
                                dev(pos, torch.int32), dev(slots, torch.int64),
                                dev(self.weight, torch.bfloat16), self.cache, self.scales, ws,
                                mass=self.mass if with_mass else None, dev_status=self.status)
        torch.cuda.synchronize()
        if check:
            self.check(before, x, k, pos, slots, with_mass)

    def check(self, before, x, k, pos, slots, with_mass):
        (c0, r0), s0, m0 = before
        want_c, want_r, want_s = P.write(c0, r0, s0, x, k, pos, slots, self.weight, 1e-6, 10000.0, self.inter)
        got_c, got_r = split_cache(self.cache)
        got_s = self.scales.cpu().double().numpy()
        assert np.array_equal(got_s, want_s)
        new = np.full((self.nb, self.bs), -1)
        for t, s in enumerate(slots):
            if 0 <= s < self.nb * self.bs:
                new.reshape(-1)[s] = t
        written = new >= 0
        assert np.array_equal(got_c[~written], want_c[~written]), "rows beside the written ones"
        assert np.array_equal(got_r[~written], want_r[~written])
        diff = (got_c != want_c) & written[..., None]
        if diff.any():
            c_hat = np.zeros((self.nb, self.bs, 512))
            c_hat[written] = O.rms_norm(x, self.weight, 1e-6)[new[written]]
            v = (c_hat / np.where(want_s > 0, want_s, 1)[:, None, None])[diff]
            mid = (O.e4m3_decode(got_c[diff]) + O.e4m3_decode(want_c[diff])) / 2
            assert np.all(np.abs(v - mid) <= 1e-5 * np.abs(v) + 1e-12)
        # x1 cos - x2 sin may cancel, so a bf16 step of the result alone does
        # not bound it: the angle, reduced in fp32, is off by a few 1e-7
        # absolute, cos and sin by an fp32 step each, the two products and
        # their sum by half a step each: in all below 2^-20 (|x1| + |x2|)
        near = np.zeros_like(want_r)
        i = np.arange(32)
        a, b = (2 * i, 2 * i + 1) if self.inter else (i, i + 32)
        size = np.abs(np.asarray(k, np.float64))
        pair = np.zeros_like(size)
        pair[:, a] = pair[:, b] = size[:, a] + size[:, b]
        near[written] = 2.0 ** -20 * pair[new[written]]
        assert np.all(np.abs(got_r - want_r)[written] <= (bf16_ulp(want_r) + near)[written])
        mass = self.mass.cpu()
        assert torch.equal(mass[torch.from_numpy(~written)], m0[torch.from_numpy(~written)])
        if with_mass:
            assert np.all(mass.numpy()[written] == 0)


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 1000, 1024, 1025, 2048, 2049, 2500])
def test_write_fills_pages(bs, n):
    w = Writer(nb=n // bs + 3, bs=bs, seed=n + bs, interleaved=bool(n & 1))
    w.write(np.arange(n) + bs // 2, outliers=0.02)
    assert status_bits(w.status) == 0


@pytest.mark.parametrize("bs", [16, 64])
def test_write_appends_and_grows_scales(bs):
    w = Writer(nb=12, bs=bs, seed=3)
    for step in range(6):     # one token into each of ten pages, larger ones now and then
        w.write([p * bs + step for p in range(10)], outliers=0.3, with_mass=bool(step & 1))
    w.write([5 * bs + 3, 5 * bs + 4], outliers=1.0)      # rewritten rows
    assert status_bits(w.status) == 0


@pytest.mark.parametrize("n", [300, 3000])
def test_write_in_any_order_with_repeats_and_padding(n):
    w = Writer(nb=n // 16 + 2, bs=16, seed=n)
    slots = w.rng.permutation(n)
    slots[w.rng.random(n) < 0.1] = -1
    slots[5:9] = slots[20]                               # the last of them stays
    slots[n - 1] = slots[30]
    w.write(slots, outliers=0.05)
    assert status_bits(w.status) == 0


@pytest.mark.parametrize("nb", [200, 1024, 1025, 1100, 2600])
def test_prompts_scattered_over_small_and_large_caches(nb):
    """Either side of where the last tokens go by slot or by page, in any order
    with slots named twice, twice into the same pages."""
    w = Writer(nb=nb, bs=16, seed=nb)
    for _ in range(2):
        w.write(w.rng.integers(-1, nb * 16, 2051), outliers=0.01)
    assert status_bits(w.status) == 0


@pytest.mark.parametrize("n", [40, 1500])
def test_write_flags_slots_past_the_cache(n):
    w = Writer(nb=4, bs=16, seed=8)
    slots = np.full(n, -1)
    slots[:6] = [3, 64, 5, 1 << 40, 40, 63]
    w.write(slots)
    assert status_bits(w.status) == L.DEV_BAD_SLOT


def test_write_twice_is_the_same_and_a_nan_token_stays_alone():
    w = Writer(nb=3, bs=16, seed=9)
    w.write(np.arange(20))
    c1, s1 = w.cache.clone(), w.scales.clone()
    x, k = w.tokens(2)
    x[1, 100] = np.nan
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    args = [dev(x, torch.bfloat16), dev(k, torch.bfloat16), dev([1, 2], torch.int32),
            dev([21, 22], torch.int64), dev(w.weight, torch.bfloat16)]
    for _ in range(2):
        L.mla_page8_cache_write(w.cfg, *args, w.cache, w.scales, ws)
    codes, _ = split_cache(w.cache)
    assert np.isnan(O.e4m3_decode(codes[1, 6])).all()
    assert not np.isnan(O.e4m3_decode(codes[1, 5])).any()
    assert torch.equal(w.cache[0], c1[0]) and torch.equal(w.scales[0], s1[0])
    if torch.equal(w.scales[1], s1[1]):
        assert torch.equal(w.cache[1, :4], c1[1, :4])


# ----------------------------------------------------------------- decode
CASES = {
    "tails_bs64": ([1, 63, 64, 65, 127, 128, 129, 1000], [1] * 8, 16, 64),
    "bs16_h32": ([5, 40, 200, 16], [1] * 4, 32, 16),
    "bs32_h64": ([33, 97, 2, 300], [1] * 4, 64, 32),
    "h128": ([500, 1, 77], [1] * 3, 128, 64),
    "empty_rows": ([0, 5, 0, 70, 9], [0, 1, 0, 1, 0], 16, 64),
    "chunks": ([150, 64, 3, 200], [40, 1, 3, 130], 16, 64),
    "chunks_h32_bs16": ([90, 17], [33, 17], 32, 16),
    "chunk_h128": ([70], [9], 128, 32),
    "many_rows": ([700, 20], [300, 1], 16, 64),
    "speculative": ([130, 500, 2, 66], [2, 3, 2, 1], 16, 32),
    "mixed": ([300, 64, 5, 1, 190], [100, 1, 1, 1, 33], 16, 16),
    "long": ([9000], [1], 16, 64),
    # the splits merged in the decode itself: pairs, single rows, wide groups
    "merged_pairs": ([700, 20, 9], [450, 1, 9], 16, 64),
    "merged_rows": ([3 + 7 * i % 150 for i in range(450)], [1] * 450, 16, 16),
    "merged_h128": ([200, 70, 130], [33, 20, 10], 128, 64),
    "merged_h32": ([260, 90], [200, 40], 32, 32),
}


def _step(name, num_ctas=0, with_mass=False, seed=11, sharp=True):
    lens, qs, H, bs = CASES[name]
    w = W.make("p8_" + name, lens, qs, H, bs, "bf16", seed, extra_blocks=2)
    rng = np.random.default_rng(seed)
    if sharp:   # some heads look at a few tokens, some at all
        w.q_nope = W.round_to_dtype(w.q_nope * np.exp2(rng.uniform(-2, 2, (1, H, 1))), "bf16")
    size = np.where(rng.random(w.num_tokens) < 0.05, 40.0, 1.0)
    w.c_kv_raw[:, 5] = W.round_to_dtype(w.c_kv_raw[:, 5] * size, "bf16")
    s = MlaDecodeStep(w, device=DEV, num_ctas=num_ctas)
    s.page8_setup(with_mass=with_mass)
    s.p8_cache.fill_(0x7F)                 # NaN wherever nothing is written
    if with_mass:
        s.p8_mass.copy_(torch.from_numpy(rng.random(tuple(s.p8_mass.shape)).astype(np.float32)))
    keep = None if s.p8_mass is None else s.p8_mass.clone()
    s.page8_populate()
    if with_mass:
        s.p8_mass.copy_(keep)
    s.absorb()
    return w, s


def oracle_rows(s):
    codes, rope = split_cache(s.p8_cache)
    return P.rows_of(codes, rope, s.p8_scales.cpu().numpy())


def check_out(w, s, got, rows, table=None, lens=None, rows_q=None):
    q = to_f64(s.q_abs)
    W_uv = to_f64(s.W_uv)
    table = w.block_table if table is None else table
    lens = w.seq_lens if lens is None else lens
    got = to_f64(got)
    num = den = 0.0
    for b in range(w.batch):
        qr = w.q_range(b)
        n = int(lens[b])
        if qr.stop == qr.start:
            continue
        kv = O.gather_paged(rows, table[b], n, w.block_size)
        pos = np.arange(n - (qr.stop - qr.start), n)
        o, lse = O.latent_attention(q[qr], kv, pos, w.softmax_scale)
        sc = w.softmax_scale * np.einsum("nhk,tk->nht", q[qr], kv)
        p = np.exp(sc - lse[..., None]) * (np.arange(n)[None, None] <= pos[:, None, None])
        want = O.out_proj(o, W_uv)
        size = O.out_proj(np.einsum("nht,tc->nhc", p, np.abs(kv[:, :512])), np.abs(W_uv))
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * O.out_proj(np.abs(o), np.abs(W_uv)) + 2.0 ** -9 * size
        err = np.abs(got[qr] - want)
        assert np.all(err <= bound), (b, float((err / bound).max()))
        num += float((err ** 2).sum())
        den += float((want ** 2).sum())
    assert num <= (5e-3) ** 2 * den, (num / den) ** 0.5


@pytest.mark.parametrize("num_ctas", [0, 1, 7, 500])
@pytest.mark.parametrize("name", sorted(CASES))
def test_decode_vs_oracle(name, num_ctas):
    w, s = _step(name, num_ctas)
    outs = []
    for _ in range(2):
        s.out.fill_(float("nan"))
        outs.append(s.page8_decode().clone())
    torch.cuda.synchronize()
    assert status_bits(s.p8_ws) == 0 and status_bits(s.status) == 0
    assert torch.equal(outs[0], outs[1])
    check_out(w, s, outs[0], oracle_rows(s))


@pytest.mark.parametrize("decay", [0.0, 0.75, 1.0])
@pytest.mark.parametrize("name", ["tails_bs64", "bs16_h32", "h128", "empty_rows", "chunks", "many_rows", "long",
                                  "merged_pairs", "merged_h128"])
def test_mass_vs_oracle(name, decay):
    w, s = _step(name, 0 if name != "chunks" else 5, with_mass=True)
    if decay == 0:
        s.p8_mass.fill_(float("nan"))      # the old value is not read
    m0 = s.p8_mass.cpu().double().numpy()
    s.page8_decode(decay)
    torch.cuda.synchronize()
    assert status_bits(s.p8_ws) == 0
    rows = oracle_rows(s)
    check_out(w, s, s.out, rows)
    q = to_f64(s.q_abs)
    _, want = P.decode(q, np.nan_to_num(rows), w.block_table, w.seq_lens, w.query_start_loc,
                       w.softmax_scale, to_f64(s.W_uv), m0, decay)
    got = s.p8_mass.cpu().double().numpy()
    seen = np.zeros_like(got, bool)
    size = 0.0
    for b in range(w.batch):
        n, qr = int(w.seq_lens[b]), w.q_range(b)
        if qr.stop > qr.start:
            pages = w.block_table[b][:(n + w.block_size - 1) // w.block_size]
            at = (pages[:, None] * w.block_size + np.arange(w.block_size)).reshape(-1)[:n]
            seen.reshape(-1)[at] = True
            kv = O.gather_paged(rows, w.block_table[b], n, w.block_size)
            size = max(size, w.softmax_scale * float(
                np.einsum("nhk,tk->nht", np.abs(q[qr]), np.abs(kv)).max()))
    assert np.array_equal(got[~seen], m0[~seen], equal_nan=True)
    tol = 2.0 ** -18 * size + 2.0 ** -20
    assert np.all(np.abs(got - want)[seen] <= tol * np.abs(want)[seen])


def test_decode_reads_out_of_range_pages_as_absent():
    w, s = _step("tails_bs64", with_mass=True)
    bad = w.block_table.copy()
    bad[7, 3] = -5
    bad[7, 9] = 1 << 20
    s.p8_table = dev(bad, torch.int32)
    m0 = s.p8_mass.clone()
    s.page8_decode(1.0)
    torch.cuda.synchronize()
    assert status_bits(s.p8_ws) == L.DEV_BAD_BLOCK
    rows = oracle_rows(s)
    # the oracle's view: the tokens of those pages do not exist
    keep = [t for t in range(1000) if t // 64 not in (3, 9)]
    kv = O.gather_paged(rows, w.block_table[7], 1000, 64)[keep]
    o, _ = O.latent_attention(to_f64(s.q_abs)[7:8], kv, [len(keep)], w.softmax_scale)
    want = O.out_proj(o, to_f64(s.W_uv))
    err = np.linalg.norm(to_f64(s.out)[7:8] - want) / np.linalg.norm(want)
    assert err <= 5e-3
    for p in (3, 9):
        page = int(w.block_table[7, p])
        assert torch.equal(s.p8_mass[page], m0[page])


def test_decode_skips_sequences_longer_than_their_table():
    w, s = _step("bs16_h32")
    lens = w.seq_lens.copy()
    lens[1] = 16 * w.max_blocks_per_seq + 1
    s.p8_lens = dev(lens, torch.int32)
    s.page8_decode()
    torch.cuda.synchronize()
    assert status_bits(s.p8_ws) == L.DEV_BAD_SEQ
    assert torch.all(s.out[1] == 0) and torch.all(s.out[0].float().abs().sum() > 0)


def test_a_nan_query_stays_in_its_head_and_a_nan_key_in_its_sequence():
    w, s = _step("chunks")
    s.page8_decode()
    clean = s.out.clone()
    s.q_abs[2, 3, 17] = float("nan")
    s.q_abs[5, 4, 540] = float("inf")
    page = int(w.block_table[1, 0])
    s.p8_cache[page, 10, 30] = 0x7F
    s.page8_decode()
    torch.cuda.synchronize()
    got = s.out.float()
    assert torch.isnan(got[2, 3]).all() and torch.isnan(got[5, 4]).all()
    assert torch.isnan(got[w.q_range(1)]).all()
    fine = torch.ones(w.num_q, 16, dtype=torch.bool)
    fine[2, 3] = fine[5, 4] = False
    fine[w.q_range(1)] = False
    assert torch.equal(s.out.cpu()[fine], clean.cpu()[fine])


@pytest.mark.parametrize("name,far", [("many_rows", 10), ("many_rows", 1), ("many_rows", 7), ("chunks", 3),
                                      ("chunks_h32_bs16", 5)])
def test_a_token_ahead_of_a_row_may_hold_anything(name, far):
    # the chunk's last tokens are NaN: earlier rows do not see them
    w, s = _step(name)
    s.page8_decode()
    clean = s.out.clone()
    n, q, bs = int(w.seq_lens[0]), int(w.q_lens[0]), w.block_size
    for t in range(n - far, n):
        s.p8_cache[int(w.block_table[0, t // bs]), t % bs] = 0x7F
    s.page8_decode()
    torch.cuda.synchronize()
    assert torch.equal(s.out[:q - far], clean[:q - far])
    assert torch.isnan(s.out[q - far:q].float()).all()
    assert torch.equal(s.out[q:], clean[q:])


def test_a_nan_query_row_leaves_the_row_beside_it():
    w, s = _step("chunks")
    s.page8_decode()
    clean = s.out.clone()
    for n in (0, 7, 39, 44):
        s.q_abs[n] = float("nan")
    s.page8_decode()
    torch.cuda.synchronize()
    fine = torch.ones(w.num_q, dtype=torch.bool)
    fine[[0, 7, 39, 44]] = False
    assert torch.isnan(s.out[~fine].float()).all()
    assert torch.equal(s.out[fine], clean[fine])


def test_scales_may_differ_widely_between_pages():
    w, s = _step("tails_bs64")
    rng = np.random.default_rng(5)
    f = np.exp2(rng.integers(-3, 3, s.p8_blocks)).astype(np.float32)
    s.p8_scales *= dev(f, torch.float32)
    s.page8_decode()
    torch.cuda.synchronize()
    check_out(w, s, s.out, oracle_rows(s))


def test_one_token_that_takes_most_of_the_weight_before_a_long_tail():
    # a first token with weight of about 0.9, and 8,999 small ones that carry the rest
    w, s = _step("long", sharp=False)
    rows = oracle_rows(s)
    kv = O.gather_paged(rows, w.block_table[0], 9000, 64)
    k0 = kv[0, 512:]
    q = to_f64(s.q_abs)
    base = w.softmax_scale * np.einsum("hk,tk->ht", q[0], kv)
    lse = np.log(np.exp(base[:, 1:]).sum(1))
    want = lse + np.log(9.0)                            # weight 9 : 1
    q[0, :, 512:] += ((want - base[:, 0]) / (w.softmax_scale * (k0 @ k0)))[:, None] * k0[None]
    s.q_abs.copy_(dev(q, torch.bfloat16))
    s.page8_decode()
    torch.cuda.synchronize()
    check_out(w, s, s.out, rows)


def test_rows_beyond_two_gigabytes_of_cache():
    bs, nb = 64, 56000                                  # 2.29 GB of pages
    cfg = L.make_config(16, bs, "bf16")
    w = W.make("p8_far", [150], [1], 16, bs, "bf16", 4)
    s = MlaDecodeStep(w, device=DEV)
    s.page8_setup(with_mass=True, spare_blocks=nb - w.num_blocks)
    table = np.array([[nb - 1, nb - 7, nb - 3]], np.int32)
    slots = table[0][np.arange(150) // bs].astype(np.int64) * bs + np.arange(150) % bs
    s.slot_mapping = dev(slots, torch.int64)
    s.page8_populate()
    s.absorb()
    near = s.page8_decode().clone()                     # (another, unwritten, page table)
    s.p8_table = dev(table, torch.int32)
    s.page8_decode()
    far = s.out.clone()
    small = MlaDecodeStep(w, device=DEV)
    small.page8_setup(with_mass=True)
    small.page8_populate()
    small.absorb()
    small.page8_decode()
    torch.cuda.synchronize()
    assert torch.equal(far, small.out) and not torch.equal(near, far)
    assert torch.equal(s.p8_mass[table[0]], small.p8_mass[w.block_table[0]])
    keep = torch.empty((1, 70), dtype=torch.int32, device=DEV)
    n = torch.empty(1, dtype=torch.int32, device=DEV)
    L.mla_evict_select(cfg, s.p8_mass, s.p8_table, s.p8_lens, 2, 10, keep, n)
    dst = dev(np.array([[nb - 11, nb - 12]]), torch.int32)
    L.mla_page8_compact(cfg, s.p8_cache, s.p8_scales, s.p8_mass, s.p8_table, keep, n, dst)
    torch.cuda.synchronize()
    k = keep[0].long().cpu()
    src = torch.from_numpy(slots)[k]
    assert torch.equal(s.p8_mass[nb - 11].cpu(), s.p8_mass.view(-1)[src[:64].to(DEV)].cpu())
    rope = s.p8_cache.view(-1, 640)[:, 512:]
    assert torch.equal(rope[(nb - 11) * bs:(nb - 11) * bs + 64], rope[src[:64].to(DEV)])


# ----------------------------------------------------------------- select
def _select(mass, table, lens, sinks, recent, budget, bs):
    cfg = L.make_config(16, bs, "bf16")
    keep = torch.full((len(lens), budget), -7, dtype=torch.int32, device=DEV)
    new = torch.full((len(lens),), -7, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    L.mla_evict_select(cfg, dev(mass, torch.float32), dev(table, torch.int32), dev(lens, torch.int32),
                       sinks, recent, keep, new, dev_status=status)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), new.cpu().numpy(), status_bits(status)


def _masses(rng, nb, bs, kind):
    m = rng.standard_normal((nb, bs)).astype(np.float32)
    if kind == "positive":
        m = np.exp(2 * m)
    elif kind == "ties":
        m = np.round(m)
    elif kind == "equal":
        m[:] = 0.25
    elif kind == "odd":
        u = rng.random((nb, bs))
        for i, v in enumerate([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, np.float32(3.4e38)]):
            m[(u >= i * 0.1) & (u < (i + 1) * 0.1)] = v
    elif kind == "near":                     # keys that differ in the last bits only
        m = (np.float32(1.0).view(np.uint32) + rng.integers(0, 300, (nb, bs)).astype(np.uint32)).view(np.float32)
    return m.astype(np.float32)


@pytest.mark.parametrize("kind", ["positive", "signed", "ties", "equal", "odd", "near"])
@pytest.mark.parametrize("bs,sinks,recent,budget", [(16, 0, 0, 1), (64, 4, 30, 100), (32, 0, 7, 8),
                                                    (16, 3, 0, 64), (64, 20, 44, 64), (32, 1, 1, 1500)])
def test_select_vs_oracle(kind, bs, sinks, recent, budget):
    rng = np.random.default_rng(budget + bs)
    lens = [0, 1, 63, 64, 65, 100, 101, 1023, 1024, 1025, 2500, budget, budget + 1]
    most = max(lens) // bs + 2
    need = [(n + bs - 1) // bs for n in lens]
    perm = rng.permutation(sum(need) + 3)
    table, at = np.full((len(lens), most), -1, np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    mass = _masses(rng, len(perm), bs, kind)
    keep, new, bits = _select(mass, table, lens, sinks, recent, budget, bs)
    want_keep, want_new = P.select(mass, table, lens, sinks, recent, budget)
    assert bits == 0
    assert np.array_equal(new, want_new)
    assert np.array_equal(keep, want_keep)


@pytest.mark.parametrize("n,budget,kind", [(70001, 5000, "positive"), (131072, 131071, "ties"),
                                           (200000, 33333, "equal"), (300011, 8191, "odd"),
                                           (1000000, 1000, "near")])
def test_select_long(n, budget, kind):
    rng = np.random.default_rng(n)
    nb = (n + 63) // 64
    table = rng.permutation(nb).astype(np.int32)[None]
    mass = _masses(rng, nb, 64, kind)
    keep, new, bits = _select(mass, table, [n], 5, 100, budget, 64)
    m = mass[table[0]].reshape(-1)[:n].astype(np.float64)
    nan = np.isnan(m)
    mid = np.arange(5, n - 100)
    order = mid[np.lexsort((mid, -np.where(nan, 0, m)[mid], nan[mid]))]
    want = np.sort(np.concatenate([np.arange(5), np.arange(n - 100, n), order[:budget - 105]]))
    assert bits == 0 and new[0] == budget
    assert np.array_equal(keep[0], want)


@pytest.mark.parametrize("batch,n", [(1, 900), (3, 3000), (20, 9000), (160, 1500), (300, 700)])
@pytest.mark.parametrize("kind", ["positive", "equal"])
def test_select_at_every_split(batch, n, kind):
    """Every number of CTAs a sequence and of CTAs an SM, ragged lengths (some
    below the budget), with few keys of the first digit and with all of them."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, n + 1, batch)
    lens[0] = n
    most = (n + 31) // 32
    table = rng.permutation(batch * most).reshape(batch, most).astype(np.int32)
    mass = _masses(rng, batch * most, 32, kind)
    keep, new, bits = _select(mass, table, lens.tolist(), 3, 17, 300, 32)
    want_keep, want_new = P.select(mass, table, lens, 3, 17, 300)
    assert bits == 0
    assert np.array_equal(new, want_new)
    assert np.array_equal(keep, want_keep)


def test_select_flags_bad_tables_and_lengths():
    rng = np.random.default_rng(1)
    mass = _masses(rng, 8, 16, "positive")
    table = np.array([[0, 1, 2], [3, -1, 99], [5, 6, 7]], np.int32)
    keep, new, bits = _select(mass, table, [49, 48, -1], 0, 0, 20, 16)
    assert bits == L.DEV_BAD_SEQ | L.DEV_BAD_BLOCK
    assert new.tolist() == [0, 20, 0]
    assert np.all(keep[0] == -1) and np.all(keep[2] == -1)
    # the page that exists comes first; then the absent ones' tokens in order
    assert keep[1].tolist() == list(range(20))


# ---------------------------------------------------------------- compact
def _random_cache(rng, nb, bs):
    codes = rng.integers(0, 256, (nb, bs, 512)).astype(np.uint8)
    rope = rng.integers(0, 256, (nb, bs, 128)).astype(np.uint8)
    scales = np.exp2(rng.integers(-12, 3, nb)).astype(np.float32)
    return codes, rope, scales, rng.random((nb, bs)).astype(np.float32)


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("with_mass", [True, False])
def test_compact_vs_oracle(bs, with_mass):
    rng = np.random.default_rng(bs)
    lens, kept = [200, 1, 70, 0, 333, 64], [130, 1, 64, 0, 1, 63]
    nb, most = 90, 333 // bs + 2
    perm, at = rng.permutation(nb), 0
    table = np.full((6, most), -1, np.int32)
    dst = np.full((6, 130 // bs + 1), -1, np.int32)
    for b in range(6):
        k = (lens[b] + bs - 1) // bs
        table[b, :k] = perm[at:at + k]
        at += k
        k = (kept[b] + bs - 1) // bs
        dst[b, :k] = perm[at:at + k]
        at += k
    keep = np.full((6, 131), -1, np.int32)
    for b in range(6):
        keep[b, :kept[b]] = np.sort(rng.permutation(lens[b])[:kept[b]])
    codes, rope, scales, mass = _random_cache(rng, nb, bs)
    cache = dev(np.concatenate([codes, rope], -1), torch.uint8)
    sc, ms = dev(scales, torch.float32), dev(mass, torch.float32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cfg = L.make_config(16, bs, "bf16")
    L.mla_page8_compact(cfg, cache, sc, ms if with_mass else None, dev(table, torch.int32),
                        dev(keep, torch.int32), dev(kept, torch.int32), dev(dst, torch.int32),
                        dev_status=status)
    torch.cuda.synchronize()
    c2, r2, s2, m2 = P.compact(codes, rope, scales, mass, table, keep, kept, dst)
    got = cache.cpu().numpy()
    assert status_bits(status) == 0
    assert np.array_equal(sc.cpu().numpy(), s2)
    assert np.array_equal(got[..., 512:], r2)
    assert np.array_equal(ms.cpu().numpy(), m2 if with_mass else mass)
    nan = np.isnan(O.e4m3_decode(c2))
    assert np.array_equal(np.isnan(O.e4m3_decode(got[..., :512])), nan)
    # a recoded zero may have either sign
    assert np.array_equal(O.e4m3_decode(got[..., :512])[~nan], O.e4m3_decode(c2)[~nan])


def test_compact_flags_and_skips_bad_entries():
    rng = np.random.default_rng(2)
    codes, rope, scales, mass = _random_cache(rng, 12, 16)
    scales[:] = 1
    cache = dev(np.concatenate([codes, rope], -1), torch.uint8)
    before = cache.clone()
    table = np.array([[0, 1], [2, -1], [3, 4], [5, 0]], np.int32)
    keep = np.array([[0, 40, 5], [1, 17, 3], [0, 1, 2], [2, 1, 0]], np.int32)
    dst = np.array([[6], [7], [99], [8]], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cfg = L.make_config(16, 16, "bf16")
    L.mla_page8_compact(cfg, cache, dev(scales, torch.float32), None, dev(table, torch.int32),
                        dev(keep, torch.int32), dev([3, 3, 3, 4], torch.int32), dev(dst, torch.int32),
                        dev_status=status)
    torch.cuda.synchronize()
    assert status_bits(status) == L.DEV_BAD_SLOT | L.DEV_BAD_BLOCK | L.DEV_BAD_SEQ
    want = before.clone()
    want[6, 0], want[6, 2] = before[0, 0], before[0, 5]
    want[7, 0], want[7, 2] = before[2, 1], before[2, 3]
    assert torch.equal(cache, want)


# --------------------------------------------------- a run of them together
def _run_together(s, w, dst, budget, stream=None):
    s.page8_write_new(stream=stream)
    s.absorb(stream=stream)
    s.page8_decode(0.9, stream=stream)
    first = s.out.clone()
    keep, lens = s.page8_evict(budget, 4, 20, dst, stream=stream)
    s.page8_decode(0.9, stream=stream)
    return first, keep, lens


def _together(seed=21):
    w = W.make("p8_run", [400, 130, 64, 900], [1, 1, 1, 1], 16, 32, "bf16", seed)
    s = MlaDecodeStep(w, device=DEV)
    budget = 150
    per = (budget + 31) // 32
    s.page8_setup(with_mass=True, spare_blocks=4 * per)
    s.page8_populate()
    dst = dev(np.arange(4 * per).reshape(4, per) + w.num_blocks, torch.int32)
    return w, s, dst, budget


def test_write_decode_evict_decode():
    w, s, dst, budget = _together()
    first, keep, lens = _run_together(s, w, dst, budget)
    torch.cuda.synchronize()
    assert status_bits(s.p8_ws) == 0 and status_bits(s.status) == 0
    rows = oracle_rows(s)
    check_out(w, s, first, rows)
    table, n = dst.cpu().numpy(), lens.cpu().numpy()
    assert n.tolist() == [150, 130, 64, 150]
    check_out(w, s, s.out, rows, table, n)
    # the kept tokens' rope keys are the old rows' own, bit for bit
    for b in range(4):
        old = O.gather_paged(rows, w.block_table[b], int(w.seq_lens[b]), 32)
        new = O.gather_paged(rows, table[b], int(n[b]), 32)
        assert np.array_equal(new[:, 512:], old[keep.cpu().numpy()[b, :n[b]], 512:])


def test_evict_needs_weights():
    _, s = _step("bs16_h32")
    with pytest.raises(ValueError, match="with_mass"):
        s.page8_evict(8, 0, 0, s.block_table)


def test_evict_on_a_stream_writes_memory_that_no_other_stream_still_uses():
    w, s, dst, budget = _together()
    side = torch.cuda.Stream()
    s.page8_decode(0.9)
    torch.cuda.synchronize()
    old = torch.empty((4, budget), dtype=torch.int32, device=DEV)   # as keep will be
    torch.cuda._sleep(100_000_000)
    old.fill_(-7)
    del old
    keep, lens = s.page8_evict(budget, 4, 20, dst, stream=side)
    torch.cuda.synchronize()
    for b, n in enumerate(lens.tolist()):
        k = keep[b].tolist()
        assert n == min(budget, int(w.seq_lens[b])) and -7 not in k
        assert k[:n] == sorted(set(k[:n])) and k[n:] == [-1] * (budget - n)


def test_the_same_run_on_another_stream_and_captured():
    w, s, dst, budget = _together()
    _run_together(s, w, dst, budget)
    torch.cuda.synchronize()
    want, want_mass = s.out.clone(), s.p8_mass.clone()
    w, s2, dst, budget = _together()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run_together(s2, w, dst, budget)
    side.synchronize()
    assert torch.equal(s2.out, want) and torch.equal(s2.p8_mass, want_mass)
    # captured: the calls on fixed buffers, replayed twice from the same state
    w, s3, dst, budget = _together()
    state = [t.clone() for t in (s3.p8_cache, s3.p8_scales, s3.p8_mass)]
    keep = torch.empty((4, budget), dtype=torch.int32, device=DEV)
    lens = torch.empty(4, dtype=torch.int32, device=DEV)

    def calls():
        s3.page8_write_new()
        s3.absorb()
        s3.page8_decode(0.9)
        L.mla_evict_select(s3.cfg, s3.p8_mass, s3.p8_table, s3.p8_lens, 4, 20, keep, lens)
        L.mla_page8_compact(s3.cfg, s3.p8_cache, s3.p8_scales, s3.p8_mass, s3.p8_table, keep, lens, dst)
        L.mla_page8_decode_mass(s3.cfg, s3.q_abs, s3.p8_cache, s3.p8_scales, dst, lens,
                                s3.query_start_loc, s3.W_uv, s3.p8_mass, 0.9, s3.p8_ws, s3.out)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(2):
        for t, v in zip((s3.p8_cache, s3.p8_scales, s3.p8_mass), state):
            t.copy_(v)
        s3.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s3.out, want) and torch.equal(s3.p8_mass, want_mass)


def test_two_calls_at_once_on_two_streams():
    """Different caches and workspaces; every call fills the device, so parts
    of the two run side by side and behind one another."""
    wants, runs = [], []
    for name, seed in (("many_rows", 5), ("h128", 6)):
        w, s = _step(name, with_mass=True, seed=seed)
        m0 = s.p8_mass.clone()
        s.page8_decode(0.5)
        torch.cuda.synchronize()
        wants.append((s.out.clone(), s.p8_mass.clone()))
        s.p8_mass.copy_(m0)
        s.out.fill_(float("nan"))
        runs.append((s, m0, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, m0, st in runs:
            with torch.cuda.stream(st):
                s.p8_mass.copy_(m0)
                s.page8_decode(0.5)
    torch.cuda.synchronize()
    for (s, _, _), (out, mass) in zip(runs, wants):
        assert torch.equal(s.out, out) and torch.equal(s.p8_mass, mass)


def test_two_captured_graphs_that_share_a_workspace():
    """Two batches of different size, a workspace that fits either, the graphs
    replayed in turn on one stream: neither finds what the other left."""
    ws, wws, steps = None, None, []
    for name in ("chunks", "speculative"):
        w, s = _step(name)
        steps.append(s)
        if ws is None or s.p8_ws.numel() > ws.numel():
            ws = s.p8_ws
        if wws is None or s.p8_write_ws.numel() > wws.numel():
            wws = s.p8_write_ws
    wants, graphs = [], []
    for s in steps:
        s.p8_ws, s.p8_write_ws = ws, wws
        state = s.p8_cache.clone()
        s.page8_write_new()
        wants.append(s.page8_decode().clone())
        torch.cuda.synchronize()
        s.p8_cache.copy_(state)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.page8_write_new()
            s.page8_decode()
        graphs.append(g)
    for k in (0, 1, 1, 0, 0, 1):
        steps[k].out.fill_(float("nan"))
        graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(steps[k].out, wants[k])
    assert status_bits(ws) == 0


def test_sequences_may_share_pages_and_repeat_them():
    """A common prefix in two block tables, and one page three times in a row."""
    w, s = _step("tails_bs64")
    table = w.block_table.copy()
    table[7, :2] = table[6, :2]
    table[7, 3:6] = table[7, 2]
    s.block_table.copy_(dev(table, torch.int32))
    got = s.page8_decode()
    torch.cuda.synchronize()
    assert status_bits(s.p8_ws) == 0
    check_out(w, s, got, oracle_rows(s), table)


def test_rows_behind_the_last_sequence_are_zeros():
    """A padded batch: more rows than query_start_loc names (as the other
    decodes: a row that sees no token is zeros), in each split's form."""
    for name in ("speculative", "h128", "many_rows"):
        w, s = _step(name)
        qsl = w.query_start_loc.copy()
        qsl[-1] = qsl[-2]                       # the last sequence's rows belong to none
        want = s.page8_decode().clone()
        s.query_start_loc.copy_(dev(qsl, torch.int32))
        s.out.fill_(float("nan"))
        got = s.page8_decode()
        torch.cuda.synchronize()
        assert status_bits(s.p8_ws) == 0
        n = int(qsl[-1])
        assert torch.all(got[n:] == 0)
        err = (got[:n].double() - want[:n].double()).abs().max() / want[:n].double().abs().max()
        assert err <= 2.0 ** -7                 # (another split, another order of sums)


def test_a_token_kept_twice_is_moved_twice():
    w, s = _step("tails_bs64", with_mass=True)
    b, n = 7, 5
    keep = dev(np.array([[3, 3, 700, 3, 12]]), torch.int32)
    lens = dev(np.array([n]), torch.int32)
    dst = dev(np.array([[w.num_blocks]]), torch.int32)
    s2 = torch.zeros((1, w.block_size, 640), dtype=torch.uint8, device=DEV)
    cache = torch.cat([s.p8_cache, s2])
    scales = torch.cat([s.p8_scales, s.p8_scales.new_zeros(1)])
    mass = torch.cat([s.p8_mass, s.p8_mass.new_zeros((1, w.block_size))])
    L.mla_page8_compact(s.cfg, cache, scales, mass, s.block_table[b:b + 1].contiguous(), keep, lens, dst,
                        dev_status=s.status)
    torch.cuda.synchronize()
    assert status_bits(s.status) == 0
    for row, t in enumerate([3, 3, 700, 3, 12]):
        p, r = int(w.block_table[b][t // w.block_size]), t % w.block_size
        assert torch.equal(cache[-1, row, 512:], cache[p, r, 512:])
        assert float(mass[-1, row]) == float(mass[p, r])
        if float(scales[p]) == float(scales[-1]):
            assert torch.equal(cache[-1, row], cache[p, r])


def test_select_on_two_streams_at_once_and_replayed_with_other_lengths():
    cfg = L.make_config(16, 32, "bf16")
    rng = np.random.default_rng(4)
    sets = []
    for batch, n, budget in ((3, 40000, 500), (40, 3000, 700)):
        most = (n + 31) // 32
        table = rng.permutation(batch * most).reshape(batch, most).astype(np.int32)
        mass = rng.random((batch * most, 32)).astype(np.float32)
        lens = rng.integers(budget // 2, n + 1, batch)
        s = dict(mass=dev(mass, torch.float32), table=dev(table, torch.int32), lens=dev(lens, torch.int32),
                 keep=torch.zeros((batch, budget), dtype=torch.int32, device=DEV),
                 new=torch.zeros(batch, dtype=torch.int32, device=DEV), stream=torch.cuda.Stream())
        sets.append((s, mass, table, lens, budget, n))

    def call(s):
        L.mla_evict_select(cfg, s["mass"], s["table"], s["lens"], 2, 50, s["keep"], s["new"])

    def check(s, mass, table, lens, budget):
        want, want_n = P.select(mass, table, lens, 2, 50, budget)
        assert np.array_equal(s["new"].cpu().numpy(), want_n)
        assert np.array_equal(s["keep"].cpu().numpy(), want)

    torch.cuda.synchronize()
    for _ in range(5):
        for s, *_ in sets:
            with torch.cuda.stream(s["stream"]):
                call(s)
    torch.cuda.synchronize()
    for s, mass, table, lens, budget, _ in sets:
        check(s, mass, table, lens, budget)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for s, *_ in sets:
            call(s)
    for _ in range(2):
        new = [rng.integers(0, n + 1, len(lens)) for _, _, _, lens, _, n in sets]
        for (s, *_), lens in zip(sets, new):
            s["lens"].copy_(dev(lens, torch.int32))
            s["keep"].fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        for (s, mass, table, _, budget, _), lens in zip(sets, new):
            check(s, mass, table, lens, budget)
