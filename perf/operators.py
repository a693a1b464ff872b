"""Operators of the page-scaled 8-bit latent cache, as one pass of a user's program each.

  write    kv_a_layernorm, RoPE and the write of new tokens into pages of e4m3 codes, one
           power-of-two scale to a page, which grows with the page's largest value
  decode   latent attention of absorbed queries over those pages, merged and projected to
           v_head_dim; with a decay, each cached token's attention weight, summed over rows and
           heads, is accumulated beside it
  select   which tokens of each sequence stay: the first ones, the last ones and those of most
           accumulated weight
  compact  the kept rows moved into fresh pages

A cache row is 640 bytes: 512 e4m3 codes of c_hat / page scale, then 64 bf16 rope values.
"""

import math
import random

import numpy as np
import torch

own = False

DC, DR, DV, ROW8 = 512, 64, 128, 640
EMIN, EMAX = -64, 64          # exponents a page scale can have
EPS, BASE = 1e-6, 10000.0
DEV = "cuda"


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # 64 prompts of 4096 tokens filling fresh pages
        {"name": "write_prompts", "op": "write", "batch": 64, "past": 0, "new": 4096, "vary": 0, "bs": 64, "inter": False, "lens": 1},
        # the step's one new token of each of 64 sequences, into part-filled pages
        {"name": "write_step", "op": "write", "batch": 64, "past": 1000, "new": 1, "vary": 900, "bs": 64, "inter": False, "lens": 2},
        # the serving batch: 64 sequences of 4096 tokens, one row each
        {"name": "decode_serving", "op": "decode", "batch": 64, "heads": 16, "len": 4096, "vary": 0, "q": 1, "bs": 64, "decay": -1.0, "lens": 3},
        # one request a few hundred tokens in: latency
        {"name": "decode_single", "op": "decode", "batch": 1, "heads": 16, "len": 333, "vary": 0, "q": 1, "bs": 16, "decay": -1.0, "lens": 4},
        # many heads over ragged lengths up to 32768
        {"name": "decode_ragged_h128", "op": "decode", "batch": 32, "heads": 128, "len": 32768, "vary": 32767, "q": 1, "bs": 64, "decay": -1.0, "lens": 5},
        # prefill chunks of 512 rows on about 2000 cached tokens
        {"name": "decode_chunks", "op": "decode", "batch": 4, "heads": 16, "len": 2560, "vary": 301, "q": 512, "bs": 64, "decay": -1.0, "lens": 6},
        # the serving batch of a program that evicts: the weights accumulate as well
        {"name": "decode_mass_serving", "op": "decode", "batch": 64, "heads": 16, "len": 4096, "vary": 0, "q": 1, "bs": 64, "decay": 1.0, "lens": 7},
        # two long contexts with decaying weights, small pages
        {"name": "decode_mass_long", "op": "decode", "batch": 2, "heads": 32, "len": 100001, "vary": 20000, "q": 1, "bs": 32, "decay": 0.9, "lens": 8},
        # every sequence of the serving batch cut to half
        {"name": "select_serving", "op": "select", "batch": 64, "len": 4096, "vary": 0, "budget": 2048, "sinks": 4, "recent": 256, "bs": 64, "lens": 9},
        # a few long contexts cut to an odd budget
        {"name": "select_long", "op": "select", "batch": 3, "len": 131072, "vary": 50000, "budget": 8191, "sinks": 16, "recent": 1000, "bs": 32, "lens": 10},
        {"name": "compact_serving", "op": "compact", "batch": 64, "len": 4096, "vary": 0, "budget": 2048, "bs": 64, "lens": 11},
        {"name": "compact_long", "op": "compact", "batch": 3, "len": 131072, "vary": 50000, "budget": 8191, "bs": 16, "lens": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "decode", "select", "compact"])
    c = {"op": op, "batch": _log(rng, 1, 64), "bs": rng.choice([16, 32, 64]), "lens": rng.randrange(1 << 20)}
    if op == "write":
        c["past"] = rng.choice([0, _log(rng, 1, 3000)])
        c["new"] = _log(rng, 1, max(1, min(4096, 200000 // c["batch"])))
        c["vary"] = rng.randrange(c["past"] // 2 + 1)
        c["inter"] = rng.random() < 0.5
        return c
    if op == "decode":
        c["heads"] = rng.choice([16, 32, 64, 128])
        c["q"] = rng.choice([1, 1, 2, _log(rng, 2, 400)])
        most = min(32768, 30_000_000 // (c["batch"] * c["heads"] * c["q"]))
        if most < max(64, c["q"]):
            c["batch"] = 1
            most = min(32768, 30_000_000 // (c["heads"] * c["q"]))
        c["len"] = max(c["q"], _log(rng, 1, most))
        c["vary"] = rng.randrange(c["len"] - c["q"] + 1)
        c["decay"] = rng.choice([-1.0, -1.0, 0.0, 0.75, 1.0])
        return c
    least = 40 if op == "select" else 1
    c["len"] = _log(rng, least, min(131072, 262144 // c["batch"]))
    c["vary"] = rng.randrange(c["len"] // 2 + 1)
    c["budget"] = rng.randint((least + 3) // 4, max(1, c["len"] * 3 // 4))
    if op == "select":  # some tokens go by their weight
        c["sinks"] = rng.randint(0, min(16, c["budget"] // 3))
        c["recent"] = rng.randint(0, c["budget"] // 2)
    return c


def _lens(case, key="len"):
    """Each sequence's length: it goes by the case alone."""
    r = random.Random(case["lens"])
    return [case[key] - (r.randint(0, case["vary"]) if case["vary"] else 0) for _ in range(case["batch"])]


def _kept(case):
    return [min(n, case["budget"]) for n in _lens(case)]


def work(case):
    op = case["op"]
    if op == "write":
        t = case["batch"] * case["new"]
        return {"bytes": t * ((DC + DR) * 2 + ROW8 + 8 + 4) + 2 * DC, "flops": t * (6 * DC + 6 * DR)}
    lens = _lens(case)
    n = sum(lens)
    if op == "decode":
        h, q = case["heads"], case["q"]
        nq = case["batch"] * q
        seen = sum(q * m - q * (q - 1) // 2 for m in lens)
        b = n * ROW8 + sum(-(-m // case["bs"]) for m in lens) * 8 + nq * h * ((DC + DR) * 2 + DV * 2) + h * DC * DV * 2
        if case["decay"] >= 0:
            b += n * 4 * (2 if case["decay"] > 0 else 1)
        return {"bytes": b, "flops": seen * h * 2 * (2 * DC + DR) + nq * h * 2 * DC * DV}
    k = sum(_kept(case))
    if op == "select":
        return {"bytes": n * 4 + case["batch"] * case["budget"] * 4, "flops": n}
    return {"bytes": k * (2 * ROW8 + 2 * 4 + 4), "flops": k}


# --------------------------------------------------------------------------------- inputs
class _State:
    pass


def _pages(case, lens, gen, spare=0):
    """A random page table: [batch, most pages], -1 where a sequence has none; the page count."""
    bs = case["bs"]
    need = torch.tensor([-(-n // bs) for n in lens])
    most, total = max(1, int(need.max())), int(need.sum())
    perm = torch.randperm(total + spare, generator=gen, device=DEV).to(torch.int32)
    first = torch.cumsum(need, 0) - need
    at = first[:, None] + torch.arange(most)[None]
    live = torch.arange(most)[None] < need[:, None]
    table = torch.where(live.to(DEV), perm[at.clamp(max=max(total - 1, 0)).to(DEV)], -1)
    return table.to(torch.int32).contiguous(), total + spare, perm[total:]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _fill_cache(s, gen):
    """Pages of codes and their scales: normal latents, here and there a token of much larger size."""
    nb, bs = s.nb, s.bs
    s.cache8 = torch.empty(nb, bs, ROW8, dtype=torch.uint8, device=DEV)
    s.scales = torch.empty(nb, dtype=torch.float32, device=DEV)
    for i in range(0, nb, 4096):  # a block of pages at a time: the fp32 values are large
        k = min(4096, nb - i)
        x = _randn(gen, k, bs, DC)
        x *= torch.where(torch.rand(k, bs, 1, generator=gen, device=DEV) < 0.005, 30.0, 1.0)
        e = _need(x.abs().amax((1, 2)))
        s.scales[i:i + k] = torch.exp2(e.float())
        x /= s.scales[i:i + k, None, None]
        s.cache8[i:i + k, :, :DC] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        s.cache8[i:i + k, :, DC:] = _randn(gen, k, bs, DR).bfloat16().view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = _State()
    s.op, s.bs, s.case = case["op"], case["bs"], dict(case)
    if s.op == "write":
        _prepare_write(s, case, gen)
    else:
        lens = _lens(case)
        spare = sum(-(-k // s.bs) for k in _kept(case)) if s.op == "compact" else 0
        s.table, s.nb, rest = _pages(case, lens, gen, spare)
        s.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s.batch, s.most = len(lens), s.table.shape[1] * s.bs
        {"decode": _prepare_decode, "select": _prepare_select, "compact": _prepare_compact}[s.op](s, case, gen, lens, rest)
    if own:
        _prepare_own(s)
    return s


def _prepare_write(s, case, gen):
    b, new, bs = case["batch"], case["new"], s.bs
    past = _lens(case, "past")
    s.table, s.nb, _ = _pages(case, [p + new for p in past], gen)
    pos = torch.tensor(past, device=DEV)[:, None] + torch.arange(new, device=DEV)[None]
    page = torch.gather(s.table.long(), 1, pos // bs)
    s.slots = (page * bs + pos % bs).reshape(-1).contiguous()
    s.pos = pos.reshape(-1).to(torch.int32).contiguous()
    s.inter = bool(case["inter"])
    t = b * new
    size = torch.where(torch.rand(t, 1, generator=gen, device=DEV) < 0.01, 3.0, 1.0)
    s.c_kv = (_randn(gen, t, DC) * (0.05 + torch.rand(t, 1, generator=gen, device=DEV))).bfloat16()
    s.c_kv[:, 7] *= size[:, 0].bfloat16() * 4  # one channel is large, and in some tokens larger
    s.k_pe = _randn(gen, t, DR).bfloat16()
    s.w = (1 + 0.1 * _randn(gen, DC)).bfloat16()
    if case["past"]:
        _fill_cache(s, gen)
    else:
        s.cache8 = torch.zeros(s.nb, bs, ROW8, dtype=torch.uint8, device=DEV)
        s.scales = torch.zeros(s.nb, dtype=torch.float32, device=DEV)


def _prepare_decode(s, case, gen, lens, rest):
    _fill_cache(s, gen)
    s.heads, s.q = case["heads"], case["q"]
    nq = s.batch * s.q
    s.qsl = torch.arange(0, nq + 1, s.q, dtype=torch.int32, device=DEV)
    # some heads look at a few tokens, some at all of them
    sharp = torch.exp2(torch.rand(1, s.heads, 1, generator=gen, device=DEV) * 4 - 2)
    s.q_abs = (_randn(gen, nq, s.heads, DC + DR) * sharp * torch.cat([torch.full((DC,), 0.5), torch.ones(DR)]).to(DEV)).bfloat16()
    s.W_uv = (_randn(gen, s.heads, DC, DV) / math.sqrt(DC)).bfloat16()
    s.out = torch.empty(nq, s.heads, DV, dtype=torch.bfloat16, device=DEV)
    s.decay = float(case["decay"])
    s.mass = torch.rand(s.nb, s.bs, generator=gen, device=DEV) * 2 if s.decay >= 0 else None


def _masses(s, gen):
    """Accumulated weights: heavy tails, many small ones that are equal."""
    m = torch.exp(2 * _randn(gen, s.nb, s.bs) - 3)
    return torch.where(m < 0.01, 0.0, m)


def _prepare_select(s, case, gen, lens, rest):
    s.mass = _masses(s, gen)
    s.budget, s.sinks, s.recent = case["budget"], case["sinks"], case["recent"]
    s.keep = torch.empty(s.batch, s.budget, dtype=torch.int32, device=DEV)
    s.new_lens = torch.empty(s.batch, dtype=torch.int32, device=DEV)


def _prepare_compact(s, case, gen, lens, rest):
    _fill_cache(s, gen)
    s.mass = _masses(s, gen)
    s.budget = case["budget"]
    kept = _kept(case)
    # a random ascending choice for each sequence
    r = torch.rand(s.batch, s.most, generator=gen, device=DEV)
    t = torch.arange(s.most, device=DEV)[None]
    r = torch.where(t < s.lens[:, None], r, 2.0)
    new = torch.tensor(kept, device=DEV)
    at = torch.argsort(r, 1)[:, :s.budget]
    j = torch.arange(at.shape[1], device=DEV)[None]
    at = torch.where(j < new[:, None], at, s.most).sort(1).values
    s.keep = torch.full((s.batch, s.budget), -1, dtype=torch.int32, device=DEV)
    s.keep[:, :at.shape[1]] = torch.where(j < new[:, None], at, -1).to(torch.int32)
    s.new_lens = new.to(torch.int32)
    pages = torch.tensor([-(-k // s.bs) for k in kept])
    first, most = torch.cumsum(pages, 0) - pages, max(1, int(pages.max()))
    i = first[:, None] + torch.arange(most)[None]
    live = torch.arange(most)[None] < pages[:, None]
    s.dst = torch.where(live.to(DEV), rest[i.clamp(max=len(rest) - 1).to(DEV)], -1).to(torch.int32).contiguous()


def _prepare_own(s):
    """What the framework's calls need beside the data: a configuration, workspaces, a status word."""
    from mla_latent_kv_03_gb300 import libmla as L
    s.L = L
    s.cfg = L.make_config(getattr(s, "heads", 16), s.bs, "bf16", rms_eps=EPS, rope_base=BASE, rope_interleaved=getattr(s, "inter", False))
    s.status = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = 0
    if s.op == "write":
        n = L.mla_page8_write_workspace_size(s.cfg, s.slots.shape[0], s.nb)
    elif s.op == "decode":
        n = L.mla_page8_decode_workspace_size(s.cfg, s.q_abs.shape[0], s.batch, s.table.shape[1], s.decay >= 0)
    if n:
        s.ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        L.mla_workspace_init(s.ws)


# ------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        _OWN[s.op](s)
    else:
        _PLAIN[s.op](s)
    return _OUT[s.op](s)


def _own_write(s):
    s.L.mla_page8_cache_write(s.cfg, s.c_kv, s.k_pe, s.pos, s.slots, s.w, s.cache8, s.scales, s.ws, dev_status=s.status)


def _own_decode(s):
    if s.mass is None:
        s.L.mla_page8_decode(s.cfg, s.q_abs, s.cache8, s.scales, s.table, s.lens, s.qsl, s.W_uv, s.ws, s.out)
    else:
        s.L.mla_page8_decode_mass(s.cfg, s.q_abs, s.cache8, s.scales, s.table, s.lens, s.qsl, s.W_uv, s.mass, s.decay, s.ws, s.out)


def _own_select(s):
    s.L.mla_evict_select(s.cfg, s.mass, s.table, s.lens, s.sinks, s.recent, s.keep, s.new_lens, dev_status=s.status)


def _own_compact(s):
    s.L.mla_page8_compact(s.cfg, s.cache8, s.scales, s.mass, s.table, s.keep, s.new_lens, s.dst, dev_status=s.status)


def _cache_out(s):
    return {"codes": s.cache8[..., :DC].view(torch.float8_e4m3fn), "rope": s.cache8[..., DC:].view(torch.bfloat16), "scales": s.scales}


_OWN = {"write": _own_write, "decode": _own_decode, "select": _own_select, "compact": _own_compact}
_OUT = {
    "write": _cache_out,
    "decode": lambda s: {"out": s.out} if s.mass is None else {"out": s.out, "mass": s.mass},
    "select": lambda s: {"keep": s.keep, "new_lens": s.new_lens},
    "compact": lambda s: dict(_cache_out(s), mass=s.mass),
}


# ------------------------------------------------------------- the plain forms, in 32 bits
def _need(amax):
    """The smallest e with amax <= 448 * 2^e, from the float's own fraction and exponent."""
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    return torch.where(amax > 0, e, EMIN).clamp(EMIN, EMAX)


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(c8):
    return c8.view(torch.float8_e4m3fn).float()


def _plain_write(s):
    x = s.c_kv.float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s.w.float()
    page = s.slots // s.bs
    # the page's scale: as large as the rows in it need, and never smaller than it was
    need = torch.exp2(_need(y.abs().amax(1)).float())
    old = s.scales.clone()
    s.scales.index_reduce_(0, page, need, "amax")
    # rows that are there already keep their values in the page's new scale
    shift = torch.where(s.scales > 0, old / s.scales, 1.0)
    grown = torch.where((shift > 0) & (shift < 1), shift, 1.0)
    s.cache8[..., :DC] = _codes(_values(s.cache8[..., :DC].contiguous()) * grown[:, None, None])
    rows = s.cache8.view(-1, ROW8)
    i = torch.arange(DR // 2, device=DEV, dtype=torch.float64)
    ang = s.pos.double()[:, None] * BASE ** (-2 * i / DR)[None]
    cos, sin = ang.cos().float(), ang.sin().float()
    k = s.k_pe.float()
    x1, x2 = (k[:, 0::2], k[:, 1::2]) if s.inter else (k[:, :DR // 2], k[:, DR // 2:])
    r1, r2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    rot = torch.stack([r1, r2], 2).reshape(-1, DR) if s.inter else torch.cat([r1, r2], 1)
    new = torch.cat([_codes(y / s.scales[page][:, None]), rot.bfloat16().view(torch.uint8)], 1)
    rows.index_copy_(0, s.slots, new)


def _plain_decode(s):
    b, h, q, bs = s.batch, s.heads, s.q, s.bs
    pages = s.table.clamp(min=0).long()
    lat = _values(s.cache8[pages][..., :DC].contiguous()) * s.scales[pages][..., None, None]
    lat = lat.reshape(b, s.most, DC)
    rope = s.cache8[pages][..., DC:].contiguous().view(torch.bfloat16).float().reshape(b, s.most, DR)
    qs = s.q_abs.float().reshape(b, q * h, DC + DR)
    sc = torch.bmm(qs[..., :DC], lat.transpose(1, 2))
    sc += torch.bmm(qs[..., DC:], rope.transpose(1, 2))
    sc = sc.reshape(b, q, h, s.most).mul_(192.0 ** -0.5)
    t = torch.arange(s.most, device=DEV)
    last = s.lens.long()[:, None] - q + torch.arange(q, device=DEV)[None]
    sc.masked_fill_((t[None, None] > last[..., None])[:, :, None], -math.inf)
    sc -= sc.amax(3, keepdim=True)
    sc.exp_()
    sc /= sc.sum(3, keepdim=True)
    o = torch.bmm(sc.reshape(b, q * h, s.most), lat).reshape(b * q, h, DC)
    s.out.copy_(torch.bmm(o.transpose(0, 1), s.W_uv.float()).transpose(0, 1))
    if s.mass is None:
        return
    add = sc.sum((1, 2))
    slots = torch.where(t[None] < s.lens[:, None], pages.repeat_interleave(bs, 1) * bs + t[None] % bs, s.nb * bs)
    m = torch.cat([s.mass.reshape(-1), s.mass.new_zeros(1)])
    m = m.scatter(0, slots.reshape(-1), (s.decay * m[slots] + add).reshape(-1))
    s.mass.copy_(m[:-1].view_as(s.mass))


def _plain_select(s):
    t = torch.arange(s.most, device=DEV)[None]
    m = s.mass[s.table.clamp(min=0).long()].reshape(s.batch, s.most)
    n = s.lens[:, None]
    forced = (t < s.sinks) | (t >= n - s.recent)
    m = torch.where(t < n, torch.where(forced, math.inf, m), -math.inf)
    rank = torch.argsort(torch.sort(m, dim=1, descending=True, stable=True).indices, 1)
    kept = (rank < s.budget) & (t < n)
    at = torch.where(kept, torch.cumsum(kept, 1) - 1, s.budget)
    keep = torch.full((s.batch, s.budget + 1), -1, dtype=torch.int32, device=DEV)
    keep.scatter_(1, at, t.expand_as(at).to(torch.int32))
    keep[:, s.budget] = -1
    s.keep.copy_(keep[:, :s.budget])
    s.new_lens.copy_(kept.sum(1))


def _plain_compact(s):
    b, bs = s.batch, s.bs
    j = torch.arange(s.dst.shape[1] * bs, device=DEV)[None]
    live = j < s.new_lens[:, None]
    k = torch.nn.functional.pad(s.keep, (0, max(0, j.shape[1] - s.budget)), value=-1)[:, :j.shape[1]].long()
    k = torch.where(live, k, 0)
    src = torch.gather(s.table.long(), 1, k // bs)
    sc = torch.where(live, s.scales[src], 0.0)
    page_sc = sc.reshape(b, -1, bs).amax(2)
    to = torch.where(live, s.dst.long().repeat_interleave(bs, 1) * bs + j % bs, s.nb * bs)
    rows = s.cache8.view(-1, ROW8)[src * bs + k % bs]
    ratio = torch.where(live, sc / page_sc.repeat_interleave(bs, 1), 1.0)
    rows[..., :DC] = _codes(_values(rows[..., :DC].contiguous()) * ratio[..., None])
    # the rows behind the kept ones go to one row past the end, which is dropped
    all8 = torch.cat([s.cache8.view(-1, ROW8), rows.new_zeros(1, ROW8)])
    mass = torch.cat([s.mass.reshape(-1), s.mass.new_zeros(1)])
    moved = mass[src * bs + k % bs]
    all8.index_copy_(0, to.reshape(-1), rows.reshape(-1, ROW8))
    mass.scatter_(0, to.reshape(-1), moved.reshape(-1))
    s.cache8.view(-1, ROW8).copy_(all8[:-1])
    s.mass.copy_(mass[:-1].view_as(s.mass))
    scales = torch.cat([s.scales, s.scales.new_zeros(1)])
    scales.scatter_(0, torch.where(s.dst >= 0, s.dst, s.nb).long().reshape(-1), page_sc.reshape(-1))
    s.scales.copy_(scales[:-1])


_PLAIN = {"write": _plain_write, "decode": _plain_decode, "select": _plain_select, "compact": _plain_compact}


# ------------------------------------------------------- the definitions, in 64 bits
def _e4m3(x):
    """Round a float64 tensor to e4m3 values: 4 significant bits, steps of 2^-9 at least, to even, at most 448."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def _table64():
    """The value of each of the 256 e4m3 codes, from its bit fields."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = math.nan if c & 127 == 127 else (-a if c >> 7 else a)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "decode": _exact_decode, "select": _exact_select, "compact": _exact_compact}[s.op](s)


def _ceil_exp(amax):
    """The exponent of a page scale, in Python's integers: the least e with amax <= 448 * 2^e."""
    if not amax > 0:
        return EMIN
    e = math.floor(math.log2(amax)) - 9
    while amax > math.ldexp(448.0, e):
        e += 1
    return max(EMIN, min(EMAX, e))


def _exact_write(s):
    tab = _table64()
    x = s.c_kv.double()
    y = x / torch.sqrt(x.square().sum(1, keepdim=True) / DC + EPS) * s.w.double()
    slots = s.slots.cpu().numpy()
    top = y.abs().max(1).values.cpu().numpy()
    scale = s.scales.double().cpu().numpy()
    old = scale.copy()
    best = np.zeros(s.nb)
    np.maximum.at(best, slots // s.bs, top)
    for p in np.unique(slots // s.bs):
        scale[p] = max(scale[p], 2.0 ** _ceil_exp(best[p]))
    shrink = torch.tensor(np.where(old > 0, old / np.where(scale > 0, scale, 1), 1.0), device=DEV)
    scale = torch.tensor(scale, device=DEV)
    val = tab[s.cache8[..., :DC].long()]
    val = torch.where((shrink < 1)[:, None, None], _e4m3(val * shrink[:, None, None]), val).view(-1, DC)
    val[s.slots] = _e4m3(y / scale[s.slots // s.bs][:, None])
    rope = s.cache8[..., DC:].contiguous().view(torch.bfloat16).double().view(-1, DR)
    k, new = s.k_pe.double(), torch.empty_like(s.k_pe, dtype=torch.float64)
    for i in range(DR // 2):
        a, b = (2 * i, 2 * i + 1) if s.inter else (i, i + DR // 2)
        ang = s.pos.double() / BASE ** (2 * i / DR)
        new[:, a] = k[:, a] * torch.cos(ang) - k[:, b] * torch.sin(ang)
        new[:, b] = k[:, a] * torch.sin(ang) + k[:, b] * torch.cos(ang)
    rope[s.slots] = new
    return {"codes": val.view(s.nb, s.bs, DC), "rope": rope.view(s.nb, s.bs, DR), "scales": scale}


def _exact_decode(s):
    tab = _table64()
    out = torch.zeros(s.batch * s.q, s.heads, DV, dtype=torch.float64, device=DEV)
    mass = s.mass.double().reshape(-1) if s.mass is not None else None
    w = s.W_uv.double()
    for b, n in enumerate(s.lens.tolist()):
        pages = s.table[b, :-(-n // s.bs)].long()
        row = s.cache8[pages].reshape(-1, ROW8)[:n]
        c = tab[row[:, :DC].long()] * s.scales[pages].double().repeat_interleave(s.bs)[:n, None]
        kv = torch.cat([c, row[:, DC:].contiguous().view(torch.bfloat16).double()], 1)
        total = torch.zeros(n, dtype=torch.float64, device=DEV)
        for i in range(0, s.q, 64):
            qr = slice(b * s.q + i, b * s.q + min(s.q, i + 64))
            z = torch.einsum("qhc,tc->qht", s.q_abs[qr].double(), kv) / math.sqrt(192.0)
            seen = n - s.q + i + torch.arange(z.shape[0], device=DEV)
            z = torch.where(torch.arange(n, device=DEV)[None, None] <= seen[:, None, None], z, -math.inf)
            p = torch.softmax(z, 2)
            out[qr] = torch.einsum("qhc,hcv->qhv", torch.einsum("qht,tc->qhc", p, c), w)
            total += p.sum((0, 1))
        if mass is not None:
            at = (pages[:, None] * s.bs + torch.arange(s.bs, device=DEV)[None]).reshape(-1)[:n]
            mass[at] = s.decay * mass[at] + total
    return {"out": out} if mass is None else {"out": out, "mass": mass.view(s.nb, s.bs)}


def _exact_select(s):
    keep = np.full((s.batch, s.budget), -1, np.int32)
    lens = s.lens.cpu().numpy()
    mass, table = s.mass.double().cpu().numpy(), s.table.cpu().numpy()
    for b, n in enumerate(lens):
        m = mass[table[b, :-(-n // s.bs)]].reshape(-1)[:n].copy()
        m[:s.sinks] = np.inf
        m[max(0, n - s.recent):] = np.inf
        best = np.lexsort((np.arange(n), -m))[:s.budget]
        keep[b, :len(best)] = np.sort(best)
    return {"keep": keep, "new_lens": np.minimum(lens, s.budget).astype(np.int32)}


def _exact_compact(s):
    tab = _table64()
    codes, scale = tab[s.cache8[..., :DC].long()].view(-1, DC), s.scales.double()
    rope = s.cache8[..., DC:].contiguous().view(torch.bfloat16).double().view(-1, DR)
    mass = s.mass.double().reshape(-1)
    c2, s2, r2, m2 = codes.clone(), scale.clone(), rope.clone(), mass.clone()
    for b, n in enumerate(s.new_lens.tolist()):
        k = s.keep[b, :n].long()
        page = s.table[b].long()[k // s.bs]
        src = page * s.bs + k % s.bs
        i = torch.arange(n, device=DEV)
        dst_page = s.dst[b].long()[i // s.bs]
        to = dst_page * s.bs + i % s.bs
        top = torch.zeros(-(-n // s.bs), dtype=torch.float64, device=DEV).index_reduce_(0, i // s.bs, scale[page], "amax")
        c2[to] = _e4m3(codes[src] * (scale[page] / top[i // s.bs])[:, None])
        s2[s.dst[b, :len(top)].long()] = top
        r2[to], m2[to] = rope[src], mass[src]
    return {"codes": c2.view(s.nb, s.bs, DC), "rope": r2.view(s.nb, s.bs, DR), "scales": s2, "mass": m2.view(s.nb, s.bs)}
