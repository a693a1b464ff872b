"""Operators of a speculative step over a tree of drafted tokens, as one pass of a user's program each.

  plan    from the tree's parents: each row's position, its mask (the row and its ancestors) and
          the cache slot that its latent goes to
  attend  latent attention of absorbed queries over a paged cache whose last rows are the tree:
          all that came before is seen, of the tree what the mask says; projected to v_head_dim
  verify  which path of the tree the target's probabilities accept, from given random numbers,
          and the token that follows it
  commit  the accepted rows moved behind the past, in every layer's cache

A sequence's rows are its tree in an order in which a parent comes before its children; row 0 is
the last token that was accepted before. A cache row is 512 latents and 64 rope values in bf16.
"""

import math
import random

import torch

own = False

DC, DR, DV, ROW = 512, 64, 128, 576
STEP = 40                     # weights of a draw count in steps of 2^-40
DEV = "cuda"


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # the serving batch, 8 rows each: the step's plan
        {"name": "plan_serving", "op": "plan", "batch": 64, "nodes": 8, "spread": 3, "len": 4096, "vary": 500, "bs": 64, "lens": 1},
        # wide trees of a large batch
        {"name": "plan_wide", "op": "plan", "batch": 256, "nodes": 333, "spread": 60, "len": 2000, "vary": 1500, "bs": 16, "lens": 2},
        # the serving batch: 64 sequences of 4096 tokens, a tree of 8 rows each
        {"name": "attend_serving", "op": "attend", "batch": 64, "heads": 16, "nodes": 8, "spread": 3, "len": 4096, "vary": 0, "bs": 64, "lens": 3},
        # one request a few hundred tokens in: latency
        {"name": "attend_single", "op": "attend", "batch": 1, "heads": 16, "nodes": 6, "spread": 2, "len": 333, "vary": 0, "bs": 16, "lens": 4},
        # many rows to a sequence, lengths from 2000 to 8000
        {"name": "attend_wide", "op": "attend", "batch": 16, "heads": 16, "nodes": 61, "spread": 20, "len": 8000, "vary": 6000, "bs": 64, "lens": 5},
        # many heads over ragged lengths up to 32768
        {"name": "attend_ragged_h128", "op": "attend", "batch": 8, "heads": 128, "nodes": 4, "spread": 2, "len": 32768, "vary": 32700, "bs": 32, "lens": 6},
        # chains of five drafted tokens with their draft's probabilities
        {"name": "verify_chains", "op": "verify", "batch": 64, "nodes": 6, "spread": 0, "vocab": 102400, "draft": True, "lens": 7},
        # one request, a tree of the draft's likeliest tokens
        {"name": "verify_single", "op": "verify", "batch": 1, "nodes": 26, "spread": 8, "vocab": 32000, "draft": False, "lens": 8},
        # trees of sampled tokens: a rejected one leaves its sibling the rest of the distribution
        {"name": "verify_trees", "op": "verify", "batch": 32, "nodes": 16, "spread": 5, "vocab": 50001, "draft": True, "lens": 9},
        # the serving batch's accepted rows in 27 layers
        {"name": "commit_serving", "op": "commit", "batch": 64, "nodes": 8, "spread": 3, "len": 128, "vary": 60, "layers": 27, "bs": 64, "lens": 10},
        # one request, one layer
        {"name": "commit_single", "op": "commit", "batch": 1, "nodes": 26, "spread": 8, "len": 1000, "vary": 0, "layers": 1, "bs": 16, "lens": 11},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "attend", "attend", "attend", "verify", "verify", "commit"])
    c = {"op": op, "batch": _log(rng, 1, 64), "nodes": _log(rng, 1, 200), "lens": rng.randrange(1 << 20)}
    c["spread"] = rng.choice([0, rng.randint(1, 8), rng.randint(0, c["nodes"])])
    if op == "verify":
        c["vocab"] = _log(rng, 1000, 110000)
        c["nodes"] = _log(rng, 1, 64)
        c["batch"] = max(1, min(c["batch"], 50_000_000 // (c["nodes"] * c["vocab"])))
        c["draft"] = rng.random() < 0.6
        return c
    c["bs"] = rng.choice([16, 32, 64])
    if op == "attend":
        c["heads"] = rng.choice([16, 16, 32, 64, 128])
        room = 60_000_000 // (c["batch"] * c["heads"] * c["nodes"])
        if room < max(64, c["nodes"]):
            c["batch"] = 1
            room = 60_000_000 // (c["heads"] * c["nodes"])
        most = min(32768, room, max(64, 262144 // c["batch"])) - c["nodes"]
        c["len"] = c["nodes"] + rng.choice([0, _log(rng, 1, max(1, most)), _log(rng, 64, max(64, most))])
    else:
        c["len"] = c["nodes"] + _log(rng, 1, 4000 if op == "plan" else 200)
    c["vary"] = rng.randrange(c["len"] - c["nodes"] + 1)
    if op == "plan":
        c["batch"] = _log(rng, 1, 256)
    elif op == "commit":
        c["layers"] = max(1, min(27, _log(rng, 1, 27), 150_000 // (c["batch"] * (c["len"] + c["bs"]))))
    return c


def _lens(case):
    """Each sequence's length, its tree included: it goes by the case alone."""
    r = random.Random(case["lens"])
    return [case["len"] - (r.randint(0, case["vary"]) if case["vary"] else 0) for _ in range(case["batch"])]


def _trees(case):
    """Each sequence's tree, by the case alone: a row's parent is one of the rows shortly before it."""
    r = random.Random(case["lens"] + 1)
    return [[-1] + [r.randint(max(0, i - 1 - case["spread"]), i - 1) for i in range(1, case["nodes"])]
            for _ in range(case["batch"])]


def _depths(tree):
    d = []
    for p in tree:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _paths(case):
    """An accepted path for each sequence: from a row of the tree up to its root."""
    r = random.Random(case["lens"] + 2)
    out = []
    for tree in _trees(case):
        i, path = r.randrange(len(tree)), []
        while i >= 0:
            path.append(i)
            i = tree[i]
        out.append(path[::-1])
    return out


def _words(case):
    return (case["nodes"] + 63) // 64


def work(case):
    op, b, t = case["op"], case["batch"], case["nodes"]
    if op == "plan":
        pages = sum(-(-n // case["bs"]) - (n - t) // case["bs"] for n in _lens(case))
        return {"bytes": b * t * (4 + 8 * _words(case) + 4 + 8) + pages * 4 + b * 8, "flops": b * t}
    if op == "attend":
        lens, h = _lens(case), case["heads"]
        seen = sum(t * (n - t) + sum(d + 1 for d in _depths(tree)) for n, tree in zip(lens, _trees(case)))
        moved = sum(lens) * ROW * 2 + sum(-(-n // case["bs"]) for n in lens) * 4
        moved += b * t * (h * (ROW + DV) * 2 + 8 * _words(case)) + h * DC * DV * 2
        return {"bytes": moved, "flops": h * 2 * (seen * (ROW + DC) + b * t * DC * DV)}
    if op == "verify":
        return {"bytes": b * case["vocab"] * (8 if case["draft"] else 4) + b * t * 12, "flops": b * case["vocab"] * 3}
    rows = sum(i != p for path in _paths(case) for i, p in enumerate(path))
    return {"bytes": max(1, rows) * case["layers"] * ROW * 2 * 2 + b * 16, "flops": max(1, rows)}


# --------------------------------------------------------------------------------- inputs
class _State:
    pass


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = _State()
    s.op, s.batch, s.nodes, s.words = case["op"], case["batch"], case["nodes"], _words(case)
    s.qsl = torch.arange(0, s.batch * s.nodes + 1, s.nodes, dtype=torch.int32, device=DEV)
    trees = _trees(case)
    s.parents = _ints([p for tree in trees for p in tree])
    if s.op == "verify":
        _prepare_verify(s, case, gen, trees)
    else:
        lens, s.bs = _lens(case), case["bs"]
        s.lens = _ints(lens)
        need = [-(-n // s.bs) for n in lens]
        s.nb, s.most = sum(need), max(need)
        perm = torch.randperm(s.nb, generator=gen, device=DEV).to(torch.int32).tolist()
        table, at = [], 0
        for k in need:
            table.append(perm[at:at + k] + [-1] * (s.most - k))
            at += k
        s.table = _ints(table)
        {"plan": _prepare_plan, "attend": _prepare_attend, "commit": _prepare_commit}[s.op](s, case, gen, trees)
    if own:
        _prepare_own(s, case)
    return s


def _prepare_plan(s, case, gen, trees):
    n = s.batch * s.nodes
    s.mask = torch.empty(n, s.words, dtype=torch.int64, device=DEV)
    s.pos = torch.empty(n, dtype=torch.int32, device=DEV)
    s.slots = torch.empty(n, dtype=torch.int64, device=DEV)


def _mask(trees, words):
    """The rows' masks, in Python's integers: word w of a row holds the tree's rows 64 w and on."""
    out = []
    for tree in trees:
        seen = []
        for i, p in enumerate(tree):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        for m in seen:
            row = [(m >> 64 * w) & (1 << 64) - 1 for w in range(words)]
            out.append([x - (1 << 64) if x >> 63 else x for x in row])
    return _ints(out, torch.int64)


def _prepare_attend(s, case, gen, trees):
    s.heads = case["heads"]
    n = s.batch * s.nodes
    s.mask = _mask(trees, s.words)
    s.cache = _randn(gen, s.nb, s.bs, ROW).bfloat16()
    # what lies behind a sequence's last token was never written
    last = [n // s.bs for n in _lens(case)]
    for b, m in enumerate(_lens(case)):
        if m % s.bs:
            s.cache[s.table[b, last[b]].long(), m % s.bs:] = math.nan
    # some heads look at a few tokens, some at all of them
    sharp = torch.exp2(torch.rand(1, s.heads, 1, generator=gen, device=DEV) * 4 - 2)
    size = torch.cat([torch.full((DC,), 0.5), torch.ones(DR)]).to(DEV)
    s.q_abs = (_randn(gen, n, s.heads, ROW) * sharp * size).bfloat16()
    s.W_uv = (_randn(gen, s.heads, DC, DV) / math.sqrt(DC)).bfloat16()
    s.out = torch.empty(n, s.heads, DV, dtype=torch.bfloat16, device=DEV)


def _prepare_verify(s, case, gen, trees):
    n, v = s.batch * s.nodes, case["vocab"]
    s.vocab = v
    logits = _randn(gen, n, v) * 2.5
    s.p = torch.softmax(logits, 1)
    q = torch.softmax(logits * 0.9 + 0.7 * _randn(gen, n, v), 1)  # the draft knows the target fairly well
    base = torch.arange(s.batch, device=DEV)[:, None] * s.nodes
    up = (s.parents.view(s.batch, -1).clamp(min=0) + base).reshape(-1).long()
    if case["draft"]:  # drawn from the draft's distribution at the parent
        best = torch.empty(n, dtype=torch.int64, device=DEV)
        for i in range(0, n, 256):
            k = min(256, n - i)
            e = -torch.log(1 - torch.rand(k, v, generator=gen, device=DEV))
            best[i:i + k] = (q[up[i:i + k]] / e).argmax(1)
        s.tokens, s.q = best.to(torch.int32), q
    else:  # the draft's likeliest, one after another
        rank, most = [], 0
        for tree in trees:
            seen = {}
            for p in tree:
                rank.append(seen.get(p, 0))
                seen[p] = rank[-1] + 1
                most = max(most, seen[p])
        top = q.topk(most, 1).indices
        s.tokens = top[up, _ints(rank, torch.int64)].to(torch.int32)
        s.q = None
    s.u = torch.rand(n, generator=gen, device=DEV)
    s.u_last = torch.rand(s.batch, generator=gen, device=DEV)
    s.max_path = max(max(_depths(tree)) for tree in trees) + 1
    s.path = torch.empty(s.batch, s.max_path, dtype=torch.int32, device=DEV)
    s.path_lens = torch.empty(s.batch, dtype=torch.int32, device=DEV)
    s.next = torch.empty(s.batch, dtype=torch.int32, device=DEV)


def _prepare_commit(s, case, gen, trees):
    s.cache = torch.empty(case["layers"], s.nb, s.bs, ROW, dtype=torch.bfloat16, device=DEV)
    for i in range(case["layers"]):
        s.cache[i] = _randn(gen, s.nb, s.bs, ROW).bfloat16()
    paths = _paths(case)
    s.max_path = max(len(p) for p in paths)
    s.path = _ints([p + [-1] * (s.max_path - len(p)) for p in paths])
    s.path_lens = _ints([len(p) for p in paths])
    s.new_lens = torch.empty(s.batch, dtype=torch.int32, device=DEV)


def _prepare_own(s, case):
    """What the framework's calls need beside the data: a configuration, a workspace, a status word."""
    from mla_latent_kv_03_gb300 import libmla as L
    s.L = L
    s.status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if s.op == "verify":
        return
    s.cfg = L.make_config(getattr(s, "heads", 16), s.bs, "bf16")
    if s.op == "attend":
        n = L.mla_tree_decode_workspace_size(s.cfg, s.q_abs.shape[0], s.batch)
        s.ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        L.mla_workspace_init(s.ws)


# ------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        _OWN[s.op](s)
    else:
        _PLAIN[s.op](s)
    return _OUT[s.op](s)


def _own_plan(s):
    s.L.mla_tree_plan(s.cfg, s.parents, s.lens, s.qsl, s.table, s.nb, s.mask, s.pos, s.slots, dev_status=s.status)


def _own_attend(s):
    s.L.mla_tree_decode(s.cfg, s.q_abs, s.cache, s.table, s.lens, s.qsl, s.mask, s.W_uv, s.ws, s.out)


def _own_verify(s):
    s.L.mla_tree_verify(s.p, s.q, s.tokens, s.parents, s.qsl, s.u, s.u_last, s.path, s.path_lens, s.next, dev_status=s.status)


def _own_commit(s):
    s.L.mla_tree_commit(s.cfg, s.cache, s.table, s.lens, s.qsl, s.path, s.path_lens, s.new_lens, dev_status=s.status)


_OWN = {"plan": _own_plan, "attend": _own_attend, "verify": _own_verify, "commit": _own_commit}
_OUT = {
    "plan": lambda s: {"mask": s.mask, "positions": s.pos, "slots": s.slots},
    "attend": lambda s: {"out": s.out},
    "verify": lambda s: {"path": s.path, "path_lens": s.path_lens, "next": s.next},
    "commit": lambda s: {"cache": s.cache, "new_lens": s.new_lens},
}


# ------------------------------------------------------------------------- the plain forms
def _plain_plan(s):
    b, t = s.batch, s.nodes
    up = s.parents.view(b, t).long()
    i = torch.arange(t, device=DEV)
    seen = torch.zeros(b, t, t, dtype=torch.bool, device=DEV)
    depth = torch.full((b, t), -1, device=DEV)
    at = i.expand(b, t)
    # a step up the tree at a time; a row past its root stays outside
    for _ in range(t):
        live = at >= 0
        seen |= (at[..., None] == i) & live[..., None]
        depth += live
        at = torch.where(live, torch.gather(up, 1, at.clamp(min=0)), -1)
    bits = torch.nn.functional.pad(seen, (0, 64 * s.words - t)).view(b, t, s.words, 64)
    s.mask.copy_((bits.long() << torch.arange(64, device=DEV)).sum(3).view(b * t, s.words))
    past = (s.lens - t).long()[:, None]
    s.pos.copy_((past + depth).reshape(-1))
    where = past + i
    s.slots.copy_((torch.gather(s.table.long(), 1, where // s.bs) * s.bs + where % s.bs).reshape(-1))


def _plain_attend(s):
    b, h, t = s.batch, s.heads, s.nodes
    most = s.most * s.bs
    at = torch.arange(most, device=DEV)
    there = at < s.lens[:, None]
    kv = s.cache[s.table.clamp(min=0).long()].reshape(b, most, ROW).float()
    kv.masked_fill_(~there[..., None], 0)
    sc = torch.bmm(s.q_abs.float().reshape(b, t * h, ROW), kv.transpose(1, 2)).mul_(192.0 ** -0.5)
    sc = sc.view(b, t, h, most)
    bits = ((s.mask[:, :, None] >> torch.arange(64, device=DEV)) & 1).bool().view(b, t, -1)
    past = (s.lens - t).long()[:, None]
    j = (at - past).clamp(0, bits.shape[2] - 1)
    seen = torch.gather(bits, 2, j[:, None].expand(b, t, most)) & (at >= past)[:, None] | (at < past)[:, None]
    sc.masked_fill_(~(seen & there[:, None])[:, :, None], -math.inf)
    sc -= sc.amax(3, keepdim=True).clamp(min=-1e30)
    sc.exp_()
    sc /= sc.sum(3, keepdim=True).clamp(min=1e-30)
    o = torch.bmm(sc.view(b, t * h, most), kv[..., :DC]).view(b * t, h, DC)
    s.out.copy_(torch.bmm(o.transpose(0, 1), s.W_uv.float()).transpose(0, 1))


def _plain_verify(s):
    b, t = s.batch, s.nodes
    base = torch.arange(b, device=DEV) * t
    cur = torch.zeros(b, dtype=torch.int64, device=DEV)
    z = torch.ones(b, dtype=torch.float64, device=DEV)
    w = s.p[base].clamp(0, 1)
    up, tok = s.parents.view(b, t), s.tokens.view(b, t).long()
    s.path.fill_(-1)
    s.path[:, 0] = 0
    n = torch.ones(b, dtype=torch.int64, device=DEV)
    for i in range(1, t):  # a row is asked when its parent is the last accepted one
        x = tok[:, i, None]
        wx = torch.gather(w, 1, x)[:, 0].double()
        u = s.u[base + i].double()
        if s.q is not None:
            u = u * s.q[base + cur, x[:, 0]].double()
        asked = up[:, i] == cur
        yes, no = asked & (u * z < wx), asked & ~(u * z < wx)
        # accepted: the walk goes on from row i
        at = n.clamp(max=s.max_path - 1)[:, None]
        s.path.scatter_(1, at, torch.where(yes[:, None], i, s.path.gather(1, at)).to(torch.int32))
        n += yes
        # rejected: what the draft had is taken out of the rest
        if s.q is not None:
            less = (w.double() - z[:, None] * s.q[base + cur].double()).float().clamp(min=0)
            z = torch.where(no, (less.double() * 2.0 ** STEP).floor().sum(1).mul(2.0 ** -STEP).float().double(), z)
        else:
            less = w.scatter(1, x, 0.0)
            z = torch.where(no, (z - wx).clamp(min=0), z)
        cur = torch.where(yes, i, cur)
        w = torch.where(yes[:, None], s.p[base + cur].clamp(0, 1), torch.where(no[:, None], less, w))
        z = torch.where(yes, 1.0, z)
    k = (w.double() * 2.0 ** STEP).long()
    empty = k.sum(1) == 0
    k = torch.where(empty[:, None], (s.p[base + cur].clamp(0, 1).double() * 2.0 ** STEP).long(), k)
    upto = torch.cumsum(k, 1)
    goal = (s.u_last.double() * upto[:, -1].double()).floor().long()
    s.next.copy_((upto <= goal[:, None]).sum(1))
    s.path_lens.copy_(n)


def _plain_commit(s):
    past = (s.lens - s.nodes).long()[:, None]
    i = torch.arange(s.max_path, device=DEV)[None]

    def slot(where):
        return torch.gather(s.table.long(), 1, where // s.bs) * s.bs + where % s.bs

    live = (i < s.path_lens[:, None]).reshape(-1)
    src = slot(past + s.path.clamp(min=0)).reshape(-1)
    # the places behind a path are one row past the cache, which is dropped
    dst = torch.where(live, slot((past + i).clamp(max=s.most * s.bs - 1)).reshape(-1), s.nb * s.bs)
    for layer in s.cache:
        rows = layer.view(-1, ROW)
        all_rows = torch.cat([rows, rows.new_zeros(1, ROW)])
        all_rows[dst] = rows[src]
        rows.copy_(all_rows[:-1])
    s.new_lens.copy_(past[:, 0] + s.path_lens)


_PLAIN = {"plan": _plain_plan, "attend": _plain_attend, "verify": _plain_verify, "commit": _plain_commit}


# ------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "attend": _exact_attend, "verify": _exact_verify, "commit": _exact_commit}[s.op](s, case)


def _exact_plan(s, case):
    pos, slots, table = [], [], s.table.tolist()
    for b, (n, tree) in enumerate(zip(_lens(case), _trees(case))):
        past = n - len(tree)
        pos += [past + d for d in _depths(tree)]
        slots += [table[b][j // s.bs] * s.bs + j % s.bs for j in range(past, n)]
    return {"mask": _mask(_trees(case), s.words), "positions": _ints(pos), "slots": _ints(slots, torch.int64)}


def _exact_attend(s, case):
    out = torch.zeros(s.batch * s.nodes, s.heads, DV, dtype=torch.float64, device=DEV)
    w = s.W_uv.double()
    for b, (n, tree) in enumerate(zip(_lens(case), _trees(case))):
        kv = s.cache[s.table[b, :-(-n // s.bs)].long()].reshape(-1, ROW)[:n].double()
        past, chains = n - s.nodes, []
        for i, p in enumerate(tree):
            chains.append((chains[p] if p >= 0 else []) + [i])
        for i in range(0, s.nodes, 16):
            some = chains[i:i + 16]
            seen = torch.zeros(len(some), n, dtype=torch.bool)
            seen[:, :past] = True
            for r, c in enumerate(some):
                seen[r, [past + j for j in c]] = True
            rows = slice(b * s.nodes + i, b * s.nodes + i + len(some))
            z = torch.einsum("qhc,tc->qht", s.q_abs[rows].double(), kv) / math.sqrt(192.0)
            z = torch.where(seen.to(DEV)[:, None], z, -math.inf)
            o = torch.einsum("qht,tc->qhc", torch.softmax(z, 2), kv[:, :DC])
            out[rows] = torch.einsum("qhc,hcv->qhv", o, w)
    return {"out": out}


def _exact_verify(s, case):
    path, lens, after = [], [], []
    u, u_last, tokens = s.u.tolist(), s.u_last.tolist(), s.tokens.tolist()
    for b, tree in enumerate(_trees(case)):
        base, cur, chain, i = b * s.nodes, 0, [0], 0
        w, z = s.p[base].double().clamp(0, 1), 1.0
        while True:  # the next row, in order, whose parent is the last accepted one
            i = next((j for j in range(i + 1, s.nodes) if tree[j] == cur), None)
            if i is None:
                break
            x = tokens[base + i]
            share = s.q[base + cur, x].item() if s.q is not None else 1.0
            if u[base + i] * share * z < w[x].item():
                cur = i
                chain.append(i)
                w, z = s.p[base + cur].double().clamp(0, 1), 1.0
            elif s.q is not None:
                w = (w - z * s.q[base + cur].double()).float().double().clamp(min=0)
                z = float(torch.tensor((w * 2.0 ** STEP).long().sum().item() * 2.0 ** -STEP, dtype=torch.float32))
            else:
                z = max(z - w[x].item(), 0.0)
                w[x] = 0
        k = (w * 2.0 ** STEP).long()
        if not k.sum().item():
            k = (s.p[base + cur].double().clamp(0, 1) * 2.0 ** STEP).long()
        goal = math.floor(u_last[b] * k.sum().item())
        after.append(int(torch.nonzero(torch.cumsum(k, 0) > goal)[0]))
        path.append(chain + [-1] * (s.max_path - len(chain)))
        lens.append(len(chain))
    return {"path": _ints(path), "path_lens": _ints(lens), "next": _ints(after)}


def _exact_commit(s, case):
    new, lens = s.cache.clone(), []
    table = s.table.tolist()
    for b, (n, path) in enumerate(zip(_lens(case), _paths(case))):
        past = n - s.nodes
        for i, p in enumerate(path):
            a, c = past + i, past + p
            new[:, table[b][a // s.bs], a % s.bs] = s.cache[:, table[b][c // s.bs], c % s.bs]
        lens.append(past + len(path))
    return {"cache": new, "new_lens": _ints(lens)}
