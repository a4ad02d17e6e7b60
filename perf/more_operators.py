"""Measured cases of the verify pass of a tree of drafted tokens: attention of the tree over a
cache (with a sliding window and first rows that stay visible), penalties, biases and masks on
its logits, the counts those penalties read, the path that is accepted, and the move of that
path's cache rows.

``run`` computes each operator in elementary torch operations where ``own`` is false and
through the framework's entry points where it is true. Lengths follow from the case alone,
trees and values from the seed.

Definitions. A tree has n nodes; node 0 is its root (the last committed token), parent[0] = -1
and 0 <= parent[j] < j; depth counts the steps from the root; anc(j) is j and all nodes above.
  attention  row j (at position ctx + depth) sees cache row p < ctx if there is no window, if
             p > ctx + depth - window or if p < sinks, and row ctx + a of a in anc(j) by the same
             rule at position ctx + depth(a); softmax(q K^T / sqrt(hd)) V over what it sees
  logits     c = generated count of the token, the drafted nodes of anc(j) with it included; seen
             if c > 0 or the prompt has it: y = x / rep (x > 0) or x * rep where seen, then
             - freq c - pres [c > 0] + its biases; -inf where not allowed; ids the argmax
  counts     bit 31: the prompt has the token; bits 0 to 30: times it was generated
  accept     from the root to the lowest child whose token is target[node], until there is none
  commit     cache rows ctx + path[t] move to ctx + t, in every layer
"""
import math

import numpy as np
import torch

own = False

BLOCK = 64            # rows of a page
QWEN3 = dict(heads=32, kv_heads=8, hd=128)   # the drafters' attention shape
VOCAB = 151936        # and vocabulary
LAYERS = 5
PROMPT = -(1 << 31)   # the prompt's bit of a count


def _case(name, op, nb, rows, **kw):
    return dict(name=name, op=op, nb=nb, rows=rows, **kw)


def _attention(name, nb, rows, lo, hi, window=0, sinks=0, paged=True, tree=True, ragged=False, **kw):
    return _case(name, "attention_tree", nb, rows, ctx_lo=lo, ctx_hi=hi, window=window, sinks=sinks, paged=paged,
                 tree=tree, ragged=ragged, **{**QWEN3, **kw})


def listed():
    return [
        # a single user's decode step: latency
        _attention("tree attention one token", 1, 1, 2046, 2046, tree=False),
        # the verify pass of a serving batch: trees of 16 nodes over ragged contexts
        _attention("tree attention trees paged", 64, 16, 1024, 8191),
        # a layer with a sliding window whose first rows stay visible, ragged trees
        _attention("tree attention window", 32, 25, 1024, 8191, window=1024, sinks=4, ragged=True),
        # one very long document under the largest tree
        _attention("tree attention long", 1, 64, 262083, 262083, paged=False),
        # one decoded token with penalties and some biases: latency
        _case("logits one row", "logits_adjust", 1, 1, vocab=VOCAB, bias=32, mask=False, tree=False, ragged=False,
              write=True),
        # the verify pass's logits under penalties, biases and a grammar
        _case("logits trees", "logits_adjust", 64, 16, vocab=VOCAB, bias=300, mask=True, tree=True, ragged=False,
              write=True),
        # what one round emitted in a serving batch
        _case("counts round", "token_counts", 64, 5, vocab=VOCAB, prompt=False, ragged=True),
        # prompts of new requests, some tokens very frequent
        _case("counts prompts", "token_counts", 8, 8189, vocab=VOCAB, prompt=True, ragged=True),
        # one user's tree
        _case("accept one tree", "accept_tree", 1, 16, vocab=VOCAB, ragged=False),
        # a batch of the largest trees
        _case("accept trees", "accept_tree", 64, 64, vocab=VOCAB, ragged=True),
        # the accepted path of one user's tree, every layer
        _case("commit one path", "kv_commit", 1, 16, ctx_lo=2046, ctx_hi=2046, layers=LAYERS, paged=True, ragged=False,
              **QWEN3),
        # a batch of the largest trees
        _case("commit paths", "kv_commit", 64, 64, ctx_lo=200, ctx_hi=900, layers=LAYERS, paged=True, ragged=True,
              **QWEN3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention_tree"] * 4 + ["logits_adjust"] * 3 + ["token_counts", "accept_tree", "kv_commit"])
    nb = _log_int(rng, 1, 64)
    rows = _log_int(rng, 1, 64)
    c = dict(op=op, nb=nb, rows=rows, ragged=rng.random() < 0.5)
    if op in ("attention_tree", "kv_commit"):
        kv = rng.choice([1, 2, 4, 8])
        c.update(QWEN3 if rng.random() < 0.4 else
                 dict(heads=kv * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads=kv, hd=rng.choice([64, 128])))
        c["paged"] = rng.random() < 0.6
    if op == "attention_tree":
        # no more key rows and no more products than the longest listed case has
        most = min(262000, 262083 * 64 * 32 // (rows * c["heads"])) // nb
        hi = _log_int(rng, 1, max(1, most))
        window = rng.random() < 0.4
        c.update(ctx_lo=rng.randint(0, hi), ctx_hi=hi, tree=rng.random() < 0.7,
                 window=_log_int(rng, 1, 8192) if window else 0, sinks=rng.choice([0, 1, 4, 4, 64, 100]) if window else 0)
    elif op == "kv_commit":
        hi = _log_int(rng, 1, 900)
        c.update(ctx_lo=rng.randint(0, hi), ctx_hi=hi, layers=rng.randint(1, LAYERS))
    elif op == "logits_adjust":
        c["rows"] = rows = min(rows, 1024 // nb)
        c.update(vocab=rng.choice([VOCAB, 4096, _log_int(rng, 1000, 151936)]), bias=rng.choice([0, 7, 300]),
                 mask=rng.random() < 0.5, tree=rng.random() < 0.6, write=rng.random() < 0.7)
    elif op == "token_counts":
        c.update(vocab=rng.choice([VOCAB, 4096]), prompt=rng.random() < 0.5)
        c["rows"] = _log_int(rng, 1, 65536 // nb)
    else:
        c["vocab"] = VOCAB
    return c


def _spread(nb):
    return [(0.6180339887 * i + 0.31) % 1.0 for i in range(nb)]


def _lengths(c):
    """(rows in the cache, nodes or tokens) of each sequence, spread over the case's range."""
    g = _spread(c["nb"])
    ctx = [c.get("ctx_lo", 0) + int(u * (c.get("ctx_hi", 0) - c.get("ctx_lo", 0) + 1)) for u in g]
    new = [c["rows"] - (int(((7 * u) % 1.0) * c["rows"]) if c["ragged"] else 0) for u in g]
    return ctx, new


def _pages(c):
    ctx, _ = _lengths(c)
    return -(-(max(ctx) + c["rows"]) // BLOCK) + 1


def work(case):
    c = case
    ctx, new = _lengths(c)
    n = sum(new)
    if c["op"] == "attention_tree":
        hq, hkv, hd = c["heads"], c["kv_heads"], c["hd"]
        w, s = c["window"], c["sinks"]
        # context rows that the root sees (deeper rows see fewer of them), and the tree's own
        old = [a if not w else min(a, w - 1 + min(s, max(0, a - w + 1))) for a in ctx]
        keys = sum(a + b for a, b in zip(old, new))
        pairs = sum(b * (a + 1) for a, b in zip(old, new))
        return {"bytes": keys * hkv * hd * 4 + 4 * n * hq * hd, "flops": 4 * pairs * hq * hd}
    if c["op"] == "logits_adjust":
        v = c["vocab"]
        per_row = 4 * v + (4 * v if c["write"] else 0) + (v // 8 if c["mask"] else 0) + 4
        return {"bytes": n * per_row + c["nb"] * (4 * v + 8 * c["bias"] + 12), "flops": 6 * n * v}
    if c["op"] == "token_counts":
        return {"bytes": 12 * n, "flops": n}
    if c["op"] == "accept_tree":
        return {"bytes": 12 * n + c["nb"] * (8 * c["rows"] + 16), "flops": 2 * n}
    # a path has some eight nodes here, the root among them
    moved = sum(min(b, 8) - 1 for b in new)
    return {"bytes": moved * c["layers"] * c["kv_heads"] * c["hd"] * 8 + 4 * n, "flops": 1}


# ------------------------------------------------------------------ inputs

def _tree(nb, rows, g, dev):
    """Parents of random trees, later nodes more often than earlier ones: some ten levels for 64 nodes."""
    j = torch.arange(rows, device=dev)
    up = (j * torch.rand(nb, rows, generator=g, device=dev).sqrt()).long()
    return torch.where(j > 0, torch.minimum(up, (j - 1).clamp(min=0)), -1).to(torch.int32)


def _zipf(shape, vocab, g, dev):
    """Token ids, low ranks more frequent, ranks spread over the vocabulary."""
    rank = (vocab ** torch.rand(shape, generator=g, device=dev, dtype=torch.float64)).long().clamp(max=vocab - 1)
    return (rank * 7919 % vocab).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    nb, rows = c["nb"], c["rows"]
    ctx, new = _lengths(c)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=g, device=dev)  # noqa: E731
    normal = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    s = {"case": c, "ctx": i32(ctx), "new": i32(new), "longest": max(ctx)}
    hq, hkv, hd, pages, cmax = c.get("heads", 4), c.get("kv_heads", 4), c.get("hd", 64), 0, 64
    if c["op"] in ("attention_tree", "kv_commit"):
        # contiguous caches [layers][nb][kv heads][cmax][hd], or pools [layers][pages][kv heads][64][hd] and a block table
        s["pps"] = pps = _pages(c)
        s["cmax"] = cmax = pps * BLOCK
        s["table"] = None
        if c["paged"]:
            pages = nb * pps + 3
            s["table"] = torch.randperm(pages, generator=g, device=dev)[:nb * pps].to(torch.int32).view(nb, pps)
        shape = (c.get("layers", 1),) + ((pages, hkv) if c["paged"] else (nb, hkv * pps)) + (BLOCK, hd)
        # some key channels stand out
        stand_out = 1.0 + 5.0 * (uni(hd) < 0.05)
        s["kc"] = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g) * stand_out.to(torch.bfloat16)
        s["vc"] = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    if c["op"] == "attention_tree":
        s["q"] = normal(nb, rows, hq, hd).to(torch.bfloat16)
        s["out"] = torch.zeros(nb, rows, hq, hd, dtype=torch.bfloat16, device=dev)
        s["parent"] = _tree(nb, rows, g, dev) if c["tree"] else None
    elif c["op"] == "logits_adjust":
        v = c["vocab"]
        s["logits"] = 3 * normal(nb * rows, v)
        # counts after a prompt and some generated text
        counts = torch.zeros(nb, v, dtype=torch.int32, device=dev)
        said = _zipf((nb, 600), v, g, dev).long()
        counts.scatter_add_(1, said, torch.ones_like(said, dtype=torch.int32))
        heard = _zipf((nb, 3000), v, g, dev).long()
        s["counts"] = counts | torch.zeros_like(counts).scatter_(1, heard, PROMPT)
        s["penalties"] = torch.stack([1 + 0.3 * uni(nb), 0.5 * uni(nb), 0.5 * uni(nb)], dim=1)
        s["bias_ids"] = s["bias"] = s["allowed"] = s["parent"] = s["tokens"] = s["y"] = None
        if c["bias"]:
            s["bias_ids"] = torch.randint(v, (nb, c["bias"]), generator=g, device=dev).to(torch.int32)
            s["bias_ids"][:, -1] = s["bias_ids"][:, 0]        # one id twice
            s["bias"] = 2 * normal(nb, c["bias"])
        if c["mask"]:
            # grammars that allow about half of the tokens
            s["allowed"] = torch.randint(-(1 << 31), 1 << 31, (nb * rows, -(-v // 32)), generator=g,
                                         device=dev).to(torch.int32)
        if c["tree"]:
            s["parent"] = _tree(nb, rows, g, dev)
            s["tokens"] = _zipf((nb, rows), v, g, dev)
        if c["write"]:
            s["y"] = torch.zeros_like(s["logits"])
        s["ids"] = torch.zeros(nb * rows, dtype=torch.int32, device=dev)
    elif c["op"] == "token_counts":
        s["tokens"] = _zipf((nb, rows), c["vocab"], g, dev)
        s["counts"] = torch.zeros(nb, c["vocab"], dtype=torch.int32, device=dev)
    elif c["op"] == "accept_tree":
        # the target follows one of most nodes' children
        s["parent"] = _tree(nb, rows, g, dev)
        s["tokens"] = torch.randint(c["vocab"], (nb, rows), generator=g, device=dev).to(torch.int32)
        j = torch.arange(rows, device=dev)
        wins = torch.where((uni(nb, rows) < 0.9) & (j > 0), j, 0)
        child = torch.zeros(nb, rows, dtype=torch.long, device=dev).scatter_reduce(
            1, s["parent"].long().clamp(min=0), wins, "amax")
        other = torch.randint(c["vocab"], (nb, rows), generator=g, device=dev).to(torch.int32)
        s["target"] = torch.where(child > 0, torch.gather(s["tokens"], 1, child), other)
        s["path"], s["emitted"] = (torch.zeros(nb, rows, dtype=torch.int32, device=dev) for _ in range(2))
        s["tau"], s["bonus"] = (torch.zeros(nb, dtype=torch.int32, device=dev) for _ in range(2))
    else:
        # the path to one of the nodes, as the walk leaves it, and the lengths behind it
        parent = _tree(nb, rows, g, dev)
        end = (uni(nb) * s["new"]).long()
        on = _ancestors(parent)[torch.arange(nb, device=dev), end]
        s["path"], s["tau"] = _path_of(on)
        s["ctx"] = s["ctx"] + s["tau"]
    if own:
        from block_diffusion_speculative_project_gb300 import dflash as D
        cfg = D.dflash_config(D=64 * hkv, Dt=64, L=1, N=c.get("layers", 1), Hq=hq, Hkv=hkv, hd=hd, F=64,
                              V=c.get("vocab", 64), B=2, k_top=1, rope_base=1.0e4, eps=1.0e-6, mask_id=0, Cmax=cmax,
                              max_batch=nb, max_proj_rows=1, conv_group=16, sel_dim=256, flags=0, max_spin=0,
                              film_dim=0, num_pages=pages)
        s["D"], s["h"] = D, D.dflash_create(cfg)
        if s.get("table") is not None:
            D.dflash_set_block_table(s["h"], s["table"])
        s["ws"] = torch.zeros(D.dflash_workspace_size(s["h"]), dtype=torch.uint8, device=dev)
        if c["op"] == "logits_adjust":
            s["rules"] = D.logit_rules(penalties=s["penalties"], counts=s["counts"], bias_ids=s["bias_ids"],
                                       bias=s["bias"], allowed=s["allowed"], parent=s["parent"], tokens=s["tokens"])
    return s


# ------------------------------------------------------------------ plain forms

def _ancestors(parent):
    """[nb, n, n] truth values: node a is node j or above it, at [j, a]."""
    nb, n = parent.shape
    step = torch.zeros(nb, n, n + 1, dtype=torch.float64, device=parent.device)
    step.scatter_(2, parent.long()[..., None] % (n + 1), 1.0)     # a root's step ends beside the tree
    one = torch.eye(n, dtype=torch.float64, device=parent.device)
    return torch.linalg.matrix_power(step[..., :n] + one, max(1, n - 1)) > 0.5


def _path_of(on):
    """The nodes of a path [nb, n] in order, -1 behind them, and their number."""
    n = on.shape[1]
    path = torch.where(on, torch.arange(n, device=on.device), n).sort(dim=1).values
    return torch.where(path < n, path, -1).to(torch.int32), on.sum(dim=1).to(torch.int32)


def _row_index(s, pos):
    """Flat cache row (in units of hd, within a layer) of every kv head at pos [nb, n]: [nb, n, kv heads]."""
    c = s["case"]
    hkv, pps = c["kv_heads"], s["pps"]
    pos = pos.clamp(max=s["cmax"] - 1)
    blk = pos // BLOCK
    if s["table"] is not None:
        first, step = torch.gather(s["table"].long(), 1, blk) * hkv, 1
    else:
        first, step = torch.arange(c["nb"], device=pos.device)[:, None] * (hkv * pps) + blk, pps
    heads = first[..., None] + step * torch.arange(hkv, device=pos.device)
    return heads * BLOCK + (pos % BLOCK)[..., None]


def _plain_attention(s):
    c = s["case"]
    nb, R, hq, hkv, hd, w = c["nb"], c["rows"], c["heads"], c["kv_heads"], c["hd"], c["window"]
    dev = s["ctx"].device
    ctx, new = s["ctx"].long(), s["new"].long()
    j = torch.arange(R, device=dev)
    anc = (j[:, None] >= j).expand(nb, R, R) if s["parent"] is None else _ancestors(s["parent"])
    depth = anc.sum(dim=2) - 1
    L = -(-(s["longest"] + R) // BLOCK) * BLOCK
    p = torch.arange(L, device=dev)
    node = p - ctx[:, None]                                                   # [nb, L], the tree's rows from 0 on
    at = torch.where(node < 0, p, ctx[:, None] + torch.gather(depth, 1, node.clamp(0, R - 1)))
    own_row = torch.gather(anc, 2, node.clamp(0, R - 1)[:, None].expand(nb, R, L))
    seen = torch.where((node < 0)[:, None], True, own_row & (node < new[:, None])[:, None])
    if w:
        lo = ctx[:, None] + depth - w
        seen = seen & ((at[:, None] > lo[..., None]) | (at < c["sinks"])[:, None])
    row = _row_index(s, p.expand(nb, L))
    k, v = (s[name].view(-1, hd)[row].float().transpose(1, 2) for name in ("kc", "vc"))   # [nb, hkv, L, hd]
    G = hq // hkv
    q = s["q"].float().view(nb, R, hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(nb, hkv, R * G, hd)
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(hd)
    x = x.masked_fill(~seen.repeat_interleave(G, dim=1)[:, None], float("-inf"))
    e = torch.exp(x - x.amax(dim=-1, keepdim=True))
    o = torch.matmul(e, v) / e.sum(dim=-1, keepdim=True)
    o = o.view(nb, hkv, R, G, hd).permute(0, 2, 1, 3, 4).reshape(nb, R, hq, hd).to(torch.bfloat16)
    s["out"].copy_(torch.where((j < new[:, None])[..., None, None], o, s["out"]))
    return {"o": s["out"]}


def _plain_logits(s):
    c = s["case"]
    nb, R, v = c["nb"], c["rows"], c["vocab"]
    x = s["logits"].view(nb, R, v)
    drafted = torch.zeros(nb, R, v, dtype=torch.int32, device=x.device)
    if c["tree"]:
        on = _ancestors(s["parent"]) & (torch.arange(R, device=x.device) > 0)
        drafted.scatter_add_(2, s["tokens"].long()[:, None].expand(nb, R, R), on.to(torch.int32))
    counts = s["counts"][:, None]
    gen = (counts & 0x7FFFFFFF) + drafted
    rep, freq, pres = (s["penalties"][:, k, None, None] for k in range(3))
    y = torch.where((counts != 0) | (drafted > 0), torch.where(x > 0, x / rep, x * rep), x)
    y = y - (freq * gen + pres * (gen > 0))
    if c["bias"]:
        y = y + torch.zeros(nb, v, device=x.device).scatter_add_(1, s["bias_ids"].long(), s["bias"])[:, None]
    if c["mask"]:
        at = torch.arange(v, device=x.device)
        y = y.masked_fill(((s["allowed"].view(nb, R, -1)[..., at // 32] >> (at % 32).to(torch.int32)) & 1) == 0,
                          float("-inf"))
    live = torch.arange(R, device=x.device) < s["new"][:, None]
    best = y.amax(dim=-1, keepdim=True)
    at = torch.arange(v, device=x.device, dtype=torch.int32)
    ids = torch.where(y == best, at, v).amin(dim=-1)
    ids = torch.where(best[..., 0] > float("-inf"), ids, -1).to(torch.int32)
    s["ids"].copy_(torch.where(live, ids, s["ids"].view(nb, R)).view(-1))
    if c["write"]:
        s["y"].copy_(torch.where(live[..., None], y, s["y"].view(nb, R, v)).view(-1, v))
    return {"y": s["y"], "ids": s["ids"]}


def _plain(s):
    c = s["case"]
    nb, R = c["nb"], c["rows"]
    dev = s["ctx"].device
    if c["op"] == "attention_tree":
        return _plain_attention(s)
    if c["op"] == "logits_adjust":
        return _plain_logits(s)
    j = torch.arange(R, device=dev)
    live = j < s["new"][:, None]
    if c["op"] == "token_counts":
        t = s["tokens"].long()
        now = torch.zeros_like(s["counts"]).scatter_add_(1, t, live.to(torch.int32))
        s["counts"].copy_(s["counts"] | torch.where(now > 0, PROMPT, 0) if c["prompt"] else s["counts"] + now)
        return {"counts": s["counts"]}
    if c["op"] == "accept_tree":
        up = s["parent"].long().clamp(min=0)
        fits = (s["tokens"] == torch.gather(s["target"], 1, up)) & live & (j > 0)
        # of the children that fit the lowest alone
        first = torch.full((nb, R), R, device=dev).scatter_reduce(1, up, torch.where(fits, j, R), "amin")
        fits = fits & (torch.gather(first, 1, up) == j) | (j == 0) & live
        on = (fits[:, None] | ~_ancestors(s["parent"])).all(dim=2)
        path, tau = _path_of(on)
        s["path"].copy_(path)
        s["tau"].copy_(tau)
        last = torch.gather(path, 1, (tau.long() - 1).clamp(min=0)[:, None]).long().clamp(min=0)
        s["bonus"].copy_(torch.gather(s["target"], 1, last)[:, 0])
        step = torch.gather(s["tokens"], 1, path.long().clamp(min=0).roll(-1, dims=1))
        s["emitted"].copy_(torch.where(j < tau[:, None] - 1, step, torch.where(j == tau[:, None] - 1, s["bonus"][:, None], -1)))
        s["ctx"] += tau
        return {"tau": s["tau"], "bonus": s["bonus"], "path": s["path"], "emitted": s["emitted"], "ctx": s["ctx"]}
    # rows behind the path write row 0 again, to its own place
    t = torch.where(j < s["tau"][:, None], j, 0)
    base = (s["ctx"] - s["tau"]).long()[:, None]
    src = _row_index(s, base + torch.gather(s["path"].long(), 1, t))
    dst = _row_index(s, base + t)
    for name in ("kc", "vc"):
        flat = s[name].view(c["layers"], -1, c["hd"])
        flat[:, dst] = flat[:, src]
    return {"k": s["kc"], "v": s["vc"]}


def run(s):
    if not own:
        return _plain(s)
    c, D, h = s["case"], s["D"], s["h"]
    nb, R = c["nb"], c["rows"]
    if c["op"] == "attention_tree":
        D.dflash_attention_tree(h, nb, 0, R, s["q"], s["kc"], s["vc"], s["parent"], s["new"], s["ctx"], s["longest"],
                                c["window"], c["sinks"], s["out"], s["ws"])
        return {"o": s["out"]}
    if c["op"] == "logits_adjust":
        v = c["vocab"]
        D.dflash_logits_adjust(h, nb, R, s["logits"], v, s["rules"], s["new"], s["y"], v, s["ids"], s["ws"])
        return {"y": s["y"], "ids": s["ids"]}
    if c["op"] == "token_counts":
        D.dflash_token_counts(h, nb, R, s["tokens"], R, s["new"], int(c["prompt"]), s["counts"], s["ws"])
        return {"counts": s["counts"]}
    if c["op"] == "accept_tree":
        D.dflash_accept_tree(h, nb, R, s["parent"], s["tokens"], s["target"], s["new"], s["ctx"], s["tau"], s["bonus"],
                             s["path"], s["emitted"], s["ws"])
        return {"tau": s["tau"], "bonus": s["bonus"], "path": s["path"], "emitted": s["emitted"], "ctx": s["ctx"]}
    D.dflash_kv_commit(h, nb, R, s["path"], s["tau"], s["ctx"], s["kc"], s["vc"], s["ws"])
    return {"k": s["kc"], "v": s["vc"]}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _up(parents, j):
    """j and the nodes above it, of one tree."""
    found = [j]
    while parents[found[-1]] >= 0:
        found.append(parents[found[-1]])
    return found


def exact(case, seed):
    if case["op"] not in ("attention_tree", "logits_adjust") or case["op"] == "logits_adjust" and not case["write"]:
        return None     # whole numbers and rows as they are
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = s["case"]
    nb, R = c["nb"], c["rows"]
    ctx, new = _lengths(c)
    parents = s["parent"].tolist() if s["parent"] is not None else [[j - 1 for j in range(R)]] * nb
    if c["op"] == "logits_adjust":
        if sum(new) * c["vocab"] > 6e7:
            return None
        v = c["vocab"]
        y = torch.zeros(nb * R, v, dtype=torch.float64, device=s["ctx"].device)
        for i in range(nb):
            said = s["counts"][i].long()
            rep, freq, pres = s["penalties"][i].double()
            add = np.zeros(v)
            if c["bias"]:
                np.add.at(add, s["bias_ids"][i].cpu().numpy(), s["bias"][i].double().cpu().numpy())
            add = torch.from_numpy(add).to(y.device)
            for j in range(new[i]):
                count, heard = said % (1 << 31), said != 0
                if c["tree"]:
                    for a in _up(parents[i], j)[:-1]:
                        t = int(s["tokens"][i, a])
                        count[t] += 1
                        heard[t] = True
                x = s["logits"][i * R + j].double()
                z = torch.where(heard, torch.where(x > 0, x / rep, x * rep), x)
                z = z - freq * count - pres * (count > 0) + add
                if c["mask"]:
                    bits = s["allowed"][i * R + j].cpu().numpy().view(np.uint8)
                    ok = torch.from_numpy(np.unpackbits(bits, bitorder="little")[:v].astype(bool)).to(y.device)
                    z = torch.where(ok, z, torch.full_like(z, -math.inf))
                y[i * R + j] = z
        return {"y": y, "ids": None}
    hq, hkv, hd, w = c["heads"], c["kv_heads"], c["hd"], c["window"]
    if sum(a + b for a, b in zip(ctx, new)) * hq * R > 4e8:
        return None     # minutes in 64 bits
    table = None if s["table"] is None else s["table"].tolist()
    out = s["out"].double()
    G = hq // hkv
    for i in range(nb):
        n = ctx[i] + new[i]
        nblk = -(-n // BLOCK)
        lines = [_up(parents[i], j) for j in range(new[i])]
        depth = [len(a) - 1 for a in lines]
        seen = torch.zeros(new[i], n, dtype=torch.bool)
        place = torch.tensor(list(range(ctx[i])) + [ctx[i] + d for d in depth])
        for j, line in enumerate(lines):
            seen[j, :ctx[i]] = True
            seen[j, [ctx[i] + a for a in line]] = True
            if w:
                seen[j] &= (place > ctx[i] + depth[j] - w) | (place < c["sinks"])
        hide = ~seen.to(out.device)
        for h in range(hkv):
            at = [(table[i][b], h) if table else (i, h * s["pps"] + b) for b in range(nblk)]
            a0, a1 = [a[0] for a in at], [a[1] for a in at]
            K, V = (s[name][0][a0, a1].double().view(-1, hd)[:n] for name in ("kc", "vc"))
            q = s["q"][i, :new[i], h * G:(h + 1) * G].double()
            x = torch.einsum("jgd,td->jgt", q, K) * hd ** -0.5
            x = x.masked_fill(hide[:, None], -math.inf)
            out[i, :new[i], h * G:(h + 1) * G] = torch.einsum("jgt,td->jgd", torch.softmax(x, dim=-1), V)
    return {"o": out}
