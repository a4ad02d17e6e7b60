"""Trees of drafted tokens through the C ABI: attention over the bf16 caches with a tree's mask, a sliding
window and first rows that stay visible; penalties, biases and masks on logits; token counts; the accepted
path and the move of its cache rows. Against the fp64 oracle.

Tolerances (u = half a step of a type relative to the value: bf16 2^-8, f32 2^-24):
  attention  one bf16 rounding 2^-8 |o|; every probability rounded to bf16, 2^-8 sum p|v|; scores: hd
             products and sums in fp32, hd 2^-24 max sum|q k| / sqrt(hd), which move p by twice that at
             most; exponents up to 2^7 in fp32 steps, the fast exp2 and the sums over the keys: below
             2^-14 of sum p|v|
  logits     a quotient or product, a product with a sum, a difference and one sum for each bias, each 2^-24 of
             at most |x| max(rep, 1/rep) + freq c + pres + sum|bias|: (4 + biases of the token) 2^-24 of it
  the rest   exact
"""
import numpy as np
import pytest
import torch

from oracle import dflash_oracle as orc

pytestmark = pytest.mark.gpu

PR = orc.PAGE_ROWS


def lib():
    from block_diffusion_speculative_project_gb300 import dflash
    return dflash


def i32(a):
    return None if a is None else torch.tensor(np.asarray(a, np.int32), device="cuda")


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Target:
    """A handle with bf16 caches of seeded values, and their numpy view."""

    def __init__(self, Hq=4, Hkv=2, hd=64, Cmax=256, nb=2, N=1, B=2, V=64, paged=True, spare=2, seed=0, max_spin=0,
                 flags=0):
        D = lib()
        self.D, self.Hq, self.Hkv, self.hd, self.Cmax, self.nb, self.N, self.V = D, Hq, Hkv, hd, Cmax, nb, N, V
        self.pps = -(-Cmax // PR)
        rng = np.random.default_rng(seed)
        P = nb * self.pps + spare if paged else 0
        self.table = rng.permutation(P)[:nb * self.pps].reshape(nb, self.pps) if paged else None
        cfg = D.dflash_config(D=64, Dt=64, L=1, N=N, Hq=Hq, Hkv=Hkv, hd=hd, F=64, V=V, B=B, k_top=1, rope_base=1e4,
                              eps=1e-6, mask_id=0, Cmax=Cmax, max_batch=nb, max_proj_rows=1, conv_group=16,
                              sel_dim=256, flags=flags, max_spin=max_spin, film_dim=0, num_pages=P)
        self.h = D.dflash_create(cfg)
        if paged:
            self.dev_table = i32(self.table)
            D.dflash_set_block_table(self.h, self.dev_table)
        self.ws = torch.zeros(D.dflash_workspace_size(self.h), dtype=torch.uint8, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (N, P, Hkv, PR, hd) if paged else (N, nb, Hkv, Cmax, hd)
        self.kc, self.vc = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))

    def __del__(self):
        try:
            self.D.dflash_destroy(self.h)
        except Exception:
            pass

    def rows(self, t, layer, i, n):
        """Rows [0, n) of sequence i, [Hkv, n, hd] (a copy)."""
        if self.table is None:
            return t[layer, i, :, :n].clone()
        return t[layer][i32(self.table[i]).long()].transpose(0, 1).reshape(self.Hkv, -1, self.hd)[:, :n].clone()

    def put(self, t, layer, i, rows, value):
        for r in np.atleast_1d(rows):
            if self.table is None:
                t[layer, i, :, r] = value
            else:
                t[layer, int(self.table[i, r // PR]), :, r % PR] = value

    def status(self):
        return self.D.dflash_status(self.h, self.ws)

    def attend(self, m, q, parent, n, ctx, window=0, sinks=0, hint=0, out=None, nb=None, layer=0, stream=None):
        nb = nb or self.nb
        out = torch.full((nb, m, self.Hq, self.hd), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        keep = [t if t is None or isinstance(t, torch.Tensor) else i32(t) for t in (parent, n, ctx)]
        self.D.dflash_attention_tree(self.h, nb, layer, m, q, self.kc, self.vc, *keep, hint, window, sinks, out,
                                     self.ws, stream)
        return out


def trees(nb, m, seed, kind="tree"):
    """Parents [nb, m], None for chains; `wide`: all nodes below the root."""
    rng = np.random.default_rng(seed)
    if kind == "chain":
        return None
    par = np.full((nb, m), -1, np.int32)
    for j in range(1, m):
        par[:, j] = 0 if kind == "wide" else (j * np.sqrt(rng.random(nb))).astype(int).clip(0, j - 1)
    return par


def queries(nb, m, Hq, hd, seed, big=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    return (big * torch.randn(nb, m, Hq, hd, generator=g, device="cuda")).to(torch.bfloat16)


def check_attention(t, m, q, parent, n, ctx, window=0, sinks=0, hint=0, layer=0, out=None, seqs=None):
    out = t.attend(m, q, parent, n, ctx, window, sinks, hint, layer=layer) if out is None else out
    assert t.status() == 0
    got, qq = f64(out), f64(q)
    for i in range(t.nb) if seqs is None else seqs:
        ni = m if n is None else n[i]
        assert (got[i, ni:] == 7.0).all(), "rows behind the tree were written"
        if ni == 0:
            continue
        par = list(range(-1, ni - 1)) if parent is None else parent[i][:ni]
        L = ctx[i] + ni
        K, V = (f64(t.rows(c, layer, i, L)) for c in (t.kc, t.vc))
        o, mag, dot = orc.attention_tree(qq[i, :ni], K, V, orc.tree_visible(par, ctx[i], window, sinks))
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -14 + 2 * t.hd * 2.0 ** -24 * dot[..., None]) * mag
        assert np.isfinite(got[i, :ni]).all(), f"sequence {i}: not finite"
        worst = (np.abs(got[i, :ni] - o) / tol).max()
        assert worst <= 1, f"sequence {i}: {worst:.2f} of the tolerance"
    return out


SHAPES = [  # Hq, Hkv, hd, paged
    (4, 4, 64, True), (8, 2, 128, True), (8, 2, 128, False), (14, 2, 64, False), (5, 1, 128, True), (16, 2, 64, True)]


@pytest.mark.parametrize("Hq,Hkv,hd,paged", SHAPES)
@pytest.mark.parametrize("m,kind", [(1, "chain"), (7, "chain"), (16, "tree"), (33, "tree"), (64, "tree"), (64, "wide"),
                                    (64, "chain")])
def test_attention_of_trees(Hq, Hkv, hd, paged, m, kind):
    nb = 5
    t = Target(Hq, Hkv, hd, Cmax=448, nb=nb, paged=paged, seed=m)
    ctx = [0, 1, 63, 130, 448 - m]
    n = [m, max(1, m // 2), m, 0, m]
    check_attention(t, m, queries(nb, m, Hq, hd, m), trees(nb, m, m, kind), n, ctx)


@pytest.mark.parametrize("Hq,Hkv,hd,paged", SHAPES)
@pytest.mark.parametrize("m,window,sinks", [(1, 1, 0), (1, 64, 4), (9, 3, 2), (16, 65, 64), (40, 130, 70), (64, 20, 300),
                                            (64, 1, 1), (64, 2 ** 31 - 1, 5), (30, 200, 2 ** 31 - 1)])
def test_attention_with_a_window_and_sinks(Hq, Hkv, hd, paged, m, window, sinks):
    nb = 6
    t = Target(Hq, Hkv, hd, Cmax=512, nb=nb, paged=paged, seed=m + window % 1000)
    ctx = [0, 2, 64, 191, 320, 512 - m]
    n = [m, m, max(1, m - 3), m, m, max(1, m // 3)]
    for kind in ("tree", "chain"):
        check_attention(t, m, queries(nb, m, Hq, hd, m), trees(nb, m, m, kind), n, ctx, window, sinks, hint=512 - m)


def test_scores_that_grow_and_peak():
    """Row maxima that rise by more than 2^8 many times, and rows where one key has all the weight."""
    t = Target(8, 2, 128, Cmax=1024, nb=2, paged=False, seed=3)
    ramp = torch.linspace(0.05, 6, 1024, device="cuda")[None, None, None, :, None]
    t.kc = (t.kc.float().abs() * ramp).to(torch.bfloat16)
    q = queries(2, 20, 8, 128, 4).abs() * 2
    check_attention(t, 20, q, trees(2, 20, 5), [20, 13], [1000, 517])
    check_attention(t, 20, -q, trees(2, 20, 5), [20, 13], [1000, 517], window=300, sinks=10)


@pytest.mark.parametrize("Hq,Hkv,m", [(64, 1, 1), (64, 1, 3), (64, 1, 64), (10, 2, 51), (6, 2, 43), (9, 1, 29)])
def test_attention_of_many_heads_and_uneven_tiles(Hq, Hkv, m):
    t = Target(Hq, Hkv, 64, Cmax=320, nb=2, paged=True, seed=m)
    check_attention(t, m, queries(2, m, Hq, 64, m), trees(2, m, m), [m, max(1, m - 2)], [250, 77])


def test_many_sequences_of_uneven_lengths():
    """More sequences than a CTA keeps lengths of, some without rows, first and last among them."""
    nb, m = 150, 5
    t = Target(4, 2, 64, Cmax=320, nb=nb, paged=True, seed=9)
    rng = np.random.default_rng(1)
    ctx = rng.integers(0, 315, nb)
    n = rng.integers(0, m + 1, nb)
    n[[0, 63, 64, 65, 120, 149]] = 0
    check_attention(t, m, queries(nb, m, 4, 64, 9), trees(nb, m, 9), n.tolist(), ctx.tolist())
    out = t.attend(m, queries(nb, m, 4, 64, 9), trees(nb, m, 9), np.zeros(nb), ctx)
    assert (out == 7).all() and t.status() == 0
    few = t.attend(m, queries(nb, m, 4, 64, 9), trees(nb, m, 9), n, ctx, nb=70)
    assert t.status() == 0 and few.shape[0] == 70


def test_a_long_context_over_every_sm():
    t = Target(8, 2, 128, Cmax=20480, nb=1, paged=True, seed=2)
    for m, window in ((1, 0), (48, 0), (48, 5000)):
        check_attention(t, m, queries(1, m, 8, 128, 3), trees(1, m, 3), None, [20480 - m], window, 3)


# Hq, Hkv, hd, sequences, nodes, window: many units a CTA, so that ranges begin and end anywhere in a pair and before its
# first unit; more pairs than CTAs, and fewer; one tile, two, two groups of two
@pytest.mark.parametrize("Hq,Hkv,hd,nb,m,window", [
    (16, 8, 64, 24, 20, 0), (32, 8, 128, 20, 64, 0), (32, 8, 64, 12, 64, 0), (64, 8, 64, 10, 64, 0), (8, 8, 128, 22, 9, 1500),
    (24, 8, 128, 20, 43, 2000), (16, 8, 128, 9, 64, 0)])
def test_ranges_of_many_units(Hq, Hkv, hd, nb, m, window):
    t = Target(Hq, Hkv, hd, Cmax=4096, nb=nb, paged=True, seed=m + nb)
    t.ws[256:].fill_(0xFF)   # behind the status word a workspace may hold anything
    rng = np.random.default_rng(nb)
    ctx, n = rng.integers(1200, 4096 - m, nb), rng.integers(1, m + 1, nb)
    ctx[[1, nb - 2]], n[[0, nb // 2, nb - 1]] = (0, 64), 0
    check_attention(t, m, queries(nb, m, Hq, hd, 4), trees(nb, m, 4), n.tolist(), ctx.tolist(), window, 70)


@pytest.mark.parametrize("Hq,m,paged", [(8, 1, True), (32, 16, True), (32, 25, False), (32, 33, True)])
def test_segments_of_many_units(Hq, m, paged):
    """Some 60 units of one pair in a row: every ring goes round many times, pages are looked up more than once."""
    nb = 8
    t = Target(Hq, 8, 128, Cmax=9216, nb=nb, paged=paged, seed=m)
    ctx, n = [8960 - 64 * i for i in range(nb)], [m - i % m for i in range(nb)]
    check_attention(t, m, queries(nb, m, Hq, 128, 4), trees(nb, m, 4), n, ctx, seqs=[0, 3, 7])


def test_graphs_of_one_workspace_and_handles_at_once():
    """Two captured calls that share a workspace, replayed in turn; two handles, each on a stream of its own, at once."""
    nb = 6
    ts = [Target(32, 8, 128, Cmax=2048, nb=nb, paged=True, seed=s) for s in (1, 2)]
    calls = []   # shape, inputs, the output alone
    for m, window in ((64, 0), (7, 300)):
        args = (m, queries(nb, m, 32, 128, m), i32(trees(nb, m, m)), i32([m - k for k in range(nb)]),
                i32([1900 - 300 * k for k in range(nb)]), window, 4)
        calls.append((args, [t.attend(*args) for t in ts]))
    torch.cuda.synchronize()
    graphs = []
    for args, want in calls:
        out, g = torch.empty_like(want[0]), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ts[0].attend(*args, out=out)
        graphs.append((g, out, want[0]))
    for k in range(6):
        for g, out, want in graphs[::1 if k % 2 else -1]:
            out.fill_(7)
            g.replay()
    for _, out, want in graphs:
        assert torch.equal(out, want)
    streams = [torch.cuda.Stream() for _ in ts]
    outs = [[torch.full_like(w[k], 7.0) for _, w in calls] for k in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                for (args, _), out in zip(calls, outs[k]):
                    ts[k].attend(*args, out=out)
    torch.cuda.synchronize()
    for k, t in enumerate(ts):
        assert t.status() == 0
        for (_, want), out in zip(calls, outs[k]):
            assert torch.equal(out, want[k])


@pytest.mark.parametrize("Hq,Hkv,Cmax", [(1, 1, 8192), (2, 1, 8192), (3, 1, 8192), (4, 2, 40), (5, 1, 8192), (32, 1, 8192)])
def test_scratch_of_the_partials(Hq, Hkv, Cmax):
    """Partials of two slots a SM hold the rows that a tree of the handle's can have, no more; the longest trees fit."""
    D = lib()
    t = Target(Hq, Hkv, 128, Cmax=Cmax, nb=1, paged=False, V=64)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = min(256, Hq // Hkv * min(64, Cmax))
    assert t.ws.numel() <= 2 * sms * rows * (128 * 4 + 8) + (1 << 20)   # the rest of so small a handle: below 1 MB
    for m in (min(64, Cmax), 33, 1):
        check_attention(t, m, queries(1, m, Hq, 128, m), trees(1, m, m), None, [Cmax - m])
    assert D.dflash_status(t.h, t.ws) == 0


@pytest.mark.parametrize("Hq,m,kind", [(4, 64, "wide"), (8, 64, "tree"), (4, 1, "chain"), (4, 40, "chain")])
def test_the_widest_window_is_none(Hq, m, kind):
    nb = 4
    t = Target(Hq, 2, 64, Cmax=448, nb=nb, paged=True, seed=m)
    q, par, ctx = queries(nb, m, Hq, 64, m), trees(nb, m, m, kind), [0, 70, 129, 448 - m]
    want = check_attention(t, m, q, par, None, ctx)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (448, 5), (1, 2 ** 31 - 1)):
        assert torch.equal(t.attend(m, q, par, None, ctx, window, sinks), want) and t.status() == 0


@pytest.mark.parametrize("Hq,m", [(2, 1), (2, 17), (4, 40)])
def test_a_quarter_million_rows(Hq, m):
    t = Target(Hq, 1, 64, Cmax=262144, nb=1, paged=False, seed=m)
    check_attention(t, m, queries(1, m, Hq, 64, 3), trees(1, m, 3), None, [262144 - m])
    check_attention(t, m, queries(1, m, Hq, 64, 5), trees(1, m, 5), None, [262144 - m], 200000, 130)


@pytest.mark.parametrize("Hq,Hkv,hd,m", [(4, 2, 64, 1), (8, 2, 128, 33), (16, 2, 64, 50), (3, 3, 128, 64)])
def test_contiguous_caches_of_odd_length(Hq, Hkv, hd, m):
    """Pages of the last rows reach into the next head's, sequence's and layer's, and past the cache's end."""
    nb, Cmax = 3, 397
    t = Target(Hq, Hkv, hd, Cmax=Cmax, nb=nb, N=2, paged=False, seed=m)
    ctx, n, par = [Cmax - m, 320, 0], [m, max(1, m - 3), m], trees(nb, m, m)
    q = queries(nb, m, Hq, hd, m)
    for layer in (0, 1):
        for window in (0, 90):
            check_attention(t, m, q, par, n, ctx, window, 5, layer=layer)
    want = [[t.rows(c, layer, i, Cmax) for c in (t.kc, t.vc)] for layer in (0, 1) for i in range(nb)]
    path = [list(range(0, k, 2)) for k in n]
    tau = [len(w) for w in path]
    t.D.dflash_kv_commit(t.h, nb, m, i32([w + [-1] * (m - len(w)) for w in path]), i32(tau),
                         i32([c + k for c, k in zip(ctx, tau)]), t.kc, t.vc, t.ws)
    assert t.status() == 0
    for layer in (0, 1):
        for i in range(nb):
            for c, was in zip((t.kc, t.vc), want[layer * nb + i]):
                was[:, ctx[i]:ctx[i] + tau[i]] = was[:, [ctx[i] + a for a in path[i]]]
                assert torch.equal(t.rows(c, layer, i, Cmax), was)


@pytest.mark.parametrize("Hq,Hkv,hd,m", [(4, 2, 64, 1), (32, 8, 128, 16), (32, 8, 128, 64), (64, 8, 64, 64)])
def test_probabilities_that_change_from_unit_to_unit(Hq, Hkv, hd, m):
    """No row's maximum grows by 2^8, so O is never rescaled, while the probabilities of a unit are about 1 or about 2^-6,
    in turns of no one length: a unit's in the place of another's would show."""
    t = Target(Hq, Hkv, hd, Cmax=4096, nb=2, paged=True, seed=m)
    unit = torch.arange(t.kc.shape[1] * PR, device="cuda").view(-1, 1, PR, 1) // PR
    high = (unit % 2 == 0) | (unit % 5 < 2)
    d = torch.where(torch.rand(hd, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.5, -1.0, 1.0)
    t.kc.copy_((torch.where(high, 1.0, 0.25) * d).to(torch.bfloat16).expand_as(t.kc[0]))
    for i in range(2):
        t.put(t.kc, 0, i, 0, d.to(torch.bfloat16))
    q = (0.25 * queries(2, m, Hq, hd, m).float() + 6 / hd ** 0.5 * d).to(torch.bfloat16)
    ctx, n, par = [4096 - m, 2500], [m, max(1, m - 5)], trees(2, m, m)
    want = check_attention(t, m, q, par, n, ctx)
    for _ in range(20):
        assert torch.equal(t.attend(m, q, par, n, ctx), want)
    assert t.status() == 0


def test_rows_that_nobody_sees_may_hold_anything():
    """NaN and infinities in keys and values outside the window, behind the tree and in the nodes of other branches."""
    nb, m, window, sinks = 3, 16, 100, 4
    for Hq in (4, 24):   # one tile and two
        t = Target(Hq, 2, 128, Cmax=512, nb=nb, paged=True, seed=5)
        ctx, n, par = [0, 300, 401], [16, 9, 16], trees(nb, m, 5)
        for i in range(nb):
            dead = [r for r in range(512) if r >= ctx[i] + n[i] or (sinks <= r <= ctx[i] - window)]
            for c, v in ((t.kc, float("nan")), (t.vc, float("inf"))):
                t.put(c, 0, i, dead, v)
            t.put(t.vc, 0, i, dead[::2], float("nan"))
        q = queries(nb, m, Hq, 128, 6)
        out = check_attention(t, m, q, par, n, ctx, window, sinks)
        # a leaf with values that are not finite: only its own row shows it
        for i in range(nb):
            leaf = n[i] - 1
            t.put(t.vc, 0, i, ctx[i] + leaf, float("-inf"))
            t.put(t.kc, 0, i, ctx[i] + leaf, float("nan"))
        again = t.attend(m, q, par, n, ctx, window, sinks)
        assert t.status() == 0
        for i in range(nb):
            leaf = n[i] - 1
            assert not again[i, leaf].isfinite().any()
            assert torch.equal(again[i, :leaf], out[i, :leaf]) and torch.equal(again[i, n[i]:], out[i, n[i]:])


def test_values_that_are_seen_and_not_finite_show():
    t = Target(4, 2, 64, Cmax=256, nb=1, paged=False, seed=7)
    q = queries(1, 6, 4, 64, 7)
    par = [[-1, 0, 0, 1, 1, 2]]
    clean = t.attend(6, q, par, None, [200])
    t.vc[0, 0, 0, 201, 5] = float("inf")     # node 1 of kv head 0: nodes 1, 3 and 4 of heads 0 and 1
    got = t.attend(6, q, par, None, [200])
    assert t.status() == 0
    hit = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    hit[[1, 3, 4], :2] = True
    assert not got[0, ..., 5][hit].isfinite().any()
    assert torch.equal(got[0][~hit], clean[0][~hit])
    t.vc[0, 0, 0, 20, 9] = float("nan")      # a context row that every node sees
    got = t.attend(6, q, par, None, [200])
    assert got[0, :, :2, 9].isnan().all() and torch.equal(got[0, :, 2:], clean[0, :, 2:])


def test_output_in_place_layers_and_a_context_hint():
    t = Target(8, 2, 128, Cmax=448, nb=3, N=3, paged=True, seed=11)
    q, par, ctx = queries(3, 20, 8, 128, 1), trees(3, 20, 1), [7, 300, 428]
    for layer in range(3):
        want = check_attention(t, 20, q, par, None, ctx, layer=layer, hint=428)
        same = q.clone()
        t.attend(20, same, par, None, ctx, layer=layer, out=same)
        assert torch.equal(same, want)


def test_attention_past_32_bit_offsets():
    """A pool of 5 GB a cache whose pages in use lie at its end."""
    pages, Hkv, hd = 40000, 8, 128
    D = lib()
    t = Target(16, Hkv, hd, Cmax=256, nb=1, paged=True, spare=pages - 4, seed=1)
    t.table = np.array([[pages - 1, pages - 3, 2, pages - 2]])
    t.dev_table = i32(t.table)
    D.dflash_set_block_table(t.h, t.dev_table)
    q, par = queries(1, 20, 16, hd, 1), trees(1, 20, 2)
    check_attention(t, 20, q, par, None, [230])
    path, tau = i32([[0, 3, 9] + [-1] * 17]), i32([3])
    before = t.rows(t.kc, 0, 0, 256)
    D.dflash_kv_commit(t.h, 1, 20, path, tau, i32([233]), t.kc, t.vc, t.ws)
    after = t.rows(t.kc, 0, 0, 256)
    want = before.clone()
    want[:, 231], want[:, 232] = before[:, 233], before[:, 239]
    assert torch.equal(after, want) and t.status() == 0


def test_captured_calls_and_streams():
    """A captured call follows the lengths, trees and queries of each replay; another stream gives the same."""
    nb, m = 4, 24
    t = Target(8, 2, 128, Cmax=640, nb=nb, paged=True, seed=12)
    q, par = queries(nb, m, 8, 128, 1), i32(trees(nb, m, 1))
    ctx, n, out = i32([10, 200, 400, 616]), i32([m] * nb), torch.empty(nb, m, 8, 128, dtype=torch.bfloat16, device="cuda")
    t.attend(m, q, par, n, ctx, 100, 4, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.attend(m, q, par, n, ctx, 100, 4, out=out)
    for k in range(3):
        p2, c2, n2 = trees(nb, m, 20 + k), [k, 333, 64 * k, 616], [m - k, m, 0, 1 + k]
        q.copy_(queries(nb, m, 8, 128, 30 + k))
        par.copy_(i32(p2))
        ctx.copy_(i32(c2))
        n.copy_(i32(n2))
        out.fill_(7)
        g.replay()
        check_attention(t, m, q, p2, n2, c2, 100, 4, out=out)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = t.attend(m, q, par, n, ctx, 100, 4)
        s.synchronize()
        assert torch.equal(other, out)


def test_lengths_trees_and_pages_out_of_range_are_reported():
    D = lib()
    t = Target(4, 2, 64, Cmax=256, nb=2, paged=True, seed=13)
    q, par = queries(2, 8, 4, 64, 1), trees(2, 8, 1)
    for ctx, n, hint in (([249, 0], None, 0), ([-1, 3], None, 0), ([10, 3], [9, 1], 0), ([10, 3], [1, -1], 0),
                         ([101, 3], None, 100)):
        t.attend(8, q, par, n, ctx, hint=hint)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
    for bad in ((0, 0), (3, 3), (3, 7), (3, -1), (3, -2), (7, 2 ** 31 - 1)):
        p2 = par.copy()
        p2[1, bad[0]] = bad[1]
        t.attend(8, q, p2, [8, 8], [100, 50])
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK, bad
    t.attend(8, q, [[-1] + list(range(7)), [-1, 0, 9, 9, 9, 9, 9, 9]], [8, 2], [100, 50])   # behind the tree: not read
    assert t.status() == 0
    t.dev_table[0, 1] = t.nb * t.pps + 2
    t.attend(8, q, par, None, [100, 50])
    assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
    t.attend(8, q, par, None, [40, 50])
    assert t.status() == 0


@pytest.mark.parametrize("n,ctx", [(8, 2 ** 31 - 1), (8, -2 ** 31), (2 ** 31 - 1, 5), (-2 ** 31, 5), (-2 ** 31, 2 ** 31 - 1),
                                   (2 ** 31 - 1, -2 ** 31)])
def test_lengths_at_the_ends_of_their_type(n, ctx):
    """Counts and lengths that no cache has: reported, and the other sequence's rows as without them."""
    D = lib()
    t = Target(4, 2, 64, Cmax=256, nb=2, paged=True, seed=14)
    for m in (8, 64):
        q, par = queries(2, m, 4, 64, 1), trees(2, m, 1)
        for window in (0, 60):
            want = check_attention(t, m, q, par, [8, 0], [100, 0], window, 2)
            got = t.attend(m, q, par, [8, n], [100, ctx], window, 2)
            assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
            assert torch.equal(got[0], want[0])
        before = t.kc.clone(), t.vc.clone()
        path = i32([[0, 2, 3] + [-1] * (m - 3)] * 2)
        D.dflash_kv_commit(t.h, 2, m, path, i32([0, n]), i32([0, ctx]), t.kc, t.vc, t.ws)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
        assert torch.equal(t.kc, before[0]) and torch.equal(t.vc, before[1])
        for d_ctx in (i32([0, ctx]), None):
            tau, bonus = i32([7, 7]), i32([7, 7])
            D.dflash_accept_tree(t.h, 2, m, i32(par), i32(np.zeros((2, m))), i32(np.full((2, m), -1)), i32([1, n]), d_ctx,
                                 tau, bonus, None, None, t.ws)
            assert (t.status() == 0) == (n == 8)
            assert tau.tolist() == [1, int(n > 0)]
    V = 64
    counts = i32(np.zeros((2, V)))
    D.dflash_token_counts(t.h, 2, 3, i32([[1, 2, 3]] * 2), 3, i32([1, n]), 0, counts, t.ws)
    assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
    assert counts.sum(1).tolist() == [1, 3 if n > 0 else 0]


def test_a_wait_that_runs_out_is_reported():
    D = lib()
    t = Target(4, 2, 64, Cmax=256, nb=2, max_spin=50, flags=D.FLAG_TEST_STALL)
    for m in (1, 20, 64):
        t.attend(m, queries(2, m, 4, 64, 1), trees(2, m, 1), None, [100, 50])
        assert t.status() == D.DFLASH_ERR_TIMEOUT
    t = Target(4, 2, 64, Cmax=256, nb=2)
    check_attention(t, 20, queries(2, 20, 4, 64, 1), trees(2, 20, 1), None, [100, 50])


def test_a_wait_that_runs_out_leaves_the_workspace_usable():
    """What calls before left in the workspace, or anything, is no harm to a call whose waits run out, nor that to the next."""
    D = lib()
    good = Target(8, 2, 64, Cmax=1024, nb=3, seed=3)
    stall = Target(8, 2, 64, Cmax=1024, nb=3, seed=3, max_spin=50, flags=D.FLAG_TEST_STALL)
    assert good.ws.numel() == stall.ws.numel()
    stall.ws = good.ws
    for fill in (None, 0xFF, 0x01):
        for m, then in ((64, 20), (20, 64), (9, 9), (1, 3)):
            q, par = queries(3, m, 8, 64, m), trees(3, m, m)
            check_attention(good, m, q, par, None, [900, 300, 5])
            if fill is not None:
                good.ws[256:].fill_(fill)
            out = stall.attend(then, queries(3, then, 8, 64, 1), trees(3, then, 1), None, [700, 50, 0])
            assert stall.status() == D.DFLASH_ERR_TIMEOUT and out.shape[1] == then
            check_attention(good, m, q, par, None, [900, 300, 5])


def refused(code, f):
    with pytest.raises(lib().DflashError) as e:
        f()
    assert e.value.code == code


def test_refusals():
    D = lib()
    t = Target(4, 2, 64, Cmax=128, nb=2, paged=True)
    A, U = D.DFLASH_ERR_INVALID_ARG, D.DFLASH_ERR_UNSUPPORTED_SHAPE
    q, out, ctx = queries(2, 8, 4, 64, 1), torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([1, 2])
    par, ids, tau = i32(trees(2, 8, 1)), i32(np.zeros((2, 8))), i32([1, 1])

    def att(nb=2, layer=0, m=8, q=q, kc=t.kc, vc=t.vc, par=par, n=None, ctx=ctx, hint=0, w=0, s=0, o=out, ws=t.ws):
        D.dflash_attention_tree(t.h, nb, layer, m, q, kc, vc, par, n, ctx, hint, w, s, o, ws)
    att()
    att(nb=0, q=None), att(m=0, q=None)
    for kw in (dict(nb=-1), dict(nb=3), dict(layer=1), dict(layer=-1), dict(m=-1), dict(m=65), dict(hint=-1), dict(hint=129),
               dict(w=-1), dict(s=-1), dict(q=None), dict(o=None), dict(kc=None), dict(vc=None), dict(ctx=None),
               dict(q=q.view(-1)[1:]), dict(o=out.view(-1)[4:]), dict(o=q.view(-1)[8:]), dict(ws=t.ws[:256]),
               dict(ws=t.ws[16:])):
        refused(A, lambda: att(**kw))
    bare = Target(4, 2, 64, Cmax=128, nb=2, paged=False)
    small = Target(4, 2, 64, Cmax=40, nb=1, paged=False)
    refused(A, lambda: small.attend(41, q, None, None, [0]))
    assert bare.status() == 0
    nt = object.__new__(Target)
    nt.D, nt.h = D, D.dflash_create(D.dflash_config(D=64, Dt=64, L=1, N=1, Hq=4, Hkv=2, hd=64, F=64, V=64, B=2, k_top=1, rope_base=1e4,
                                                    eps=1e-6, mask_id=0, Cmax=128, max_batch=2, max_proj_rows=1, conv_group=16,
                                                    sel_dim=256, num_pages=6))
    refused(A, lambda: D.dflash_attention_tree(nt.h, 2, 0, 8, q, t.kc, t.vc, par, None, ctx, 0, 0, 0, out, t.ws))
    refused(A, lambda: D.dflash_kv_commit(nt.h, 2, 8, ids, tau, ctx, t.kc, t.vc, t.ws))   # no table registered

    def acc(nb=2, m=8, par=par, tok=ids, tgt=ids, n=None, ctx=None, tau=tau, bonus=tau.clone(), path=None, out=None, ws=t.ws):
        D.dflash_accept_tree(t.h, nb, m, par, tok, tgt, n, ctx, tau, bonus, path, out, ws)
    acc()
    acc(nb=0, tau=None), acc(m=0, par=None, tok=None, tgt=None)
    for kw in (dict(nb=-1), dict(m=65), dict(m=-1), dict(par=None), dict(tok=None), dict(tgt=None), dict(tau=None),
               dict(bonus=None), dict(ws=t.ws[:256])):
        refused(A, lambda: acc(**kw))

    def com(nb=2, m=8, path=ids, tau=tau, ctx=ctx, kc=t.kc, vc=t.vc, ws=t.ws):
        D.dflash_kv_commit(t.h, nb, m, path, tau, ctx, kc, vc, ws)
    com()
    com(nb=0, path=None), com(m=0, path=None)
    for kw in (dict(nb=-1), dict(nb=3), dict(m=65), dict(path=None), dict(tau=None), dict(ctx=None), dict(kc=None),
               dict(vc=t.vc.view(-1)[3:]), dict(ws=t.ws[:256])):
        refused(A, lambda: com(**kw))

    counts = torch.zeros(2, 64, dtype=torch.int32, device="cuda")

    def cnt(nb=2, n=8, tok=ids, ld=8, nt=None, counts=counts, ws=t.ws):
        D.dflash_token_counts(t.h, nb, n, tok, ld, nt, 0, counts, ws)
    cnt()
    cnt(nb=0, tok=None), cnt(n=0, tok=None)
    for kw in (dict(nb=-1), dict(n=-1), dict(ld=7), dict(tok=None), dict(counts=None), dict(ws=t.ws[:256])):
        refused(A, lambda: cnt(**kw))
    refused(U, lambda: cnt(nb=65536))

    x = torch.zeros(16, 64, device="cuda")
    rules = D.logit_rules(counts=counts)

    def adj(nb=2, m=8, x=x, ld=64, rules=rules, n=None, y=x, ldy=64, ids=ids, ws=t.ws):
        D.dflash_logits_adjust(t.h, nb, m, x, ld, rules, n, y, ldy, ids, ws)
    adj()
    adj(nb=0, x=None), adj(m=0, x=None)
    half = D.logit_rules(parent=par)
    lone = D.logit_rules()
    lone.n_bias = 3
    many = D.logit_rules(bias_ids=i32(np.zeros((2, 1025))), bias=torch.zeros(2, 1025, device="cuda"))
    minus = D.logit_rules()
    minus.n_bias = -1
    buf = torch.zeros(4096, device="cuda")
    for kw in (dict(nb=-1), dict(m=65), dict(ld=63), dict(ldy=63), dict(x=None), dict(y=None, ids=None), dict(rules=None),
               dict(rules=half), dict(rules=lone), dict(rules=minus), dict(ws=t.ws[:256]), dict(x=buf, y=buf, ldy=65),
               dict(x=buf, y=buf[8:])):
        refused(A, lambda: adj(**kw))
    refused(U, lambda: adj(rules=many))
    refused(U, lambda: adj(nb=2 ** 20 + 1))
    assert t.status() == 0


# ------------------------------------------------------------------ the walk and the move

@pytest.mark.parametrize("nb,m", [(1, 1), (3, 5), (9, 16), (70, 33), (130, 64)])
def test_accepted_paths(nb, m):
    D = lib()
    t = Target(nb=1)
    rng = np.random.default_rng(m)
    for kind in ("tree", "deep", "wide"):
        par = trees(nb, m, m, kind if kind != "deep" else "tree")
        if kind == "deep":   # chains in rising order of random nodes
            par[:, 1:] = np.maximum(np.arange(m - 1) - rng.integers(0, 2, (nb, m - 1)), 0)
        tokens = rng.integers(0, 6, (nb, m))
        target = rng.integers(-1, 6, (nb, m))
        for j in range(m - 1, 0, -1):   # most nodes have a child that fits
            fit = rng.random(nb) < 0.8
            target[np.arange(nb)[fit], par[fit, j]] = tokens[fit, j]
        n = rng.integers(0, m + 1, nb)
        ctx = rng.integers(0, 1000, nb)
        dev, d_ctx = [i32(a) for a in (par, tokens, target)], i32(ctx)
        tau, bonus = i32(np.zeros(nb)), i32(np.zeros(nb))
        path, out = i32(np.zeros((nb, m))), i32(np.zeros((nb, m)))
        D.dflash_accept_tree(t.h, nb, m, *dev, i32(n), d_ctx, tau, bonus, path, out, t.ws)
        assert t.status() == 0
        for i in range(nb):
            want, emitted = orc.accept_tree(par[i, :n[i]], tokens[i, :n[i]], target[i])
            k = len(want)
            assert int(tau[i]) == k and int(d_ctx[i]) == ctx[i] + k
            assert int(bonus[i]) == (emitted[-1] if k else -1)
            assert path[i].tolist() == want + [-1] * (m - k) and out[i].tolist() == emitted + [-1] * (m - k)
        t2, b2 = tau.clone().zero_(), bonus.clone().zero_()
        D.dflash_accept_tree(t.h, nb, m, *dev, i32(n), None, t2, b2, None, None, t.ws)
        assert torch.equal(t2, tau) and torch.equal(b2, bonus)


def test_paths_of_the_most_sequences():
    """2^31 - 1 sequences without nodes: 8.6 GB for each output."""
    D = lib()
    t, nb = Target(nb=1), 2 ** 31 - 1
    tau, bonus = (torch.full((nb,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    D.dflash_accept_tree(t.h, nb, 0, None, None, None, None, None, tau, bonus, None, None, t.ws)
    assert t.status() == 0
    assert int(tau.min()) == int(tau.max()) == 0 and int(bonus.min()) == int(bonus.max()) == -1


def test_trees_that_are_none_are_reported_and_end_the_walk():
    D = lib()
    t = Target(nb=1)
    m = 6
    tokens, target = [[0, 1, 2, 3, 4, 5]], [[1, 2, 3, 4, 5, 6]]
    chain = [-1, 0, 1, 2, 3, 4]
    for j, up, tau in ((0, 0, 6), (3, 3, 3), (3, 5, 3), (3, -1, 3), (5, 2 ** 31 - 1, 5), (1, -7, 1)):
        par = list(chain)
        par[j] = up
        out = i32([0]), i32([0]), i32([[0] * m]), i32([[0] * m])
        D.dflash_accept_tree(t.h, 1, m, i32([par]), i32(tokens), i32(target), None, None, *out, t.ws)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK and int(out[0]) == tau, (j, up)
    for n in (-1, 7):
        D.dflash_accept_tree(t.h, 1, m, i32([chain]), i32(tokens), i32(target), i32([n]), None, *out, t.ws)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK and int(out[0]) == max(0, min(n, 6))


@pytest.mark.parametrize("hd,paged,nb,m", [(64, True, 5, 16), (128, True, 4, 64), (128, False, 3, 64), (64, False, 2, 1),
                                           (64, False, 6, 40)])
def test_committed_rows(hd, paged, nb, m):
    D = lib()
    Cmax = 250 if not paged else 256
    t = Target(6, 3, hd, Cmax=Cmax, nb=nb, N=2, paged=paged, seed=m)
    rng = np.random.default_rng(m)
    path, tau, base = np.full((nb, m), -1), np.zeros(nb, int), np.zeros(nb, int)
    for i in range(nb):
        tau[i] = [m, 0, min(m, 2)][i] if i < 3 else rng.integers(1, m + 1)
        if tau[i]:
            # rising, from the root; the last sequence's is dense at the end
            rest = np.sort(rng.choice(np.arange(1, m), tau[i] - 1, replace=False)) if m > 1 else []
            path[i, :tau[i]] = [0] + list(rest)
        base[i] = [Cmax - m, 17, 60, 0, 127, 64][i]
    before = [t.kc.clone(), t.vc.clone()]
    D.dflash_kv_commit(t.h, nb, m, i32(path), i32(tau), i32(base + tau), t.kc, t.vc, t.ws)
    assert t.status() == 0
    want = [b.clone() for b in before]
    for c, b, now in zip(want, before, (t.kc, t.vc)):
        for layer in range(2):
            for i in range(nb):
                old = t.rows(b, layer, i, Cmax)
                for k in range(tau[i]):
                    r = base[i] + k
                    new = old[:, base[i] + path[i, k]]
                    if paged:
                        c[layer, int(t.table[i, r // PR]), :, r % PR] = new
                    else:
                        c[layer, i, :, r] = new
        assert torch.equal(now.view(torch.int16), c.view(torch.int16))


def test_paths_that_are_none_are_reported_and_not_moved():
    D = lib()
    t = Target(4, 2, 64, Cmax=128, nb=1, paged=True)
    before = t.kc.clone()
    for path, tau, ln in (([0, 5, 4, 7], 4, 50), ([0, 8, 9, 10], 4, 50), ([1, 1, 2, 3], 3, 50), ([0, -1, 2, 3], 3, 50),
                          ([0, 1, 2, 3], 9, 50), ([0, 1, 2, 3], -1, 50), ([0, 1, 2, 3], 4, 3), ([0, 1, 2, 7], 4, 126),
                          ([0, 1, 2, 3], 4, 129)):
        t.kc.copy_(before)
        full = path + [-1] * 4
        D.dflash_kv_commit(t.h, 1, 8, i32([full]), i32([tau]), i32([ln]), t.kc, t.vc, t.ws)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK, (path, tau, ln)
    t.kc.copy_(before)
    D.dflash_kv_commit(t.h, 1, 8, i32([[0, 5, 4, 7] + [-1] * 4]), i32([4]), i32([50]), t.kc, t.vc, t.ws)
    a, b = t.rows(before, 0, 0, 128), t.rows(t.kc, 0, 0, 128)   # base 46: row 1 from 5, row 2 stays, row 3 from 7
    assert torch.equal(b[:, 47], a[:, 51]) and torch.equal(b[:, 48], a[:, 48]) and torch.equal(b[:, 49], a[:, 53])
    assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
    t.kc.copy_(before)
    t.dev_table[0, 1] = -1
    D.dflash_kv_commit(t.h, 1, 8, i32([[0, 1, 3, 7] + [-1] * 4]), i32([4]), i32([62 + 4]), t.kc, t.vc, t.ws)
    assert t.status() == D.DFLASH_ERR_DEVICE_CHECK and torch.equal(t.kc, before)


# ------------------------------------------------------------------ counts and logits

@pytest.mark.parametrize("nb,n,ld,V", [(1, 1, 1, 64), (5, 7, 9, 64), (3, 1000, 1000, 4099), (2, 5000, 5003, 151936)])
def test_counts_of_tokens(nb, n, ld, V):
    D = lib()
    t = Target(nb=1, V=V)
    rng = np.random.default_rng(n)
    tokens = (V ** rng.random((nb, ld))).astype(int) - 1
    tokens[:, 0] = 7
    num = rng.integers(0, n + 1, nb)
    num[0] = n
    start = rng.integers(0, 3, (nb, V)).astype(np.int32)
    counts = i32(start)
    D.dflash_token_counts(t.h, nb, n, i32(tokens), ld, i32(num), 0, counts, t.ws)
    want = start.copy()
    for i in range(nb):
        np.add.at(want[i], tokens[i, :num[i]], 1)
    assert np.array_equal(counts.cpu().numpy(), want) and t.status() == 0
    D.dflash_token_counts(t.h, nb, n, i32(tokens), ld, None, 1, counts, t.ws)
    for i in range(nb):
        want[i, tokens[i, :n]] |= np.int32(-2 ** 31)
    assert np.array_equal(counts.cpu().numpy(), want) and t.status() == 0
    for bad in (-1, V, 2 ** 31 - 1):
        tokens[nb - 1, 0] = bad
        D.dflash_token_counts(t.h, nb, 1, i32(tokens), ld, None, 0, counts, t.ws)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
        want[:nb - 1, 7] += 1
        assert np.array_equal(counts.cpu().numpy(), want)
    D.dflash_token_counts(t.h, nb, n, i32(tokens), ld, i32([n + 1] + [0] * (nb - 1)), 0, counts, t.ws)
    assert t.status() == D.DFLASH_ERR_DEVICE_CHECK


def test_counts_of_the_longest_row():
    """A row of 2^31 - 1 tokens: 8.6 GB."""
    D = lib()
    n, V = 2 ** 31 - 1, 64
    t = Target(nb=1, V=V)
    tokens = torch.full((n,), 5, dtype=torch.int32, device="cuda")
    tokens[0], tokens[2 ** 31 - 257], tokens[n - 1] = 1, 2, 3
    for num, want in ((None, {1: 1, 2: 1, 3: 1, 5: n - 3}), (n, {1: 1, 2: 1, 3: 1, 5: n - 3}), (n - 1, {1: 1, 2: 1, 5: n - 3}),
                      (9, {1: 1, 5: 8})):
        counts = i32(np.zeros((1, V)))
        D.dflash_token_counts(t.h, 1, n, tokens, n, None if num is None else i32([num]), 0, counts, t.ws)
        assert t.status() == 0 and {v: c for v, c in enumerate(counts[0].tolist()) if c} == want


def pack(allowed):
    rows, V = allowed.shape
    pad = np.zeros((rows, -(-V // 32) * 32), bool)
    pad[:, :V] = allowed
    return torch.from_numpy(np.packbits(pad, axis=1, bitorder="little").view(np.int32)).cuda()


class Row:
    """Seeded logits and rules; `want` gives the oracle's rows and their tolerances."""

    def __init__(self, nb, m, V, seed, penalties=True, counts=True, n_bias=0, mask=False, tree=False, ragged=False):
        rng = np.random.default_rng(seed)
        self.nb, self.m, self.V = nb, m, V
        self.x = (3 * rng.standard_normal((nb * m, V))).astype(np.float32)
        self.pen = np.stack([1 + rng.random(nb), rng.random(nb), rng.random(nb)], axis=1).astype(np.float32) if penalties else None
        self.counts = None
        if counts:
            self.counts = (rng.integers(1, 5, (nb, V)) * (rng.random((nb, V)) < 0.1)).astype(np.uint32)
            self.counts |= (rng.random((nb, V)) < 0.1).astype(np.uint32) << 31
        self.bias_ids = self.bias = None
        if n_bias:
            self.bias_ids = rng.integers(-3, V + 3, (nb, n_bias))
            self.bias_ids[:, n_bias // 2:] = np.where(rng.random((nb, n_bias - n_bias // 2)) < 0.3, self.bias_ids[:, :1],
                                                      self.bias_ids[:, n_bias // 2:])
            self.bias = (4 * rng.standard_normal((nb, n_bias))).astype(np.float32)
        self.allowed = rng.random((nb * m, V)) < 0.5 if mask else None
        self.parent = trees(nb, m, seed) if tree else None
        self.tokens = rng.integers(0, min(V, 40), (nb, m)) if tree else None
        self.n = [m - (i * 5) % (m + 1) for i in range(nb)] if ragged else None

    def rules(self):
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return lib().logit_rules(dev(self.pen), None if self.counts is None else dev(self.counts.view(np.int32)),
                                 i32(self.bias_ids), dev(self.bias), None if self.allowed is None else pack(self.allowed),
                                 i32(self.parent), i32(self.tokens))

    def want(self, i, j):
        r = i * self.m + j
        x = self.x[r].astype(np.float64)
        word = np.zeros(self.V, np.uint32) if self.counts is None else self.counts[i]
        c = (word & 0x7FFFFFFF).astype(np.int64)
        if self.parent is not None:
            for a in orc.tree_lines(self.parent[i][:j + 1])[j][:-1]:
                c[self.tokens[i, a]] += 1
        rep, freq, pres = (1.0, 0.0, 0.0) if self.pen is None else self.pen[i].astype(np.float64)
        y = np.where((c > 0) | (word >> 31 > 0), np.where(x > 0, x / rep, x * rep), x) - freq * c - pres * (c > 0)
        mag = np.abs(x) * max(rep, 1 / rep) + freq * c + pres
        steps = np.full(self.V, 4.0)
        if self.bias is not None:
            for t, b in zip(self.bias_ids[i], self.bias[i]):
                if 0 <= t < self.V:
                    y[t] += b
                    mag[t] += abs(b)
                    steps[t] += 1
        if self.allowed is not None:
            y = np.where(self.allowed[r], y, -np.inf)
        return y, steps * 2.0 ** -24 * mag

    def check(self, y, ids, fill=7.0):
        y, ids = None if y is None else y.double().cpu().numpy(), None if ids is None else ids.cpu().numpy()
        for i in range(self.nb):
            for j in range(self.m):
                r = i * self.m + j
                if self.n is not None and j >= self.n[i]:
                    assert y is None or (y[r] == fill).all()
                    assert ids is None or ids[r] == 7
                    continue
                w, tol = self.want(i, j)
                if y is not None:
                    fin = np.isfinite(w)
                    assert np.array_equal(y[r][~fin], w[~fin], equal_nan=True), (i, j)
                    assert (np.abs(y[r] - w)[fin] <= tol[fin]).all(), (i, j, (np.abs(y[r] - w) / tol)[fin].max())
                if ids is not None:
                    if y is not None:   # the lowest id of the largest value of its own row
                        assert ids[r] == orc.greedy(y[r])
                    best = orc.greedy(w)
                    assert ids[r] == best or (best >= 0 and w[ids[r]] >= w[best] - tol[best] - tol[ids[r]]), (i, j)


def test_the_tests_own_rows_are_the_oracles():
    r = Row(2, 6, 90, 1, n_bias=9, mask=True, tree=True)
    for i in range(2):
        for j in range(6):
            line = orc.tree_lines(r.parent[i][:j + 1])[j][:-1]
            w = orc.adjust_logits(r.x[i * 6 + j], r.counts[i], r.pen[i].astype(np.float64), r.tokens[i][line],
                                  r.bias_ids[i], r.bias[i].astype(np.float64), r.allowed[i * 6 + j])
            assert np.allclose(w, r.want(i, j)[0], rtol=1e-12, atol=1e-12)


def run_row(r, t, ld=None, ldy=None, inplace=False, out=True, ids=True, shift=0):
    D = lib()
    ld, rows = ld or r.V, r.nb * r.m
    x = torch.full((rows * ld + 8,), 3.0, device="cuda")[shift:shift + rows * ld].view(rows, ld)
    x[:, :r.V] = torch.from_numpy(r.x).cuda()
    before = x.clone()
    ldy = ld if inplace else ldy or r.V
    y = x if inplace else torch.full((rows, ldy), 7.0, device="cuda") if out else None
    g = torch.full((rows,), 7, dtype=torch.int32, device="cuda") if ids else None
    D.dflash_logits_adjust(t.h, r.nb, r.m, x, ld, r.rules(), i32(r.n), y, ldy, g, t.ws)
    assert t.status() == 0
    if not inplace:
        assert torch.equal(x.view(torch.int32), before.view(torch.int32))
    if y is not None:
        assert (y[:, r.V:] == (3.0 if inplace else 7.0)).all()
    return y, g


@pytest.mark.parametrize("V", [64, 1000, 4099])
@pytest.mark.parametrize("nb,m", [(1, 1), (3, 4), (2, 64), (60, 10)])
def test_adjusted_logits(V, nb, m):
    if nb * m * V > 700000:
        V = 257
    t = Target(nb=1, V=V)
    for k, kw in enumerate((dict(), dict(n_bias=20), dict(mask=True), dict(tree=True, ragged=True),
                            dict(n_bias=13, mask=True, tree=True, ragged=True),
                            dict(counts=False, tree=True), dict(penalties=False, n_bias=3), dict(penalties=False, counts=False))):
        r = Row(nb, m, V, 10 * k + m, **kw)
        y, g = run_row(r, t)
        r.check(y[:, :V], g)
        y2, g2 = run_row(r, t, out=False)
        assert torch.equal(g2, g)
        y3, _ = run_row(r, t, ids=False)
        assert torch.equal(y3, y)


@pytest.mark.parametrize("nb,m", [(2, 3), (40, 8)])
def test_adjusted_logits_of_any_stride_and_in_place(nb, m):
    V = 1000
    t = Target(nb=1, V=V)
    r = Row(nb, m, V, 5, n_bias=9, mask=True, tree=True)
    y, g = run_row(r, t)
    r.check(y, g)
    for kw in (dict(ld=1003), dict(ld=1004, ldy=1008), dict(ld=1000, ldy=1001), dict(ld=1000, shift=1), dict(ld=1004, inplace=True),
               dict(ld=1001, inplace=True)):
        z, g2 = run_row(r, t, **kw)
        assert torch.equal(z[:, :V], y) and torch.equal(g2, g), kw


def test_a_whole_vocabulary():
    V = 151936
    t = Target(nb=1, V=V)
    for nb, m, seed in ((1, 1, 1), (2, 5, 2), (5, 32, 3)):
        r = Row(nb, m, V, seed, n_bias=300, mask=True, tree=True, ragged=nb > 1)
        y, g = run_row(r, t)
        if nb * m > 20:     # the rows of two sequences
            r.nb, y, g = 2, y[:2 * m], g[:2 * m]
        r.check(y, g)


def test_biases_of_one_slice_and_of_one_token():
    V = 151936
    t = Target(nb=1, V=V)
    r = Row(2, 2, V, 3, n_bias=1024)
    r.bias_ids[0] = 19000 + np.arange(1024) % 700     # ids of one part of the vocabulary, some twice
    r.bias_ids[1] = 151935
    r.bias[1] = 2.0 ** -6 * (np.arange(1024) % 7)     # sums that are exact
    r.check(*run_row(r, t))


# Sequences, rows and vocabularies of serving batches: several groups of rows a CTA, eight tiles a warp with one row and
# with two at a time, values one by one; and more sequences than the handle's scratch holds
@pytest.mark.parametrize("nb,m,V,most", [(64, 16, 151936, 64), (64, 15, 151936, 64), (64, 1, 151936, 64), (16, 64, 32003, 16),
                                         (64, 16, 151935, 64), (64, 1, 151935, 64), (8, 16, 151936, 8), (1, 64, 151936, 1),
                                         (64, 16, 32003, 37), (64, 1, 151936, 37), (300, 3, 4096, 300), (16, 64, 4096, 16)])
def test_adjusted_logits_of_serving_batches(nb, m, V, most):
    """All rules, ragged, in place and not: three sequences against the oracle, and every sequence of the batch, which has
    the rules and logits of one of them, as the handle of one sequence gives it, whose work is split otherwise."""
    D = lib()
    k = min(3, nb)
    r = Row(k, m, V, nb + m, n_bias=50, mask=True, tree=True)
    y, g = run_row(r, Target(nb=1, V=V))
    r.check(y, g)
    want, want_g = y.view(torch.int32).view(k, m, V), g.view(k, m)
    tile = lambda a: a.repeat(-(-nb // k), *[1] * (a.dim() - 1))  # noqa: E731
    rules = D.logit_rules(*[tile(a)[:nb * a.shape[0] // k].contiguous() for a in r.rules().tensors])
    n = [m - (i * 5) % (m + 1) for i in range(nb)]
    t = Target(nb=most, V=V, Cmax=64, paged=False)
    x = tile(torch.from_numpy(r.x).cuda())[:nb * m].contiguous()
    same = x.clone()
    out, ids, only = torch.full_like(x, 7.0), i32(np.full(nb * m, 7)), i32(np.full(nb * m, 7))
    D.dflash_logits_adjust(t.h, nb, m, x, V, rules, i32(n), out, V, ids, t.ws)
    D.dflash_logits_adjust(t.h, nb, m, x, V, rules, i32(n), None, V, only, t.ws)
    assert torch.equal(x, same) and torch.equal(ids, only)
    D.dflash_logits_adjust(t.h, nb, m, same, V, rules, i32(n), same, V, None, t.ws)
    assert t.status() == 0
    left = torch.tensor(7.0).view(torch.int32).item()
    for i in range(nb):
        rows, behind = slice(i * m, i * m + n[i]), slice(i * m + n[i], (i + 1) * m)
        assert torch.equal(out[rows].view(torch.int32), want[i % k, :n[i]]), i
        assert torch.equal(same[rows].view(torch.int32), want[i % k, :n[i]]), i
        assert torch.equal(ids[rows], want_g[i % k, :n[i]]), i
        assert (out[behind].view(torch.int32) == left).all() and (ids[behind] == 7).all(), i
        assert torch.equal(same[behind], x[behind]), i


@pytest.mark.parametrize("nb,m,V", [(1, 1, 64), (256, 64, 64), (200, 64, 1024), (90, 64, 1025), (5, 3, 151936),
                                    (1, 1, 2 ** 21), (2, 64, 2 ** 21)])
def test_scratch_of_the_ids(nb, m, V):
    """A sequence's scratch follows the vocabulary: at most a pair of words for each row and 1024 tokens. Nothing is
    written behind the workspace's end, where that scratch lies."""
    D = lib()
    t, one = Target(nb=nb, V=V, Cmax=64, paged=False), Target(nb=1, V=V, Cmax=64, paged=False)
    per = (t.ws.numel() - one.ws.numel()) / max(nb - 1, 1)
    assert per <= 8 * 64 * min(256, -(-V // 1024)) + 16384   # the rest of these small handles: below 16 KB a sequence
    size = t.ws.numel()
    ws = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    ws[:size] = 0
    x = torch.randint(-1000, 1000, (nb * m, V), generator=torch.Generator(device="cuda").manual_seed(V), device="cuda").float()
    ids = i32(np.full(nb * m, 7))
    D.dflash_logits_adjust(t.h, nb, m, x, V, D.logit_rules(), None, None, V, ids, ws)
    assert D.dflash_status(t.h, ws) == 0 and (ws[size:] == 0x5A).all()
    first = torch.arange(V, dtype=torch.int32, device="cuda").where(x == x.max(1, keepdim=True).values, V).min(1).values
    assert torch.equal(ids, first)


@pytest.mark.parametrize("nb,m", [(3, 2), (40, 8)])
def test_special_values_and_ties(nb, m):
    V = 520
    t = Target(nb=1, V=V)
    r = Row(nb, m, V, 4, penalties=False, counts=False, mask=True)
    r.x = np.round(2 * r.x) / 2           # many ties
    r.x[:, 5] = np.nan
    r.x[0] = -np.inf
    r.x[1] = np.nan
    r.x[2, 100] = r.x[2, 300] = np.inf
    r.allowed[2, [100, 300]] = True
    r.allowed[3] = False
    r.x[4] = 1.0
    r.allowed[4, :] = True
    y, g = run_row(r, t)
    for i in range(nb * m):
        w, _ = r.want(i // m, i % m)
        assert np.array_equal(y[i].double().cpu().numpy(), w, equal_nan=True)
        assert int(g[i]) == orc.greedy(w)
    assert g[:5].tolist()[:2] == [-1, -1] and g[2:5].tolist() == [100, -1, 0]
    # penalties of infinities and NaN stay what they are
    r = Row(2, 1, V, 4, mask=False)
    r.x[:, :260] = np.array([np.inf, -np.inf, np.nan, 0.0] * 65)
    y, g = run_row(r, t)
    r.check(y, None)


def test_logits_out_of_range_rows_and_trees_are_reported():
    D = lib()
    t = Target(nb=1, V=64)
    r = Row(2, 4, 64, 1, tree=True)
    for n in ([5, 1], [1, -1]):
        r.n = n
        x = torch.zeros(8, 64, device="cuda")
        D.dflash_logits_adjust(t.h, 2, 4, x, 64, r.rules(), i32(n), x, 64, None, t.ws)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK
    r.n = None
    for j, up in ((0, 1), (2, 2), (3, -1)):
        r2 = Row(2, 4, 64, 1, tree=True)
        r2.parent[1, j] = up
        D.dflash_logits_adjust(t.h, 2, 4, x, 64, r2.rules(), None, x, 64, None, t.ws)
        assert t.status() == D.DFLASH_ERR_DEVICE_CHECK


def test_a_captured_round_of_logits_walk_and_counts():
    """Greedy tokens of adjusted logits, the walk along them and the counts of what it emitted, in one graph."""
    D = lib()
    nb, m, V = 6, 12, 4096
    t = Target(nb=1, V=V)
    r = Row(nb, m, V, 8, n_bias=30, mask=True, tree=True)
    x, ids = torch.from_numpy(r.x).cuda(), i32(np.zeros((nb, m)))
    rules = r.rules()
    counts, par, tok = rules.tensors[1], rules.tensors[5], rules.tensors[6]
    tau, bonus, path, out, ctx = (i32(np.zeros(s)) for s in (nb, nb, (nb, m), (nb, m), nb))

    def call():
        D.dflash_logits_adjust(t.h, nb, m, x, V, rules, None, None, V, ids, t.ws)
        D.dflash_accept_tree(t.h, nb, m, par, tok, ids, None, ctx, tau, bonus, path, out, t.ws)
        D.dflash_token_counts(t.h, nb, m, out, m, tau, 0, counts, t.ws)
    keep = counts.clone()
    call()
    counts.copy_(keep)
    ctx.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    total = np.zeros(nb, int)
    for k in range(3):
        want = [[orc.greedy(r.want(i, j)[0]) for j in range(m)] for i in range(nb)]
        g.replay()
        assert t.status() == 0 and ids.tolist() == want
        for i in range(nb):
            p, e = orc.accept_tree(r.parent[i], r.tokens[i], want[i])
            total[i] += len(p)
            assert out[i].tolist()[:len(e)] == e and int(tau[i]) == len(e)
            np.add.at(r.counts[i], e, 1)
        assert np.array_equal(counts.cpu().numpy(), r.counts.view(np.int32)) and ctx.tolist() == total.tolist()
        # the next round: the first sequences' trees hold what will be emitted
        nxt = [[orc.greedy(r.want(i, 0)[0])] for i in range(nb)]
        r.tokens[:3, 1] = [n[0] for n in nxt[:3]]
        tok.copy_(i32(r.tokens))


# ------------------------------------------------------------------ a run of them together

@pytest.mark.parametrize("paged,window", [(True, 0), (False, 0), (True, 40)])
def test_tree_rounds_emit_what_single_tokens_emit(paged, window):
    """A small two-layer target with penalties decodes by trees of guesses, some right: what it emits are the tokens
    that it gives one by one, and the cache rows at the end are theirs."""
    D = lib()
    nb, Hq, Hkv, hd, N, V, C0, steps = 3, 4, 2, 64, 2, 96, 21, 40
    dim = Hq * hd
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    E, W_lm = rnd(V, dim), rnd(V, dim) / dim ** 0.5
    W_qkv = [rnd((Hq + 2 * Hkv) * hd, dim) / dim ** 0.5 for _ in range(N)]
    pen = torch.tensor([[1.2, 0.3, 0.2]] * nb, device="cuda")
    prompt = torch.randint(V, (nb, C0), generator=g, device="cuda").to(torch.int32)

    class Text:
        def __init__(self):
            self.t = Target(Hq, Hkv, hd, Cmax=192, nb=nb, N=N, V=V, paged=paged, seed=1)
            self.ctx, self.counts = i32(np.zeros(nb)), i32(np.zeros((nb, V)))
            D.dflash_token_counts(self.t.h, nb, C0, prompt, C0, None, 1, self.counts, self.t.ws)
            for at in range(0, C0 - 1, 10):
                self.forward(prompt[:, at:min(at + 10, C0 - 1)].contiguous(), None, None)
                self.ctx += min(at + 10, C0 - 1) - at
            self.root = prompt[:, -1:].contiguous()

        def forward(self, tokens, parent, depth):
            """Logits behind every row; rows are appended at ctx."""
            t, m = self.t, tokens.shape[1]
            depth = torch.arange(m, dtype=torch.int32, device="cuda").expand(nb, m) if depth is None else depth
            pos = (self.ctx[:, None] + depth).contiguous().view(-1)
            x = E[tokens.long()]
            for layer in range(N):
                qkv = (x.view(nb * m, dim) @ W_qkv[layer].t()).to(torch.bfloat16)
                q, k, v = qkv.split([Hq * hd, Hkv * hd, Hkv * hd], dim=1)
                qr = torch.empty(nb, m, Hq, hd, dtype=torch.bfloat16, device="cuda")
                kr = torch.empty(nb * m, Hkv * hd, dtype=torch.bfloat16, device="cuda")
                ld = qkv.stride(0)
                D.dflash_qk_norm_rope(t.h, nb * m, 1, q, ld, k, ld, None, None, pos, qr, kr)
                D.dflash_kv_append(t.h, nb, layer, m, kr, Hkv * hd, v, ld, None, 0, None, self.ctx, t.kc, t.vc, t.ws)
                o = t.attend(m, qr, parent, None, self.ctx, window, 3 if window else 0, layer=layer)
                x = x + o.view(nb, m, dim).float()
            return x.view(nb * m, dim) @ W_lm.t()

        def round(self, tokens, parent=None, depth=None):
            """Logits, greedy tokens, the walk, the move of the rows and the counts; (tau, emitted, adjusted logits)."""
            t, m = self.t, tokens.shape[1]
            par = i32([[-1]] * nb) if parent is None else parent
            z = self.forward(tokens, par, depth).contiguous()
            ids, tau, bonus = i32(np.zeros((nb, m))), i32(np.zeros(nb)), i32(np.zeros(nb))
            path, out = i32(np.zeros((nb, m))), i32(np.zeros((nb, m)))
            D.dflash_logits_adjust(t.h, nb, m, z, V, D.logit_rules(pen, self.counts, parent=par, tokens=tokens), None, z, V,
                                   ids, t.ws)
            D.dflash_accept_tree(t.h, nb, m, par, tokens, ids, None, self.ctx, tau, bonus, path, out, t.ws)
            D.dflash_kv_commit(t.h, nb, m, path, tau, self.ctx, t.kc, t.vc, t.ws)
            D.dflash_token_counts(t.h, nb, m, out, m, tau, 0, self.counts, t.ws)
            assert t.status() == 0
            self.root = bonus[:, None].contiguous()
            return tau.tolist(), out.tolist(), z

        def forced(self, tokens):
            """Adjusted logits behind the root, and `tokens` taken instead of their greedy ones."""
            t = self.t
            z = self.forward(self.root, i32([[-1]] * nb), None).contiguous()
            D.dflash_logits_adjust(t.h, nb, 1, z, V, D.logit_rules(pen, self.counts), None, z, V, None, t.ws)
            self.root = i32(tokens)[:, None].contiguous()
            self.ctx += 1
            D.dflash_token_counts(t.h, nb, 1, self.root, 1, None, 0, self.counts, t.ws)
            assert t.status() == 0
            return z

    one, text = Text(), [[] for _ in range(nb)]
    for _ in range(steps):
        _, out, _ = one.round(one.root)
        for i in range(nb):
            text[i].append(out[i][0])
    many, done, rng = Text(), [[] for _ in range(nb)], np.random.default_rng(2)
    taus = []
    while min(len(d) for d in done) < steps - 12:
        m = 12
        par, tok = trees(nb, m, int(rng.integers(1000))), rng.integers(0, V, (nb, m))
        depth = np.array([[len(line) - 1 for line in orc.tree_lines(par[i])] for i in range(nb)])
        for i in range(nb):
            tok[i, 0] = int(many.root[i])
            for j in range(1, m):   # the token that single steps gave at its depth, two times in three
                k = len(done[i]) + depth[i, j] - 1
                if rng.random() < 0.67 and k < steps:
                    tok[i, j] = text[i][k]
        tau, out, _ = many.round(i32(tok), i32(par), i32(depth))
        taus += tau
        for i in range(nb):
            done[i] += out[i][:tau[i]]
    assert max(taus) >= 3, "no tree was accepted far"
    # The same text token by token: each of its tokens is the greedy one, or one that the attention's rounding
    # cannot tell from it. An output is off by (2^-8 + 2^-8) sum p|v| <= 2^-7 max|v| on either side, 2^-6 * 4 = 2^-4
    # in every channel at the most; over W_lm's rows of norm 1 with signs of their own the two layers' logits
    # are off by 2^-4 each, and by as much through the second layer's inputs: 3 * 2^-4. Keys and values likewise.
    n = min(len(d) for d in done)
    force = Text()
    for k in range(n):
        z = force.forced([d[k] for d in done])
        for i in range(nb):
            assert float(z[i].max() - z[i, done[i][k]]) <= 3 * 2.0 ** -4, (i, k)
    for layer in range(N):
        for a, b in ((force.t.kc, many.t.kc), (force.t.vc, many.t.vc)):
            for i in range(nb):
                x, y = (f64(c.rows(s, layer, i, C0 - 1 + n)) for c, s in ((force.t, a), (many.t, b)))
                assert (np.abs(x - y) <= 3 * 2.0 ** -4 + 2.0 ** -7 * np.abs(x)).all(), (layer, i)


@pytest.mark.parametrize("paged", [False, True])
def test_a_drafters_round(paged):
    """The calls of a round through Drafter, every layer: attention, ids, walk and the moved rows against the oracle."""
    import dflash_inputs as di
    from block_diffusion_speculative_project_gb300 import drafter
    w = di.TINY
    nb, Cmax, m = 2, 192, 12
    Hq, Hkv, hd, V = w.Hq, w.Hkv, w.hd, w.V
    dev = {k: drafter.to_device_bf16(v) for k, v in di.make_weights(w, 0).items()}
    pps = Cmax // PR
    dr = drafter.Drafter(w, dev, nb, Cmax, w.B, num_pages=nb * pps + 1 if paged else 0)
    table = np.random.default_rng(1).permutation(nb * pps + 1)[:nb * pps].reshape(nb, pps)
    if paged:
        dr.set_block_table(i32(table))
    lens = [100, 3]
    ctx, par = i32(lens), trees(nb, m, 1)
    depth = i32([[len(line) - 1 for line in orc.tree_lines(par[i])] for i in range(nb)])
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)

    def rows(t, layer, i, n):
        if paged:
            return t[layer][i32(table[i]).long()].transpose(0, 1).reshape(Hkv, -1, hd)[:, :n].clone()
        return t[layer, i, :, :n].clone()

    pos = (ctx[:, None] + depth).view(-1)
    for layer in range(w.N):
        k, v = rnd(nb * 100, Hkv * hd), rnd(nb * 100, Hkv * hd)
        dr.kv_append(nb, layer, 100, k, v, i32([0, 0]), n_rows=ctx)
        q, k, v = rnd(nb * m, (Hq + 2 * Hkv) * hd).split([Hq * hd, Hkv * hd, Hkv * hd], dim=1)
        q_rot, k_rot = rnd(nb, m, Hq, hd), rnd(nb * m, Hkv * hd)
        dr.qk_norm_rope(nb * m, 1, q, k, pos, q_rot, k_rot)
        dr.kv_append(nb, layer, m, k_rot, v, ctx, rotate=False)
        out = torch.empty_like(q_rot)
        dr.attention_tree(nb, layer, m, q_rot, ctx, out, parent=i32(par), window=50, sinks=4)
        for i in range(nb):
            K, V_ = (f64(rows(c, layer, i, lens[i] + m)) for c in (dr.kcache, dr.vcache))
            o, mag, dot = orc.attention_tree(f64(q_rot[i]), K, V_, orc.tree_visible(par[i], lens[i], 50, 4))
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -14 + 2 * hd * 2.0 ** -24 * dot[..., None]) * mag
            assert (np.abs(f64(out[i]) - o) <= tol).all()
    r = Row(nb, m, V, 3, n_bias=5, mask=True, tree=True)
    r.parent = par
    want = [[orc.greedy(r.want(i, j)[0]) for j in range(m)] for i in range(nb)]
    for i in range(nb):   # some nodes hold what will be asked for; a drafted token changes only rows below it
        for j in range(1, m, 2):
            r.tokens[i, j] = orc.greedy(r.want(i, int(par[i, j]))[0])
        want[i] = [orc.greedy(r.want(i, j)[0]) for j in range(m)]
    rules = r.rules().tensors
    x = torch.from_numpy(r.x).cuda()
    ids, tau, bonus = i32(np.zeros((nb, m))), i32(np.zeros(nb)), i32(np.zeros(nb))
    path, emitted = i32(np.zeros((nb, m))), i32(np.zeros((nb, m)))
    old = [[[rows(c, layer, i, lens[i] + m) for c in (dr.kcache, dr.vcache)] for i in range(nb)] for layer in range(w.N)]
    dr.logits_adjust(nb, m, x, None, ids, *rules)
    dr.accept_tree(nb, m, rules[5], rules[6], ids, tau, bonus, out_path=path, out_tokens=emitted, ctx_len=ctx)
    dr.kv_commit(nb, m, path, tau, ctx)
    dr.token_counts(nb, m, emitted, rules[1], n_tokens=tau)
    assert dr.status() == 0 and ids.tolist() == want
    counts = r.counts.copy()
    for i in range(nb):
        walk, said = orc.accept_tree(par[i], r.tokens[i], want[i])
        assert path[i].tolist()[:len(walk)] == walk and emitted[i].tolist()[:len(said)] == said
        assert int(ctx[i]) == lens[i] + len(walk) and int(bonus[i]) == said[-1]
        np.add.at(counts[i], said, 1)
        keep = list(range(lens[i])) + [lens[i] + a for a in walk]
        for layer in range(w.N):
            for c, was in zip((dr.kcache, dr.vcache), old[layer][i]):
                assert torch.equal(rows(c, layer, i, len(keep)), was[:, keep])
    assert np.array_equal(rules[1].cpu().numpy(), counts.view(np.int32))
