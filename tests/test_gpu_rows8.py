"""Per-head norm and rotation, cache appends in bf16 and 8 bits, and attention over the 8-bit
cache, through the C ABI against the fp64 oracle.

Tolerances (u = half a step of a type relative to the value: bf16 2^-8, f16 2^-11, e4m3 2^-4,
f32 2^-24):
  rows       one bf16 rounding 2^-8 |y|; the fp32 steps before it: norm sum of hd <= 128 squares
             (128 u), its root, reciprocal and two products (< 16 u): 2^-16 |x| for each of the two
             rotated values a, b; sine and cosine to 2^-20.  2^-8 |y| + (2^-16 + 2^-19)(|a| + |b|)
  8 bits     half a step of e4m3: 2^-4 |y| for normal values, scale * 2^-10 for subnormal ones,
             and the same fp32 steps; scales are exact where amax is not within 2^-15 of a border
             (checked on the oracle's side). Rows that stay are exact.
  attention  one bf16 rounding 2^-8 |o|; probabilities rounded to f16, 2^-11 p, then to a sum of three
             e5m2 terms: the first keeps 3 bits, so the rest is below 2^-2 of p's power of two, the
             second rounds that rest to 3 bits (at most 2^-6 off), the third what is then left, at
             most 2^-6, to 3 bits: at most 2^-10 off. Scores: hd products and sums in fp32,
             hd * 2^-24 * sum|q k| / sqrt(hd), which move p by twice that at most; exponent and log2
             steps below 2^-16 of p; e5m2's smallest step is 2^-16, half of it 2^-24 of the largest
             p * scale (2^7 at the least) for every key: rows * 2^-24 * max|v|.
"""
import numpy as np
import pytest
import torch

import dflash_inputs as di
from oracle import dflash_oracle as orc

pytestmark = pytest.mark.gpu

PR = orc.PAGE_ROWS
EPS, BASE = 1e-6, 1e4


def lib():
    from block_diffusion_speculative_project_gb300 import dflash
    return dflash


def i32(a):
    return None if a is None else torch.tensor(np.asarray(a, np.int32), device="cuda")


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Cache:
    """A handle with its four kinds of caches, filled with seeded values, and their numpy view."""

    def __init__(self, Hq, Hkv, hd, Cmax, nb, N=2, B=16, paged=True, spare=2, seed=0, max_spin=0, flags=0):
        D = lib()
        self.D, self.Hq, self.Hkv, self.hd, self.Cmax, self.nb, self.N = D, Hq, Hkv, hd, Cmax, nb, N
        self.pps = Cmax // PR
        rng = np.random.default_rng(seed)
        P = nb * self.pps + spare if paged else 0
        self.table = rng.permutation(P)[:nb * self.pps].reshape(nb, self.pps) if paged else None
        self.cfg = D.dflash_config(D=64, Dt=64, L=1, N=N, Hq=Hq, Hkv=Hkv, hd=hd, F=64, V=64, B=B, k_top=1,
                                   rope_base=BASE, eps=EPS, mask_id=0, Cmax=Cmax, max_batch=nb, max_proj_rows=1,
                                   conv_group=16, sel_dim=256, flags=flags, max_spin=max_spin, film_dim=0,
                                   num_pages=P)
        self.h = D.dflash_create(self.cfg)
        if paged:
            self.dev_table = i32(self.table)
            D.dflash_set_block_table(self.h, self.dev_table)
        self.ws = torch.zeros(D.dflash_workspace_size(self.h), dtype=torch.uint8, device="cuda")
        lead = (N, P, Hkv) if paged else (N, nb, Hkv, self.pps)
        self.lead = lead
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.kc, self.vc = (r(*lead, PR, hd).to(torch.bfloat16) for _ in range(2))
        self.k8, self.v8 = ((100 * r(*lead, PR, hd)).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2))
        self.ks, self.vs = (torch.exp2(torch.randint(-8, -5, lead, generator=g, device="cuda").float())
                            for _ in range(2))

    def at(self, i, b):
        """Index of sequence i's block b in a cache [N, ...lead..., 64, hd], without layer and head."""
        return (int(self.table[i, b]), slice(None)) if self.table is not None else (i, slice(None), b)

    def rows(self, t, layer, i, n, scale=None):
        """Rows [0, n) of sequence i, [Hkv, n, hd] in 64 bits (times the block scales)."""
        out = []
        for b in range(-(-n // PR)):
            x = f64(t[layer][self.at(i, b)])
            out.append(x if scale is None else x * f64(scale[layer][self.at(i, b)])[:, None, None])
        return np.concatenate(out, axis=1)[:, :n]

    def status(self):
        return self.D.dflash_status(self.h, self.ws)

    def append8(self, layer, R, k, v, n, ctx, g=None, rotate=1, nb=None):
        self.D.dflash_kv_append8(self.h, nb or self.nb, layer, R, k, k.stride(0), v, v.stride(0), g, rotate, i32(n),
                                 i32(ctx), self.k8, self.v8, self.ks, self.vs, self.ws)

    def append(self, layer, R, k, v, n, ctx, g=None, rotate=1, nb=None):
        self.D.dflash_kv_append(self.h, nb or self.nb, layer, R, k, k.stride(0), v, v.stride(0), g, rotate, i32(n),
                                i32(ctx), self.kc, self.vc, self.ws)

    def attend(self, layer, m, q, n, ctx, causal, hint=0, out=None, nb=None):
        nb = nb or self.nb
        out = torch.full((nb, m, self.Hq, self.hd), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        self.D.dflash_attention8(self.h, nb, layer, m, q, self.k8, self.v8, self.ks, self.vs, i32(n), i32(ctx), hint,
                                 int(causal), out, self.ws)
        return out


def fused(nb, R, Hq, Hkv, hd, seed, big=None):
    """Rows of a fused q|k|v projection, and views of its parts; big = (row, scale) makes a row large."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(nb * R, (Hq + 2 * Hkv) * hd, generator=g, device="cuda")
    if big:
        x[big[0]] *= big[1]
    x = x.to(torch.bfloat16)
    q, k, v = x.split([Hq * hd, Hkv * hd, Hkv * hd], dim=1)
    gq, gk = ((1 + 0.2 * torch.randn(hd, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    return q, k, v, gq, gk


def want_rows(x, nb, R, heads, hd, g, pos, rotate=True):
    """[nb, R, heads, hd] in 64 bits, and the fp32 part of the tolerance (2^-16 + 2^-19)(|a| + |b|)."""
    x = f64(x).reshape(nb * R, heads, hd)
    gg = None if g is None else f64(g)
    normed = orc.head_rows(x, gg, np.zeros(nb * R), BASE, EPS, rotate=False)
    y = orc.head_rows(x, gg, np.asarray(pos).reshape(-1), BASE, EPS, rotate=rotate)
    a = np.abs(normed)
    slack = (a + np.roll(a, hd // 2, axis=-1)) * (2.0 ** -16 + 2.0 ** -19)
    return y.reshape(nb, R, heads, hd), slack.reshape(nb, R, heads, hd)


def assert_within(got, want, tol, what=""):
    assert np.isfinite(got).all(), f"{what}: not finite"
    bad = np.abs(got - want) > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{(np.abs(got - want) / np.maximum(tol, 1e-300)).max():.2f} of the tolerance")


# ------------------------------------------------------------------ refusals (no launch)

def test_refusals():
    D = lib()
    c = Cache(4, 2, 64, 128, 2, B=4)
    q, k, v, gq, gk = fused(2, 4, 4, 2, 64, 1)
    ctx = i32([0, 0])
    out_q = torch.empty(2, 4, 4, 64, dtype=torch.bfloat16, device="cuda")
    out_k = torch.empty(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    ld = q.stride(0)

    def norm(nb=2, R=4, q=q, ldq=ld, k=k, ldk=ld, pos=ctx, oq=out_q, ok=out_k, g=gq):
        D.dflash_qk_norm_rope(c.h, nb, R, q, ldq, k, ldk, g, gk, pos, oq, ok)

    def app8(nb=2, layer=0, R=4, k=k, ldk=ld, v=v, ldv=ld, ctx=ctx, k8=c.k8, ks=c.ks, ws=c.ws):
        D.dflash_kv_append8(c.h, nb, layer, R, k, ldk, v, ldv, gk, 1, None, ctx, k8, c.v8, ks, c.vs, ws)

    def app(nb=2, layer=0, R=4, k=k, ldk=ld, v=v, ldv=ld, ctx=ctx, kc=c.kc, ws=c.ws):
        D.dflash_kv_append(c.h, nb, layer, R, k, ldk, v, ldv, gk, 1, None, ctx, kc, c.vc, ws)

    def att(nb=2, layer=0, m=4, q=out_q, k8=c.k8, ks=c.ks, ctx=ctx, hint=0, o=out_q, ws=c.ws):
        D.dflash_attention8(c.h, nb, layer, m, q, k8, c.v8, ks, c.vs, None, ctx, hint, 0, o, ws)

    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    odd = out_q.view(-1)[1:]
    for f, kw in ((norm, dict(nb=-1)), (norm, dict(R=-1)), (norm, dict(q=None)), (norm, dict(ldq=4 * 64 - 8)),
                  (norm, dict(ldq=ld + 4)), (norm, dict(ldk=64)), (norm, dict(pos=None)), (norm, dict(oq=None)),
                  (norm, dict(ok=None)), (norm, dict(k=None)), (norm, dict(q=odd)), (norm, dict(g=gq[1:])),
                  (app8, dict(nb=3)), (app8, dict(nb=-1)), (app8, dict(layer=2)), (app8, dict(layer=-1)),
                  (app8, dict(R=129)), (app8, dict(R=-1)), (app8, dict(k=None)), (app8, dict(ldv=64)),
                  (app8, dict(ctx=None)), (app8, dict(k8=None)), (app8, dict(ks=None)), (app8, dict(ws=small)),
                  (app, dict(nb=3)), (app, dict(layer=2)), (app, dict(R=129)), (app, dict(v=None)),
                  (app, dict(ldk=ld + 1)), (app, dict(kc=None)), (app, dict(ws=small)), (app, dict(ctx=None)),
                  (att, dict(nb=3)), (att, dict(layer=5)), (att, dict(m=5)), (att, dict(m=-1)), (att, dict(q=None)),
                  (att, dict(q=odd)), (att, dict(k8=None)), (att, dict(ks=None)), (att, dict(ctx=None)),
                  (att, dict(hint=-1)), (att, dict(hint=129)), (att, dict(o=None)), (att, dict(ws=small))):
        with pytest.raises(D.DflashError) as e:
            f(**kw)
        assert e.value.code == D.DFLASH_ERR_INVALID_ARG, (f.__name__, kw, e.value)
    for f, kw in ((norm, dict(nb=0)), (norm, dict(R=0)), (app8, dict(nb=0)), (app8, dict(R=0)), (app, dict(R=0)),
                  (att, dict(m=0)), (att, dict(nb=0))):
        f(**kw)  # nothing to do
    assert c.status() == 0
    bare = D.dflash_config.from_buffer_copy(c.cfg)
    bare.num_pages, bare.Cmax = 0, 100
    h = D.dflash_create(bare)
    ws = torch.zeros(D.dflash_workspace_size(h), dtype=torch.uint8, device="cuda")
    with pytest.raises(D.DflashError) as e:
        D.dflash_kv_append8(h, 1, 0, 4, k, ld, v, ld, None, 1, None, ctx, c.k8, c.v8, c.ks, c.vs, ws)
    assert e.value.code == D.DFLASH_ERR_UNSUPPORTED_SHAPE  # 8-bit blocks: Cmax % 64
    D.dflash_destroy(h)
    bare.num_pages, bare.Cmax = 4, 128
    h = D.dflash_create(bare)
    for call in (lambda: D.dflash_kv_append8(h, 1, 0, 4, k, ld, v, ld, None, 1, None, ctx, c.k8, c.v8, c.ks, c.vs,
                                             c.ws),
                 lambda: D.dflash_attention8(h, 1, 0, 4, out_q, c.k8, c.v8, c.ks, c.vs, None, ctx, 0, 0, out_q, c.ws)):
        with pytest.raises(D.DflashError) as e:
            call()
        assert e.value.code == D.DFLASH_ERR_INVALID_ARG  # no block table
    D.dflash_destroy(h)


# ------------------------------------------------------------------ norm and rotation

@pytest.mark.parametrize("Hq,Hkv,hd,nb,R,base", [(4, 4, 64, 1, 1, 0), (32, 8, 128, 1, 1, 4095), (8, 2, 128, 3, 5, 7),
                                                 (1, 1, 64, 2, 17, 1), (32, 8, 128, 2, 300, 60), (7, 7, 64, 5, 33, 9),
                                                 (32, 8, 128, 1, 3, 2000000000), (16, 2, 64, 2, 700, 131071)])
@pytest.mark.parametrize("norm", [True, False])
def test_qk_norm_rope(Hq, Hkv, hd, nb, R, base, norm):
    c = Cache(Hq, Hkv, hd, 128, nb)
    q, k, _, gq, gk = fused(nb, R, Hq, Hkv, hd, seed=R, big=(0, 1e4))
    pos0 = np.array([base + 37 * i for i in range(nb)])
    pos = pos0[:, None] + np.arange(R)
    oq = torch.zeros(nb, R, Hq, hd, dtype=torch.bfloat16, device="cuda")
    ok = torch.zeros(nb, R, Hkv, hd, dtype=torch.bfloat16, device="cuda")
    g = (gq, gk) if norm else (None, None)
    c.D.dflash_qk_norm_rope(c.h, nb, R, q, q.stride(0), k, k.stride(0), *g, i32(pos0), oq, ok)
    for got, x, n, gg in ((oq, q, Hq, g[0]), (ok, k, Hkv, g[1])):
        want, slack = want_rows(x, nb, R, n, hd, gg, pos)
        assert_within(f64(got), want, 2.0 ** -8 * np.abs(want) + slack)
    # queries alone, in place
    only = q.contiguous()
    c.D.dflash_qk_norm_rope(c.h, nb, R, only, only.stride(0), None, 0, g[0], None, i32(pos0), only, None)
    assert torch.equal(only.view_as(oq), oq)


def test_norm_of_one_tensor_only_and_of_zeros():
    c = Cache(4, 2, 128, 128, 1)
    q, k, _, gq, gk = fused(1, 9, 4, 2, 128, seed=3)
    q = q.clone()
    q[3] = 0
    oq, ok = torch.empty(1, 9, 4, 128, dtype=torch.bfloat16, device="cuda"), \
        torch.empty(1, 9, 2, 128, dtype=torch.bfloat16, device="cuda")
    for g in ((gq, None), (None, gk)):
        c.D.dflash_qk_norm_rope(c.h, 1, 9, q, q.stride(0), k, k.stride(0), *g, i32([11]), oq, ok)
        for got, x, n, gg in ((oq, q, 4, g[0]), (ok, k, 2, g[1])):
            want, slack = want_rows(x, 1, 9, n, 128, gg, 11 + np.arange(9))
            assert_within(f64(got), want, 2.0 ** -8 * np.abs(want) + slack)
        assert not oq[0, 3].any()


# ------------------------------------------------------------------ appends

APPENDS = [(4, 64, 1, 1, [0], [1], True), (2, 128, 3, 5, [63, 64, 0], [5, 0, 3], True),
           (1, 128, 2, 64, [0, 64], [64, 63], False), (8, 128, 3, 130, [1, 63, 100], [130, 129, 2], True),
           (2, 64, 2, 200, [56, 17], [200, 66], False), (3, 64, 4, 16, [240, 255, 0, 128], [16, 1, 16, 0], True)]


@pytest.mark.parametrize("Hkv,hd,nb,R,ctx,n,paged", APPENDS)
@pytest.mark.parametrize("norm,rotate", [(True, 1), (False, 1), (False, 0)])
def test_kv_append(Hkv, hd, nb, R, ctx, n, paged, norm, rotate):
    c = Cache(Hkv, Hkv, hd, 256, nb, paged=paged, seed=R)
    _, k, v, _, gk = fused(nb, R, 1, Hkv, hd, seed=5)
    k = k.clone()
    v = v.clone()
    for i in range(nb):  # rows beyond n are padding
        k[i * R + n[i]:(i + 1) * R] = float("nan")
        v[i * R + n[i]:(i + 1) * R] = float("nan")
    before = {name: getattr(c, name).clone() for name in ("kc", "vc")}
    c.append(1, R, k, v, n, ctx, gk if norm else None, rotate)
    assert c.status() == 0
    pos = np.array(ctx)[:, None] + np.arange(R)
    wk, slack = want_rows(torch.nan_to_num(k), nb, R, Hkv, hd, gk if norm else None, pos, bool(rotate))
    wv = f64(torch.nan_to_num(v)).reshape(nb, R, Hkv, hd)
    same = {name: before[name].clone() for name in before}
    for i in range(nb):
        got_k, got_v = c.rows(c.kc, 1, i, ctx[i] + n[i])[:, ctx[i]:], c.rows(c.vc, 1, i, ctx[i] + n[i])[:, ctx[i]:]
        w = wk[i, :n[i]].transpose(1, 0, 2)
        assert_within(got_k, w, 2.0 ** -8 * np.abs(w) + slack[i, :n[i]].transpose(1, 0, 2), f"keys {i}")
        assert np.array_equal(got_v, wv[i, :n[i]].transpose(1, 0, 2))
        for b in range(c.pps):  # what the call may write
            lo, hi = max(ctx[i], b * PR) - b * PR, min(ctx[i] + n[i], (b + 1) * PR) - b * PR
            if lo < hi:
                for name in same:
                    same[name][1][c.at(i, b)][:, lo:hi] = getattr(c, name)[1][c.at(i, b)][:, lo:hi]
    for name in same:
        assert torch.equal(getattr(c, name).view(torch.int16), same[name].view(torch.int16)), name


def check_append8(c, layer, R, k, v, n, ctx, gk, rotate, before):
    """Compares the 8-bit caches with the oracle's append to `before`; returns how many scales grew."""
    nb, Hkv, hd = c.nb, c.Hkv, c.hd
    pos = np.array(ctx)[:, None] + np.arange(R)
    wk, slack = want_rows(torch.nan_to_num(k, posinf=0, neginf=0), nb, R, Hkv, hd, gk, pos, bool(rotate))
    if not torch.isfinite(k).all():  # rows of infinities and NaN are given without norm and rotation
        assert gk is None and not rotate
        wk = f64(k).reshape(nb, R, Hkv, hd)
    wv = f64(v).reshape(nb, R, Hkv, hd)
    grew = 0
    for cache, scale, want, sl in (("k8", "ks", wk, slack), ("v8", "vs", wv, np.zeros_like(wv))):
        exp_c, exp_s = before[cache].clone(), before[scale].clone()
        for i in range(nb):
            for b in range(ctx[i] // PR, -(-(ctx[i] + n[i]) // PR) if n[i] else 0):
                lo, hi = max(ctx[i], b * PR), min(ctx[i] + n[i], (b + 1) * PR)
                kept = lo - b * PR
                old, s_old = f64(before[cache][layer][c.at(i, b)]), f64(before[scale][layer][c.at(i, b)])
                got, s_got = f64(getattr(c, cache)[layer][c.at(i, b)]), f64(getattr(c, scale)[layer][c.at(i, b)])
                for h in range(Hkv):
                    x = want[i, lo - ctx[i]:hi - ctx[i], h]
                    y, s = orc.append8_block(old[h], s_old[h], kept, x)
                    assert s_got[h] == s, f"{scale} {i} {b} {h}: {s_got[h]} instead of {s}"
                    grew += bool(kept) and s > s_old[h]
                    assert np.array_equal(got[h, :kept], y[:kept], equal_nan=True), f"{cache} rows that stay"
                    nan = np.isnan(x)
                    assert np.array_equal(np.isnan(got[h, kept:kept + len(x)]), nan)
                    x = np.where(nan, 0, np.clip(x, -448 * s, 448 * s))
                    err = np.abs(np.where(nan, 0, got[h, kept:kept + len(x)]) * s - x)
                    tol = np.maximum(2.0 ** -4 * np.abs(x), s * 2.0 ** -10) + sl[i, lo - ctx[i]:hi - ctx[i], h]
                    assert (err <= tol * (1 + 1e-9)).all(), f"{cache} {i} {b} {h}: {(err / tol).max()}"
                exp_c[layer][c.at(i, b)][:, kept:hi - b * PR] = getattr(c, cache)[layer][c.at(i, b)][:, kept:hi - b * PR]
                exp_c[layer][c.at(i, b)][:, :kept] = getattr(c, cache)[layer][c.at(i, b)][:, :kept]
                exp_s[layer][c.at(i, b)] = getattr(c, scale)[layer][c.at(i, b)]
        assert torch.equal(getattr(c, cache).view(torch.uint8), exp_c.view(torch.uint8)), f"{cache}: other rows"
        assert torch.equal(getattr(c, scale), exp_s), f"{scale}: other blocks"
    return grew


def snap(c):
    return {x: getattr(c, x).clone() for x in ("k8", "v8", "ks", "vs")}


@pytest.mark.parametrize("Hkv,hd,nb,R,ctx,n,paged", APPENDS)
@pytest.mark.parametrize("norm,rotate", [(True, 1), (False, 1), (False, 0)])
def test_kv_append8(Hkv, hd, nb, R, ctx, n, paged, norm, rotate):
    c = Cache(Hkv, Hkv, hd, 256, nb, paged=paged, seed=R)
    # the first sequence's last row is large: the block it joins has to grow
    _, k, v, _, gk = fused(nb, R, 1, Hkv, hd, seed=6, big=(max(n[0] - 1, 0), 300.0))
    before = snap(c)
    c.append8(1, R, k, v, n, ctx, gk if norm else None, rotate)
    assert c.status() == 0
    grew = check_append8(c, 1, R, k, v, n, ctx, gk if norm else None, rotate, before)
    if (ctx[0] + n[0] - 1) // PR == ctx[0] // PR and ctx[0] % PR and n[0]:
        assert grew > 0


def test_append8_one_row_at_a_time_then_rollback():
    """65 single rows of growing and shrinking size, then the context set back into the first block."""
    c = Cache(2, 2, 128, 128, 1, seed=9)
    rng = np.random.default_rng(4)
    grew = 0
    for t in list(range(65)) + [20, 21]:
        _, k, v, _, gk = fused(1, 1, 1, 2, 128, seed=100 + t, big=(0, float(np.exp2(rng.integers(-12, 6)))))
        before = snap(c)
        c.append8(0, 1, k, v, None, [t], None, 1)
        grew += check_append8(c, 0, 1, k, v, [1], [t], None, 1, before)
    assert c.status() == 0
    assert grew > 0  # counted on the oracle: the draws do make blocks grow


def test_append8_infinities_nan_and_zeros():
    c = Cache(1, 1, 64, 128, 3)
    x = torch.zeros(3 * 4, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 3], x[0, 4], x[1, 5], x[2] = float("inf"), float("-inf"), float("nan"), 2.0
    x[5] = 1e38
    before = snap(c)
    c.append8(0, 4, x, x, None, [0, 60, 64], None, 0)
    check_append8(c, 0, 4, x, x, [4, 4, 4], [0, 60, 64], None, 0, before)
    assert c.status() == 0
    assert float(c.ks[0][c.at(2, 1)][0]) == 2.0 ** -100


def test_appends_report_lengths_and_pages_out_of_range():
    for bits8 in (True, False):
        c = Cache(2, 2, 64, 128, 2)
        _, k, v, _, _ = fused(2, 8, 1, 2, 64, seed=2)
        call = c.append8 if bits8 else c.append
        names = ("k8", "v8") if bits8 else ("kc", "vc")
        for n, ctx in (([9, 0], [0, 0]), ([-1, 0], [0, 0]), ([0, 0], [-1, 0]), ([0, 8], [0, 128]), ([0, 0], [0, 129])):
            before = {x: getattr(c, x).clone() for x in names}
            call(0, 8, k, v, n, ctx)
            assert c.status() == c.D.DFLASH_ERR_DEVICE_CHECK, (n, ctx)
            if n != [9, 0]:
                for x in names:
                    assert torch.equal(getattr(c, x).view(torch.uint8), before[x].view(torch.uint8)), (n, ctx)
        call(0, 8, k, v, [0, 8], [0, 124])  # four rows fit
        assert c.status() == c.D.DFLASH_ERR_DEVICE_CHECK
        for bad in (-1, c.cfg.num_pages):
            c.dev_table[1, 1] = bad
            before = {x: getattr(c, x).clone() for x in names}
            call(0, 8, k, v, [0, 8], [0, 70])
            assert c.status() == c.D.DFLASH_ERR_DEVICE_CHECK
            for x in names:
                assert torch.equal(getattr(c, x).view(torch.uint8), before[x].view(torch.uint8))
        call(0, 8, k, v, [8, 8], [70, 0])  # that page is not reached
        assert c.status() == 0


# ------------------------------------------------------------------ attention

def check_attention(c, layer, m, q, n, ctx, causal, out, what=""):
    for i in range(len(ctx)):
        K = c.rows(c.k8, layer, i, ctx[i] + n[i], c.ks) if n[i] else None
        V = c.rows(c.v8, layer, i, ctx[i] + n[i], c.vs) if n[i] else None
        if n[i]:
            o, mag, dot = orc.attention8(f64(q[i, :n[i]]), K, V, ctx[i], causal)
            tol = (2.0 ** -8 * np.abs(o) + mag * (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -16 + 2 * c.hd * 2.0 ** -24 * dot[..., None])
                   + K.shape[1] * 2.0 ** -24 * np.abs(V).max())
            assert_within(f64(out[i, :n[i]]), o, tol, f"{what} sequence {i}")
        assert (out[i, n[i]:] == 7.0).all(), f"{what}: rows behind sequence {i}"


def queries(c, m, seed=0, std=1.0, nb=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(nb or c.nb, m, c.Hq, c.hd, generator=g, device="cuda")).to(torch.bfloat16)


SHAPES = [(4, 4, 64), (8, 1, 64), (8, 2, 128), (16, 2, 128), (1, 1, 128), (6, 2, 64)]


@pytest.mark.parametrize("Hq,Hkv,hd", SHAPES)
@pytest.mark.parametrize("m", [1, 2, 7, 16])
@pytest.mark.parametrize("paged,causal", [(True, False), (False, True)])
def test_attention8(Hq, Hkv, hd, m, paged, causal):
    c = Cache(Hq, Hkv, hd, 384, 6, paged=paged, seed=m)
    q = queries(c, m, seed=m)
    ctx = [0, 64 - m, 63, 384 - m, 130, 5]
    for n in ([m] * 6, [1, m, 0, max(1, m - 1), m, (m + 1) // 2]):
        out = c.attend(1, m, q, n, ctx, causal)
        assert c.status() == 0
        check_attention(c, 1, m, q, n, ctx, causal, out)
    every = c.attend(0, m, q, None, ctx, causal, hint=384)
    check_attention(c, 0, m, q, [m] * 6, ctx, causal, every, "n_rows NULL")


@pytest.mark.parametrize("hd,Hq,Hkv,nb,m,L", [(128, 8, 2, 2, 3, 20000), (64, 4, 4, 1, 1, 9001), (128, 32, 8, 1, 16, 4096),
                                              (64, 2, 1, 70, 2, 700), (128, 2, 2, 33, 1, 1500)])
def test_attention8_many_units(hd, Hq, Hkv, nb, m, L):
    """Pairs split over many CTAs, and many pairs for one CTA; ragged, one sequence empty."""
    Cmax = -(-(L + m) // PR) * PR
    c = Cache(Hq, Hkv, hd, Cmax, nb, N=1, seed=nb)
    q = queries(c, m, seed=1)
    ctx = [(L * (i + 1)) // nb if i % 3 else L for i in range(nb)]
    n = [m if i != 1 else 0 for i in range(nb)]
    for causal in (False, True):
        out = c.attend(0, m, q, n, ctx, causal, hint=L)
        assert c.status() == 0
        check_attention(c, 0, m, q, n, ctx, causal, out)
        assert torch.equal(out, c.attend(0, m, q, n, ctx, causal, hint=L))  # reproducible


@pytest.mark.parametrize("hd", [64, 128])
def test_attention8_growing_scores_sinks_and_scales(hd):
    """Scores that grow along the context (the running maximum moves often), a first key that takes
    most of the weight, blocks whose scales differ by 2^40, and one of scale zero."""
    c = Cache(4, 1, hd, 1024, 2, N=1, seed=7)
    m = 4
    q = queries(c, m, seed=2)
    ctx = [1020, 700]
    grow = torch.ones(hd, device="cuda")
    for i in range(2):
        for b in range(c.pps):
            x = torch.randn(PR, hd, device="cuda") + (0.02 * b) * q[i, 0, 0].float() * grow
            c.k8[0][c.at(i, b)] = (x * 16).clamp(-448, 448).to(torch.float8_e4m3fn)
            c.ks[0][c.at(i, b)] = 2.0 ** -4 * (1.0 + 0.25 * (b % 3))  # any positive scale
            c.vs[0][c.at(i, b)] = 2.0 ** (-20 + (b % 5) * 10)
        c.vs[0][c.at(i, 3)] = 0.0
        c.ks[0][c.at(i, 4)] = 0.0
    c.k8[0][c.at(1, 0)][:, 0] = (4 * q[1, 1, 1].float()).clamp(-448, 448).to(torch.float8_e4m3fn)
    for causal in (False, True):
        out = c.attend(0, m, q, None, ctx, causal)
        check_attention(c, 0, m, q, [m, m], ctx, causal, out)
    assert c.status() == 0


def test_attention8_large_queries_and_special_values():
    c = Cache(4, 2, 128, 256, 3, N=1, seed=3)
    m = 2
    q = queries(c, m, seed=4)
    q[0, 0] *= 3e4          # beyond f16's range
    q[0, 1] *= 1e-6
    q[1, 0, 0] = 0
    q[2, 1, 3] = float("nan")
    ctx = [200, 100, 60]
    # whatever lies beyond the rows attended to
    for i in range(3):
        t = ctx[i] + m
        for b in range(c.pps):
            for name in ("k8", "v8"):
                raw = getattr(c, name).view(torch.uint8)[0][c.at(i, b)]
                if (b + 1) * PR > t:
                    raw[:, max(0, t - b * PR):] = 0x7F
            if b * PR >= t:
                c.ks[0][c.at(i, b)] = float("nan")
                c.vs[0][c.at(i, b)] = float("inf")
    out = c.attend(0, m, q, None, ctx, True)
    assert torch.isnan(out[2, 1, 3]).all()
    out[2, 1, 3] = 0
    q[2, 1, 3] = 0
    ref = c.attend(0, m, q, None, ctx, True)
    out[2, 1, 3] = ref[2, 1, 3]
    assert torch.equal(out, ref)
    check_attention(c, 0, m, q, [m] * 3, ctx, True, ref)
    # a NaN among the values of a row that is attended to reaches every query that sees it
    c.v8.view(torch.uint8)[0][c.at(1, 0)][0, 5, 9] = 0x7F
    out = c.attend(0, m, q, None, ctx, False)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, :, :2, 9] = True
    assert torch.equal(torch.isnan(out), bad)
    assert c.status() == 0


def test_attention8_reports_lengths_and_pages_out_of_range():
    c = Cache(4, 2, 64, 256, 2, N=1, B=4)
    q = queries(c, 4)
    check = c.D.DFLASH_ERR_DEVICE_CHECK
    for n, ctx, hint in (([5, 1], [0, 0], 0), ([-1, 1], [0, 0], 0), ([1, 1], [-1, 0], 0), ([1, 1], [0, 256], 0),
                         ([4, 4], [253, 0], 0), ([1, 1], [9, 0], 8)):
        out = c.attend(0, 4, q, n, ctx, False, hint)
        assert c.status() == check, (n, ctx, hint)
        assert torch.isfinite(out.float()).all()
    c.dev_table[1, 2] = c.cfg.num_pages
    out = c.attend(0, 4, q, None, [20, 200], False)
    assert c.status() == check
    out = c.attend(0, 4, q, None, [20, 100], False)
    assert c.status() == 0
    check_attention(c, 0, 4, q, [4, 4], [20, 100], False, out)


def test_attention8_other_stream_and_captured():
    """The calls run on the stream they are given, and replay from a graph with new lengths and rows."""
    c = Cache(8, 2, 128, 512, 3, N=1, seed=5)
    D, m = c.D, 2
    qr, k, v, gq, gk = fused(3, m, 8, 2, 128, seed=8)
    n, ctx = i32([2, 1, 2]), i32([10, 63, 300])
    q = torch.empty(3, m, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, m, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")

    def step():
        D.dflash_qk_norm_rope(c.h, 3, m, qr, qr.stride(0), None, 0, gq, None, ctx, q, None)
        D.dflash_kv_append8(c.h, 3, 0, m, k, k.stride(0), v, v.stride(0), gk, 1, n, ctx, c.k8, c.v8, c.ks, c.vs, c.ws)
        D.dflash_attention8(c.h, 3, 0, m, q, c.k8, c.v8, c.ks, c.vs, n, ctx, 0, 1, out, c.ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    check_attention(c, 0, m, q, [2, 1, 2], [10, 63, 300], True, out, "other stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([40, 0, 449], [509, 127, 64]):
        ctx.copy_(i32(lens))
        qr.copy_(torch.randn_like(qr, dtype=torch.float32))
        out.fill_(7.0)
        graph.replay()
        check_attention(c, 0, m, q, [2, 1, 2], lens, True, out, "replayed")
    assert c.status() == 0


def test_decode_loop_over_the_8_bit_cache():
    """Prompt, then tokens one at a time and a block of candidates of which some are taken back, through
    the public calls, against the oracle fed with the cache's own rows; two layers."""
    nb, N, m = 3, 2, 4
    c = Cache(8, 2, 128, 256, nb, N=N, seed=11)
    lens = np.array([0, 0, 0])
    prompt = np.array([70, 1, 63])
    for step, (R, n) in enumerate([(70, prompt), (1, [1, 1, 1]), (1, [1, 0, 1]), (m, [4, 4, 2]), (1, [1, 1, 1])]):
        n = np.array(n)
        for layer in range(N):
            qr, k, v, gq, gk = fused(nb, R, 8, 2, 128, seed=10 * step + layer)
            before = snap(c)
            c.append8(layer, R, k, v, n, lens, gk, 1)
            check_append8(c, layer, R, k, v, n, list(lens), gk, 1, before)
            if R > 16:
                continue
            q = torch.empty(nb, R, 8, 128, dtype=torch.bfloat16, device="cuda")
            c.D.dflash_qk_norm_rope(c.h, nb, R, qr, qr.stride(0), None, 0, gq, None, i32(lens), q, None)
            out = c.attend(layer, R, q, n, lens, True, hint=int(lens.max()))
            check_attention(c, layer, R, q, n, lens, True, out, f"step {step} layer {layer}")
        lens = lens + (np.minimum(n, 2) if R == m else n)  # two of the candidates are accepted
    assert c.status() == 0


def test_attention8_wait_limit_is_reported():
    """With the producer held back every wait runs out after max_spin polls: the status says so, the
    kernels return, and the context stays usable."""
    D = lib()
    c = Cache(8, 2, 128, 512, 3, N=1, max_spin=2000, flags=1 << 30)
    q = queries(c, 4)
    c.attend(0, 4, q, None, [100, 0, 400], False)
    assert c.status() == D.DFLASH_ERR_TIMEOUT
    assert c.status() == D.DFLASH_OK


# ------------------------------------------------------------------ splits of the work

@pytest.mark.parametrize("Hkv,hd,nb,R,paged", [(3, 128, 3, 1, True), (33, 64, 2, 2, False), (3, 128, 2, 3, True),
                                               (5, 64, 2, 16, True), (3, 128, 2, 17, False), (33, 64, 1, 70, True),
                                               (7, 128, 5, 700, True), (4, 64, 6, 1100, False)])
def test_append8_row_slots_and_head_groups(Hkv, hd, nb, R, paged):
    """Every number of row slots, single heads and several in a CTA, also a number that groups do not divide;
    rows behind a sequence's own hold NaN."""
    c = Cache(Hkv, Hkv, hd, -(-(R + 140) // PR) * PR, nb, N=1, paged=paged, seed=R)
    _, k, v, _, gk = fused(nb, R, 1, Hkv, hd, seed=R, big=(0, 200.0))
    k, v = k.clone(), v.clone()
    ctx = [(61, 0, 130, 64, 63, 1)[i] for i in range(nb)]
    n = [max(R - 5 * i, 0) for i in range(nb)]
    for i in range(nb):
        k[i * R + n[i]:(i + 1) * R] = float("nan")
        v[i * R + n[i]:(i + 1) * R] = float("nan")
    before = snap(c)
    c.append8(0, R, k, v, n, ctx, gk, 1)
    assert c.status() == 0
    check_append8(c, 0, R, torch.nan_to_num(k), torch.nan_to_num(v), n, ctx, gk, 1, before)


@pytest.mark.parametrize("Hq,hd,m,L", [(1, 128, 1, 20000), (16, 64, 1, 30001), (4, 128, 7, 20011), (8, 64, 16, 19990)])
def test_attention8_one_pair_over_all_sms(Hq, hd, m, L):
    """One sequence and one kv head: more parts to join than a warp has lanes."""
    c = Cache(Hq, 1, hd, -(-(L + m) // PR) * PR, 1, N=1, B=max(m, 2), seed=m)
    q = queries(c, m, seed=L)
    out = c.attend(0, m, q, None, [L], True, hint=L)
    assert c.status() == 0
    check_attention(c, 0, m, q, [m], [L], True, out)


@pytest.mark.parametrize("hd,Hq,m", [(64, 2, 2), (128, 4, 8)])
def test_attention8_many_short_sequences(hd, Hq, m):
    """300 sequences of zero to four blocks, every third without rows, some all the way at the front."""
    nb = 300
    c = Cache(Hq, 1, hd, 256, nb, N=1, seed=m)
    q = queries(c, m, seed=3)
    rng = np.random.default_rng(m)
    ctx = [0 if i % 7 == 0 else int(x) for i, x in enumerate(rng.integers(0, 256 - m, nb))]
    n = [0 if i % 3 == 1 or i < 2 else int(x) for i, x in enumerate(rng.integers(1, m + 1, nb))]
    out = c.attend(0, m, q, n, ctx, True)
    assert c.status() == 0
    check_attention(c, 0, m, q, n, ctx, True, out)


def test_calls_on_two_streams_and_two_graphs_of_one_workspace():
    """Handles with workspaces of their own work side by side, and graphs captured with the same handle and
    workspace replay in turn, each with its own lengths: all bitwise as one after the other."""
    D, m = lib(), 4
    sides = []
    for s in range(2):
        c = Cache(8, 2, 128, 4096, 3, N=1, seed=20 + s)
        qr, k, v, gq, gk = fused(3, m, 8, 2, 128, seed=30 + s)
        sides.append((c, qr, k, v, gq, gk, torch.empty(3, m, 8, 128, dtype=torch.bfloat16, device="cuda")))

    def step(side, ctx, out):
        c, qr, k, v, gq, gk, q = side
        D.dflash_qk_norm_rope(c.h, 3, m, qr, qr.stride(0), None, 0, gq, None, ctx, q, None)
        c.D.dflash_kv_append8(c.h, 3, 0, m, k, k.stride(0), v, v.stride(0), gk, 1, None, ctx, c.k8, c.v8, c.ks, c.vs,
                              c.ws)
        D.dflash_attention8(c.h, 3, 0, m, q, c.k8, c.v8, c.ks, c.vs, None, ctx, 0, 1, out, c.ws)

    lens = [i32([4000, 1, 700]), i32([64, 3000, 2222])]
    new = lambda: torch.full((3, m, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    want = [[new() for _ in lens] for _ in sides]
    for s, side in enumerate(sides):
        for _ in range(2):  # each length's rows lie in what the other reads: from the second round on they are there
            for a, ctx in enumerate(lens):
                step(side, ctx, want[s][a])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    got = [[new() for _ in lens] for _ in sides]
    torch.cuda.synchronize()
    for a, ctx in enumerate(lens):
        for s, side in enumerate(sides):
            with torch.cuda.stream(streams[s]):
                step(side, ctx, got[s][a])
    torch.cuda.synchronize()
    for s in range(2):
        for a in range(2):
            assert torch.equal(got[s][a], want[s][a]), (s, a)
    graphs, outs = [], [new() for _ in lens]
    for ctx, out in zip(lens, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(sides[0], ctx, out)
    for a in (0, 1, 0, 1):
        outs[a].fill_(7.0)
        graphs[a].replay()
        assert torch.equal(outs[a], want[0][a])
    assert all(side[0].status() == 0 for side in sides)


@pytest.mark.parametrize("paged", [False, True])
def test_drafter_with_both_caches(paged):
    """Drafter(cache8=True): a prompt and a block appended to the bf16 and the 8-bit caches of one layer,
    then the same rotated queries over either, each against the oracle on the rows that its cache
    holds. The bf16 attention rounds its probabilities to bf16: 2^-8 of each."""
    from block_diffusion_speculative_project_gb300 import drafter
    w = di.TINY
    nb, Cmax, m, layer = 2, 192, w.B, 1
    dev = {k: drafter.to_device_bf16(v) for k, v in di.make_weights(w, 0).items()}
    pps = Cmax // PR
    dr = drafter.Drafter(w, dev, nb, Cmax, w.B, num_pages=nb * pps + 1 if paged else 0, cache8=True)
    if paged:
        table = np.random.default_rng(1).permutation(nb * pps + 1)[:nb * pps].reshape(nb, pps)
        dr.set_block_table(i32(table))
    lens, none = [100, 5], i32([0, 0])
    ctx = i32(lens)
    for R, n, at, seed in ((100, i32(lens), none, 1), (m, None, ctx, 2)):
        q, k, v, gq, gk = fused(nb, R, w.Hq, w.Hkv, w.hd, seed=seed)
        dr.kv_append(nb, layer, R, k, v, at, n_rows=n, g_k=gk)
        dr.kv_append8(nb, layer, R, k, v, at, n_rows=n, g_k=gk)
    rot = torch.empty(nb, m, w.Hq, w.hd, dtype=torch.bfloat16, device="cuda")
    o16, o8 = torch.empty_like(rot), torch.empty_like(rot)
    dr.qk_norm_rope(nb, m, q, None, ctx, rot, None, g_q=gq)
    dr.attention(nb, layer, rot, ctx, o16)
    dr.attention8(nb, layer, m, rot, ctx, o8)
    assert dr.status() == 0

    def rows(t, i, scale=None):
        if paged:
            x = f64(t[layer][table[i].tolist()]).transpose(1, 0, 2, 3)           # [Hkv, pps, 64, hd]
            s = None if scale is None else f64(scale[layer][table[i].tolist()]).T
        else:
            x = f64(t[layer][i]).reshape(w.Hkv, pps, PR, w.hd)
            s = None if scale is None else f64(scale[layer][i])
        return (x if s is None else x * s[:, :, None, None]).reshape(w.Hkv, Cmax, w.hd)[:, :lens[i] + m]

    for i in range(nb):
        for out, K, V, step in ((o16, rows(dr.kcache, i), rows(dr.vcache, i), 2.0 ** -8),
                                (o8, rows(dr.kcache8, i, dr.kscale), rows(dr.vcache8, i, dr.vscale),
                                 2.0 ** -11 + 2.0 ** -10)):
            o, mag, dot = orc.attention8(f64(rot[i]), K, V, lens[i], False)
            tol = (2.0 ** -8 * np.abs(o) + mag * (step + 2.0 ** -16 + 2 * w.hd * 2.0 ** -24 * dot[..., None])
                   + K.shape[1] * 2.0 ** -24 * np.abs(V).max())
            assert_within(f64(out[i]), o, tol, f"sequence {i}")


@pytest.mark.parametrize("n,ctx", [(130, 2 ** 31 - 1), (130, 2 ** 31 - 64), (2 ** 31 - 1, 0), (-2 ** 31, 0),
                                   (130, -2 ** 31), (130, 2 ** 31 - 200)])
def test_lengths_at_the_ends_of_their_type(n, ctx):
    """Counts and lengths that no cache has: reported, and nothing beyond the rows that exist is touched."""
    c = Cache(2, 2, 64, 256, 2, N=1)
    _, k, v, _, _ = fused(2, 130, 1, 2, 64, seed=2)
    q = queries(c, 4)
    writes = 0 <= ctx < 256 and n > 0
    for call, names in ((c.append8, ("k8", "v8", "ks", "vs")), (c.append, ("kc", "vc"))):
        before = {x: getattr(c, x).clone() for x in names}
        call(0, 130, k, v, [0, n], [0, ctx])
        assert c.status() == c.D.DFLASH_ERR_DEVICE_CHECK
        for x in names:
            same = torch.equal(getattr(c, x).view(torch.uint8), before[x].view(torch.uint8))
            assert same != writes, x
    out = c.attend(0, 4, q, [0, n], [0, ctx], True)
    assert c.status() == c.D.DFLASH_ERR_DEVICE_CHECK
    assert torch.isfinite(out.float()).all() and (out[0] == 7.0).all()


@pytest.mark.parametrize("Hq,Hkv,hd,m", [(8, 2, 128, 4), (4, 2, 64, 7), (8, 2, 128, 8), (8, 2, 64, 16), (8, 1, 128, 16)])
@pytest.mark.parametrize("paged", [False, True])
def test_attention8_causal_rows_do_not_see_a_later_nan(Hq, Hkv, hd, m, paged):
    """NaN among the values of the call's own rows: in its column for the rows that attend to it, nowhere else;
    new rows that end a block, begin one and lie on both sides of a border."""
    ctx = [62, 640 - m, 64, 0, 505, 127]
    nb = len(ctx)
    c = Cache(Hq, Hkv, hd, 640, nb, N=1, paged=paged, seed=hd + m)
    q = queries(c, m, seed=4)
    n = [m, m, max(m - 1, 1), m, m, 1]
    rng = np.random.default_rng(m)
    nan = np.zeros((nb, Hkv, m, hd), bool)
    for i in range(nb):
        for h in range(Hkv):
            for t in rng.permutation(n[i])[:2] if (i + h) % 3 else []:  # some heads keep all their values
                nan[i, h, t, rng.permutation(hd)[:5]] = True
    bytes8 = c.v8.view(torch.uint8)

    def put(values):
        for i, h, t, d in zip(*np.nonzero(nan)):
            b, row = divmod(ctx[i] + int(t), PR)
            bytes8[0][c.at(i, b)][h, row, int(d)] = values
    put(0)
    want = []
    for i in range(nb):
        K, V = (c.rows(x, 0, i, ctx[i] + n[i], s) for x, s in ((c.k8, c.ks), (c.v8, c.vs)))
        want.append(orc.attention8(f64(q[i, :n[i]]), K, V, ctx[i], True) + (np.abs(V).max(), K.shape[1]))
    for byte in (0x7F, 0xFF):
        put(byte)
        out = c.attend(0, m, q, n, ctx, True)
        assert c.status() == 0
        for i in range(nb):
            o, mag, dot, vmax, L = want[i]
            sees = np.repeat(np.cumsum(nan[i, :, :n[i]], axis=1).transpose(1, 0, 2) > 0, Hq // Hkv, axis=1)
            got = f64(out[i, :n[i]])
            assert np.array_equal(np.isnan(got), sees), f"sequence {i}"
            tol = (2.0 ** -8 * np.abs(o) + mag * (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -16 + 2 * hd * 2.0 ** -24 * dot[..., None])
                   + L * 2.0 ** -24 * vmax)
            assert_within(np.where(sees, o, got), o, tol, f"sequence {i}")
            assert (out[i, n[i]:] == 7.0).all()
    every = c.attend(0, m, q, n, ctx, False)  # without the mask every row attends to them
    for i in range(nb):
        sees = np.repeat(nan[i, :, :n[i]].any(axis=1), Hq // Hkv, axis=0)
        assert np.array_equal(np.isnan(f64(every[i, :n[i]])), np.broadcast_to(sees, (n[i], Hq, hd))), f"sequence {i}"


@pytest.mark.parametrize("Hq,Hkv,hd,m", [(8, 2, 128, 4), (8, 2, 64, 16), (8, 1, 128, 16)])
def test_attention8_causal_rows_do_not_see_a_later_nan_key(Hq, Hkv, hd, m):
    """A key of NaN: the rows that attend to it are NaN, those before it as without it."""
    ctx, nb, t = [62, 320 - m, 64], 3, 2
    c = Cache(Hq, Hkv, hd, 320, nb, N=1, seed=m)
    q = queries(c, m, seed=4)
    bytes8 = c.k8.view(torch.uint8)
    for i in range(nb):
        b, row = divmod(ctx[i] + t, PR)
        bytes8[0][c.at(i, b)][:, row, 3] = 0x7F
    out = c.attend(0, m, q, None, ctx, True)
    assert c.status() == 0
    assert torch.isnan(out[:, t:]).all()
    for i in range(nb):
        K, V = (c.rows(x, 0, i, ctx[i] + t, s) for x, s in ((c.k8, c.ks), (c.v8, c.vs)))
        o, mag, dot = orc.attention8(f64(q[i, :t]), K, V, ctx[i], True)
        tol = (2.0 ** -8 * np.abs(o) + mag * (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -16 + 2 * hd * 2.0 ** -24 * dot[..., None])
               + (K.shape[1] + m) * 2.0 ** -24 * np.abs(V).max())
        assert_within(f64(out[i, :t]), o, tol, f"sequence {i}")
