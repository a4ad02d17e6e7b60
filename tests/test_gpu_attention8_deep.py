"""The 8-bit attention in the state that long contexts put it in, in both of its forms (up to 16 query
rows of a kv head, and more: up to 64 and up to 128): tens of pairs of units in one CTA, references that
move inside a segment, attention sinks, scales far apart, queries with a channel that stands out.

The reference is the formula in 64 bits on the device. Tolerances, besides those that
test_gpu_rows8.py derives (one bf16 rounding 2^-8 |o|; of each probability 2^-11, 2^-10 and 2^-16;
scores hd * 2^-24 * sum|q k| / sqrt(hd), which move a probability by twice that at most):
  small probabilities  P is at least 2^8 (2^7 in the form for many rows) for the key that set the
             reference. f16's smallest step is 2^-24, half of it 2^-25; in the form for few rows the
             last e5m2 term has the smallest step 2^-16 after a factor 2^7: half of it 2^-24. Together
             below 2^-31 of the largest p * V scale for every key: rows * 2^-31 * max p * max|e4m3 V| *
             max scale
  queries    bf16 exactly for what is at least 2^-13 of a row's largest value
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_rows8 import PR, Cache, lib, queries

pytestmark = pytest.mark.gpu


def held(c, name, scale, i, rows):
    """[Hkv, rows, hd] of sequence i's cache in layer 0 in 64 bits, without and with the block scales."""
    nblk = -(-rows // PR)
    if c.table is not None:
        idx = torch.as_tensor(c.table[i, :nblk], device="cuda").long()
        x, s = getattr(c, name)[0][idx].transpose(0, 1), getattr(c, scale)[0][idx].t()
    else:
        x, s = getattr(c, name)[0][i, :, :nblk], getattr(c, scale)[0][i, :, :nblk]
    raw = x.to(torch.float32).double()
    full = (raw * s.double()[..., None, None]).reshape(c.Hkv, nblk * PR, c.hd)[:, :rows]
    return raw.reshape(c.Hkv, nblk * PR, c.hd)[:, :rows], full, s.double()


def check(c, q, n, ctx, causal, out, what=""):
    """Every row of out against 64 bits; rows at n and behind hold 7."""
    worst = 0.0
    m, G = q.shape[1], c.Hq // c.Hkv
    for i in range(len(ctx)):
        assert (out[i, n[i]:] == 7.0).all(), f"{what}: rows behind sequence {i}"
        if n[i] == 0:
            continue
        L = ctx[i] + n[i]
        _, K, _ = held(c, "k8", "ks", i, L)
        V8, V, vs = held(c, "v8", "vs", i, L)
        pos = torch.arange(L, device="cuda")
        end = (torch.arange(n[i], device="cuda") + ctx[i] + 1 if causal
               else torch.full((n[i],), L, device="cuda")).repeat_interleave(G)
        for h in range(c.Hkv):
            qh = q[i, :n[i], h * G:(h + 1) * G].double().reshape(-1, c.hd)
            x = qh @ K[h].t() / math.sqrt(c.hd)
            x.masked_fill_(pos[None] >= end[:, None], -math.inf)
            p = torch.softmax(x, dim=-1)
            del x
            o, mag = p @ V[h], p @ V[h].abs()
            dot = (qh.abs() @ K[h].abs().t()).amax(dim=-1, keepdim=True) / math.sqrt(c.hd)
            floor = L * 2.0 ** -31 * p.amax(dim=-1, keepdim=True) * V8[h].abs().max() * vs[h].max()
            tol = 2.0 ** -8 * o.abs() + mag * (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -16 + 2 * c.hd * 2.0 ** -24 * dot) + floor
            got = out[i, :n[i], h * G:(h + 1) * G].double().reshape(-1, c.hd)
            assert torch.isfinite(got).all(), f"{what}: sequence {i} head {h} not finite"
            r = ((got - o).abs() / tol.clamp(min=1e-300)).max().item()
            worst = max(worst, r)
            assert r <= 1, f"{what}: sequence {i} kv head {h}: {r:.2f} of the tolerance"
    return worst


def block(c, name, i, b):
    return getattr(c, name)[0][c.at(i, b)]


def put8(t, value):
    t.copy_(torch.full(t.shape, value, device="cuda").to(torch.float8_e4m3fn))


def poison():
    """An attention over nothing but NaN, whose bytes stay in the SMs' shared memory."""
    for Hq, m in ((1, 1), (8, 8)):
        c = Cache(Hq, 1, 128, 64 * 400, 1, N=1, B=max(m, 2))
        for name in ("k8", "v8"):
            getattr(c, name).view(torch.uint8).fill_(0x7F)
        c.attend(0, m, queries(c, m), None, [64 * 400 - m], False)


# (hd, Hq, Hkv, rows m): 1, 16 and 14 rows of a kv head in the form for few, 32 and 63 in the form for up to 64,
# 96 and 128 in the one for more
FORMS = [(128, 2, 2, 1), (64, 4, 1, 4), (128, 4, 2, 7), (128, 16, 2, 4), (64, 7, 1, 9), (128, 8, 1, 12), (64, 8, 1, 16)]


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
@pytest.mark.parametrize("paged,causal", [(True, False), (False, True)])
def test_a_hundred_units_in_one_cta(hd, Hq, Hkv, m, paged, causal):
    """Two sequences of together 152 * 100 units and more: every CTA has some fifty pairs, the rings wrap several
    times and the scales come in four chunks. Scores are flat but for one key in every 37 units, which
    lies 2^14 to 2^15.5 above for half of the query heads: the reference moves inside every CTA's segment,
    and what was added before it still weighs about a tenth of what the key does."""
    units = 152 * 104 // Hkv
    L = [PR * (units * 2 // 3) - 5 - m, PR * (units // 3) + 9]
    c = Cache(Hq, Hkv, hd, PR * (units * 2 // 3) + PR, 2, N=1, B=max(m, 2), paged=paged, seed=m)
    g = torch.Generator(device="cuda").manual_seed(m)
    c.k8.copy_((8 * torch.randn(c.k8.shape, generator=g, device="cuda")).to(torch.float8_e4m3fn))
    c.v8.copy_((100 + 20 * torch.randn(c.v8.shape, generator=g, device="cuda")).to(torch.float8_e4m3fn))
    c.k8.view(torch.uint8)[..., 0] = 0
    q = queries(c, m, seed=1, std=0.25)
    q[..., 0] = 0
    q[:, :, ::2, 0] = 8.0
    c.ks.fill_(2.0 ** -4)
    step = math.log(2) * math.sqrt(hd) / 8.0            # of channel 0, for one power of two
    for i in range(2):
        for x, b in enumerate(range(30, (L[i] + m) // PR, 37)):
            k = block(c, "k8", i, b)
            put8(k[:, (x * 11) % PR, 0], (14 + x % 4 * 0.5) * step * 16)
            put8(block(c, "v8", i, b)[:, (x * 11) % PR], -60.0)
    n = [m, max(m - 1, 1)]
    out = c.attend(0, m, q, n, L, causal)
    assert c.status() == 0
    check(c, q, n, L, causal, out)
    poison()
    again = c.attend(0, m, q, n, L, causal)
    assert torch.equal(out, again)


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
def test_many_segments_of_many_units(hd, Hq, Hkv, m):
    """40 ragged sequences, so that a CTA's chunks of 32 scales begin anywhere in a segment; some odd, some
    empty, one of a single row."""
    nb = 40
    c = Cache(Hq, Hkv, hd, PR * 1200 // Hkv, nb, N=1, B=max(m, 2), seed=m)
    rng = np.random.default_rng(m)
    ctx = [int(x) for x in rng.integers(PR * 150 // Hkv, PR * 1100 // Hkv, nb)]
    n = [int(x) for x in rng.integers(0, m + 1, nb)]
    ctx[7], n[7] = 0, 1
    q = queries(c, m, seed=5)
    out = c.attend(0, m, q, n, ctx, True)
    assert c.status() == 0
    check(c, q, n, ctx, True, out)


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
@pytest.mark.parametrize("below", [20.3, 23.54])
def test_a_sink_whose_value_is_zero(hd, Hq, Hkv, m, below):
    """The first key takes 2^below times the weight of each other, and its value is zero: the output is
    what the others add up to."""
    nb = 160 // Hkv
    c = Cache(Hq, Hkv, hd, PR * 96, nb, N=1, B=max(m, 2), seed=3)
    g = torch.Generator(device="cuda").manual_seed(3)
    c.k8.view(torch.uint8).zero_()
    c.v8.copy_((67 + 3 * torch.rand(c.v8.shape, generator=g, device="cuda")).to(torch.float8_e4m3fn))
    c.ks.fill_(1.0)
    c.vs.fill_(2.0 ** -6)
    q = torch.zeros(nb, m, Hq, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 5] = 1.0
    # score of the sink in powers of two: k / sqrt(hd) / ln 2 * scale
    for i in range(nb):
        put8(block(c, "k8", i, 0)[:, 0, 5], 1.0)
        put8(block(c, "v8", i, 0)[:, 0], 0.0)
        block(c, "ks", i, 0)[:] = below * math.log(2) * math.sqrt(hd)
    ctx = [PR * 95 - 3 * i for i in range(nb)]
    out = c.attend(0, m, q, None, ctx, False)
    assert c.status() == 0
    check(c, q, [m] * nb, ctx, False, out)


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
def test_queries_with_a_channel_that_stands_out(hd, Hq, Hkv, m):
    """One channel of every query row is 2^10 to 2^13 times the others that count, and the keys are zero in
    it: the scores are those of the small ones, which bf16 holds to 8 bits. Rows of one kv head differ
    by up to 2^3."""
    nb = 12
    c = Cache(Hq, Hkv, hd, 128, nb, N=1, B=max(m, 2), seed=4)
    g = torch.Generator(device="cuda").manual_seed(4)
    u = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    sign = lambda *s: torch.where(u(*s) < 0.5, -1.0, 1.0)  # noqa: E731
    q = torch.zeros(nb, m, Hq, hd, device="cuda")
    top = torch.exp2(torch.floor(u(nb, m, Hq) * 4))
    q[..., 0] = top * 1.5
    q[..., 1:4] = sign(nb, m, Hq, 3) * (1 + u(nb, m, Hq, 3)) * top[..., None] * torch.exp2(-10 - torch.floor(u(nb, m, Hq, 3) * 3))
    q = q.to(torch.bfloat16)
    c.k8.view(torch.uint8).zero_()
    c.k8[..., 1:4] = (sign(*c.k8.shape[:-1], 3) * (200 + 248 * u(*c.k8.shape[:-1], 3))).to(torch.float8_e4m3fn)
    c.ks.fill_(16.0)
    ctx = [1 + i % 5 for i in range(nb)]
    out = c.attend(0, m, q, None, ctx, True)
    assert c.status() == 0
    check(c, q, [m] * nb, ctx, True, out)


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
@pytest.mark.parametrize("few", [True, False])
def test_value_scales_far_apart(hd, Hq, Hkv, m, few):
    """Blocks of equal scores whose values' scales are 2^-100 (what an append of zeros gives), 2^60 and in
    between weigh the same in the sum of the softmax; a scale of zero takes nothing from the others'
    small values. In one CTA, or one unit a CTA joined by the merge."""
    nb = 1 if few else 152 // Hkv + 8
    for scales in ([2.0 ** -100, 2.0 ** 60, 1.0, 2.0 ** -100, 2.0 ** -40], [2.0 ** -100], [2.0 ** -30, 0.0, 2.0 ** -31],
                   [0.0], [2.0 ** 80, 2.0 ** -100, 2.0 ** -19]):
        c = Cache(Hq, Hkv, hd, PR * 24, nb, N=1, B=max(m, 2), seed=6)
        g = torch.Generator(device="cuda").manual_seed(6)
        c.k8.copy_(torch.randn(c.k8.shape, generator=g, device="cuda").to(torch.float8_e4m3fn))
        c.ks.fill_(0.25)
        for i in range(nb):
            for b in range(c.pps):
                c.vs[0][c.at(i, b)] = scales[(b + i) % len(scales)]
        q = queries(c, m, seed=7)
        ctx = [PR * 23 - 7 * i % 500 for i in range(nb)]
        out = c.attend(0, m, q, None, ctx, False)
        assert c.status() == 0
        check(c, q, [m] * nb, ctx, False, out, str(scales))


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
def test_a_nan_byte_in_a_block_of_scale_zero(hd, Hq, Hkv, m):
    """An element is its e4m3 value times the scale: NaN times zero is NaN, for any number of query rows."""
    c = Cache(Hq, Hkv, hd, 256, 2, N=1, B=max(m, 2), seed=8)
    q = queries(c, m, seed=8)
    for i in range(2):
        c.vs[0][c.at(i, 1)] = 0.0
    ctx = [200, 100]
    clean = c.attend(0, m, q, None, ctx, False)
    check(c, q, [m, m], ctx, False, clean)
    block(c, "v8", 1, 1).view(torch.uint8)[:, 5, 9] = 0x7F
    out = c.attend(0, m, q, None, ctx, False)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[1, :, :, 9] = True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want])
    assert c.status() == 0


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
def test_growing_scores_and_scales_of_keys_and_values(hd, Hq, Hkv, m):
    """Scores that grow by far more than any reference allows within a CTA's units, for some rows only; scales
    2^40 apart; blocks of key scale and of value scale zero."""
    nb = 152 // Hkv + 5
    c = Cache(Hq, Hkv, hd, PR * 17, nb, N=1, B=max(m, 2), seed=9)
    q = queries(c, m, seed=9)
    g = torch.Generator(device="cuda").manual_seed(9)
    for i in range(nb):
        for b in range(c.pps):
            x = torch.randn(Hkv, PR, hd, generator=g, device="cuda") + 0.12 * b * q[i, 0, 0].float()
            block(c, "k8", i, b).copy_((x * 16).clamp(-448, 448).to(torch.float8_e4m3fn))
            c.ks[0][c.at(i, b)] = 2.0 ** -4 * (1.0 + 0.25 * (b % 3))
            c.vs[0][c.at(i, b)] = 2.0 ** (-20 + (b % 5) * 10)
        c.vs[0][c.at(i, 3)] = 0.0
        c.ks[0][c.at(i, 4)] = 0.0
    ctx = [PR * 17 - m - i % 70 for i in range(nb)]
    for causal in (False, True):
        out = c.attend(0, m, q, None, ctx, causal)
        check(c, q, [m] * nb, ctx, causal, out)
    assert c.status() == 0


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS[1:])
def test_large_small_zero_and_nan_query_rows(hd, Hq, Hkv, m):
    c = Cache(Hq, Hkv, hd, 256, 3, N=1, B=max(m, 2), seed=3)
    q = queries(c, m, seed=4)
    q[0, 0] *= 3e4
    q[0, 1] *= 1e-6
    q[0, 2] *= 1e-30
    q[1, 0, 0] = 0
    ctx = [200, 100, 60]
    ref = c.attend(0, m, q, None, ctx, True)
    check(c, q, [m] * 3, ctx, True, ref)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[2, 1, Hq - 1, 7] = bad
        out = c.attend(0, m, q2, None, ctx, True)
        assert torch.isnan(out[2, 1, Hq - 1]).all()
        out[2, 1, Hq - 1] = ref[2, 1, Hq - 1]
        check(c, q, [m] * 3, ctx, True, out)  # (an infinite row changes the scaling of those beside it)
        assert bad == math.inf or torch.equal(out, ref)
    assert c.status() == 0


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
@pytest.mark.parametrize("L", [40, 20000])
def test_the_output_may_be_the_queries(hd, Hq, Hkv, m, L):
    """Written whole by one CTA, or joined from many: a pair's queries are read before its rows are written."""
    c = Cache(Hq, Hkv, hd, -(-(L + m) // PR) * PR, 3, N=1, B=max(m, 2), seed=2)
    q = queries(c, m, seed=2)
    n, ctx = [m, max(m - 1, 0), m], [L, L // 2, L // 3]
    want = c.attend(0, m, q, n, ctx, True)
    got = q.clone()
    c.attend(0, m, got, n, ctx, True, out=got)
    want[1, n[1]:] = q[1, n[1]:]
    assert torch.equal(got, want)
    both = torch.zeros(2 * q.numel(), dtype=torch.bfloat16, device="cuda")
    for shift in (8, q.numel() - 8):
        with pytest.raises(c.D.DflashError) as e:  # some rows would be written over before they are read
            c.attend(0, m, both[:q.numel()].view_as(q), n, ctx, True, out=both[shift:shift + q.numel()].view_as(q))
        assert e.value.code == c.D.DFLASH_ERR_INVALID_ARG
    assert c.status() == 0


@pytest.mark.parametrize("hd,Hq,Hkv,m", FORMS)
def test_wait_limit_in_every_form(hd, Hq, Hkv, m):
    """No loads are issued, so every wait runs out after 2000 polls: reported, and a handle without the
    flag works right afterwards."""
    D = lib()
    c = Cache(Hq, Hkv, hd, 512, 3, N=1, B=max(m, 2), max_spin=2000, flags=1 << 30)
    q = queries(c, m)
    ctx = [100, 0, 400]
    c.attend(0, m, q, None, ctx, False)
    assert c.status() == D.DFLASH_ERR_TIMEOUT
    assert c.status() == D.DFLASH_OK
    c = Cache(Hq, Hkv, hd, 512, 3, N=1, B=max(m, 2))
    out = c.attend(0, m, q, None, ctx, False)
    assert c.status() == 0
    check(c, q, [m] * 3, ctx, False, out)
