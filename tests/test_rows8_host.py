"""Host side of the row and 8-bit cache calls, without a GPU: the oracle's definitions against
brute force, and the refusals that need no device."""
import numpy as np
import pytest

from oracle import dflash_oracle as orc


def test_e4m3_round_is_the_nearest_code():
    vals = orc.e4m3_values()
    fin = np.unique(vals[np.isfinite(vals)])
    assert fin.max() == 448 and len(fin) == 253  # +-0 are one value
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(2000) * np.exp2(rng.integers(-12, 10, 2000)), fin,
                        (fin[1:] + fin[:-1]) / 2, [1e9, -1e9, np.inf, -np.inf]])
    got = orc.e4m3_round(x)
    d = np.abs(np.clip(x, -448, 448)[:, None] - fin)
    assert np.array_equal(np.abs(np.clip(x, -448, 448) - got), d.min(axis=1))
    # a value halfway between two codes goes to the one with the even mantissa
    code = {v: c for c, v in enumerate(vals) if np.isfinite(v) and c < 128}
    mid = np.array([(a + b) / 2 for a, b in zip(fin[126:-1], fin[127:])])
    assert all(code[abs(v)] % 2 == 0 for v in orc.e4m3_round(mid[mid > 0]))
    assert np.isnan(orc.e4m3_round(np.array([np.nan])))[0]


def test_torch_e4m3_codes_are_the_oracles():
    torch = pytest.importorskip("torch")
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, orc.e4m3_values(), equal_nan=True)


def test_block_scale_is_the_smallest_power_of_two_that_fits():
    rng = np.random.default_rng(1)
    amax = np.concatenate([np.exp2(rng.uniform(-20, 20, 500)), 448 * np.exp2(np.arange(-10.0, 10)),
                           np.nextafter(448 * np.exp2(np.arange(-10.0, 10)), np.inf)])
    for a in amax:
        s = orc.block_scale(a)
        assert a / s <= 448 < a / (s / 2)
    assert orc.block_scale(0.0) == 2.0 ** -100 and orc.block_scale(1e-38) == 2.0 ** -100


def test_append8_block_keeps_and_rescales():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((10, 8))
    old, s0 = orc.append8_block(np.zeros((64, 8)), 123.0, 0, x)
    assert s0 == orc.block_scale(np.abs(x).max())  # a block without earlier rows begins afresh
    same, s1 = orc.append8_block(old, s0, 10, np.full((3, 8), 1e-3))
    assert s1 == s0 and np.array_equal(same[:10], old[:10])
    grown, s2 = orc.append8_block(old, s0, 10, np.full((3, 8), 100.0))
    assert s2 > s0 and np.abs(grown[:10] * s2 - old[:10] * s0).max() <= s2 * 2.0 ** -10


def test_attention8_of_equal_keys_is_the_mean_of_the_values():
    rng = np.random.default_rng(3)
    q, V = rng.standard_normal((2, 4, 8)), rng.standard_normal((2, 7, 8))
    K = np.ones((2, 7, 8))
    o, _, _ = orc.attention8(q, K, V, 5, causal=True)
    assert np.allclose(o[0, 1], V[0, :6].mean(axis=0)) and np.allclose(o[1, 3], V[1].mean(axis=0))


def test_null_handles_are_refused():
    from block_diffusion_speculative_project_gb300 import dflash as d
    i, N = 0, None
    calls = [lambda: d.LIB.dflash_qk_norm_rope(N, 1, 1, N, 64, N, 64, N, N, N, N, N, N),
             lambda: d.LIB.dflash_kv_append(N, 1, 0, 1, N, 64, N, 64, N, 1, N, N, N, N, N, i, N),
             lambda: d.LIB.dflash_kv_append8(N, 1, 0, 1, N, 64, N, 64, N, 1, N, N, N, N, N, N, N, i, N),
             lambda: d.LIB.dflash_attention8(N, 1, 0, 1, N, N, N, N, N, N, N, 0, 0, N, N, i, N)]
    for f in calls:
        assert f() == d.DFLASH_ERR_INVALID_ARG


def stub_drafter(monkeypatch, calls):
    """A Drafter without a handle on the CPU whose calls are noted instead of made."""
    from types import SimpleNamespace

    import torch

    from block_diffusion_speculative_project_gb300 import drafter
    dr = object.__new__(drafter.Drafter)
    dr.h, dr.ws, dr.shape = None, torch.zeros(1), SimpleNamespace(Hq=4, Hkv=2, hd=64)
    dr.kcache = dr.vcache = dr.kcache8 = dr.vcache8 = dr.kscale = dr.vscale = None
    for name in ("qk_norm_rope", "kv_append", "kv_append8", "attention8"):
        monkeypatch.setattr(drafter._d, "dflash_" + name, lambda *a, name=name: calls.append((name, a)))
    return dr


def test_drafter_refuses_rows_that_its_calls_would_read_past(monkeypatch):
    """A row stride is taken from a tensor only if its rows are [nb * R, heads * hd]: the stride of a
    [nb, R, heads * hd] tensor is R rows, and R times its length would be read."""
    import torch
    calls = []
    dr = stub_drafter(monkeypatch, calls)
    nb, R, bf16 = 2, 3, torch.bfloat16
    i32 = torch.zeros(nb, dtype=torch.int32)
    wide = torch.zeros(nb * R, 8 * 64, dtype=bf16)
    q, k, v = wide.split([256, 128, 128], dim=1)
    oq, ok = torch.zeros(nb, R, 4, 64, dtype=bf16), torch.zeros(nb, R, 2, 64, dtype=bf16)
    g = torch.ones(64, dtype=bf16)

    def norm(q=q, k=k, pos=i32, oq=oq, ok=ok, g=g):
        dr.qk_norm_rope(nb, R, q, k, pos, oq, ok, g_q=g, g_k=g)

    def both(k=k, v=v, ctx=i32, n=i32, g=g):
        dr.kv_append(nb, 0, R, k, v, ctx, n_rows=n, g_k=g)

    def app8(k=k, v=v, ctx=i32, n=i32, g=g):
        dr.kv_append8(nb, 0, R, k, v, ctx, n_rows=n, g_k=g)

    def att(q=oq, ctx=i32, o=oq, n=i32):
        dr.attention8(nb, 0, R, q, ctx, o, n_rows=n)

    for f in (norm, both, app8, att):
        f()
    assert [c[0] for c in calls] == ["qk_norm_rope", "kv_append", "kv_append8", "attention8"]
    assert calls[0][1][4] == calls[0][1][6] == calls[1][1][5] == calls[2][1][7] == 8 * 64  # the row strides
    norm(k=None, ok=None)
    one = torch.zeros(1, 1, 128, dtype=bf16).expand(1, 1, 128)[:, 0]
    dr.kv_append(1, 0, 1, one, one, i32)  # a single row has any stride
    assert calls[-1][1][5] == 128
    del calls[:]
    three = torch.zeros(nb, R, 128, dtype=bf16)
    longs = torch.zeros(nb, dtype=torch.int64)
    rows = [three, three[:, 0], k[:nb * R - 1], k[:, :64], k.float(), torch.zeros(128, nb * R, dtype=bf16).t(),
            torch.zeros(nb * R, 256, dtype=bf16)[:, ::2], k.to("meta")]
    for x in rows:
        for f, kw in ((norm, dict(k=x)), (both, dict(k=x)), (both, dict(v=x)), (app8, dict(k=x)), (app8, dict(v=x))):
            with pytest.raises(ValueError):
                f(**kw)
    for f, kw in ((norm, dict(q=oq.view(nb, R, 256))), (norm, dict(q=k)), (norm, dict(pos=longs)), (norm, dict(pos=i32[:1])),
                  (norm, dict(oq=oq[:1])), (norm, dict(ok=ok[..., :32])), (norm, dict(g=g[:32])), (norm, dict(g=g.float())),
                  (both, dict(ctx=longs)), (both, dict(n=i32[:1])), (app8, dict(n=longs)), (app8, dict(g=g[:8])),
                  (att, dict(q=ok)), (att, dict(o=oq[:, :2])), (att, dict(q=oq.transpose(1, 2))), (att, dict(o=oq.float())),
                  (att, dict(ctx=longs)), (att, dict(n=i32[:1]))):
        with pytest.raises(ValueError):
            f(**kw)
    assert not calls


def test_the_binding_needs_torch_only_for_a_stream():
    import os
    import subprocess
    import sys
    code = ("import sys; sys.modules['torch'] = None; from block_diffusion_speculative_project_gb300 import dflash as d; "
            "assert d.DFLASH_PAGE_ROWS == 64")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)
