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
