"""Appends of keys that the caller has rotated already (dflash_kv_append with rotate = 0)."""
import pytest
import torch

from test_gpu_rows8 import Cache, fused

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_keys_that_are_not_rotated(hd, norm):
    """rotate = 0: without a gain the keys go to the bf16 cache bit for bit, infinities, NaN and -0 too; with
    one, a value reaches only its own place and its row's norm."""
    R, Hkv = 9, 3
    c = Cache(Hkv, Hkv, hd, 128, 1, N=1, seed=1)
    _, k, v, _, gk = fused(1, R, 1, Hkv, hd, seed=5)
    k, v = k.clone(), v.clone()
    at = k.view(R, Hkv, hd)
    at[0, 0, 3], at[1, 1, hd - 2], at[2, 2, hd // 2] = float("inf"), float("-inf"), float("nan")
    at[3, :, ::3] = -0.0
    v.view(R, Hkv, hd)[4, 0, 1] = float("nan")
    c.append(0, R, k, v, None, [30], gk if norm else None, 0)
    assert c.status() == 0
    got = c.kc[0][c.at(0, 0)][:, 30:30 + R].transpose(0, 1)
    assert torch.equal(c.vc[0][c.at(0, 0)][:, 30:30 + R].transpose(0, 1).reshape(R, -1).view(torch.int16),
                       v.view(torch.int16))
    if not norm:
        assert torch.equal(got.reshape(R, -1).view(torch.int16), k.view(torch.int16))
        return
    x = at.double()
    y = x * gk.double() / (x.square().mean(dim=-1, keepdim=True) + 1e-6).sqrt()  # inf / inf is NaN, x / inf zero
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    live = ~torch.isnan(y)
    # one bf16 rounding; the norm's fp32 steps, 2^-16 (test_gpu_rows8.py)
    assert ((got.double() - y).abs()[live] <= (2.0 ** -8 + 2.0 ** -16) * y.abs()[live]).all()
    assert torch.equal(torch.signbit(got[3]), torch.signbit(at[3]))
