"""The cache calls on pools whose offsets pass 32 bits, on pages that two sequences share, and on contiguous
caches that end inside a block (bf16)."""
import numpy as np
import pytest
import torch

from test_gpu_attention8_deep import check
from test_gpu_rows8 import PR, Cache, f64, fused, i32, lib, queries, want_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,m", [(1, 4), (4, 8), (8, 16)])
def test_pages_at_the_end_of_a_large_pool(G, m):
    """70,001 pages of 8 heads of 128: 4.6e9 elements. The same rows in a small pool give the same bits."""
    D, Hkv, hd, nb = lib(), 8, 128, 2
    c = Cache(G * Hkv, Hkv, hd, 4 * PR, nb, N=1, seed=m)
    cfg = D.dflash_config.from_buffer_copy(c.cfg)
    cfg.num_pages = 70001
    h = D.dflash_create(cfg)
    table = cfg.num_pages - 1 - c.table            # its pages in the other order, at the very end
    big_table = i32(table)
    D.dflash_set_block_table(h, big_table)
    ws = torch.zeros(D.dflash_workspace_size(h), dtype=torch.uint8, device="cuda")
    small = {x: getattr(c, x) for x in ("kc", "vc", "k8", "v8", "ks", "vs")}
    big = {x: torch.empty(1, cfg.num_pages, *t.shape[2:], dtype=t.dtype, device="cuda") for x, t in small.items()}
    src, dst = (torch.as_tensor(np.ascontiguousarray(t).reshape(-1), device="cuda").long() for t in (c.table, table))
    bits = lambda t: t if t.dtype == torch.float32 else t.view({1: torch.uint8, 2: torch.int16}[t.element_size()])  # noqa: E731
    for x in small:
        bits(big[x])[0][dst] = bits(small[x])[0][src]
    qr, k, v, gq, gk = fused(nb, m, G * Hkv, Hkv, hd, seed=m)
    q = torch.empty(nb, m, G * Hkv, hd, dtype=torch.bfloat16, device="cuda")
    ctx, n = i32([4 * PR - m, 60]), i32([m, m - 1])
    outs = []
    for hh, t, w in ((c.h, small, c.ws), (h, big, ws)):
        D.dflash_qk_norm_rope(hh, nb, m, qr, qr.stride(0), None, 0, gq, None, ctx, q, None)
        D.dflash_kv_append(hh, nb, 0, m, k, k.stride(0), v, v.stride(0), gk, 1, n, ctx, t["kc"], t["vc"], w)
        D.dflash_kv_append8(hh, nb, 0, m, k, k.stride(0), v, v.stride(0), gk, 1, n, ctx, t["k8"], t["v8"], t["ks"],
                            t["vs"], w)
        outs.append(torch.full_like(q, 7.0))
        D.dflash_attention8(hh, nb, 0, m, q, t["k8"], t["v8"], t["ks"], t["vs"], n, ctx, 0, 1, outs[-1], w)
        assert D.dflash_status(hh, w) == 0
    for x in small:
        assert torch.equal(bits(big[x])[0][dst], bits(small[x])[0][src]), x
    assert torch.equal(*outs)
    check(c, q, [m, m - 1], [4 * PR - m, 60], True, outs[0])
    D.dflash_destroy(h)


@pytest.mark.parametrize("G,m", [(2, 3), (4, 7)])
def test_two_sequences_share_the_pages_of_their_prefix(G, m):
    """Whole pages of a common prefix, each sequence's own rows behind them."""
    Hkv, hd = 2, 64
    c = Cache(G * Hkv, Hkv, hd, 4 * PR, 2, N=1, seed=5)
    c.table[1, :2] = c.table[0, :2]
    c.dev_table.copy_(i32(c.table))
    before = c.k8.clone()
    _, k, v, _, gk = fused(2, m, 1, Hkv, hd, seed=1)
    ctx = [2 * PR, 2 * PR]
    c.append8(0, m, k, v, None, ctx, gk, 1)
    for b in range(2):
        assert torch.equal(c.k8[0][c.at(0, b)].view(torch.uint8), before[0][c.at(0, b)].view(torch.uint8))
    q = queries(c, m, seed=2)
    out = c.attend(0, m, q, None, ctx, True)
    assert c.status() == 0
    check(c, q, [m, m], ctx, True, out)


def test_append_to_contiguous_caches_that_end_inside_a_block():
    """The bf16 caches take any length; rows behind it are reported and not written."""
    D, nb, Hkv, hd, Cmax, R = lib(), 3, 3, 64, 101, 7
    cfg = D.dflash_config.from_buffer_copy(Cache(Hkv, Hkv, hd, 128, 1).cfg)
    cfg.num_pages, cfg.Cmax, cfg.max_batch, cfg.N = 0, Cmax, nb, 1
    h = D.dflash_create(cfg)
    ws = torch.zeros(D.dflash_workspace_size(h), dtype=torch.uint8, device="cuda")
    kc, vc = (torch.full((nb, Hkv, Cmax, hd), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _, k, v, _, gk = fused(nb, R, 1, Hkv, hd, seed=3)
    ctx = [Cmax - R, 0, Cmax - 2]
    for n, code in (([R, R, 2], 0), ([R, R, R], D.DFLASH_ERR_DEVICE_CHECK)):
        D.dflash_kv_append(h, nb, 0, R, k, k.stride(0), v, v.stride(0), gk, 1, i32(n), i32(ctx), kc, vc, ws)
        assert D.dflash_status(h, ws) == code
        want, slack = want_rows(k, nb, R, Hkv, hd, gk, np.array(ctx)[:, None] + np.arange(R))
        for i, fit in enumerate((R, R, 2)):
            got = f64(kc[i, :, ctx[i]:ctx[i] + fit]).transpose(1, 0, 2)
            assert (np.abs(got - want[i, :fit]) <= 2.0 ** -8 * np.abs(want[i, :fit]) + slack[i, :fit]).all()
            assert torch.equal(vc[i, :, ctx[i]:ctx[i] + fit], v.reshape(nb, R, Hkv, hd)[i, :fit].transpose(0, 1))
            rest = torch.ones(Cmax, dtype=torch.bool, device="cuda")
            rest[ctx[i]:ctx[i] + fit] = False
            assert (kc[i, :, rest] == 3.0).all() and (vc[i, :, rest] == 3.0).all()
    D.dflash_destroy(h)
