"""Host side of the calls on trees of drafted tokens, without a GPU: the oracle's definitions against
hand cases and brute force, and the refusals that need no device."""
import numpy as np
import pytest

from oracle import dflash_oracle as orc

#        0
#      1   2
#     3 4   5
#     6
PARENT = [-1, 0, 0, 1, 1, 2, 3]


def test_lines_and_visibility_of_a_hand_tree():
    assert orc.tree_lines(PARENT) == [[0], [1, 0], [2, 0], [3, 1, 0], [4, 1, 0], [5, 2, 0], [6, 3, 1, 0]]
    seen = orc.tree_visible(PARENT, 3, 0, 0)
    assert seen[:, :3].all()
    assert [np.flatnonzero(r[3:]).tolist() for r in seen] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 4], [0, 2, 5],
                                                              [0, 1, 3, 6]]
    # window 2: a node and its parent; the root also the last context row; sinks 1: cache row 0 for all
    seen = orc.tree_visible(PARENT, 3, 2, 1)
    assert [np.flatnonzero(r).tolist() for r in seen] == [[0, 2, 3], [0, 3, 4], [0, 3, 5], [0, 4, 6], [0, 4, 7],
                                                          [0, 5, 8], [0, 6, 9]]
    # sinks beyond the context: nodes at the first positions stay visible to those below them
    seen = orc.tree_visible(PARENT, 1, 1, 3)
    assert [np.flatnonzero(r).tolist() for r in seen] == [[0, 1], [0, 1, 2], [0, 1, 3], [0, 1, 2, 4], [0, 1, 2, 5],
                                                          [0, 1, 3, 6], [0, 1, 2, 7]]


def test_a_chain_is_causal_and_a_wide_window_hides_nothing():
    chain = list(range(-1, 5))
    causal = np.tril(np.ones((6, 10)), 4) > 0
    assert np.array_equal(orc.tree_visible(chain, 4, 0, 0), causal)
    assert np.array_equal(orc.tree_visible(chain, 4, 10, 0), causal)
    assert not np.array_equal(orc.tree_visible(chain, 4, 9, 0), causal)


def test_attention_of_a_path_equals_the_chain_of_its_rows():
    """A node's output is that of causal attention over its own line laid out as a chain."""
    rng = np.random.default_rng(0)
    ctx, n, Hq, Hkv, hd = 5, len(PARENT), 4, 2, 8
    q = rng.standard_normal((n, Hq, hd))
    K, V = rng.standard_normal((2, Hkv, ctx + n, hd))
    o, _, _ = orc.attention_tree(q, K, V, orc.tree_visible(PARENT, ctx, 0, 0))
    for j, line in enumerate(orc.tree_lines(PARENT)):
        rows = list(range(ctx)) + [ctx + a for a in reversed(line)]
        want, _, _ = orc.attention8(q[line[::-1]], K[:, rows], V[:, rows], ctx, causal=True)
        assert np.allclose(o[j], want[-1])


def test_adjusted_logits_of_a_hand_row():
    x = np.array([2.0, -2.0, 1.0, 4.0, -np.inf, np.nan, 3.0])
    counts = np.array([2, 0, 1 << 31, 0, 1, 0, (1 << 31) + 3], np.uint32).astype(np.int32)
    y = orc.adjust_logits(x, counts, (2.0, 0.5, 0.25), drafted=[1, 0], bias_ids=[3, 9, 3, -1], bias=[1, 5, -4, 7],
                          allowed=[1, 1, 1, 1, 1, 1, 0])
    assert np.array_equal(y, [1.0 - 1.5 - 0.25, -4.0 - 0.5 - 0.25, 0.5, 1.0, -np.inf, np.nan, -np.inf], equal_nan=True)
    assert orc.greedy(y) == 3
    assert orc.greedy(np.array([np.nan, -np.inf])) == -1 and orc.greedy(np.array([1.0, 3, 3])) == 1


def test_accepted_path_of_a_hand_tree():
    tokens = [10, 20, 21, 30, 30, 31, 40]
    # 0 -> 20 (node 1) -> 30 (node 3, the lower of two) -> 40 (node 6) -> 99
    path, out = orc.accept_tree(PARENT, tokens, [20, 30, 7, 40, 8, 9, 99])
    assert path == [0, 1, 3, 6] and out == [20, 30, 40, 99]
    assert orc.accept_tree(PARENT, tokens, [5] * 7) == ([0], [5])
    assert orc.accept_tree(PARENT, [-1] * 7, [-1] * 7) == ([0], [-1])
    assert orc.accept_tree([], [], []) == ([], [])
    # a chain accepts as the block's rule does
    draft, target = [4, 5, 6], [4, 5, 9, 2]
    tau, bonus = orc.accept(np.array([draft]), np.array([target]))
    path, out = orc.accept_tree([-1, 0, 1, 2], [1] + draft, target)
    assert len(path) == tau[0] and out[-1] == bonus[0]


def test_null_handles_and_rules_are_refused():
    from block_diffusion_speculative_project_gb300 import dflash as d
    N, r = None, d.logit_rules()
    calls = [lambda: d.LIB.dflash_attention_tree(N, 1, 0, 1, N, N, N, N, N, N, 0, 0, 0, N, N, 0, N),
             lambda: d.LIB.dflash_logits_adjust(N, 1, 1, N, 64, r, N, N, 64, N, N, 0, N),
             lambda: d.LIB.dflash_token_counts(N, 1, 1, N, 1, N, 0, N, N, 0, N),
             lambda: d.LIB.dflash_accept_tree(N, 1, 1, N, N, N, N, N, N, N, N, N, N, 0, N),
             lambda: d.LIB.dflash_kv_commit(N, 1, 1, N, N, N, N, N, N, 0, N)]
    for f in calls:
        assert f() == d.DFLASH_ERR_INVALID_ARG


def test_drafter_refuses_tensors_that_its_calls_would_read_past(monkeypatch):
    from types import SimpleNamespace

    import torch

    from block_diffusion_speculative_project_gb300 import drafter
    calls = []
    dr = object.__new__(drafter.Drafter)
    dr.h, dr.ws, dr.shape = None, torch.zeros(1), SimpleNamespace(Hq=4, Hkv=2, hd=64, V=50)
    dr.kcache = dr.vcache = None
    for name in ("attention_tree", "logits_adjust", "token_counts", "accept_tree", "kv_commit"):
        monkeypatch.setattr(drafter._d, "dflash_" + name, lambda *a, name=name: calls.append((name, a)))
    nb, m, V = 2, 3, 50
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(nb, m, 4, 64, dtype=torch.bfloat16)
    wide = torch.zeros(nb * m, 64)

    def att(q=q, o=q, ctx=i32(nb), parent=i32(nb, m), n=i32(nb)):
        dr.attention_tree(nb, 0, m, q, ctx, o, parent=parent, n_rows=n)

    def adj(x=wide[:, :V], y=wide[:, :V], **kw):
        args = dict(out_ids=i32(nb * m), penalties=torch.zeros(nb, 3), counts=i32(nb, V), bias_ids=i32(nb, 4),
                    bias=torch.zeros(nb, 4), allowed=i32(nb * m, 2), parent=i32(nb, m), tokens=i32(nb, m), n_rows=i32(nb))
        dr.logits_adjust(nb, m, x, out=y, **{**args, **kw})

    def cnt(t=i32(nb, 7)[:, :5], c=i32(nb, V), n=i32(nb)):
        dr.token_counts(nb, 5, t, c, n_tokens=n)

    def acc(parent=i32(nb, m), tokens=i32(nb, m), target=i32(nb, m), tau=i32(nb), bonus=i32(nb), path=i32(nb, m),
            out=i32(nb, m), ctx=i32(nb)):
        dr.accept_tree(nb, m, parent, tokens, target, tau, bonus, out_path=path, out_tokens=out, ctx_len=ctx)

    def com(path=i32(nb, m), tau=i32(nb), ctx=i32(nb)):
        dr.kv_commit(nb, m, path, tau, ctx)

    for f in (att, adj, cnt, acc, com):
        f()
    assert [c[0] for c in calls] == ["attention_tree", "logits_adjust", "token_counts", "accept_tree", "kv_commit"]
    assert calls[1][1][4] == calls[1][1][8] == 64 and calls[2][1][4] == 7
    del calls[:]
    long = torch.zeros(nb * m, dtype=torch.int64)
    for f, kw in ((att, dict(q=q[:1])), (att, dict(o=q.float())), (att, dict(parent=i32(nb, 2))), (att, dict(n=i32(1))),
                  (att, dict(ctx=long)), (adj, dict(x=wide[:, :V - 1])), (adj, dict(x=wide[:5, :V])),
                  (adj, dict(y=wide[:, :V].double())), (adj, dict(x=torch.zeros(V, nb * m).t())),
                  (adj, dict(x=torch.zeros(1, V).expand(nb * m, V))), (adj, dict(out_ids=i32(5))),
                  (adj, dict(penalties=torch.zeros(nb, 2))), (adj, dict(counts=i32(nb, V - 1))),
                  (adj, dict(bias=torch.zeros(nb, 3))), (adj, dict(bias=None)), (adj, dict(bias_ids=i32(1, 4), bias=torch.zeros(1, 4))),
                  (adj, dict(allowed=i32(nb * m, 1))), (adj, dict(allowed=long)), (adj, dict(tokens=i32(nb, 2))),
                  (cnt, dict(t=i32(nb, 4))), (cnt, dict(t=i32(1, 5))), (cnt, dict(t=i32(7, nb).t())), (cnt, dict(c=i32(V))),
                  (cnt, dict(n=long)), (acc, dict(tokens=i32(nb, 2))), (acc, dict(tau=i32(1))), (acc, dict(ctx=long)),
                  (acc, dict(path=i32(nb))), (com, dict(path=i32(nb, 2))), (com, dict(tau=long)), (com, dict(ctx=i32(1)))):
        with pytest.raises(ValueError):
            f(**kw)
    assert not calls
