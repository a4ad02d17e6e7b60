"""Holder for one libdflash handle: device weights, KV caches and workspace.

PyTorch supplies device memory and the stream; every step is a call into the C ABI
(see dflash.py). Weight tensors are borrowed by the handle and kept alive here.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import dflash as _d


def to_device_bf16(bits: np.ndarray, device="cuda") -> torch.Tensor:
    """bf16 bit patterns (uint16 numpy) -> bf16 torch tensor on the device."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    return t.to(device).view(torch.bfloat16)


class Drafter:
    """One handle with its caches [N, max_batch, Hkv, Cmax, hd] and workspace; with
    ``num_pages`` > 0 the caches are page pools [N, num_pages, Hkv, 64, hd] read and
    written through the block table given to ``set_block_table``.

    ``shape`` is any object with the workload fields D, Dt, L, N, Hq, Hkv, hd, F, V,
    B, k_top, rope_base, eps, mask_id, flags, conv_group, sel_dim and film_width.
    ``cache8`` adds the 8-bit caches kcache8, vcache8 (e4m3, laid out as the bf16 ones) and their
    scales kscale, vscale, for ``kv_append8`` and ``attention8``.

    ``weights`` maps the weight names of dflash_inputs.weight_shapes to bf16 device
    tensors.
    """

    def __init__(self, shape, weights: dict, max_batch: int, Cmax: int, max_proj_rows: int,
                 max_spin: int = 0, device="cuda", num_pages: int = 0, cache8: bool = False):
        self.shape = shape
        s = shape
        self.cfg = _d.dflash_config(
            D=s.D, Dt=s.Dt, L=s.L, N=s.N, Hq=s.Hq, Hkv=s.Hkv, hd=s.hd, F=s.F, V=s.V, B=s.B,
            k_top=s.k_top, rope_base=s.rope_base, eps=s.eps, mask_id=s.mask_id, Cmax=Cmax,
            max_batch=max_batch, max_proj_rows=max_proj_rows, conv_group=s.conv_group,
            sel_dim=s.sel_dim, flags=s.flags, max_spin=max_spin, film_dim=s.film_width,
            num_pages=num_pages)
        self.h = _d.dflash_create(self.cfg)
        self.weights = weights
        P = lambda name: ctypes.c_void_p(weights[name].data_ptr()) if name in weights else None
        layers = (_d.dflash_layer_weights * s.N)()
        for n in range(s.N):
            p = f"layer{n}."
            L = layers[n]
            for f in ("W_qkv", "Wk_c", "Wv_c", "W_o", "W_gate", "W_up", "W_down", "g_attn", "g_ffn"):
                setattr(L, f, P(p + f))
            for q in range(4):
                L.conv_W0[q] = P(p + f"conv{q}.W0")
                L.conv_W1[q] = P(p + f"conv{q}.W1")
                L.conv_base[q] = P(p + f"conv{q}.base")
        self._layers = layers
        self.wstruct = _d.dflash_weights(W_c=P("W_c"), g_ctx=P("g_ctx"), E=P("E"), W_lm=P("W_lm"),
                                         g_final=P("g_final"), W_A=P("W_A"), W_B=P("W_B"),
                                         W_G=P("W_G"), layers=layers, film_W1=P("film.W1"),
                                         film_W2=P("film.W2"))
        _d.dflash_set_weights(self.h, self.wstruct)
        nbytes = _d.dflash_workspace_size(self.h)
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        cshape = ((s.N, num_pages, s.Hkv, _d.DFLASH_PAGE_ROWS, s.hd) if num_pages > 0
                  else (s.N, max_batch, s.Hkv, Cmax, s.hd))
        self.kcache = torch.zeros(cshape, dtype=torch.bfloat16, device=device)
        self.vcache = torch.zeros(cshape, dtype=torch.bfloat16, device=device)
        self.kcache8 = self.vcache8 = self.kscale = self.vscale = None
        if cache8:
            if Cmax % _d.DFLASH_PAGE_ROWS:
                raise ValueError(f"8-bit caches need Cmax % {_d.DFLASH_PAGE_ROWS} == 0, got {Cmax}")
            self.kcache8 = torch.zeros(cshape, dtype=torch.float8_e4m3fn, device=device)
            self.vcache8 = torch.zeros(cshape, dtype=torch.float8_e4m3fn, device=device)
            sshape = cshape[:3] if num_pages > 0 else cshape[:3] + (Cmax // _d.DFLASH_PAGE_ROWS,)
            self.kscale = torch.ones(sshape, dtype=torch.float32, device=device)
            self.vscale = torch.ones(sshape, dtype=torch.float32, device=device)
        self.max_batch, self.Cmax, self.max_proj_rows = max_batch, Cmax, max_proj_rows
        self.num_pages = num_pages
        self.block_table = None

    def set_block_table(self, table: torch.Tensor):
        """Register the int32 device block table [max_batch, Cmax / 64] (kept alive here)."""
        assert table.dtype == torch.int32 and table.is_cuda and table.is_contiguous()
        assert tuple(table.shape) == (self.max_batch, self.Cmax // _d.DFLASH_PAGE_ROWS)
        self.block_table = table
        _d.dflash_set_block_table(self.h, table)

    def __del__(self):
        try:
            if getattr(self, "h", None):
                _d.dflash_destroy(self.h)
                self.h = None
        except Exception:
            pass

    # thin forwards -------------------------------------------------------------
    def ctx_project(self, nb, R, hv, n_commit, ctx_len, relay_a=None, x0_relay=None, stream=None,
                    relay_b=None, relay_y=None):
        if relay_b is not None or relay_y is not None:
            _d.dflash_ctx_project_film(self.h, nb, R, hv, n_commit, relay_a, relay_b, relay_y, ctx_len,
                                       self.kcache, self.vcache, x0_relay, self.ws, stream)
        else:
            _d.dflash_ctx_project(self.h, nb, R, hv, n_commit, relay_a, ctx_len, self.kcache,
                                  self.vcache, x0_relay, self.ws, stream)

    def draft_block(self, nb, block_ids, ctx_len, out_hidden, x0_relay=None, max_ctx_hint=0,
                    stream=None):
        _d.dflash_draft_block(self.h, nb, block_ids, x0_relay, self.kcache, self.vcache, ctx_len,
                              max_ctx_hint, out_hidden, self.ws, stream)

    def lm_head_topk(self, nb, hidden, k, out_ids, out_vals, out_logits=None, stream=None):
        _d.dflash_lm_head_topk(self.h, nb, hidden, k, out_ids, out_vals, out_logits, self.ws, stream)

    def accept(self, nb, draft, target, out_tau, out_bonus, stream=None):
        _d.dflash_accept(self.h, nb, draft, target, out_tau, out_bonus, stream)

    def accept_topk(self, nb, topk_ids, k, target, out_tau, out_bonus, stream=None):
        _d.dflash_accept_topk(self.h, nb, topk_ids, k, target, out_tau, out_bonus, stream)

    def sample(self, rows, logits, temperature, seed, out_ids, out_lse, out_logq=None, row0=0,
               stream=None):
        _d.dflash_sample(self.h, rows, logits, temperature, seed, row0, out_ids, out_lse, out_logq,
                         self.ws, stream)

    def lm_head_sample(self, nb, hidden, temperature, seed, out_cand, out_lse, out_logq=None,
                       out_logits=None, k=0, out_ids=None, out_vals=None, stream=None):
        _d.dflash_lm_head_sample(self.h, nb, hidden, temperature, seed, out_cand, out_lse, out_logq,
                                 out_logits, k, out_ids, out_vals, self.ws, stream)

    def verify_sample(self, nb, draft_logits, draft_lse, cand, target_logits, temperature, seed,
                      out_tau, out_token, stream=None):
        _d.dflash_verify_sample(self.h, nb, draft_logits, draft_lse, cand, target_logits, temperature,
                                seed, out_tau, out_token, self.ws, stream)

    def conv(self, layer, which, nb, x, stream=None):
        _d.dflash2_conv(self.h, layer, which, nb, x, self.ws, stream)

    def select(self, nb, k, topk_ids, topk_vals, hidden, block_ids, out_path, stream=None):
        _d.dflash2_select(self.h, nb, k, topk_ids, topk_vals, hidden, block_ids, out_path, self.ws,
                          stream)

    def select_sample(self, nb, k, topk_ids, topk_vals, hidden, block_ids, temperature, seed, out_path,
                      out_walk_logq, stream=None):
        _d.dflash2_select_sample(self.h, nb, k, topk_ids, topk_vals, hidden, block_ids, temperature, seed,
                                 out_path, out_walk_logq, self.ws, stream)

    def verify_sample_walk(self, nb, k, cand_ids, walk_logq, path, target_logits, temperature, seed,
                           out_tau, out_token, stream=None):
        _d.dflash_verify_sample_walk(self.h, nb, k, cand_ids, walk_logq, path, target_logits, temperature,
                                     seed, out_tau, out_token, self.ws, stream)

    def recall_at_k(self, nb, k, cand_ids, target, hits, eligible, stream=None):
        _d.dflash_recall_at_k(self.h, nb, k, cand_ids, target, hits, eligible, stream)

    def attention(self, nb, layer, q, ctx_len, out_o, max_ctx_hint=0, stream=None):
        _d.dflash_attention(self.h, nb, layer, q, self.kcache, self.vcache, ctx_len, max_ctx_hint,
                            out_o, self.ws, stream)

    def _rows(self, name, t, rows, heads):
        """Row stride of t, which has to be bf16 [rows or more, heads * hd] with dense rows."""
        self._mine(name, t, torch.bfloat16)
        width = heads * self.shape.hd
        if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != width or t.stride(1) != 1:
            raise ValueError(f"{name}: rows [{rows}, {width}] with values side by side, "
                             f"got {tuple(t.shape)} with strides {t.stride()}")
        return t.stride(0) if t.shape[0] > 1 else width

    def _dense(self, name, t, count, dtype=torch.bfloat16):
        self._mine(name, t, dtype)
        if t.numel() < count or not t.is_contiguous():
            raise ValueError(f"{name}: {count} values without gaps, got {tuple(t.shape)} with strides {t.stride()}")

    def _mine(self, name, t, dtype):
        if t.dtype != dtype or t.device != self.ws.device:
            raise ValueError(f"{name}: {dtype} on {self.ws.device}, got {t.dtype} on {t.device}")

    def _append_rows(self, nb, R, k, v, ctx_len, n_rows, g_k):
        s = self.shape
        ldk, ldv = self._rows("k", k, nb * R, s.Hkv), self._rows("v", v, nb * R, s.Hkv)
        self._dense("ctx_len", ctx_len, nb, torch.int32)
        if n_rows is not None:
            self._dense("n_rows", n_rows, nb, torch.int32)
        if g_k is not None:
            self._dense("g_k", g_k, s.hd)
        return ldk, ldv

    def qk_norm_rope(self, nb, R, q, k, pos0, out_q, out_k, g_q=None, g_k=None, stream=None):
        """q, k: rows [nb * R, heads * hd] of any row stride (k and out_k may be None)."""
        s = self.shape
        ldq, ldk = self._rows("q", q, nb * R, s.Hq), 0
        self._dense("out_q", out_q, nb * R * s.Hq * s.hd)
        self._dense("pos0", pos0, nb, torch.int32)
        if k is not None:
            ldk = self._rows("k", k, nb * R, s.Hkv)
        if out_k is not None:
            self._dense("out_k", out_k, nb * R * s.Hkv * s.hd)
        for name, g in (("g_q", g_q), ("g_k", g_k)):
            if g is not None:
                self._dense(name, g, s.hd)
        _d.dflash_qk_norm_rope(self.h, nb, R, q, ldq, k, ldk, g_q, g_k, pos0, out_q, out_k, stream)

    def kv_append(self, nb, layer, R, k, v, ctx_len, n_rows=None, g_k=None, rotate=True, stream=None):
        """k, v: rows [nb * R, Hkv * hd] of any row stride."""
        ldk, ldv = self._append_rows(nb, R, k, v, ctx_len, n_rows, g_k)
        _d.dflash_kv_append(self.h, nb, layer, R, k, ldk, v, ldv, g_k, int(rotate), n_rows, ctx_len,
                            self.kcache, self.vcache, self.ws, stream)

    def kv_append8(self, nb, layer, R, k, v, ctx_len, n_rows=None, g_k=None, rotate=True, stream=None):
        ldk, ldv = self._append_rows(nb, R, k, v, ctx_len, n_rows, g_k)
        _d.dflash_kv_append8(self.h, nb, layer, R, k, ldk, v, ldv, g_k, int(rotate), n_rows, ctx_len,
                             self.kcache8, self.vcache8, self.kscale, self.vscale, self.ws, stream)

    def attention8(self, nb, layer, m, q, ctx_len, out_o, n_rows=None, causal=False, max_ctx_hint=0, stream=None):
        s = self.shape
        self._dense("q", q, nb * m * s.Hq * s.hd)
        self._dense("out_o", out_o, nb * m * s.Hq * s.hd)
        self._dense("ctx_len", ctx_len, nb, torch.int32)
        if n_rows is not None:
            self._dense("n_rows", n_rows, nb, torch.int32)
        _d.dflash_attention8(self.h, nb, layer, m, q, self.kcache8, self.vcache8, self.kscale, self.vscale, n_rows,
                             ctx_len, max_ctx_hint, int(causal), out_o, self.ws, stream)

    def topk(self, rows, cols, logits, k, out_ids, out_vals, stream=None):
        _d.dflash_topk(self.h, rows, cols, logits, k, out_ids, out_vals, None, stream)

    def status(self, stream=None) -> int:
        return _d.dflash_status(self.h, self.ws, stream)
