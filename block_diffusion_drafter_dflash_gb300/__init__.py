"""GB300 (sm_103a) DFlash draft cycle: thin Python binding over the C ABI.

The functions below carry the C ABI's names and only marshal arguments (torch
tensors -> device pointers, the current torch stream -> cudaStream_t); every
step of the cycle — context fusion, K/V injection, the non-causal drafter
pass, the LM head argmax and greedy verification — runs in the CUDA library
``libdflash_gb300.so`` built from ``csrc/``.  There is no CPU fallback: if the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import Optional

import torch

from . import _abi
from ._abi import DFlashError, check, lib

__all__ = ["DFlashError", "Model", "Cache", "lib", "dflash_model_create", "dflash_cache_init",
           "dflash_workspace_bytes", "dflash_workspace", "dflash_inject_context", "dflash_draft_block",
           "dflash_verify_greedy", "dflash_draft_cycle", "dflash_get_status", "dflash_clear_status", "dflash_version",
           "dflash_launch_count", "dflash_profile_start", "dflash_profile_stop", "dflash_inject_context_noalloc",
           "dflash_selftest_wait_timeout", "dflash_sampling_workspace", "dflash_verify_sampled", "dflash_sample_tokens",
           "BlockPolicy", "dflash_packed_attention_workspace", "dflash_packed_block_attention",
           "dflash_packed_attention_status", "dflash_token_logprobs", "dflash_token_logprobs_backward",
           "dflash_clip_workspace", "dflash_clip_grad_norm", "dflash_packed_attention_backward_workspace",
           "dflash_packed_block_attention_backward", "dflash_linear_cross_entropy_workspace",
           "dflash_linear_cross_entropy", "dflash_linear_cross_entropy_backward_workspace",
           "dflash_linear_cross_entropy_backward", "dflash_linear_cross_entropy_status", "dflash_embed_tokens",
           "dflash_embed_tokens_backward_workspace", "dflash_embed_tokens_backward"]


# The current stream's handle without a Stream object (microseconds a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _config_struct(cfg) -> _abi.Config:
    mask = cfg.mask_id if hasattr(cfg, "mask_id") else cfg.mask_token_id
    return _abi.Config(hidden=cfg.hidden, layers=cfg.layers, n_q_heads=cfg.n_q_heads, n_kv_heads=cfg.n_kv_heads,
                       head_dim=cfg.head_dim, ffn=cfg.ffn, vocab=cfg.vocab, n_target_feats=cfg.n_target_feats,
                       max_block=cfg.max_block, rope_theta=float(cfg.rope_theta), rms_eps=float(cfg.rms_eps),
                       mask_token_id=int(mask), dtype=_abi.DTYPE_F32 if cfg.dtype == "fp32" else _abi.DTYPE_BF16,
                       qk_norm=1 if getattr(cfg, "qk_norm", False) else 0,
                       input_fusion=1 if getattr(cfg, "input_fusion", False) else 0,
                       kv_bf16=1 if getattr(cfg, "kv_bf16", False) else 0,
                       head_bf16=1 if getattr(cfg, "head_bf16", False) else 0)


def dflash_version() -> int:
    return lib().dflash_version()


class Model:
    """A created dflash_model; keeps the borrowed weight tensors alive."""

    def __init__(self, cfg, weights: dict):
        self.cfg = cfg
        self.weights = weights
        self.dtype = torch.float32 if cfg.dtype == "fp32" else torch.bfloat16
        tensors = [weights[k] for k in ("embed", "lm_head", "w_c", "g_c", "g_final")]
        for lw in weights["layers"]:
            tensors += list(lw.values())
        for t in tensors:
            if t.dtype != self.dtype or not t.is_cuda or not t.is_contiguous():
                raise ValueError("weights must be contiguous CUDA tensors of the model dtype")
        self._layers = (_abi.LayerWeights * cfg.layers)(*[
            _abi.LayerWeights(**{k: (lw[k].data_ptr() if k in lw else None)
                                 for k in ("g_in", "w_q", "w_k", "w_v", "w_o", "g_post", "w_g", "w_u", "w_d", "g_q",
                                           "g_k")})
            for lw in weights["layers"]])
        w = _abi.Weights(embed=weights["embed"].data_ptr(), lm_head=weights["lm_head"].data_ptr(),
                         w_c=weights["w_c"].data_ptr(), g_c=weights["g_c"].data_ptr(),
                         g_final=weights["g_final"].data_ptr(), layers=self._layers)
        self._cfg = _config_struct(cfg)
        h = ctypes.c_void_p()
        check(lib().dflash_model_create(ctypes.byref(self._cfg), ctypes.byref(w), ctypes.byref(h)),
              "dflash_model_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            lib().dflash_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Cache:
    """A dflash_cache carved out of a torch-owned device buffer."""

    def __init__(self, model: Model, batch: int, capacity: int, stream=None):
        self.model, self.batch, self.capacity = model, batch, capacity
        nbytes = lib().dflash_cache_bytes(ctypes.byref(model._cfg), batch, capacity)
        if nbytes == 0:
            raise ValueError("invalid cache shape")
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        h = ctypes.c_void_p()
        check(lib().dflash_cache_init(model.handle, self.buffer.data_ptr(), nbytes, batch, capacity,
                                      _stream_ptr(stream), ctypes.byref(h)), "dflash_cache_init")
        self.handle = h
        k, v, ln = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        check(lib().dflash_cache_layout(h, ctypes.byref(k), ctypes.byref(v), ctypes.byref(ln)), "dflash_cache_layout")
        self.k_off, self.v_off, self.len_off = k.value, v.value, ln.value

    def _kv_view(self, off: int, hd_major: bool = False) -> torch.Tensor:
        c = self.model.cfg
        B, L, H, cap, hd = self.batch, c.layers, c.n_kv_heads, self.capacity, c.head_dim
        if self.model.dtype == torch.float32:
            raw = self.buffer[off:off + B * L * H * cap * hd * 4]
            return raw.view(torch.float32).view(B, L, H, cap, hd)
        P = 1 if getattr(c, "kv_bf16", False) else 2   # bf16 planes of each value
        if hd_major:   # bf16 V: [B][L][H][P][hd][pitch], pitch = capacity rounded up to 8
            pitch = (cap + 7) // 8 * 8
            raw = self.buffer[off:off + B * L * H * P * hd * pitch * 2]
            planes = raw.view(torch.bfloat16).view(B, L, H, P, hd, pitch)[..., :cap].transpose(-1, -2)
        else:
            raw = self.buffer[off:off + B * L * H * P * cap * hd * 2]
            planes = raw.view(torch.bfloat16).view(B, L, H, P, cap, hd)
        return planes.float().sum(dim=3)

    def k(self) -> torch.Tensor:
        """Context keys as fp32 [batch][layers][n_kv_heads][capacity][head_dim]
        (a view for fp32 models; the sum of the bf16 planes otherwise)."""
        return self._kv_view(self.k_off)

    def v(self) -> torch.Tensor:
        """Context values as fp32 [batch][layers][n_kv_heads][capacity][head_dim]
        (bf16 models store them head-dim-major; this returns them position-major)."""
        return self._kv_view(self.v_off, hd_major=True)

    def ctx_len(self) -> torch.Tensor:
        return self.buffer[self.len_off:self.len_off + 4 * self.batch].view(torch.int32)

    def set_lengths(self, lengths, stream=None):
        arr = (ctypes.c_int32 * self.batch)(*[int(v) for v in lengths])
        check(lib().dflash_cache_set_lengths(self.handle, arr, _stream_ptr(stream)), "dflash_cache_set_lengths")

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            lib().dflash_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dflash_model_create(cfg, weights: dict) -> Model:
    return Model(cfg, weights)


def dflash_cache_init(model: Model, batch: int, capacity: int, stream=None) -> Cache:
    return Cache(model, batch, capacity, stream)


def dflash_workspace_bytes(model: Model, batch: int, capacity: int, block_size: int, max_inject_rows: int) -> int:
    return int(lib().dflash_workspace_bytes(model.handle, batch, capacity, block_size, max_inject_rows))


def dflash_workspace(model: Model, batch: int, capacity: int, block_size: int, max_inject_rows: int) -> torch.Tensor:
    n = dflash_workspace_bytes(model, batch, capacity, block_size, max_inject_rows)
    if n == 0:
        raise ValueError("invalid workspace shape")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def dflash_inject_context(model: Model, cache: Cache, feats: torch.Tensor, n_new_dev: torch.Tensor,
                          n_new_host=None, max_rows: Optional[int] = None, workspace: torch.Tensor = None,
                          stream=None) -> None:
    """feats [max_rows, m, D] (model dtype), n_new_dev int32 [batch] on the device."""
    if n_new_dev.dtype != torch.int32 or feats.dtype != model.dtype:
        raise ValueError("n_new_dev must be int32 and feats of the model dtype")
    rows = feats.shape[0] if max_rows is None else int(max_rows)
    host = None
    if n_new_host is not None:
        host = (ctypes.c_int32 * cache.batch)(*[int(v) for v in n_new_host])
    check(lib().dflash_inject_context(model.handle, cache.handle, _ptr(feats), _ptr(n_new_dev), host, rows,
                                      _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
          "dflash_inject_context")


def dflash_inject_context_noalloc(model: Model, cache: Cache, feats: torch.Tensor, n_new_dev: torch.Tensor,
                                  n_new_host=None, max_rows: Optional[int] = None, stream=None) -> None:
    """dflash_inject_context without a workspace, for callers that cannot
    allocate device memory: the library's fixed static scratch is used."""
    if n_new_dev.dtype != torch.int32 or feats.dtype != model.dtype:
        raise ValueError("n_new_dev must be int32 and feats of the model dtype")
    rows = feats.shape[0] if max_rows is None else int(max_rows)
    host = None
    if n_new_host is not None:
        host = (ctypes.c_int32 * cache.batch)(*[int(v) for v in n_new_host])
    check(lib().dflash_inject_context_noalloc(model.handle, cache.handle, _ptr(feats), _ptr(n_new_dev), host, rows,
                                              _stream_ptr(stream)), "dflash_inject_context_noalloc")


def dflash_draft_block(model: Model, cache: Cache, anchor_dev: torch.Tensor, block_size: int,
                       draft_dev: torch.Tensor, logits_dev: Optional[torch.Tensor] = None,
                       workspace: torch.Tensor = None, stream=None) -> None:
    """anchor_dev int32 [batch]; draft_dev int32 [batch, block-1]; logits_dev fp32 [batch, block-1, V] or None."""
    if anchor_dev.dtype != torch.int32 or draft_dev.dtype != torch.int32:
        raise ValueError("anchor_dev and draft_dev must be int32")
    if logits_dev is not None and logits_dev.dtype != torch.float32:
        raise ValueError("logits_dev must be float32")
    check(lib().dflash_draft_block(model.handle, cache.handle, _ptr(anchor_dev), int(block_size), _ptr(draft_dev),
                                   _ptr(logits_dev), _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
          "dflash_draft_block")


def dflash_draft_cycle(model: Model, cache: Cache, feats: torch.Tensor, n_new_dev: torch.Tensor, anchor_dev: torch.Tensor,
                       block_size: int, draft_dev: torch.Tensor, logits_dev: Optional[torch.Tensor] = None,
                       n_new_host=None, max_rows: Optional[int] = None, workspace: torch.Tensor = None,
                       stream=None) -> None:
    """Injection of feats [max_rows, m, D] (n_new_dev rows per request) then a
    drafter pass of block_size from anchor_dev; one persistent launch when
    both fit it."""
    if n_new_dev.dtype != torch.int32 or anchor_dev.dtype != torch.int32 or draft_dev.dtype != torch.int32:
        raise ValueError("n_new_dev, anchor_dev and draft_dev must be int32")
    if feats.dtype != model.dtype:
        raise ValueError("feats must be of the model dtype")
    rows = feats.shape[0] if max_rows is None else int(max_rows)
    host = None
    if n_new_host is not None:
        host = (ctypes.c_int32 * cache.batch)(*[int(v) for v in n_new_host])
    check(lib().dflash_draft_cycle(model.handle, cache.handle, _ptr(feats), _ptr(n_new_dev), host, rows,
                                   _ptr(anchor_dev), int(block_size), _ptr(draft_dev), _ptr(logits_dev),
                                   _ptr(workspace), workspace.numel(), _stream_ptr(stream)), "dflash_draft_cycle")


def dflash_verify_greedy(draft_dev: torch.Tensor, target_argmax_dev: torch.Tensor, accept_len_dev: torch.Tensor,
                         out_tokens_dev: torch.Tensor, next_anchor_dev: torch.Tensor, stream=None) -> None:
    """draft int32 [B, g-1], target int32 [B, g] -> tau [B], out [B, g], next anchor [B] (all int32)."""
    B, g = target_argmax_dev.shape
    for t in (draft_dev, target_argmax_dev, accept_len_dev, out_tokens_dev, next_anchor_dev):
        if t.dtype != torch.int32:
            raise ValueError("verify tensors must be int32")
    check(lib().dflash_verify_greedy(_ptr(draft_dev), _ptr(target_argmax_dev), B, g, _ptr(accept_len_dev),
                                     _ptr(out_tokens_dev), _ptr(next_anchor_dev), _stream_ptr(stream)),
          "dflash_verify_greedy")


def dflash_sampling_workspace(rows: int, draws: int, vocab: int) -> torch.Tensor:
    """Device scratch for dflash_verify_sampled / dflash_sample_tokens."""
    n = int(lib().dflash_sampling_workspace_bytes(int(rows), int(draws), int(vocab)))
    if n == 0:
        raise ValueError("invalid sampling workspace shape")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def dflash_verify_sampled(draft_logits: Optional[torch.Tensor], target_logits: torch.Tensor,
                          drafts: Optional[torch.Tensor], u_accept: Optional[torch.Tensor], u_sample: torch.Tensor,
                          temperature: float, accept_len: torch.Tensor, out_tokens: torch.Tensor,
                          next_anchor: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Stochastic lossless verification: draft logits fp32 [B, g-1, V], target
    logits fp32 [B, g, V], drafts int32 [B, g-1], uniforms fp32 u_accept
    [B, g-1] and u_sample [B] -> tau [B], out [B, g], next anchor [B]."""
    B, g, V = target_logits.shape
    for t in (draft_logits, target_logits, u_accept, u_sample):
        if t is not None and t.dtype != torch.float32:
            raise ValueError("logits and uniforms must be float32")
    for t in (drafts, accept_len, out_tokens, next_anchor):
        if t is not None and t.dtype != torch.int32:
            raise ValueError("token tensors must be int32")
    if workspace is None:
        workspace = dflash_sampling_workspace(B * (2 * g - 1), B, V)
    check(lib().dflash_verify_sampled(_ptr(draft_logits), _ptr(target_logits), _ptr(drafts), _ptr(u_accept),
                                      _ptr(u_sample), B, g, V, float(temperature), _ptr(accept_len),
                                      _ptr(out_tokens), _ptr(next_anchor), _ptr(workspace), workspace.numel(),
                                      _stream_ptr(stream)), "dflash_verify_sampled")


def dflash_sample_tokens(logits: torch.Tensor, temperature: float, u: torch.Tensor, tokens: torch.Tensor,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """tokens[r] = inverse-CDF draw with uniform u[r] from softmax(logits[r] / T); logits fp32 [..., V]."""
    V = logits.shape[-1]
    rows = logits.numel() // V
    if logits.dtype != torch.float32 or u.dtype != torch.float32 or tokens.dtype != torch.int32:
        raise ValueError("logits and u must be float32, tokens int32")
    if workspace is None:
        workspace = dflash_sampling_workspace(rows, rows, V)
    check(lib().dflash_sample_tokens(_ptr(logits), rows, V, float(temperature), _ptr(u), _ptr(tokens),
                                     _ptr(workspace), workspace.numel(), _stream_ptr(stream)), "dflash_sample_tokens")


def dflash_packed_attention_workspace(n_blocks: int, block: int, seq_len: int, n_q_heads: int, n_kv_heads: int,
                                      head_dim: int) -> torch.Tensor:
    n = int(lib().dflash_packed_attention_workspace_bytes(n_blocks, block, seq_len, n_q_heads, n_kv_heads, head_dim))
    if n == 0:
        raise ValueError("invalid packed attention shape")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def dflash_packed_block_attention(q: torch.Tensor, k_ctx: torch.Tensor, v_ctx: torch.Tensor, k_blk: torch.Tensor,
                                  v_blk: torch.Tensor, anchors_dev: torch.Tensor, out: torch.Tensor,
                                  workspace: torch.Tensor, anchors_host=None, stream=None,
                                  lse: Optional[torch.Tensor] = None) -> None:
    """Packed training attention: q [N, g, nq, hd], k_ctx / v_ctx [S, nkv, hd],
    k_blk / v_blk [N, g, nkv, hd] (fp32 or bf16), anchors int32 [N] -> out fp32 [N, g, nq, hd];
    lse fp32 [N, g, nq], if given, receives the log-sum-exp of each row's scores
    (what dflash_packed_block_attention_backward needs)."""
    N, g, nq, hd = q.shape
    S, nkv = k_ctx.shape[0], k_blk.shape[2]
    dt = _abi.DTYPE_F32 if q.dtype == torch.float32 else _abi.DTYPE_BF16
    for t in (k_ctx, v_ctx, k_blk, v_blk):
        if t.dtype != q.dtype:
            raise ValueError("q, k and v must share one dtype")
    if out.dtype != torch.float32 or anchors_dev.dtype != torch.int32:
        raise ValueError("out must be float32 and anchors int32")
    host = None
    if anchors_host is not None:
        host = (ctypes.c_int32 * N)(*[int(a) for a in anchors_host])
    if lse is not None:
        check(lib().dflash_packed_block_attention_lse(
            _ptr(q), _ptr(k_ctx), _ptr(v_ctx), _ptr(k_blk), _ptr(v_blk), _ptr(anchors_dev), host, N, g, S, nq, nkv, hd,
            dt, _ptr(out), _vector(lse, N * g * nq, torch.float32, q, "lse"), _ptr(workspace), workspace.numel(),
            _stream_ptr(stream)), "dflash_packed_block_attention_lse")
        return
    check(lib().dflash_packed_block_attention(_ptr(q), _ptr(k_ctx), _ptr(v_ctx), _ptr(k_blk), _ptr(v_blk),
                                              _ptr(anchors_dev), host, N, g, S, nq, nkv, hd, dt, _ptr(out),
                                              _ptr(workspace), workspace.numel(), _stream_ptr(stream)),
          "dflash_packed_block_attention")


def dflash_packed_attention_backward_workspace(n_blocks: int, block: int, seq_len: int, n_q_heads: int,
                                               n_kv_heads: int, head_dim: int, dtype: torch.dtype) -> torch.Tensor:
    """Device scratch for dflash_packed_block_attention_backward with operands of `dtype`."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("operands are float32 or bfloat16")
    n = int(lib().dflash_packed_attention_backward_workspace_bytes(
        n_blocks, block, seq_len, n_q_heads, n_kv_heads, head_dim,
        _abi.DTYPE_F32 if dtype == torch.float32 else _abi.DTYPE_BF16))
    if n == 0:
        raise ValueError("invalid packed attention shape")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def dflash_packed_block_attention_backward(q: torch.Tensor, k_ctx: torch.Tensor, v_ctx: torch.Tensor,
                                           k_blk: torch.Tensor, v_blk: torch.Tensor, anchors_dev: torch.Tensor,
                                           out: torch.Tensor, lse: torch.Tensor, d_out: torch.Tensor,
                                           d_q: torch.Tensor, d_k_ctx: torch.Tensor, d_v_ctx: torch.Tensor,
                                           d_k_blk: torch.Tensor, d_v_blk: torch.Tensor, workspace: torch.Tensor,
                                           anchors_host=None, stream=None) -> None:
    """Gradients of dflash_packed_block_attention: from its operands, its out and
    lse and d_out fp32 [N, g, nq, hd] -> d_q, d_k_ctx, d_v_ctx, d_k_blk, d_v_blk,
    shaped and typed as the operands (every element is written)."""
    _on_current_device(q)
    if q.dim() != 4 or k_ctx.dim() != 3 or k_blk.dim() != 4:
        raise ValueError("q [N, g, nq, hd], k_ctx [S, nkv, hd] and k_blk [N, g, nkv, hd] are expected")
    N, g, nq, hd = q.shape
    S, nkv = k_ctx.shape[0], k_blk.shape[2]
    dt = q.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("operands are float32 or bfloat16")
    rows, ctx, blk = N * g * nq * hd, S * nkv * hd, N * g * nkv * hd
    vec = lambda t, n, name: _vector(t, n, dt, q, name)  # noqa: E731
    host = None
    if anchors_host is not None:
        if len(anchors_host) != N:
            raise ValueError("anchors_host must have one entry per block")
        host = (ctypes.c_int32 * N)(*[int(a) for a in anchors_host])
    check(lib().dflash_packed_block_attention_backward(
        vec(q, rows, "q"), vec(k_ctx, ctx, "k_ctx"), vec(v_ctx, ctx, "v_ctx"), vec(k_blk, blk, "k_blk"),
        vec(v_blk, blk, "v_blk"), _vector(anchors_dev, N, torch.int32, q, "anchors_dev"), host, N, g, S, nq, nkv, hd,
        _abi.DTYPE_F32 if dt == torch.float32 else _abi.DTYPE_BF16, _vector(out, rows, torch.float32, q, "out"),
        _vector(lse, N * g * nq, torch.float32, q, "lse"), _vector(d_out, rows, torch.float32, q, "d_out"),
        vec(d_q, rows, "d_q"), vec(d_k_ctx, ctx, "d_k_ctx"), vec(d_v_ctx, ctx, "d_v_ctx"), vec(d_k_blk, blk, "d_k_blk"),
        vec(d_v_blk, blk, "d_v_blk"), *_workspace(workspace, q), _stream_ptr(stream)),
        "dflash_packed_block_attention_backward")


def dflash_packed_attention_status(workspace: torch.Tensor, stream=None) -> int:
    st = ctypes.c_int32(0)
    check(lib().dflash_packed_attention_status(_ptr(workspace), _stream_ptr(stream), ctypes.byref(st)),
          "dflash_packed_attention_status")
    return st.value


def _rows_of(t: torch.Tensor, name: str):
    """(rows, vocab, elements between rows) of a [..., V] tensor whose rows are evenly spaced."""
    if t.dim() == 0 or t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be a float32 or bfloat16 [..., V] tensor")
    V = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // V if V else 0), V, V
    if t.dim() > 2:
        try:
            t = t.view(-1, V)
        except RuntimeError:
            raise ValueError(f"{name}: the rows must be evenly spaced") from None
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: a row must be contiguous")
    return (1, V, V) if t.dim() == 1 else (t.shape[0], V, t.stride(0))


def _vector(t: Optional[torch.Tensor], n: int, dtype: torch.dtype, like: torch.Tensor, name: str) -> Optional[int]:
    """Address of a contiguous tensor of n values on the device of `like` (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} values on {like.device}")
    return t.data_ptr()


def _workspace(t: torch.Tensor, like: torch.Tensor):
    """(address, bytes) of a workspace on the device of `like`."""
    at = _ptr(t)
    if t is not None and t.get_device() != like.get_device():
        raise ValueError(f"the workspace must be on {like.device}")
    return at, 0 if t is None else t.numel() * t.element_size()


def _on_current_device(t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}, which is not the current device")


def dflash_token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor], temperature: float,
                          logprob: Optional[torch.Tensor], entropy: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, top_ids: Optional[torch.Tensor] = None,
                          top_logprobs: Optional[torch.Tensor] = None, stream=None) -> None:
    """Log probabilities of tokens int32 [...] under softmax(logits / T), logits
    fp32 or bf16 [..., V] with evenly spaced rows -> logprob, entropy and lse
    fp32 [...] and the likeliest tokens top_ids int32 / top_logprobs fp32
    [..., k]; what is None is not computed (tokens and logprob go together)."""
    _on_current_device(logits)
    rows, V, stride = _rows_of(logits, "logits")
    k = 0
    if top_ids is not None or top_logprobs is not None:
        if top_ids is None or top_logprobs is None or top_ids.dim() == 0:
            raise ValueError("top_ids and top_logprobs [..., k] go together")
        k = top_ids.shape[-1]
    check(lib().dflash_token_logprobs(
        logits.data_ptr(), _abi.DTYPE_F32 if logits.dtype == torch.float32 else _abi.DTYPE_BF16, stride,
        _vector(tokens, rows, torch.int32, logits, "tokens"), rows, V, float(temperature), k,
        _vector(logprob, rows, torch.float32, logits, "logprob"),
        _vector(entropy, rows, torch.float32, logits, "entropy"), _vector(lse, rows, torch.float32, logits, "lse"),
        _vector(top_ids, rows * k, torch.int32, logits, "top_ids"),
        _vector(top_logprobs, rows * k, torch.float32, logits, "top_logprobs"), _stream_ptr(stream)),
        "dflash_token_logprobs")


def dflash_token_logprobs_backward(logits: torch.Tensor, tokens: Optional[torch.Tensor], temperature: float,
                                   lse: torch.Tensor, d_logits: torch.Tensor,
                                   d_logprob: Optional[torch.Tensor] = None, entropy: Optional[torch.Tensor] = None,
                                   d_entropy: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradient of sum(d_logprob * logprob) + sum(d_entropy * entropy) with
    respect to the logits, in their type, into d_logits [..., V] (which may be
    the logits themselves); lse and entropy are dflash_token_logprobs'."""
    _on_current_device(logits)
    rows, V, stride = _rows_of(logits, "logits")
    d_rows, d_V, d_stride = _rows_of(d_logits, "d_logits")
    if d_rows != rows or d_V != V or d_logits.dtype != logits.dtype or d_logits.device != logits.device:
        raise ValueError("d_logits must have the logits' rows, type and device")
    check(lib().dflash_token_logprobs_backward(
        logits.data_ptr(), _abi.DTYPE_F32 if logits.dtype == torch.float32 else _abi.DTYPE_BF16, stride,
        _vector(tokens, rows, torch.int32, logits, "tokens"), rows, V, float(temperature),
        _vector(lse, rows, torch.float32, logits, "lse"), _vector(entropy, rows, torch.float32, logits, "entropy"),
        _vector(d_logprob, rows, torch.float32, logits, "d_logprob"),
        _vector(d_entropy, rows, torch.float32, logits, "d_entropy"), d_logits.data_ptr(), d_stride,
        _stream_ptr(stream)), "dflash_token_logprobs_backward")


_CLIP_DTYPES = {torch.float32: _abi.DTYPE_F32, torch.bfloat16: _abi.DTYPE_BF16}


def _scratch(nbytes: int, stream=None) -> torch.Tensor:
    """Device scratch of the caching allocator, ordered with the stream the call runs on."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def dflash_clip_workspace() -> torch.Tensor:
    """Device scratch for dflash_clip_grad_norm (a few kilobytes, whatever the tensors)."""
    n = int(lib().dflash_clip_workspace_bytes())
    if n == 0:
        raise ValueError("no current device")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def dflash_clip_grad_norm(grads, max_norm: float, norm: torch.Tensor, out=None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Global 2-norm of the contiguous fp32 / bf16 tensors `grads` into norm
    fp32 [1], and grads scaled by max_norm / norm where it exceeds max_norm:
    in place, or into the tensors `out` of the same types and sizes.  A norm
    that is not finite leaves the gradients as they are; max_norm = inf
    computes the norm alone."""
    _on_current_device(norm)
    n = len(grads)
    tensors = [*grads] if out is None else [*grads, *out]
    dtypes = [t.dtype for t in tensors]
    numels = list(map(torch.Tensor.numel, tensors))
    if n and (not all(map(torch.Tensor.is_contiguous, tensors)) or
              set(map(torch.Tensor.get_device, tensors)) != {norm.get_device()}):
        raise ValueError("gradients must be contiguous tensors on the norm's device")
    if out is not None and (len(out) != n or dtypes[:n] != dtypes[n:] or numels[:n] != numels[n:]):
        raise ValueError("out must have one tensor for each of grads, of its type and size")
    if not _CLIP_DTYPES.keys() >= set(dtypes):
        raise ValueError("gradients must be float32 or bfloat16")
    ptrs = array("Q", map(torch.Tensor.data_ptr, tensors))
    sizes, types = array("q", numels[:n]), array("i", [_CLIP_DTYPES[t] for t in dtypes[:n]])
    at = ptrs.buffer_info()[0]
    if workspace is None:
        workspace = _scratch(int(lib().dflash_clip_workspace_bytes()), stream)
    check(lib().dflash_clip_grad_norm(
        at, None if out is None else at + 8 * n, sizes.buffer_info()[0], types.buffer_info()[0], n, float(max_norm),
        _vector(norm, 1, torch.float32, norm, "norm"), *_workspace(workspace, norm), _stream_ptr(stream)),
        "dflash_clip_grad_norm")


def _dtype_of(t: torch.Tensor, name: str) -> int:
    code = _CLIP_DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return code


def _head_workspace(nbytes, rows: int, dim: int, vocab: int, dtype: torch.dtype) -> torch.Tensor:
    if dtype not in _CLIP_DTYPES:
        raise ValueError("hidden states and head are float32 or bfloat16")
    n = int(nbytes(rows, dim, vocab, _CLIP_DTYPES[dtype]))
    if n == 0:
        raise ValueError("invalid cross-entropy shape")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def dflash_linear_cross_entropy_workspace(rows: int, dim: int, vocab: int, dtype: torch.dtype) -> torch.Tensor:
    """Device scratch for dflash_linear_cross_entropy."""
    return _head_workspace(lib().dflash_linear_cross_entropy_workspace_bytes, rows, dim, vocab, dtype)


def dflash_linear_cross_entropy_backward_workspace(rows: int, dim: int, vocab: int, dtype: torch.dtype) -> torch.Tensor:
    """Device scratch for dflash_linear_cross_entropy_backward (a piece of the logits' gradient, not all of it)."""
    return _head_workspace(lib().dflash_linear_cross_entropy_backward_workspace_bytes, rows, dim, vocab, dtype)


def _head_operands(hidden: torch.Tensor, weight: torch.Tensor):
    """(rows, dim, vocab, elements between rows, dtype code) of hidden [..., D] against the head [V, D]."""
    _on_current_device(hidden)
    rows, D, stride = _rows_of(hidden, "hidden")
    if weight.dim() != 2 or weight.shape[1] != D:
        raise ValueError(f"the head must be [V, {D}]")
    return rows, D, weight.shape[0], stride, _dtype_of(hidden, "hidden")


def dflash_linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, loss: torch.Tensor,
                                lse: torch.Tensor, workspace: torch.Tensor, temperature: float = 1.0,
                                stream=None) -> None:
    """Softmax cross-entropy of hidden [..., D] against the LM head weight [V, D]
    (fp32 or bf16 both) for targets int32 [...], without storing the logits ->
    loss and lse fp32 [...]; a target outside [0, V) gives 0 for both."""
    rows, D, V, stride, dt = _head_operands(hidden, weight)
    check(lib().dflash_linear_cross_entropy(
        hidden.data_ptr(), dt, stride, _vector(weight, V * D, hidden.dtype, hidden, "weight"),
        _vector(targets, rows, torch.int32, hidden, "targets"), rows, D, V, float(temperature),
        _vector(loss, rows, torch.float32, hidden, "loss"), _vector(lse, rows, torch.float32, hidden, "lse"),
        *_workspace(workspace, hidden), _stream_ptr(stream)), "dflash_linear_cross_entropy")


def dflash_linear_cross_entropy_backward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                                         lse: torch.Tensor, d_loss: torch.Tensor, d_hidden: Optional[torch.Tensor],
                                         d_weight: Optional[torch.Tensor], workspace: torch.Tensor,
                                         temperature: float = 1.0, stream=None) -> None:
    """Gradients of sum(d_loss * loss): d_hidden [..., D] (which may be hidden
    itself) and d_weight [V, D], in the operands' type; either may be None.  lse
    is dflash_linear_cross_entropy's."""
    rows, D, V, stride, dt = _head_operands(hidden, weight)
    d_stride = D
    if d_hidden is not None:
        d_rows, d_D, d_stride = _rows_of(d_hidden, "d_hidden")
        if d_rows != rows or d_D != D or d_hidden.dtype != hidden.dtype or d_hidden.device != hidden.device:
            raise ValueError("d_hidden must have the hidden states' rows, type and device")
    check(lib().dflash_linear_cross_entropy_backward(
        hidden.data_ptr(), dt, stride, _vector(weight, V * D, hidden.dtype, hidden, "weight"),
        _vector(targets, rows, torch.int32, hidden, "targets"), rows, D, V, float(temperature),
        _vector(lse, rows, torch.float32, hidden, "lse"), _vector(d_loss, rows, torch.float32, hidden, "d_loss"),
        None if d_hidden is None else d_hidden.data_ptr(), d_stride,
        _vector(d_weight, V * D, hidden.dtype, hidden, "d_weight"), *_workspace(workspace, hidden),
        _stream_ptr(stream)), "dflash_linear_cross_entropy_backward")


def dflash_linear_cross_entropy_status(workspace: torch.Tensor, stream=None) -> int:
    st = ctypes.c_int32(0)
    check(lib().dflash_linear_cross_entropy_status(_ptr(workspace), _stream_ptr(stream), ctypes.byref(st)),
          "dflash_linear_cross_entropy_status")
    return st.value


def _table(t: torch.Tensor, like: torch.Tensor, D: int, name: str):
    """(address, rows) of a contiguous table [V, D] on the device of `like`."""
    if t.dim() != 2 or t.shape[1] != D:
        raise ValueError(f"{name} must be [V, {D}]")
    return _vector(t, t.numel(), t.dtype, like, name), t.shape[0]


def dflash_embed_tokens(table: torch.Tensor, tokens: torch.Tensor, out: torch.Tensor, scale: float = 1.0,
                        stream=None) -> None:
    """out [..., D] = scale * table[tokens], table [V, D] and out fp32 or bf16 each,
    tokens int32 [...]; a token outside [0, V) gives zeros."""
    _on_current_device(out)
    rows, D, stride = _rows_of(out, "out")
    at, V = _table(table, out, D, "table")
    check(lib().dflash_embed_tokens(at, _dtype_of(table, "table"), V, D, _vector(tokens, rows, torch.int32, out, "tokens"),
                                    rows, float(scale), out.data_ptr(), _dtype_of(out, "out"), stride,
                                    _stream_ptr(stream)), "dflash_embed_tokens")


def dflash_embed_tokens_backward_workspace(n_tokens: int, dim: int, vocab: int) -> torch.Tensor:
    """Device scratch for dflash_embed_tokens_backward."""
    n = int(lib().dflash_embed_tokens_backward_workspace_bytes(n_tokens, dim, vocab))
    if n == 0:
        raise ValueError("invalid embedding shape")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def dflash_embed_tokens_backward(d_out: torch.Tensor, tokens: torch.Tensor, d_table: torch.Tensor,
                                 workspace: torch.Tensor, scale: float = 1.0, accumulate: bool = False,
                                 stream=None) -> None:
    """d_table [V, D] = scale * the sum of d_out's rows [..., D] over the tokens
    int32 [...] that are each v (fp32 or bf16 each), or, with accumulate, added
    to what d_table holds."""
    _on_current_device(d_out)
    rows, D, stride = _rows_of(d_out, "d_out")
    at, V = _table(d_table, d_out, D, "d_table")
    check(lib().dflash_embed_tokens_backward(
        d_out.data_ptr(), _dtype_of(d_out, "d_out"), stride, _vector(tokens, rows, torch.int32, d_out, "tokens"), rows, V,
        D, float(scale), at, _dtype_of(d_table, "d_table"), 1 if accumulate else 0, *_workspace(workspace, d_out),
        _stream_ptr(stream)), "dflash_embed_tokens_backward")


class BlockPolicy:
    """Host block-size scheduling policy (dflash_block_policy_*): observe each
    cycle's accepted lengths, choose the next cycle's block size."""

    def __init__(self, candidates, cost_fixed_ms: float, cost_per_row_ms: float, cost_per_request_ms: float = 0.0,
                 decay: float = 0.9, prior_accept: float = 0.8, prior_weight: float = 2.0):
        cfg = _abi.PolicyConfig()
        cand = [int(c) for c in candidates]
        if len(cand) > _abi.POLICY_MAX_CANDIDATES:
            raise ValueError("too many candidates")
        cfg.n_candidates = len(cand)
        for i, c in enumerate(cand):
            cfg.candidates[i] = c
        cfg.cost_fixed_ms, cfg.cost_per_row_ms, cfg.cost_per_request_ms = cost_fixed_ms, cost_per_row_ms, \
            cost_per_request_ms
        cfg.decay, cfg.prior_accept, cfg.prior_weight = decay, prior_accept, prior_weight
        h = ctypes.c_void_p()
        check(lib().dflash_block_policy_create(ctypes.byref(cfg), ctypes.byref(h)), "dflash_block_policy_create")
        self.handle = h
        self.candidates = cand

    def observe(self, block_size: int, taus) -> None:
        arr = (ctypes.c_int32 * len(taus))(*[int(t) for t in taus])
        check(lib().dflash_block_policy_observe(self.handle, int(block_size), arr, len(taus)),
              "dflash_block_policy_observe")

    def choose(self, batch: int):
        g, e = ctypes.c_int32(0), ctypes.c_double(0.0)
        check(lib().dflash_block_policy_choose(self.handle, int(batch), ctypes.byref(g), ctypes.byref(e)),
              "dflash_block_policy_choose")
        return g.value, e.value

    def acceptance(self, n: int):
        out = (ctypes.c_double * n)()
        check(lib().dflash_block_policy_acceptance(self.handle, out, n), "dflash_block_policy_acceptance")
        return list(out)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            lib().dflash_block_policy_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dflash_synthetic_target(drafts: torch.Tensor, match: torch.Tensor, off: torch.Tensor, bonus: torch.Tensor,
                            pattern_idx: torch.Tensor, target_out: torch.Tensor, vocab: int,
                            tau: Optional[torch.Tensor] = None, tau_sum: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """Benchmark utility: the synthetic target's answer for stacked agreement
    patterns (match bool/uint8 [P,B,g-1], off int32 [P,B,g-1], bonus int32
    [P,B]) selected by the device counter pattern_idx (int64 [1])."""
    P, B = bonus.shape
    g = target_out.shape[1]
    m = match.view(torch.uint8) if match.dtype == torch.bool else match
    check(lib().dflash_synthetic_target(_ptr(drafts) if g > 1 else None, _ptr(m), _ptr(off), _ptr(bonus), P,
                                        _ptr(pattern_idx), _ptr(tau), _ptr(tau_sum), B, g, int(vocab),
                                        _ptr(target_out), _stream_ptr(stream)), "dflash_synthetic_target")


def dflash_get_status(model: Model, stream=None) -> int:
    st = ctypes.c_int32(0)
    check(lib().dflash_get_status(model.handle, _stream_ptr(stream), ctypes.byref(st)), "dflash_get_status")
    return st.value


def dflash_clear_status(model: Model, stream=None) -> None:
    check(lib().dflash_clear_status(model.handle, _stream_ptr(stream)), "dflash_clear_status")


def dflash_selftest_wait_timeout(model: Model, budget_cycles: int, stream=None) -> None:
    """Run the bounded-wait self-test: a wait that nothing completes gives up
    after budget_cycles SM cycles and sets the status word to DFLASH_ERR_TIMEOUT."""
    check(lib().dflash_selftest_wait_timeout(model.handle, int(budget_cycles), _stream_ptr(stream)),
          "dflash_selftest_wait_timeout")


def dflash_launch_count() -> int:
    """Kernel launches made by the library in this process."""
    return int(lib().dflash_launch_count())


def dflash_profile_start(model: Model, max_launches: int = 4096) -> None:
    check(lib().dflash_profile_start(model.handle, int(max_launches)), "dflash_profile_start")


def dflash_profile_stop(model: Model, stream=None) -> dict:
    """{stage: (milliseconds, launches)} recorded since dflash_profile_start."""
    n = len(_abi.STAGES)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int32 * n)()
    check(lib().dflash_profile_stop(model.handle, _stream_ptr(stream), ms, cnt, n), "dflash_profile_stop")
    return {name: (float(ms[i]), int(cnt[i])) for i, name in enumerate(_abi.STAGES)}
