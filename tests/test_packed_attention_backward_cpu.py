"""The packed attention gradient's formula against differences of the forward's
definition, and the entry points' refusals, which need no GPU."""
import ctypes
import math

import pytest
import torch

from test_abi_cpu import L  # noqa: F401  (the built library)


def forward_reference(q, kc, vc, kb, vb, anchors):
    """(out, lse, P over [context | own block]) in the operands' precision, by the mask's definition."""
    N, g, nq, hd = q.shape
    S, nkv = kc.shape[0], kb.shape[2]
    G = nq // nkv
    rep = lambda x, dim: x.repeat_interleave(G, dim=dim)
    seen = torch.arange(S, device=q.device)[None, :] < torch.as_tensor(anchors, device=q.device)[:, None]
    sc = torch.einsum("nihd,shd->nihs", q, rep(kc, 1)) / math.sqrt(hd)
    sc = torch.where(seen[:, None, None, :], sc, -math.inf)
    sb = torch.einsum("nihd,njhd->nihj", q, rep(kb, 2)) / math.sqrt(hd)
    s = torch.cat([sc, sb], dim=-1)
    lse = torch.logsumexp(s, dim=-1)
    p = (s - lse[..., None]).exp()
    out = torch.einsum("nihs,shd->nihd", p[..., :S], rep(vc, 1)) + torch.einsum("nihj,njhd->nihd", p[..., S:], rep(vb, 2))
    return out, lse, p


def backward_reference(q, kc, vc, kb, vb, anchors, d_out):
    """(d_q, d_k_ctx, d_v_ctx, d_k_blk, d_v_blk) by the formula."""
    N, g, nq, hd = q.shape
    S, nkv = kc.shape[0], kb.shape[2]
    G, c = nq // nkv, 1.0 / math.sqrt(hd)
    rep = lambda x, dim: x.repeat_interleave(G, dim=dim)
    fold = lambda x, dim: x.unflatten(dim, (nkv, G)).sum(dim + 1)       # the q heads of a kv head
    out, _, p = forward_reference(q, kc, vc, kb, vb, anchors)
    dp = torch.cat([torch.einsum("nihd,shd->nihs", d_out, rep(vc, 1)),
                    torch.einsum("nihd,njhd->nihj", d_out, rep(vb, 2))], dim=-1)
    ds = p * (dp - (d_out * out).sum(-1, keepdim=True)) * c
    dsc, dsb, pc, pb = ds[..., :S], ds[..., S:], p[..., :S], p[..., S:]
    d_q = torch.einsum("nihs,shd->nihd", dsc, rep(kc, 1)) + torch.einsum("nihj,njhd->nihd", dsb, rep(kb, 2))
    return (d_q, fold(torch.einsum("nihs,nihd->shd", dsc, q), 1), fold(torch.einsum("nihs,nihd->shd", pc, d_out), 1),
            fold(torch.einsum("nihj,nihd->njhd", dsb, q), 2), fold(torch.einsum("nihj,nihd->njhd", pb, d_out), 2))


def operands(S, N, g, nq, nkv, hd, dtype, seed, device="cpu"):
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device=device).to(dtype)
    return r(N, g, nq, hd), r(S, nkv, hd), r(S, nkv, hd), r(N, g, nkv, hd), r(N, g, nkv, hd)


@pytest.mark.parametrize("S,anchors,g,nq,nkv,hd", [(5, [0, 5, 2], 3, 4, 2, 8), (0, [0], 2, 2, 2, 4), (4, [3, 3], 1, 3, 1, 4)])
def test_formula_matches_differences(S, anchors, g, nq, nkv, hd):
    ops = operands(S, len(anchors), g, nq, nkv, hd, torch.float64, 1)
    w = torch.randn(ops[0].shape, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    grads = backward_reference(*ops, anchors, w)
    f = lambda o: float((forward_reference(*o, anchors)[0] * w).sum())
    gen, eps = torch.Generator().manual_seed(3), 1e-6
    for i, grad in enumerate(grads):
        assert grad.shape == ops[i].shape
        for _ in range(6 if grad.numel() else 0):
            e = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
            up = [o + eps * e if j == i else o for j, o in enumerate(ops)]
            down = [o - eps * e if j == i else o for j, o in enumerate(ops)]
            # central differences: O(eps^2) truncation and 2^-52 |f| / eps rounding, both under 1e-7 here
            assert abs((f(up) - f(down)) / (2 * eps) - float((grad * e).sum())) < 1e-7


P = 1 << 20


def _call(L, anchors=None, n=2, block=4, seq=8, nq=4, nkv=2, hd=64, dtype=1, ws=P, null=(), at={}):
    names = ["q", "k_ctx", "v_ctx", "k_blk", "v_blk", "anchors_dev", "out", "lse", "d_out", "d_q", "d_k_ctx", "d_v_ctx",
             "d_k_blk", "d_v_blk"]
    a = {k: None if k in null else at.get(k, P) for k in names}
    host = None if anchors is None else (ctypes.c_int32 * n)(*anchors)
    return L.dflash_packed_block_attention_backward(
        *[a[k] for k in names[:6]], host, n, block, seq, nq, nkv, hd, dtype, *[a[k] for k in names[6:]], ws, 1 << 40, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -2), (dict(block=0), -2), (dict(block=33), -2), (dict(seq=-1), -2), (dict(hd=96), -2), (dict(nq=3), -2),
    (dict(nkv=0), -2), (dict(n=40000), -2), (dict(dtype=3), -1), (dict(ws=None), -1), (dict(ws=P + 16), -1),
    (dict(n=8000, block=32, nq=8192, nkv=8, seq=0), -2),       # 2000 tiles of 128 rows, 8192 heads, two planes: 2^31 rows
    (dict(anchors=[0, 9]), -1), (dict(anchors=[-1, 3]), -1),
    *[(dict(null=(k,)), -1) for k in ("q", "k_ctx", "v_ctx", "k_blk", "v_blk", "anchors_dev", "out", "lse", "d_out", "d_q",
                                      "d_k_ctx", "d_v_ctx", "d_k_blk", "d_v_blk")],
    *[(dict(at={k: P + 8}), -1) for k in ("d_q", "d_k_ctx", "d_v_ctx", "d_k_blk", "d_v_blk")],
    *[(dict(at={k: P + 1}), -1) for k in ("q", "k_ctx", "v_ctx", "k_blk", "v_blk")],
])
def test_refusals(L, kw, code):  # noqa: F811
    assert _call(L, **kw) == code
    assert len(L.dflash_last_error()) > 0


def test_lse_is_needed_by_its_entry_point(L):  # noqa: F811
    assert L.dflash_packed_block_attention_lse(P, P, P, P, P, P, None, 2, 4, 8, 4, 2, 64, 1, P, None, P, 1 << 30, None) == -1


def test_workspace_of_an_invalid_shape_is_zero(L):  # noqa: F811
    assert L.dflash_packed_attention_backward_workspace_bytes(2, 4, 8, 4, 2, 96, 1) == 0
    assert L.dflash_packed_attention_backward_workspace_bytes(2, 4, 8, 4, 2, 64, 9) == 0
