"""dflash_packed_block_attention_backward where blocks' gradients differ far in
size: each block's own gradients against the formula in 64 bits, by norm.

Tolerances add the roundings' squares, every one at its largest (errors of
thousands of elements, independent of one another).  With u the rounding of an
operand, of P or of ds (one fp16 plane: 2^-11; hi/lo pairs: 2^-22, and 2^-22 of
each product for the lo lo part that is left out) and f = 2^-39 of the operand's
largest value (half a step of the scaled fp16 at its lower end; of 1 for P):
  dp - D   sum_d dx_d (v_d - o_d) + x_d dv_d, dx and dv = u |.| + f
  ds       P's 2u and f, 2^-20 (e^, lse) and the scores' error, dp - D's error,
           and 2^-36 of the largest norms of d_out's and v's rows: half a step,
           2^-25, of what is held as ds 2^14 2^dp, where 2^-dp <= 8 times them
and the gradient's own rounding (bf16: 2^-8).  fp32 tensors: the tensor cores
truncate by at most 2^-24 on average a step, 96 of which follow one another."""
import math

import pytest
import torch

from test_packed_attention_backward_cpu import backward_reference, forward_reference, operands

pytestmark = pytest.mark.gpu
NAMES = ("d_q", "d_k_ctx", "d_v_ctx", "d_k_blk", "d_v_blk")


def _df():
    import block_diffusion_drafter_dflash_gb300 as df
    return df


def squared_errors(ops, anchors, d_out, want, dtype):
    """Squares of the errors that d_k_ctx, d_v_ctx, d_k_blk and d_v_blk may have, element by element (64-bit operands)."""
    q, kc, vc, kb, vb = ops
    hd, S, nkv = q.shape[3], kc.shape[0], kb.shape[2]
    G, c = q.shape[2] // nkv, 1.0 / math.sqrt(hd)
    rep = lambda t, dim: t.repeat_interleave(G, dim=dim)
    fold = lambda t, dim: t.unflatten(dim, (nkv, G)).sum(dim + 1)
    both = lambda a, ctx, blk: torch.cat([torch.einsum("nihd,shd->nihs", a, rep(ctx, 1)),
                                          torch.einsum("nihd,njhd->nihj", a, rep(blk, 2))], dim=-1)
    top = lambda *t: max(float(a.abs().max()) for a in t if a.numel())
    norm = lambda *t: max(float(a.norm(dim=-1).max()) for a in t if a.numel())
    bf16 = dtype == torch.bfloat16
    u, w = (2.0 ** -11, 0.0) if bf16 else (2.0 ** -22, 2.0 ** -22)      # w: of an operand that bf16 tensors hold exactly
    f = 2.0 ** -39
    err = lambda t, r, m: (r * t) ** 2 + (f * m) ** 2
    out, lse, p = forward_reference(*ops, anchors)
    x, x2, o2 = d_out, d_out ** 2, out ** 2
    m_k, m_v = top(kc, kb), top(vc, vb)
    ex, eq = err(x, u, top(x)), err(q, w, top(q))
    ekc, ekb, evc, evb = err(kc, w, m_k), err(kb, w, m_k), err(vc, w, m_v), err(vb, w, m_v)
    es = c * c * (both(eq, kc ** 2, kb ** 2) + both(q ** 2, ekc, ekb) + w * w * both(q ** 2, kc ** 2, kb ** 2))
    d = (x * out).sum(-1, keepdim=True)
    part = both(x, vc, vb) - d
    ed = (both(ex, vc ** 2, vb ** 2) - 2 * both(ex * out, vc, vb) + (ex * o2).sum(-1, keepdim=True) + both(x2, evc, evb)
          + w * w * both(x2, vc ** 2, vb ** 2) + (2.0 ** -22 * (x * out).abs().sum(-1, keepdim=True)) ** 2)
    ds = p * part
    ep = p ** 2 * (es + 2.0 ** -40 + (2.0 ** -23 * lse[..., None]) ** 2)
    eds = (ep + 2 * (u * p) ** 2 + f * f) * part ** 2 + p ** 2 * ed + (2.0 ** -36 * norm(x) * norm(vc, vb)) ** 2
    tk = eds + (w * ds) ** 2
    q2 = q ** 2
    e = [fold(torch.einsum("nihs,nihd->shd", tk[..., :S], q2), 1) * c * c,
         fold(torch.einsum("nihs,nihd->shd", (ep + (u * p) ** 2 + f * f)[..., :S], x2)
              + torch.einsum("nihs,nihd->shd", (p ** 2)[..., :S], ex), 1),
         fold(torch.einsum("nihj,nihd->njhd", tk[..., S:], q2), 2) * c * c,
         fold(torch.einsum("nihj,nihd->njhd", (ep + (u * p) ** 2 + f * f)[..., S:], x2)
              + torch.einsum("nihj,nihd->njhd", (p ** 2)[..., S:], ex), 2)]
    for a, ds_q in ((0, torch.einsum("nihs,nihd->shd", (ds ** 2)[..., :S], eq)),
                    (2, torch.einsum("nihj,nihd->njhd", (ds ** 2)[..., S:], eq))):
        e[a] = e[a] + fold(ds_q, 1 if a == 0 else 2) * c * c
    own = 2.0 ** -8 if bf16 else 96 * 2.0 ** -24
    return [a + (own * r) ** 2 for a, r in zip(e, want[1:])]


def gradients(ops, anchors, d_out, dtype):
    """The library's gradients from the 64-bit forward's out and lse, and what they should be."""
    df = _df()
    N, g, nq, hd = ops[0].shape
    S, nkv = ops[1].shape[0], ops[3].shape[2]
    ref = [t.double() for t in ops]
    out, lse, _ = forward_reference(*ref, anchors)
    got = [torch.full_like(t, math.nan) for t in ops]
    ws = df.dflash_packed_attention_backward_workspace(N, g, S, nq, nkv, hd, dtype)
    df.dflash_packed_block_attention_backward(*ops, torch.tensor(anchors, dtype=torch.int32, device="cuda"),
                                              out.float().contiguous(), lse.float().contiguous(), d_out, *got, ws)
    assert df.dflash_packed_attention_status(ws) == 0
    want = backward_reference(*ref, anchors, d_out.double())
    return ref, [t.double() for t in got], want


def check(got, want, e2, blocks, keys, what):
    """Errors of some blocks, each by its own norm, and of some context keys together."""
    worst = 0.0
    for i, name in ((2, "d_k_blk"), (3, "d_v_blk")):
        for n in blocks:
            err, tol = float((got[1 + i][n] - want[1 + i][n]).norm()), float(e2[i][n].sum().sqrt())
            worst = max(worst, err / tol)
            assert err <= tol, f"{what} {name}[{n}]: {err / float(want[1 + i][n].norm()):.2e} of its norm"
    for i, name in ((0, "d_k_ctx"), (1, "d_v_ctx")):
        err, tol = float((got[1 + i][keys] - want[1 + i][keys]).norm()), float(e2[i][keys].sum().sqrt())
        worst = max(worst, err / tol)
        assert err <= tol, f"{what} {name}: {err / float(want[1 + i][keys].norm()):.2e} of its norm"
    print(f"{what}: worst {worst:.2f} of its tolerance")


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_blocks_far_smaller_than_others(dtype, hd):
    """Half of the blocks, and they alone see the later half of the context, have a d_out 2^-k of the others'."""
    S, N, g, nq, nkv = 300, 20, 6, 4, 2
    anchors = [(7 * n) % 150 for n in range(N // 2)] + [151 + (13 * n) % 150 for n in range(N // 2)]
    ops = operands(S, N, g, nq, nkv, hd, dtype, 12, "cuda")
    base = torch.randn(ops[0].shape, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    for k in (0, 8, 12, 16, 20):
        d_out = base.clone()
        d_out[N // 2:] *= 2.0 ** -k
        ref, got, want = gradients(ops, anchors, d_out, dtype)
        e2 = squared_errors(ref, anchors, d_out.double(), want, dtype)
        check(got, want, e2, range(N // 2, N), slice(150, S), f"2^-{k}")
        check(got, want, e2, range(N // 2), slice(0, 150), f"2^-{k}, the others")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_value_row_far_larger(dtype):
    """One row of v is 2^8 of the others and seen by the first half of the blocks; the rest have a d_out of 2^-k."""
    S, N, g, nq, nkv, hd = 300, 20, 6, 4, 2, 128
    anchors = [(7 * n) % 150 for n in range(N // 2)] + [151 + (13 * n) % 150 for n in range(N // 2)]
    ops = operands(S, N, g, nq, nkv, hd, dtype, 12, "cuda")
    ops[4][2, 3] *= 256                                   # an own value of the third block
    base = torch.randn(ops[0].shape, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    for k in (0, 8, 12):
        d_out = base.clone()
        d_out[N // 2:] *= 2.0 ** -k
        ref, got, want = gradients(ops, anchors, d_out, dtype)
        e2 = squared_errors(ref, anchors, d_out.double(), want, dtype)
        check(got, want, e2, range(N // 2, N), slice(150, S), f"2^-{k}")


@pytest.mark.parametrize("S,N,g,nq,nkv,hd,larger", [(300, 20, 6, 4, 2, 64, 1.0), (1000, 96, 7, 4, 2, 64, 1.0),
                                                    (3000, 200, 16, 8, 2, 128, 1.0), (1000, 60, 16, 8, 2, 128, 3.0)])
def test_fp32_forward_and_gradient_together(S, N, g, nq, nkv, hd, larger):
    """fp32 gradients from the library's own out and lse, by norm.  The forward's operands are bf16 hi/lo pairs: each
    product of a score is off by 2^-18 for either operand and for the lo lo part, independently, the score by e =
    sqrt(3) * 2^-18 of the root of its terms' squares (their mean over the rows, weighted by P).  lse is off by e at
    most, P by that factor, out by twice that and v's 2^-18, and ds by what P and D are off."""
    df = _df()
    anchors = torch.randint(0, S + 1, (N,), generator=torch.Generator().manual_seed(13)).tolist()
    ops = operands(S, N, g, nq, nkv, hd, torch.float32, 14, "cuda")
    ops = (ops[0] * larger, *ops[1:])
    d_out = torch.randn(ops[0].shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    a = torch.tensor(anchors, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(ops[0], math.nan), torch.full((N, g, nq), math.nan, device="cuda")
    df.dflash_packed_block_attention(*ops, a, out, df.dflash_packed_attention_workspace(N, g, S, nq, nkv, hd), lse=lse)
    got = [torch.full_like(t, math.nan) for t in ops]
    ws = df.dflash_packed_attention_backward_workspace(N, g, S, nq, nkv, hd, torch.float32)
    df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out, *got, ws)
    assert df.dflash_packed_attention_status(ws) == 0
    ref = [t.double() for t in ops]
    q2, (k2, b2) = ref[0].square(), (t.square().repeat_interleave(nq // nkv, dim=-2) for t in (ref[1], ref[3]))
    p = forward_reference(*ref, anchors)[2]
    terms = (p[..., :S] * torch.einsum("nihd,shd->nihs", q2, k2)).sum() + (p[..., S:] * torch.einsum("nihd,njhd->nihj", q2, b2)).sum()
    e = math.sqrt(3.0) * 2.0 ** -18 * math.sqrt(float(terms) / (N * g * nq) / hd)
    for name, x, w in zip(NAMES, got, backward_reference(*ref, anchors, d_out.double())):
        err = float((x.double() - w).norm() / w.norm())
        print(f"{name}: rel {err:.2e} (bound {3 * e + 2.0 ** -18 + 96 * 2.0 ** -24 + 2.0 ** -20:.1e})")
        assert err <= 3 * e + 2.0 ** -18 + 96 * 2.0 ** -24 + 2.0 ** -20, name
