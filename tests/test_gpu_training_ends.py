"""A training step from its tokens to its clipped gradient, as a drafter's trainer with
a tied table calls the operators: tokens embedded, packed attention, the
cross-entropy at the LM head without logits (position-weighted, the anchors carry no
loss: paper section 4.2, eq. 1), its gradient, the attention's gradient, the
embedding's gradient added onto the head's, clipping.  Against automatic
differentiation in 64 bits, at the hidden states that the step rounded to bf16.

Tolerance, in norms: a rounding to bf16 perturbs a tensor by at most 2^-8 of its norm.
The head's part: G and the stored gradient, two.  The table's part through the
attention: G, d_hidden, d_q (and three of 2^-11 inside, d_out, P and ds), three.  Their
sum is rounded once more, and once when clipped."""
import math

import pytest
import torch

from test_packed_attention_backward_cpu import forward_reference

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_a_training_step_with_a_tied_table():
    import block_diffusion_drafter_dflash_gb300 as df
    S, N, b, nq, nkv, hd, V, gamma, scale, max_norm = 300, 24, 8, 8, 2, 64, 1003, 4.0, 6.0, 0.25
    D = nq * hd
    g = torch.Generator(device="cuda").manual_seed(41)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    table = (rnd(V, D) / math.sqrt(D) * 2).to(BF16)
    kc, vc, kb, vb = rnd(S, nkv, hd).to(BF16), rnd(S, nkv, hd).to(BF16), rnd(N, b, nkv, hd).to(BF16), rnd(N, b, nkv, hd).to(BF16)
    anchors = torch.randint(0, S + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    tokens = torch.full((N, b), V - 1, dtype=torch.int32, device="cuda")            # the mask token
    tokens[:, 0] = torch.randint(0, V - 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    targets = torch.randint(0, V, (N, b), generator=g, device="cuda", dtype=torch.int32)
    targets[:, 0] = -1
    w = torch.exp(-(torch.arange(b, device="cuda") - 1).clamp_min(0) / gamma).expand(N, b).contiguous()

    # the library's operators
    new = lambda *s, dtype=BF16: torch.full(s, math.nan, dtype=dtype, device="cuda")  # noqa: E731
    F32 = torch.float32
    q = new(N, b, nq, hd)
    df.dflash_embed_tokens(table, tokens, q.view(N, b, D), scale=scale)
    out, alse = new(N, b, nq, hd, dtype=F32), new(N, b, nq, dtype=F32)
    df.dflash_packed_block_attention(q, kc, vc, kb, vb, anchors, out, df.dflash_packed_attention_workspace(N, b, S, nq, nkv, hd),
                                     lse=alse)
    hidden = out.view(N, b, D).to(BF16)
    loss, lse = new(N, b, dtype=F32), new(N, b, dtype=F32)
    df.dflash_linear_cross_entropy(hidden, table, targets, loss, lse,
                                   df.dflash_linear_cross_entropy_workspace(N * b, D, V, BF16))
    total = (w * loss).sum()
    d_hidden, d_table = new(N, b, D), new(V, D)
    ws = df.dflash_linear_cross_entropy_backward_workspace(N * b, D, V, BF16)
    df.dflash_linear_cross_entropy_backward(hidden, table, targets, lse, w, d_hidden, d_table, ws)
    grads = [torch.empty_like(t) for t in (q, kc, vc, kb, vb)]
    aws = df.dflash_packed_attention_backward_workspace(N, b, S, nq, nkv, hd, BF16)
    df.dflash_packed_block_attention_backward(q, kc, vc, kb, vb, anchors, out, alse, d_hidden.float().view(N, b, nq, hd),
                                              *grads, aws)
    df.dflash_embed_tokens_backward(grads[0].view(N, b, D), tokens, d_table,
                                    df.dflash_embed_tokens_backward_workspace(N * b, D, V), scale=scale, accumulate=True)
    norm = torch.empty(1, device="cuda")
    df.dflash_clip_grad_norm([d_table], max_norm, norm)
    assert df.dflash_linear_cross_entropy_status(ws) == 0 and df.dflash_packed_attention_status(aws) == 0

    # the definition in 64 bits; the table as input and as head apart
    emb, head = (table.double().requires_grad_() for _ in range(2))
    q64 = (emb[tokens.long()] * scale).view(N, b, nq, hd)
    assert torch.equal(q, q64.detach().to(BF16))
    q64 = q64 + (q.double() - q64).detach()                      # at the rounded queries and hidden states
    o64 = forward_reference(q64, *(t.double() for t in (kc, vc, kb, vb)), anchors)[0].reshape(N, b, D)
    h64 = o64 + (hidden.double() - o64).detach()
    logp = torch.log_softmax(h64 @ head.t(), dim=-1)
    picked = logp.gather(-1, targets.clamp_min(0).long()[..., None])[..., 0]
    total64 = -(w.double() * torch.where(targets >= 0, picked, 0.0)).sum()
    d_emb, d_head = torch.autograd.grad(total64, (emb, head))
    want = d_emb + d_head
    assert float(d_emb.norm()) > 0.05 * float(want.norm()) and float(d_head.norm()) > 0.05 * float(want.norm())
    assert abs(float(total) - float(total64.detach())) <= 1e-5 * abs(float(total64.detach()))
    u = 2.0 ** -8
    tol = 2 * u * float(d_head.norm()) + (3 * u + 3 * 2.0 ** -11) * float(d_emb.norm()) + u * float(want.norm())
    assert float(want.norm()) > 2 * max_norm
    assert abs(float(norm) - float(want.norm())) <= tol
    clipped = want * (max_norm / want.norm())
    off = float((d_table.double() - clipped).norm())
    # (the norm's own error scales the clipped gradient by at most tol / |want| more)
    limit = 2 * tol * max_norm / float(want.norm()) + u * max_norm
    print(f"off {off / max_norm:.2e} of the norm, limit {limit / max_norm:.2e}")
    assert off <= limit
