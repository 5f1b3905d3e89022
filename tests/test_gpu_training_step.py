"""One training step's operators together, as a drafter's trainer calls them:
packed attention with its lse, a projection to the vocabulary, the
position-weighted log-probability loss (paper section 4.2, eq. 1:
w_k = exp(-(k - 1) / gamma), the anchor has no loss), its gradient, the
attention's gradient, and clipping by the global norm.  Against automatic
differentiation of the definition in 64 bits.

Tolerance: the bf16 gradients round by at most 2^-8 of a value, twice (the
gradient and its clipped value), and their products' operands by 2^-11 three
times (d_out, P, ds), errors of independent sign in sums of terms of independent
sign: 2 * 2^-8 + 3 * 2^-11 of the norm at most, and fp32 sums far below."""
import math

import pytest
import torch

from test_packed_attention_backward_cpu import forward_reference, operands

pytestmark = pytest.mark.gpu


def test_a_training_step():
    import block_diffusion_drafter_dflash_gb300 as df
    S, N, g, nq, nkv, hd, V, gamma, temp, max_norm = 300, 24, 8, 8, 2, 64, 1003, 4.0, 1.0, 0.25
    gen = torch.Generator(device="cuda").manual_seed(31)
    ops = operands(S, N, g, nq, nkv, hd, torch.bfloat16, 30, "cuda")
    head = torch.randn((V, nq * hd), generator=gen, device="cuda") / math.sqrt(nq * hd) * 4
    anchors = torch.randint(0, S + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
    tokens = torch.randint(0, V, (N, g), generator=gen, device="cuda", dtype=torch.int32)
    tokens[:, 0] = -1                                        # the anchor's position
    w = torch.exp(-(torch.arange(g, device="cuda") - 1).clamp_min(0) / gamma).expand(N, g).contiguous()

    # the library's operators
    new = lambda *s, dtype=torch.float32: torch.full(s, math.nan, dtype=dtype, device="cuda")
    out, alse = new(N, g, nq, hd), new(N, g, nq)
    df.dflash_packed_block_attention(*ops, anchors, out, df.dflash_packed_attention_workspace(N, g, S, nq, nkv, hd), lse=alse)
    logits = (out.view(N, g, nq * hd) @ head.t()).contiguous()
    lp, ent, lse = new(N, g), new(N, g), new(N, g)
    top_ids, top = torch.empty((N, g, 4), dtype=torch.int32, device="cuda"), new(N, g, 4)
    df.dflash_token_logprobs(logits, tokens, temp, lp, entropy=ent, lse=lse, top_ids=top_ids, top_logprobs=top)
    assert torch.equal(top_ids[..., 0].long(), logits.argmax(-1))
    loss = -(w * lp).sum()
    df.dflash_token_logprobs_backward(logits, tokens, temp, lse, logits, d_logprob=-w)      # in place
    d_out = (logits @ head).view(N, g, nq, hd)
    grads = [new(*t.shape, dtype=t.dtype) for t in ops]
    ws = df.dflash_packed_attention_backward_workspace(N, g, S, nq, nkv, hd, torch.bfloat16)
    df.dflash_packed_block_attention_backward(*ops, anchors, out, alse, d_out, *grads, ws)
    norm = torch.empty(1, device="cuda")
    df.dflash_clip_grad_norm(grads, max_norm, norm)
    assert df.dflash_packed_attention_status(ws) == 0

    # the definition in 64 bits
    leaf = [t.double().requires_grad_() for t in ops]
    o64 = forward_reference(*leaf, anchors)[0]
    logp = torch.log_softmax(o64.reshape(N, g, nq * hd) @ head.double().t() / temp, dim=-1)
    picked = logp.gather(-1, tokens.clamp_min(0).long()[..., None])[..., 0]
    loss64 = -(w.double() * torch.where(tokens >= 0, picked, 0.0)).sum()
    want = torch.autograd.grad(loss64, leaf)
    norm64 = torch.sqrt(sum(t.square().sum() for t in want))
    assert float(norm64) > 2 * max_norm
    assert abs(float(loss) - float(loss64.detach())) <= 1e-5 * abs(float(loss64.detach()))
    tol = 2 * 2.0 ** -8 + 3 * 2.0 ** -11
    assert abs(float(norm) - float(norm64)) <= tol * float(norm64)
    for name, got, ref in zip(("d_q", "d_k_ctx", "d_v_ctx", "d_k_blk", "d_v_blk"), grads, want):
        ref = ref * (max_norm / norm64)
        rel = float((got.double() - ref).norm() / ref.norm())
        print(f"{name}: rel {rel:.2e}")
        assert rel <= tol, name
