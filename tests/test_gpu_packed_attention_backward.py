"""dflash_packed_block_attention_backward (and the forward's lse) against the
formula in 64 bits, element by element.

Tolerances follow the roundings.  Operands, P and ds enter their products as
scaled fp16: with u the rounding of one of them (bf16 tensors: 2^-11, q, k and v
being exact; fp32 tensors as hi/lo pairs: 3 * 2^-22 with the lo lo product that
is left out), a score carries n_s |q| |k| / sqrt(hd), P the factor e^ of that and
2^-20 (e^, lse), dp = dO v the error u |dO| |v|, and ds = P (dp - D)
  E_ds = E_P |dp - D| + P (E_dp + hd 2^-23 |dO| |O|) + u |ds|.
dv sums (E_P + 2 u P) |dO|, dq sums E_ds |k|, dk sums E_ds |q| (and u of the other
operand for fp32), each with n 2^-24 of its sum of absolute terms for n
additions, and the gradient's own rounding (bf16: 2^-8).  Scaled values under
fp16's normal range are good to 2^-38 of their largest: absolute values are
taken with 2^-16 of the largest added, P with 2^-16, ds with 2^-16 of the norms'
bound."""
import math

import pytest
import torch

from test_packed_attention_backward_cpu import backward_reference, forward_reference, operands

pytestmark = pytest.mark.gpu


def _df():
    import block_diffusion_drafter_dflash_gb300 as df
    return df


def tolerances(ops, anchors, d_out, grads, dtype):
    q, kc, vc, kb, vb = ops
    N, g, nq, hd = q.shape
    S, nkv = kc.shape[0], kb.shape[2]
    G, c = nq // nkv, 1.0 / math.sqrt(hd)
    rep = lambda x, dim: x.repeat_interleave(G, dim=dim)
    fold = lambda x, dim: x.unflatten(dim, (nkv, G)).sum(dim + 1)
    both = lambda x, ctx, blk: torch.cat([torch.einsum("nihd,shd->nihs", x, rep(ctx, 1)),
                                          torch.einsum("nihd,njhd->nihj", x, rep(blk, 2))], dim=-1)
    bf16 = dtype == torch.bfloat16
    u = 2.0 ** -11 if bf16 else 3 * 2.0 ** -22
    n_s = hd * 2.0 ** -24 + (0 if bf16 else u)
    w = 0 if bf16 else u                      # of an operand that is exact in bf16
    out, lse, p = forward_reference(*ops, anchors)
    floor = 2.0 ** -16
    size = lambda *t: max([float(x.abs().max()) for x in t if x.numel()])
    mag = lambda t, top: t.abs() + floor * top
    norm = lambda *t: max([float(x.norm(dim=-1).max()) for x in t if x.numel()])
    a = [mag(t, m) for t, m in ((kc, size(kc, kb)), (vc, size(vc, vb)), (kb, size(kc, kb)), (vb, size(vc, vb)))]
    aq, x = mag(q, size(q)), mag(d_out, size(d_out))
    e_p = p * (n_s * c * both(aq, a[0], a[2]) + 2.0 ** -20 + 2.0 ** -23 * lse.abs()[..., None])
    adov = both(x, a[1], a[3])
    d = (d_out * out).sum(-1, keepdim=True)
    dp = both(d_out, vc, vb)
    ds = p * (dp - d)
    e_dp = (u + hd * 2.0 ** -24) * adov
    e_ds = e_p * (dp - d).abs() + p * (e_dp + hd * 2.0 ** -23 * (d_out * out).abs().sum(-1, keepdim=True)) + u * mag(ds, norm(d_out) * norm(vc, vb))
    e_dv = e_p + 2 * u * (p + floor)
    n_q, n_k = (S + g) * 2.0 ** -24, N * g * G * 2.0 ** -24
    ads = (e_ds + (w + n_q) * ds.abs()) * c, (e_ds + (w + n_k) * ds.abs()) * c
    adv = e_dv + n_k * p
    t_q = torch.einsum("nihs,shd->nihd", ads[0][..., :S], rep(a[0], 1)) + torch.einsum("nihj,njhd->nihd", ads[0][..., S:],
                                                                                       rep(a[2], 2))
    tol = (t_q, fold(torch.einsum("nihs,nihd->shd", ads[1][..., :S], aq), 1),
           fold(torch.einsum("nihs,nihd->shd", adv[..., :S], x), 1),
           fold(torch.einsum("nihj,nihd->njhd", ads[1][..., S:], aq), 2),
           fold(torch.einsum("nihj,nihd->njhd", adv[..., S:], x), 2))
    own = 2.0 ** -8 if bf16 else 2.0 ** -24
    return [t * 1.02 + own * r.abs() * 1.01 + 1e-30 for t, r in zip(tol, grads)]


def run(ops, anchors, d_out, host=True, stream=None, ws=None):
    """lse and out by the forward, then the gradients; outputs start as NaN."""
    df = _df()
    q, kc, vc, kb, vb = ops
    N, g, nq, hd = q.shape
    S, nkv = kc.shape[0], kb.shape[2]
    a = torch.tensor(anchors, dtype=torch.int32, device="cuda")
    out, lse = torch.full(q.shape, math.nan, device="cuda"), torch.full((N, g, nq), math.nan, device="cuda")
    df.dflash_packed_block_attention(q, kc, vc, kb, vb, a, out, df.dflash_packed_attention_workspace(N, g, S, nq, nkv, hd),
                                     lse=lse)
    grads = [torch.full_like(t, math.nan) for t in ops]
    ws = df.dflash_packed_attention_backward_workspace(N, g, S, nq, nkv, hd, q.dtype) if ws is None else ws
    if stream is not None:
        torch.cuda.synchronize()
    df.dflash_packed_block_attention_backward(q, kc, vc, kb, vb, a, out, lse, d_out, *grads, ws,
                                              anchors_host=anchors if host else None, stream=stream)
    return out, lse, grads, ws


def anchors_of(N, S, seed):
    return torch.randint(0, S + 1, (N,), generator=torch.Generator().manual_seed(seed)).tolist()


CASES = [
    (0, [0, 0, 0], 8, 8, 2, 64),                       # no context: each block sees only itself
    (1, [1], 1, 1, 1, 64),                             # one row
    (200, [0, 200, 77, 128, 129, 5], 4, 4, 2, 64),     # anchors at both ends and at tile boundaries
    (300, [150, 10, 299, 256, 31], 16, 32, 8, 128),    # 8B-shaped heads, ragged context tiles
    (257, anchors_of(40, 257, 1), 10, 6, 2, 128),      # blocks that do not fill a row tile
    (1000, anchors_of(70, 1000, 2), 7, 4, 4, 64),
    (640, [640] * 12, 32, 8, 1, 128),                  # every block sees everything, one kv head
    (130, anchors_of(150, 130, 3), 1, 2, 2, 64),       # blocks of one row
    (384, [0] * 9, 5, 5, 1, 128),                      # nobody sees the context: its gradients are 0
    (700, anchors_of(33, 700, 4), 31, 3, 1, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,anchors,g,nq,nkv,hd", CASES)
def test_gradients_match_the_formula(S, anchors, g, nq, nkv, hd, dtype):
    N = len(anchors)
    ops = operands(S, N, g, nq, nkv, hd, dtype, S + N, "cuda")
    d_out = torch.randn(ops[0].shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    out, lse, grads, ws = run(ops, anchors, d_out)
    assert _df().dflash_packed_attention_status(ws) == 0
    ref = [t.double() for t in ops]
    o64, l64, _ = forward_reference(*ref, anchors)
    # the forward's scores carry hi/lo operands: 3 * 2^-16 of |q| |k| / sqrt(hd), and its sums a few 2^-20
    size = (ref[0].norm(dim=-1).max() * max([t.norm(dim=-1).max() for t in (ref[1], ref[3]) if t.numel()])) / math.sqrt(hd)
    assert float((lse.double() - l64).abs().max()) <= 3 * 2.0 ** -16 * float(size) + 2.0 ** -18
    want = backward_reference(*ref, anchors, d_out.double())
    tol = tolerances(ref, anchors, d_out.double(), want, dtype)
    for name, got, w, t in zip(("d_q", "d_k_ctx", "d_v_ctx", "d_k_blk", "d_v_blk"), grads, want, tol):
        if not got.numel():
            continue
        err = (got.double() - w).abs()
        worst = float((err / t).max())
        print(f"{name}: rel {float(err.norm() / w.norm().clamp_min(1e-30)):.2e}, worst {worst:.2f} of its tolerance")
        assert worst <= 1.0, name
    if max(anchors) == 0 and S:
        assert bool((grads[1] == 0).all()) and bool((grads[2] == 0).all())


def test_same_bits_every_time_other_stream_and_graph():
    """The same call gives the same bits: again, on another stream, and captured and replayed over new operands."""
    df = _df()
    S, N, g, nq, nkv, hd = 500, 60, 8, 8, 2, 128
    anchors = anchors_of(N, S, 9)
    ops = operands(S, N, g, nq, nkv, hd, torch.bfloat16, 1, "cuda")
    d_out = torch.randn(ops[0].shape, device="cuda")
    out, lse, first, ws = run(ops, anchors, d_out)
    for stream in (None, torch.cuda.Stream()):
        again = run(ops, anchors, d_out, host=False, stream=stream)[2]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    a = torch.tensor(anchors, dtype=torch.int32, device="cuda")
    fws = df.dflash_packed_attention_workspace(N, g, S, nq, nkv, hd)
    grads = [torch.full_like(t, math.nan) for t in ops]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df.dflash_packed_block_attention(*ops, a, out, fws, lse=lse)
        df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out, *grads, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, grads))
    new = operands(S, N, g, nq, nkv, hd, torch.bfloat16, 2, "cuda")
    for o, n in zip(ops, new):
        o.copy_(n)
    a.copy_(torch.tensor(anchors[::-1], dtype=torch.int32))
    graph.replay()
    other = run(new, anchors[::-1], d_out)[2]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(other, grads)) and not torch.equal(other[0], first[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_operands_far_from_one(dtype):
    """Operands and gradients of any size (their squares outside fp32): the gradients scale exactly with them."""
    S, N, g, nq, nkv, hd = 200, 20, 6, 4, 2, 64
    anchors = anchors_of(N, S, 8)
    ops = operands(S, N, g, nq, nkv, hd, dtype, 12, "cuda")
    d_out = torch.randn(ops[0].shape, device="cuda")
    want = run(ops, anchors, d_out)[2]
    for eq, ev, eo in ((40, 70, -90), (-30, -80, 60), (0, 20, -100), (60, 0, 20)):
        # q 2^eq, k 2^-eq, v 2^ev, d_out 2^eo: the scores stay, every gradient is scaled by a power of two
        f = [2.0 ** e for e in (eq, -eq, ev, -eq, ev)]
        scaled = tuple(o * s for o, s in zip(ops, f))
        df = _df()
        a = torch.tensor(anchors, dtype=torch.int32, device="cuda")
        out, lse, _, ws = run(ops, anchors, d_out)
        grads = [torch.full_like(t, math.nan) for t in ops]
        df.dflash_packed_block_attention_backward(*scaled, a, out * 2.0 ** ev, lse, d_out * 2.0 ** eo, *grads, ws)
        for got, w, e in zip(grads, want, (ev + eo - eq, ev + eo + eq, eo, ev + eo + eq, eo)):
            assert torch.equal(got, w * 2.0 ** e)


@pytest.mark.parametrize("hd", [64, 128])
def test_long_sums_of_fp32_tensors(hd):
    """Tensor-core sums truncate: by at most 2^-23 of the sum a step, 2^-24 on average.  96 steps at most follow one
    another in the context's gradients and (3,000 / 128 + 1) * 8 or (3,000 / 64 + 1) * 4 in d_q's large products: 200;
    e^ and lse add 2^-20 of independent terms, d_q's sums of both signs shrink with the square root."""
    S, N, g, nq, nkv = 3000, 200, 16, 8, 2
    anchors = anchors_of(N, S, 13)
    ops = operands(S, N, g, nq, nkv, hd, torch.float32, 14, "cuda")
    d_out = torch.randn(ops[0].shape, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    ref = [t.double() for t in ops]
    out, lse, _ = forward_reference(*ref, anchors)
    df = _df()
    grads = [torch.full_like(t, math.nan) for t in ops]
    ws = df.dflash_packed_attention_backward_workspace(N, g, S, nq, nkv, hd, torch.float32)
    df.dflash_packed_block_attention_backward(*ops, torch.tensor(anchors, dtype=torch.int32, device="cuda"), out.float().contiguous(),
                                              lse.float().contiguous(), d_out, *grads, ws)
    for name, got, w in zip(("d_q", "d_k_ctx", "d_v_ctx", "d_k_blk", "d_v_blk"), grads,
                            backward_reference(*ref, anchors, d_out.double())):
        err = float((got.double() - w).norm() / w.norm())
        print(f"{name}: rel {err:.2e}")
        assert err <= 96 * 2.0 ** -24 + 2.0 ** -20, name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_far_smaller_than_others(dtype):
    """Rows whose d_out is 2^-12 .. 1 of the others': each row's d_q is as precise as if it were alone (d_out's
    fp16 planes hold 2^-40 of their largest, 2^-28 of the smallest rows', below their own rounding)."""
    S, N, g, nq, nkv, hd = 300, 30, 6, 4, 2, 64
    anchors = anchors_of(N, S, 8)
    ops = operands(S, N, g, nq, nkv, hd, dtype, 12, "cuda")
    gen = torch.Generator(device="cuda").manual_seed(6)
    base = torch.randn(ops[0].shape, generator=gen, device="cuda")
    scale = torch.exp2(-torch.randint(0, 13, (N, g, nq, 1), generator=gen, device="cuda").float())
    grads = run(ops, anchors, base * scale)[2]
    ref = [t.double() for t in ops]
    want = backward_reference(*ref, anchors, base.double())
    tol = tolerances(ref, anchors, base.double(), want, dtype)
    worst = float(((grads[0].double() / scale - want[0]).abs() / tol[0]).max())
    print(f"worst {worst:.2f} of its tolerance")
    assert worst <= 1.0
    want = backward_reference(*ref, anchors, (base * scale).double())
    tol = tolerances(ref, anchors, (base * scale).double(), want, dtype)
    for got, w, t in zip(grads[1:], want[1:], tol[1:]):
        assert float(((got.double() - w).abs() / t).max()) <= 1.0


def test_context_that_no_block_sees_is_not_read():
    """Context rows from the last anchor on hold NaN and infinities: their gradients are 0, the others' bits stay."""
    S, N, g, nq, nkv, hd = 700, 20, 8, 4, 2, 128
    anchors = [a % 301 for a in anchors_of(N, S, 3)] + [300]
    ops = operands(S, N + 1, g, nq, nkv, hd, torch.bfloat16, 12, "cuda")
    d_out = torch.randn(ops[0].shape, device="cuda")
    out, lse, want, ws = run(ops, anchors, d_out)
    df = _df()
    for x in (math.nan, math.inf, -math.inf):
        for t in ops[1:3]:
            t[300:] = x
        got = [torch.full_like(t, math.nan) for t in ops]
        df.dflash_packed_block_attention_backward(*ops, torch.tensor(anchors, dtype=torch.int32, device="cuda"), out, lse,
                                                  d_out, *got, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool((got[1][300:] == 0).all()) and bool((got[2][300:] == 0).all())


def test_zero_gradient_and_operands():
    S, N, g, nq, nkv, hd = 100, 9, 4, 4, 2, 64
    anchors = anchors_of(N, S, 8)
    ops = operands(S, N, g, nq, nkv, hd, torch.bfloat16, 12, "cuda")
    for z in (ops, tuple(torch.zeros_like(o) for o in ops)):
        grads = run(z, anchors, torch.zeros(ops[0].shape, device="cuda"))[2]
        assert all(bool((t == 0).all()) for t in grads)


def test_many_calls_in_a_row():
    """A wait that runs out takes 0.2 s and sets the status: none does in hundreds of back-to-back calls of many
    work items, and all of them give the same bits."""
    df = _df()
    S, N, g, nq, nkv, hd = 2048, 256, 16, 16, 4, 128
    anchors = anchors_of(N, S, 4)
    ops = operands(S, N, g, nq, nkv, hd, torch.bfloat16, 21, "cuda")
    d_out = torch.randn(ops[0].shape, device="cuda")
    out, lse, first, ws = run(ops, anchors, d_out)
    a = torch.tensor(anchors, dtype=torch.int32, device="cuda")
    grads = [torch.full_like(t, math.nan) for t in ops]
    statuses = []
    for _ in range(10):
        for _ in range(40):
            df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out, *grads, ws)
        statuses.append(df.dflash_packed_attention_status(ws))
        assert all(torch.equal(x, y) for x, y in zip(first, grads))
    assert statuses == [0] * 10


def test_two_streams_at_once():
    """Calls that overlap in time, each with its own workspace: the bits of each alone."""
    df = _df()
    cases = [(900, 96, 8, 16, 4, 128, torch.bfloat16), (700, 80, 6, 8, 2, 64, torch.float32)]
    jobs = []
    for i, (S, N, g, nq, nkv, hd, dtype) in enumerate(cases):
        anchors = anchors_of(N, S, 40 + i)
        ops = operands(S, N, g, nq, nkv, hd, dtype, 50 + i, "cuda")
        d_out = torch.randn(ops[0].shape, device="cuda")
        out, lse, want, ws = run(ops, anchors, d_out)
        a = torch.tensor(anchors, dtype=torch.int32, device="cuda")
        jobs.append((torch.cuda.Stream(), ops, a, out, lse, d_out, want, [torch.full_like(t, math.nan) for t in ops], ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, ops, a, out, lse, d_out, _, got, ws in jobs:
            df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out, *got, ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, _, _, _, want, got, ws in jobs:
        assert df.dflash_packed_attention_status(ws) == 0
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_anchors_outside_the_sequence_are_clamped_and_flagged():
    df = _df()
    S, N, g, nq, nkv, hd = 64, 3, 4, 4, 2, 64
    ops = operands(S, N, g, nq, nkv, hd, torch.bfloat16, 3, "cuda")
    d_out = torch.randn(ops[0].shape, device="cuda")
    out, lse, want, ws = run(ops, [3, S, 0], d_out)
    with pytest.raises(df.DFlashError):
        df.dflash_packed_block_attention_backward(*ops, torch.zeros(N, dtype=torch.int32, device="cuda"), out, lse, d_out,
                                                  *want, ws, anchors_host=[3, S + 1, 0])
    grads = [torch.full_like(t, math.nan) for t in ops]
    bad = torch.tensor([3, S + 100, -7], dtype=torch.int32, device="cuda")
    df.dflash_packed_block_attention_backward(*ops, bad, out, lse, d_out, *grads, ws)
    assert df.dflash_packed_attention_status(ws) == -1
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    df.dflash_packed_block_attention_backward(*ops, torch.tensor([3, S, 0], dtype=torch.int32, device="cuda"), out, lse,
                                              d_out, *grads, ws)
    assert df.dflash_packed_attention_status(ws) == 0


def test_operands_at_any_alignment():
    """Operand views that start one element into their storage."""
    S, N, g, nq, nkv, hd = 150, 20, 6, 4, 2, 128
    anchors = anchors_of(N, S, 6)
    for dtype in (torch.bfloat16, torch.float32):
        ops = operands(S, N, g, nq, nkv, hd, dtype, 4, "cuda")
        d_out = torch.randn(ops[0].shape, device="cuda")
        want = run(ops, anchors, d_out)[2]
        shifted = []
        for t in (*ops, d_out):
            s = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
            shifted.append(s.copy_(t))
        got = run(tuple(shifted[:5]), anchors, shifted[5])[2]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_blocks_and_wrapper_refusals():
    df = _df()
    S, nkv, hd = 40, 2, 64
    e = lambda *s, dtype=torch.bfloat16: torch.full(s, 7.0, dtype=dtype, device="cuda")
    ws = df.dflash_packed_attention_backward_workspace(0, 4, S, 4, nkv, hd, torch.bfloat16)
    kc, dkc, dvc = e(S, nkv, hd), e(S, nkv, hd), e(S, nkv, hd)
    q, kb = e(0, 4, 4, hd), e(0, 4, nkv, hd)
    f = torch.empty((0, 4, 4, hd), device="cuda")
    df.dflash_packed_block_attention_backward(q, kc, kc, kb, kb, torch.empty(0, dtype=torch.int32, device="cuda"), f,
                                              f[..., 0], f, q, dkc, dvc, kb, kb, ws)
    assert bool((dkc == 0).all()) and bool((dvc == 0).all()) and df.dflash_packed_attention_status(ws) == 0
    ops = operands(S, 3, 4, 4, nkv, hd, torch.bfloat16, 3, "cuda")
    d_out = torch.randn(ops[0].shape, device="cuda")
    out, lse, grads, ws = run(ops, [1, 2, 3], d_out)
    a = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    for bad in (lambda: df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out.bfloat16(), *grads, ws),
                lambda: df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out, grads[0].float(), *grads[1:], ws),
                lambda: df.dflash_packed_block_attention_backward(ops[0], ops[1][:-1], *ops[2:], a, out, lse, d_out, *grads, ws),
                lambda: df.dflash_packed_block_attention_backward(*ops, a.long(), out, lse, d_out, *grads, ws),
                lambda: df.dflash_packed_attention_backward_workspace(3, 4, S, 4, nkv, hd, torch.float16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(df.DFlashError):
        df.dflash_packed_block_attention_backward(*ops, a, out, lse, d_out, *grads, ws[:256])
