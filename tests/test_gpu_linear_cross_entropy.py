"""dflash_linear_cross_entropy and its gradient against the definition in 64 bits.

Tolerances count roundings (u = 2^-24), with A = |h| |w|' the sum of a logit's
absolute terms.
  Logits.  Products of bf16 are exact; those of fp32's planes leave out less than 4u
  of a term.  A sum of the tensor cores spans at most 32 steps of 16 terms (for fp32
  tensors 160 more of terms 2^-8 smaller), each of which may truncate at 2 * 2^-23 of
  the sum (the sum and the terms' alignment), and D / 512 sums are added: off by
  c A / T with c = 4u + 33 * 4u + u D / 512.
  Exponents.  z log2(e) / T and lse log2(e) are rounded, e^ is good to 2^-22 = 4u:
  off by another 3u |z| + 3u |lse| + 4u.  (fp32 gradients carry the factor's and
  lse's residuals, so this bounds them too.)
  Exponentials below 2^-126 are flushed to 0 (ex2.approx.ftz), which is off by less than
  that times d_loss / T in a value of G; values of G below 2^-126 may count as 0 in a
  product, off by less than 2^-126 again.
  lse.  Its sum has at most 32 + 8 + parts / 16 + 16 roundings in turn, parts being
  two for 128 or 256 columns."""
import math

import pytest
import torch

from test_training_ends_cpu import loss_grad_reference, loss_reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _df():
    import block_diffusion_drafter_dflash_gb300 as df
    return df


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _c(D):
    return 4 * U + 33 * 4 * U + U * (D / 512 + 1)


def operands(R, D, V, dtype, seed, pad=0, offset=0, ignored=0.0, lean=6.0, amp=1.0):
    """Hidden states (a pad behind each row, the first `offset` elements into their storage), head, targets."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, D), generator=g, device="cuda") * 2 / math.sqrt(D)).to(dtype)
    targets = torch.randint(0, V, (R,), generator=g, device="cuda")
    store = torch.full((R * (D + pad) + offset,), math.nan, dtype=dtype, device="cuda")
    h = store[offset:].view(R, D + pad)[:, :D]
    along = lean * torch.rand((R, 1), generator=g, device="cuda") / 4
    h.copy_(amp * (torch.randn((R, D), generator=g, device="cuda") + along * w[targets].float()))
    targets = torch.where(torch.rand(R, generator=g, device="cuda") < ignored, -1, targets).to(torch.int32)
    return h, w, targets


def forward(h, w, t, temp=1.0, stream=None, ws=None):
    df = _df()
    (R, D), V = h.shape, w.shape[0]
    loss, lse = torch.full((R,), 777.0, device="cuda"), torch.full((R,), 777.0, device="cuda")
    ws = df.dflash_linear_cross_entropy_workspace(R, D, V, h.dtype) if ws is None else ws
    df.dflash_linear_cross_entropy(h, w, t, loss, lse, ws, temperature=temp, stream=stream)
    if stream is None:
        assert df.dflash_linear_cross_entropy_status(ws) == 0
    return loss, lse


def backward(h, w, t, lse, d_loss, temp=1.0, want=(True, True), stream=None, d_hidden=None, ws=None):
    df = _df()
    (R, D), V = h.shape, w.shape[0]
    if d_hidden is None and want[0]:
        d_hidden = torch.full((R, D), 777.0, dtype=h.dtype, device="cuda")
    d_weight = torch.full((V, D), 777.0, dtype=h.dtype, device="cuda") if want[1] else None
    ws = df.dflash_linear_cross_entropy_backward_workspace(R, D, V, h.dtype) if ws is None else ws
    df.dflash_linear_cross_entropy_backward(h, w, t, lse, d_loss, d_hidden, d_weight, ws, temperature=temp, stream=stream)
    if stream is None:
        assert df.dflash_linear_cross_entropy_status(ws) == 0
    return d_hidden, d_weight


def _bounds(h, w, t, temp):
    """(h, w in 64 bits with ignored rows zeroed, |z| and its error, lse and its error)."""
    inside = (t >= 0) & (t < w.shape[0])
    h, w = torch.where(inside[:, None], h.double(), 0.0), w.double()
    D, V = w.shape[1], w.shape[0]
    z = h @ w.t() / temp
    lse = torch.logsumexp(z, dim=1)
    dz = _c(D) * (h.abs() @ w.abs().t()) / temp + 3 * U * z.abs()
    e = dz + 3 * U * lse.abs()[:, None] + 4 * U
    p = torch.softmax(z, dim=1)
    parts = 2 * (V / 128 + 1)
    # the error of ln sum e^z is the mean of the exponents' errors under p
    d_lse = (p * e).sum(1) + U * (32 + 8 + parts / 16 + 16) + 2 * U * (lse.abs() + 1)
    return inside, h, w, z, dz, lse, d_lse, e, p


def check_forward(h, w, t, temp, got):
    loss, lse = (x.double() for x in got)
    want_loss, want_lse = loss_reference(h.double(), w.double(), t, temp)
    inside, _, _, z, dz, _, d_lse, _, _ = _bounds(h, w, t, temp)
    at = torch.where(inside, t, 0).long()[:, None]
    tol = torch.where(inside, d_lse + dz.gather(1, at)[:, 0] + 3 * U * (want_lse.abs() + z.gather(1, at)[:, 0].abs()), 0.0)
    assert bool(((lse - want_lse).abs() <= torch.where(inside, d_lse, 0.0)).all())
    assert bool(((loss - want_loss).abs() <= tol).all())


def check_backward(h, w, t, temp, lse, d_loss, got):
    inside, hd, wd, z, dz, _, _, e, p = _bounds(h, w, t, temp)
    want_h, want_w, g = loss_grad_reference(h.double(), w.double(), t, temp, d_loss.double())
    D, (R, V) = w.shape[1], g.shape
    gain = torch.where(inside, d_loss.double().abs(), 0.0)[:, None] / temp
    lse_off = torch.where(inside, (lse.double() - torch.logsumexp(z, dim=1)).abs(), 0.0)[:, None]
    dg = gain * p * (torch.expm1(e + lse_off) + 2 * U) + 3 * U * g.abs()
    stored = _half_step(BF16) if h.dtype == BF16 else 4 * U
    dg = dg + stored * (g.abs() + dg) + (gain + 1) * 2.0 ** -126
    # a product's sums as the logits', over V (its pieces' and shares' sums too) or the rows
    for x, ref, n, other, spread in ((got[0], want_h, V, wd, lambda m: m @ wd.abs()),
                                     (got[1], want_w, R, hd, lambda m: m.t() @ hd.abs())):
        if x is None:
            continue
        tol = spread(dg) + (_c(n) + 80 * U) * spread(g.abs() + dg)
        tol = tol + _half_step(x.dtype) * (ref.abs() + tol) + 1e-38
        off = (x.double() - ref).abs()
        assert bool((off <= tol).all()), f"{float((off / tol).max()):.3g} times the tolerance"
        if float(ref.norm()) > 0:
            print(f"rel {float((x.double() - ref).norm() / ref.norm()):.2e}", end=" ")


SHAPES = [
    (1, 8, 1), (1, 64, 300), (5, 8, 257), (128, 64, 256), (129, 72, 255), (300, 256, 1003), (257, 128, 128),
    (45, 1032, 5001), (640, 192, 2049), (2, 4096, 1000), (127, 520, 40001),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,D,V", SHAPES)
def test_loss_against_the_definition(R, D, V, dtype):
    h, w, t = operands(R, D, V, dtype, R + D + V, ignored=0.2 if R > 100 else 0.0)
    check_forward(h, w, t, 1.0, forward(h, w, t))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,D,V", SHAPES)
def test_gradients_against_the_formula(R, D, V, dtype):
    h, w, t = operands(R, D, V, dtype, R + D + V + 1, ignored=0.2 if R > 100 else 0.0)
    lse = loss_reference(h.double(), w.double(), t, 1.0)[1].float()
    d_loss = (torch.randn(R, device="cuda") / R).float()
    check_backward(h, w, t, 1.0, lse, d_loss, backward(h, w, t, lse, d_loss))


@pytest.mark.parametrize("dtype,R,D,V", [(BF16, 8100, 64, 16500), (F32, 4000, 72, 9001), (F32, 64, 4096, 9001)])
def test_vocabularies_of_several_pieces(dtype, R, D, V):
    h, w, t = operands(R, D, V, dtype, 5, ignored=0.1)
    got = forward(h, w, t)
    check_forward(h, w, t, 1.0, got)
    d_loss = torch.full((R,), 1.0 / R, device="cuda")
    check_backward(h, w, t, 1.0, got[1], d_loss, backward(h, w, t, got[1], d_loss))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,D,V", [(3, 65536, 100), (1 << 20, 8, 20), (1, 8, 70001)])
def test_the_largest_dim_and_row_count_and_the_smallest_dim(R, D, V, dtype):
    h, w, t = operands(R, D, V, dtype, 6, ignored=0.0 if R < 10 else 0.1)
    got = forward(h, w, t)
    check_forward(h, w, t, 1.0, got)
    d_loss = torch.rand(R, device="cuda") / R
    check_backward(h, w, t, 1.0, got[1], d_loss, backward(h, w, t, got[1], d_loss))


def test_a_head_past_32_bits():
    """A head of 2.4 G values, its gradient and a piece's first row past 2^31; the rows' own logits in 64 bits."""
    R, D, V = 3, 4096, 590_000
    g = torch.Generator(device="cuda").manual_seed(30)
    w = torch.empty((V, D), dtype=BF16, device="cuda")
    for v in range(0, V, 65536):
        w[v:v + 65536] = torch.randn((min(65536, V - v), D), generator=g, device="cuda") / math.sqrt(D)
    t = torch.tensor([V - 1, 7, 550_000], dtype=torch.int32, device="cuda")
    h = (torch.randn((R, D), generator=g, device="cuda") + 8 * w[t.long()].float()).to(BF16)
    got = forward(h, w, t)
    z = torch.cat([h.double() @ w[v:v + 65536].double().t() for v in range(0, V, 65536)], dim=1)
    a = torch.cat([h.double().abs() @ w[v:v + 65536].double().abs().t() for v in range(0, V, 65536)], dim=1)
    lse = torch.logsumexp(z, dim=1)
    p = torch.softmax(z, dim=1)
    dz = _c(D) * a + 3 * U * z.abs()
    e = dz + 3 * U * lse[:, None].abs() + 4 * U
    d_lse = (p * e).sum(1) + U * (32 + 8 + 2 * (V / 128 + 1) / 16 + 16) + 2 * U * (lse.abs() + 1)
    assert bool(((got[1].double() - lse).abs() <= d_lse).all())
    picked = z.gather(1, t.long()[:, None])[:, 0]
    tol = d_lse + dz.gather(1, t.long()[:, None])[:, 0] + 3 * U * (lse.abs() + picked.abs())
    assert bool(((got[0].double() - (lse - picked)).abs() <= tol).all())
    d_loss = torch.tensor([0.5, -1.0, 2.0], device="cuda")
    d_h, d_w = backward(h, w, t, lse.float(), d_loss)
    p[torch.arange(R), t.long()] -= 1.0
    gr = p * d_loss.double()[:, None]
    dg = d_loss.double().abs()[:, None] * torch.softmax(z, dim=1) * (torch.expm1(e + U * lse.abs()[:, None]) + 2 * U) + 3 * U * gr.abs()
    dg = dg + _half_step(BF16) * (gr.abs() + dg) + 3 * 2.0 ** -126
    rows = torch.cat([torch.arange(0, 200), torch.arange(549_900, 550_100), torch.arange(V - 200, V)]).cuda()
    want = gr[:, rows].t() @ h.double()
    tol = dg[:, rows].t() @ h.double().abs() + _c(R) * (gr.abs() + dg)[:, rows].t() @ h.double().abs()
    tol = tol + _half_step(BF16) * (want.abs() + tol)
    assert bool(((d_w[rows].double() - want).abs() <= tol).all())
    want, tol = 0.0, 0.0
    for v in range(0, V, 65536):
        x = w[v:v + 65536].double()
        want = want + gr[:, v:v + 65536] @ x
        tol = tol + dg[:, v:v + 65536] @ x.abs() + (_c(V) + 80 * U) * ((gr.abs() + dg)[:, v:v + 65536] @ x.abs())
    tol = tol + _half_step(BF16) * (want.abs() + tol)
    assert bool(((d_h.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,offset,temp", [(8, 0, 0.7), (3, 0, 1.5), (1, 1, 1.0), (40, 8, 1.0)])
def test_strides_alignment_and_temperature(dtype, pad, offset, temp):
    R, D, V = 200, 136, 777
    h, w, t = operands(R, D, V, dtype, 7, pad=pad, offset=offset, ignored=0.3)
    got = forward(h, w, t, temp)
    check_forward(h, w, t, temp, got)
    d_loss = torch.rand(R, device="cuda")
    store = torch.full((R * (D + pad) + offset,), 555.0, dtype=dtype, device="cuda")
    d_h = store[offset:].view(R, D + pad)[:, :D]
    check_backward(h, w, t, temp, got[1], d_loss, backward(h, w, t, got[1], d_loss, temp, d_hidden=d_h))
    assert bool((store[:offset] == 555.0).all()) and bool((store[offset:].view(R, D + pad)[:, D:] == 555.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ignored_rows_reach_nothing(dtype):
    """Targets outside the vocabulary on every side, rows of NaN and infinity behind them, lse and d_loss of NaN."""
    R, D, V = 150, 64, 500
    h, w, t = operands(R, D, V, dtype, 9)
    bad = torch.tensor([-1, V, V + 1, -(2 ** 31), 2 ** 31 - 1], dtype=torch.int32, device="cuda").repeat(20)
    rows = torch.randperm(R, device="cuda")[:100]
    t[rows] = bad
    h[rows[:50]] = math.nan
    h[rows[50:]] = math.inf
    got = forward(h, w, t)
    check_forward(h, w, t, 1.0, got)
    d_loss, lse = torch.rand(R, device="cuda"), got[1].clone()
    d_loss[rows[::2]] = math.nan
    lse[rows[1::2]] = math.nan
    d_h, d_w = backward(h, w, t, lse, d_loss)
    assert bool((d_h[rows] == 0).all())
    clean, clean_lse = d_loss.clone(), got[1]
    clean[rows] = 0.0
    check_backward(h, w, t, 1.0, clean_lse, clean, (d_h, d_w))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_all_rows_ignored(dtype):
    R, D, V = 130, 64, 300
    h, w, t = operands(R, D, V, dtype, 10, ignored=2.0)
    loss, lse = forward(h, w, t)
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    d_h, d_w = backward(h, w, t, lse, torch.ones(R, device="cuda"))
    assert bool((d_h == 0).all()) and bool((d_w == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_rows(dtype):
    h, w, t = operands(0, 64, 300, dtype, 10)
    forward(h, w, t)
    d_h, d_w = backward(h, w, t, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    assert d_h.shape == (0, 64) and bool((d_w == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_row_of_nan_spoils_its_own_results_alone(dtype):
    R, D, V = 140, 128, 600
    h, w, t = operands(R, D, V, dtype, 11)
    want = forward(h, w, t)
    d_loss = torch.rand(R, device="cuda")
    clean, _ = backward(h, w, t, want[1], d_loss, want=(True, False))
    h[5, 3], h[77, 100] = math.nan, math.inf
    loss, lse = forward(h, w, t)
    d_h, _ = backward(h, w, t, lse, d_loss, want=(True, False))
    others = torch.ones(R, dtype=torch.bool, device="cuda")
    others[[5, 77]] = False
    assert bool(loss[~others].isnan().all()) and bool(lse[~others].isnan().all()) and bool(d_h[~others].isnan().all())
    assert torch.equal(loss[others], want[0][others]) and torch.equal(lse[others], want[1][others])
    assert torch.equal(d_h[others], clean[others])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_confident_rows_and_large_logits(dtype):
    """Logits of hundreds: softmaxes of one token, losses of exactly 0 and of hundreds."""
    R, D, V = 100, 64, 900
    h, w, t = operands(R, D, V, dtype, 12, amp=60.0)
    z = h.double() @ w.double().t()
    t[::2] = z.argmax(1).to(torch.int32)[::2]
    got = forward(h, w, t)
    check_forward(h, w, t, 1.0, got)
    assert bool((got[0][::2] >= 0).all())
    d_loss = torch.rand(R, device="cuda")
    check_backward(h, w, t, 1.0, got[1], d_loss, backward(h, w, t, got[1], d_loss))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_either_gradient_alone_and_in_place(dtype):
    R, D, V = 260, 200, 1300
    h, w, t = operands(R, D, V, dtype, 13, pad=8, ignored=0.2)
    _, lse = forward(h, w, t)
    d_loss = torch.rand(R, device="cuda")
    d_h, d_w = backward(h, w, t, lse, d_loss)
    assert torch.equal(backward(h, w, t, lse, d_loss, want=(True, False))[0], d_h)
    assert torch.equal(backward(h, w, t, lse, d_loss, want=(False, True))[1], d_w)
    _, again = backward(h, w, t, lse, d_loss, d_hidden=h)       # the hidden states' place
    assert torch.equal(h, d_h) and torch.equal(again, d_w)


def test_fp32_gradient_precision():
    """fp32 gradients are good to fp32: 2e-6 of their norm (the logits' errors of at most 33 truncating steps, 2e-8
    of a sum each, and exponents of about 20 rounded to 2^-24 of themselves)."""
    R, D, V = 256, 2048, 4000
    h, w, t = operands(R, D, V, F32, 14)
    _, lse = loss_reference(h.double(), w.double(), t, 1.0)
    d_loss = torch.rand(R, device="cuda") / R
    got = backward(h, w, t, lse.float(), d_loss)
    want = loss_grad_reference(h.double(), w.double(), t, 1.0, d_loss.double())
    for x, ref in zip(got, want):
        rel = float((x.double() - ref).norm() / ref.norm())
        print(f"rel {rel:.2e}")
        assert rel <= 2e-6


def test_the_same_call_gives_the_same_bits():
    R, D, V = 500, 256, 3001
    h, w, t = operands(R, D, V, BF16, 15, ignored=0.1)
    d_loss = torch.rand(R, device="cuda")
    first = forward(h, w, t)
    grads = backward(h, w, t, first[1], d_loss)
    for _ in range(5):
        for a, b in zip(forward(h, w, t), first):
            assert torch.equal(a, b)
        for a, b in zip(backward(h, w, t, first[1], d_loss), grads):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    sets = [operands(700, 256, 2500, BF16, 16 + i, ignored=0.1 * i) for i in range(2)]
    d_loss = torch.rand(700, device="cuda")
    want = []
    for s in sets:
        f = forward(*s)
        want.append((f, backward(*s, f[1], d_loss)))
    df = _df()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [(df.dflash_linear_cross_entropy_workspace(700, 256, 2500, BF16),
           df.dflash_linear_cross_entropy_backward_workspace(700, 256, 2500, BF16)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, st, x in zip(sets, streams, ws):
            with torch.cuda.stream(st):
                f = forward(*s, stream=st, ws=x[0])
                got.append((f, backward(*s, f[1], d_loss, stream=st, ws=x[1])))
        torch.cuda.synchronize()
        for (f, b), (f0, b0) in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip((*f, *b), (*f0, *b0)))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_and_replayed(dtype):
    df = _df()
    R, D, V = 300, 128, 1500
    h, w, t = operands(R, D, V, dtype, 18, ignored=0.2)
    d_loss = torch.rand(R, device="cuda")
    new = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    loss, lse, d_h, d_w = new(R), new(R), new(R, D, dt=dtype), new(V, D, dt=dtype)
    ws = df.dflash_linear_cross_entropy_workspace(R, D, V, dtype)
    ws_b = df.dflash_linear_cross_entropy_backward_workspace(R, D, V, dtype)

    def step():
        df.dflash_linear_cross_entropy(h, w, t, loss, lse, ws)
        df.dflash_linear_cross_entropy_backward(h, w, t, lse, d_loss, d_h, d_w, ws_b)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, ignored in ((19, 0.0), (20, 0.7), (21, 2.0)):     # other kept rows than at the capture
        h2, w2, t2 = operands(R, D, V, dtype, seed, ignored=ignored)
        h.copy_(h2), w.copy_(w2), t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        want = forward(h, w, t)
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
        want = backward(h, w, t, lse, d_loss)
        assert torch.equal(d_h, want[0]) and torch.equal(d_w, want[1])


def test_binding_refusals():
    df = _df()
    h, w, t = operands(6, 64, 100, BF16, 22)
    f = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    ws = df.dflash_linear_cross_entropy_workspace(6, 64, 100, BF16)
    ok = [h, w, t, f(6), f(6), ws]
    for i, bad in ((0, h.cpu()), (0, h.half()), (1, w.float()), (1, w[:, :32]), (1, w.t()), (2, t.long()), (2, t[:5]),
                   (3, f(5)), (4, f(6, dt=BF16)), (1, w.cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            df.dflash_linear_cross_entropy(*args)
    with pytest.raises(df.DFlashError):
        df.dflash_linear_cross_entropy(*ok[:5], ws[:1024])
    wb = df.dflash_linear_cross_entropy_backward_workspace(6, 64, 100, BF16)
    for d_h, d_w in ((f(6, 64), None), (f(5, 64, dt=BF16), None), (None, f(100, 64)), (None, f(99, 64, dt=BF16))):
        with pytest.raises(ValueError):
            df.dflash_linear_cross_entropy_backward(h, w, t, f(6), f(6), d_h, d_w, wb)
    with pytest.raises(df.DFlashError):
        df.dflash_linear_cross_entropy_backward(h, w, t, f(6), f(6), None, None, wb)
    with pytest.raises(ValueError):
        df.dflash_linear_cross_entropy_workspace(6, 64, 100, torch.float16)
