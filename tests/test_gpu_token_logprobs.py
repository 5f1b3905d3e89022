"""dflash_token_logprobs and its gradient against the definition in 64 bits.

Tolerances count roundings (u = 2^-24).  w = (x - max) log2(e) / T carries 3u
|w|, e^ is good to 2^-22 = 4u, a thread adds up to V / 256 + 16 terms in turn and
a tree of at most 11 levels follows, so the sum S and t = sum e w are within
rel(V) = u (V / 256 + 16 + 11 + 4 + 3 * 60) of their values, terms with |w| > 60
being below 2^-60 of the sum.  ln S is then off by rel(V) + u |ln S|, and what is
added to it by its own roundings."""
import numpy as np
import pytest
import torch

from test_scoring_cpu import logprob_grad_reference, logprob_reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF = float("inf")


def _df():
    import block_diffusion_drafter_dflash_gb300 as df
    return df


def rel(V):
    return U * (V / 256 + 16 + 11 + 4 + 3 * 60)


def _logits(R, V, dtype, seed, pad=0, offset=0, masked=0.0):
    """Rows with a pad between them and the first `offset` elements into its storage."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    store = torch.zeros(R * (V + pad) + offset, dtype=dtype, device="cuda")
    x = torch.randn((R, V), generator=g, device="cuda") * 3
    if masked:
        keep = torch.rand((R, V), generator=g, device="cuda") >= masked
        keep[:, V // 2] = True
        x = torch.where(keep, x, -INF)
    view = store[offset:].view(R, V + pad)[:, :V]
    view.copy_(x)
    return view


def _run(x, tokens, temp, k, stream=None):
    df = _df()
    R, V = x.shape
    f = lambda *s: torch.full(s, 777.0, device="cuda")
    lp, h, lse, top = f(R), f(R), f(R), f(R, k)
    ids = torch.full((R, k), 777, dtype=torch.int32, device="cuda")
    tok = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    kw = dict(top_ids=ids, top_logprobs=top) if k else {}
    df.dflash_token_logprobs(x, tok, temp, lp, entropy=h, lse=lse, stream=stream, **kw)
    return lp, h, lse, ids, top


def _order(x, k):
    """The k largest of each row, descending, ties to the lowest id (stable sort of the negated row)."""
    return np.argsort(-x, axis=1, kind="stable")[:, :k]


def _check(x, tokens, temp, k, got):
    xd = x.double().cpu().numpy()
    V = xd.shape[1]
    lp, h, lse = logprob_reference(xd, tokens, temp)
    z = xd / temp
    m = z.max(axis=1)
    r = rel(V)
    g = [t.double().cpu().numpy() for t in got]
    ln_s = np.abs(lse - m)
    tol_s = r + 2 * U * ln_s
    assert np.all(np.abs(g[2] - lse) <= tol_s + 3 * U * (np.abs(m) + np.abs(lse)))
    for i, t in enumerate(tokens):
        if not 0 <= t < V:
            assert g[0][i] == 0.0
        elif z[i, t] == -INF:
            assert g[0][i] == -INF
        else:
            assert abs(g[0][i] - lp[i]) <= tol_s[i] + 4 * U * (m[i] - z[i, t]) + U * abs(lp[i])
    # H = ln S - ln 2 t / S: both relative errors against E|w| <= H + ln S
    assert np.all(np.abs(g[1] - h) <= tol_s + (2 * r + 4 * U) * (np.abs(h) + ln_s) + U * np.abs(h))
    if k:
        order = _order(xd, k)
        assert np.array_equal(got[3].cpu().numpy(), order)
        with np.errstate(invalid="ignore"):
            logp = (z - m[:, None]) - np.log(np.exp(z - m[:, None]).sum(axis=1, keepdims=True))
        want = np.take_along_axis(logp, order, axis=1)
        for i in range(len(want)):
            dead = want[i] == -INF
            assert np.all(g[4][i][dead] == -INF)
            got_i, want_i, far = g[4][i][~dead], want[i][~dead], (m[i] - z[i, order[i]])[~dead]
            assert np.all(np.abs(got_i - want_i) <= tol_s[i] + 4 * U * far + U * np.abs(want_i))


SIZES = [(1, 1, 0, 0), (1, 2, 0, 1), (3, 7, 0, 0), (2, 31, 1, 3), (5, 1000, 0, 0), (40, 515, 5, 1), (3, 8705, 3, 2),
         (77, 32003, 13, 0), (2, 151936, 0, 0), (1, 151936, 0, 5), (1300, 257, 0, 0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,pad,offset", SIZES)
def test_logprobs_match_the_definition(R, V, pad, offset, dtype):
    for masked, temp, k in ((0.0, 1.0, min(20, V)), (0.6, 0.7, min(32, V)), (0.95, 1.9, 1), (0.0, 1.3, 0)):
        x = _logits(R, V, dtype, R + V, pad, offset, masked)
        rng = np.random.default_rng(V)
        tokens = rng.integers(0, V, R).tolist()
        if R > 2:
            tokens[0], tokens[1] = -1, V      # padding on either side of the vocabulary
        _check(x, tokens, temp, k, _run(x, tokens, temp, k))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 3001, 40000])
def test_rows_at_the_edges(V, dtype):
    low = torch.finfo(dtype).min
    x = _logits(9, V, dtype, 5)
    x[0] = -INF                               # nothing is possible
    x[1] = low                                # everything at the type's lowest value: uniform
    x[2] = -INF
    x[2, V // 2] = 3.5                        # one token is possible
    x[3, 1::2] = low                          # masked with the lowest value
    x[4] = 0.0                                # ties everywhere
    x[4, 1::2] = -0.0                         # -0 equals 0
    x[5, V - 1] = 80.0                        # a certain token
    x[6, 1] = float("nan")
    x[7, V - 1] = INF
    x[8, ::3] = x[8, 0].clone()               # ties among others
    tokens = [1, 2, V // 2, 0, V - 1, V - 1, 2, 2, 0]
    k = min(32, V)
    lp, h, lse, ids, top = _run(x, tokens, 1.0, k)
    assert lp[0] == -INF and lse[0] == -INF and h[0] == 0 and bool((top[0] == -INF).all())
    assert ids[0].tolist() == list(range(k))
    assert bool(torch.stack([lp[6], h[6], lse[6], lp[7], h[7], lse[7]]).isnan().all())
    assert bool(top[6].isnan().all()) and bool(top[7].isnan().all())
    xd = x.double().cpu().numpy()
    numbers = np.where(np.isnan(xd[6]), -np.inf, xd[6])[None]
    assert ids[6].tolist()[:k - 1] == [i for i in _order(numbers, V)[0] if i != 1][:k - 1]
    assert ids[7, 0] == V - 1
    sane = [1, 2, 3, 4, 5, 8]
    pick = lambda t: t[sane]
    _check(x[sane], [tokens[i] for i in sane], 1.0, k, [pick(t) for t in (lp, h, lse, ids, top)])
    assert h[2] == 0 and lp[2] == 0 and lp[5] == 0


def test_all_nan_row_has_no_alternatives():
    x = torch.full((2, 40), float("nan"), device="cuda")
    lp, h, lse, ids, top = _run(x, [0, 1], 1.0, 3)
    assert bool(lp.isnan().all()) and ids.tolist() == [[-1] * 3] * 2 and bool(top.isnan().all())


def test_only_what_is_asked_for():
    df = _df()
    x = _logits(4, 1000, torch.float32, 1)
    h, lse = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    full = _run(x, [0, 1, 2, 3], 1.0, 0)
    df.dflash_token_logprobs(x, None, 1.0, None, entropy=h)
    assert torch.equal(h, full[1])
    df.dflash_token_logprobs(x.view(2, 2, 1000), None, 1.0, None, lse=lse.view(2, 2))
    assert torch.equal(lse, full[2])
    empty = torch.empty((0, 8), device="cuda")
    e = torch.empty(0, device="cuda")
    df.dflash_token_logprobs(empty, torch.empty(0, dtype=torch.int32, device="cuda"), 1.0, e, entropy=e)


def test_wrapper_refusals():
    df = _df()
    x = _logits(4, 16, torch.float32, 1)
    lp, tok = torch.empty(4, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: df.dflash_token_logprobs(x.double(), tok, 1.0, lp),
                lambda: df.dflash_token_logprobs(x.t(), tok, 1.0, lp),
                lambda: df.dflash_token_logprobs(x.cpu(), tok, 1.0, lp),
                lambda: df.dflash_token_logprobs(x, tok.long(), 1.0, lp),
                lambda: df.dflash_token_logprobs(x, tok[:3], 1.0, lp),
                lambda: df.dflash_token_logprobs(x, tok, 1.0, lp.cpu()),
                lambda: df.dflash_token_logprobs(x, tok, 1.0, lp, top_ids=tok.view(4, 1)),
                lambda: df.dflash_token_logprobs_backward(x, tok, 1.0, lp, x[:2], d_logprob=lp),
                lambda: df.dflash_token_logprobs_backward(x, tok, 1.0, lp, x.bfloat16(), d_logprob=lp)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: df.dflash_token_logprobs(x[:1].expand(4, 16), tok, 1.0, lp),     # rows on top of one another
                lambda: df.dflash_token_logprobs(x, tok, 0.0, lp),
                lambda: df.dflash_token_logprobs(x, tok, 1.0, None),
                lambda: df.dflash_token_logprobs_backward(x, tok, 1.0, lp, torch.empty_like(x))):
        with pytest.raises(df.DFlashError):
            bad()


# ---------------------------------------------------------------- gradient
def _grad_tol(xd, tokens, temp, d_lp, d_h, want, dtype):
    """p is off by u (|z| + |lse| + 2 |ln p|) from its exponent and 4u + u from e^; the sums around it by 4u."""
    z = xd / temp
    _, h, lse = logprob_reference(xd, tokens, temp)
    logp = z - lse[:, None]
    p = np.exp(logp)
    logp = np.where(p > 0, logp, 0.0)
    zz = np.where(p > 0, np.abs(z), 0.0)
    g = np.array([d if 0 <= t < z.shape[1] else 0.0 for t, d in zip(tokens, d_lp)])
    size = np.abs(g)[:, None] + (0 if d_h is None else np.abs(d_h)[:, None] * (np.abs(logp) + h[:, None]))
    e_logp = U * (2 * zz + np.abs(lse)[:, None] + 2 * np.abs(logp))
    tol = p * (size * (e_logp + 9 * U) + (0 if d_h is None else np.abs(d_h)[:, None] * (e_logp + 2 * U * h[:, None])))
    tol = tol / temp + 4 * U * np.abs(want) + 4 * U * np.abs(g)[:, None] / temp * (p > 1e-3) + 1e-37
    return tol + (np.abs(want) * 2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,pad,offset", SIZES)
def test_gradient_matches_the_formula(R, V, pad, offset, dtype):
    df = _df()
    rng = np.random.default_rng(V + 1)
    for masked, temp, with_lp, with_h, d_pad in ((0.0, 1.0, True, False, 0), (0.5, 0.7, True, True, pad),
                                                 (0.0, 1.6, False, True, 1)):
        x = _logits(R, V, dtype, R + V, pad, offset, masked)
        tokens = rng.integers(0, V, R).tolist()
        if R > 2:
            tokens[0], tokens[1] = -1, V + 3
        d_lp, d_h = rng.normal(size=R), rng.normal(size=R)
        d_lp, d_h = (torch.tensor(v, dtype=torch.float32, device="cuda") for v in (d_lp, d_h))
        xd = x.double().cpu().numpy()
        _, h, lse = logprob_reference(xd, tokens, temp)
        store = torch.full((R, V + d_pad), 55.0, dtype=dtype, device="cuda")
        d = store[:, :V]
        f = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")
        tok = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        df.dflash_token_logprobs_backward(x, tok, temp, f(lse), d, d_logprob=d_lp if with_lp else None, entropy=f(h),
                                          d_entropy=d_h if with_h else None)
        a = d_lp.double().cpu().numpy() if with_lp else np.zeros(R)
        b = d_h.double().cpu().numpy() if with_h else None
        want = logprob_grad_reference(xd, tokens, temp, a, b)
        err = np.abs(d.double().cpu().numpy() - want)
        assert np.all(err <= _grad_tol(xd, tokens, temp, a, b, want, dtype))
        assert bool((store[:, V:] == 55).all())        # nothing between the rows is written
        # in place: the same bits
        y = x.clone(memory_format=torch.preserve_format) if pad == 0 and offset == 0 else x
        df.dflash_token_logprobs_backward(y, tok, temp, f(lse), y, d_logprob=d_lp if with_lp else None, entropy=f(h),
                                          d_entropy=d_h if with_h else None)
        assert torch.equal(y, d)


def test_gradient_rows_at_the_edges():
    df = _df()
    x = _logits(4, 300, torch.float32, 3)
    x[0] = -INF
    x[1] = torch.finfo(torch.float32).min
    x[2, 7] = float("nan")
    tokens = torch.tensor([5, 5, 5, 5], dtype=torch.int32, device="cuda")
    lp, h, lse, _, _ = _run(x, [5] * 4, 1.0, 0)
    d, one = torch.empty_like(x), torch.ones(4, device="cuda")
    df.dflash_token_logprobs_backward(x, tokens, 1.0, lse, d, d_logprob=one, entropy=h, d_entropy=one)
    assert bool((d[0] == 0).all()) and bool((d[1] == 0).all())
    assert bool(d[2].isnan().all()) and bool(d[3].isfinite().all())


def test_side_stream_and_graph_replay():
    """Calls on another stream, and a captured forward and gradient replayed over new logits."""
    df = _df()
    R, V = 6, 20011
    x, new = _logits(R, V, torch.float32, 8), _logits(R, V, torch.float32, 9)
    tok = torch.arange(R, dtype=torch.int32, device="cuda")
    lp, h, lse = (torch.empty(R, device="cuda") for _ in range(3))
    ids, top = torch.empty((R, 4), dtype=torch.int32, device="cuda"), torch.empty((R, 4), device="cuda")
    d, w = torch.empty_like(x), torch.randn(R, device="cuda")

    def step(stream=None):
        df.dflash_token_logprobs(x, tok, 0.9, lp, entropy=h, lse=lse, top_ids=ids, top_logprobs=top, stream=stream)
        df.dflash_token_logprobs_backward(x, tok, 0.9, lse, d, d_logprob=w, entropy=h, d_entropy=w, stream=stream)

    outs = (lp, h, lse, ids, top, d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    first = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))
    x.copy_(new)
    graph.replay()
    again = [t.clone() for t in outs]
    step()
    assert all(torch.equal(a, b) for a, b in zip(outs, again)) and not torch.equal(again[0], first[0])
    _check(x, list(range(R)), 0.9, 4, again[:5])


def test_largest_row_count_and_vocabulary():
    R, V, k = 65535, 5, 3
    x = _logits(R, V, torch.float32, 3)
    tokens = np.random.default_rng(4).integers(-1, V + 1, R).tolist()
    _check(x, tokens, 0.9, k, _run(x, tokens, 0.9, k))
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(1, 1 << 24, dtype, 5)
        _check(x, [1 << 23], 1.0, 32, _run(x, [1 << 23], 1.0, 32))


def test_offsets_past_32_bits():
    """More than 2^31 logits: 64 rows repeated give the same bits wherever they lie, forward and gradient (in place)."""
    df = _df()
    V, n, reps = 151936, 64, 222
    base = _logits(n, V, torch.bfloat16, 9)
    x = base.repeat(reps, 1)
    assert x.numel() > 2 ** 31
    tokens = np.random.default_rng(4).integers(0, V, n).tolist()
    tok = torch.tensor(tokens * reps, dtype=torch.int32, device="cuda")
    f = lambda: torch.full((n * reps,), 777.0, device="cuda")
    lp, h, lse = f(), f(), f()
    ids = torch.full((n * reps, 2), 777, dtype=torch.int32, device="cuda")
    top = torch.full((n * reps, 2), 777.0, device="cuda")
    df.dflash_token_logprobs(x, tok, 1.0, lp, entropy=h, lse=lse, top_ids=ids, top_logprobs=top)
    for t in (lp, h, lse, ids, top):
        assert bool((t.view(reps, n, -1) == t[:n].view(n, -1)).all())
    _check(base, tokens, 1.0, 2, [t[:n] for t in (lp, h, lse, ids, top)])
    g = torch.linspace(-1, 1, n, device="cuda").repeat(reps)
    df.dflash_token_logprobs_backward(x, tok, 1.0, lse, x, d_logprob=g)
    first = x[:n].clone()
    assert all(torch.equal(x[i * n:(i + 1) * n], first) for i in range(reps))
    xd = base[:4].double().cpu().numpy()
    a = g[:4].double().cpu().numpy()
    want = logprob_grad_reference(xd, tokens[:4], 1.0, a, None)
    assert np.all(np.abs(first[:4].double().cpu().numpy() - want)
                  <= _grad_tol(xd, tokens[:4], 1.0, a, None, want, torch.bfloat16))


def test_smallest_temperature():
    """log2(e) / T near fp32's largest: the row's maxima share the probability, everything else has none."""
    x = torch.full((2, 1000), -0.5, device="cuda")
    x[0, [3, 700]] = 1.0
    x[1, 999] = 1.0
    for dtype in (torch.float32, torch.bfloat16):
        lp, h, lse, ids, top = _run(x.to(dtype), [700, 0], 4.3e-39, 3)
        ln2 = float(np.log(2.0))
        assert abs(float(lp[0]) + ln2) <= 4 * U and abs(float(h[0]) - ln2) <= 4 * U and float(h[1]) == 0
        assert float(lp[1]) < -3e38 and bool(lse.isfinite().all())
        assert ids[0, :2].tolist() == [3, 700] and int(ids[1, 0]) == 999 and float(top[1, 0]) == 0


def test_gradient_between_the_logits_rows():
    """d_logits in the gaps between the logits' rows, before and behind them, overlaps nothing: the bits of a separate
    gradient, and the logits and what lies between stay.  A gap that is one element short is refused."""
    df = _df()
    R, V = 5, 1003
    for dtype in (torch.float32, torch.bfloat16):
        for at_x, at_d in ((0, V + 1), (V, 0), (2, V + 2)):
            store = torch.full((R + 1, 2 * V + 3), 5.0, dtype=dtype, device="cuda")
            x, d = store[:R, at_x:at_x + V], store[:R, at_d:at_d + V]
            x.copy_(_logits(R, V, dtype, 3))
            kept = store.clone()
            tok = torch.arange(R, dtype=torch.int32, device="cuda")
            g, lse = torch.linspace(-1, 1, R, device="cuda"), torch.empty(R, device="cuda")
            df.dflash_token_logprobs(x, None, 0.9, None, lse=lse)
            alone = torch.empty((R, V), dtype=dtype, device="cuda")
            df.dflash_token_logprobs_backward(x, tok, 0.9, lse, alone, d_logprob=g)
            df.dflash_token_logprobs_backward(x, tok, 0.9, lse, d, d_logprob=g)
            assert torch.equal(d, alone)
            kept[:R, at_d:at_d + V] = alone
            assert torch.equal(store, kept)
            for shift in (1, 2 * V + 3 - 1):
                bad = store.view(-1)[at_x + V - 1 if shift == 1 else at_x + V + 4:]
                bad = bad.as_strided((R, V), (2 * V + 3, 1), bad.storage_offset())
                with pytest.raises(df.DFlashError):
                    df.dflash_token_logprobs_backward(x, tok, 0.9, lse, bad, d_logprob=g)
