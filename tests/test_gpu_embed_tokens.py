"""dflash_embed_tokens and its gradient against the definition in 64 bits.

Tolerances (u = 2^-24): a looked-up value is one fp32 product, rounded to the output's
type.  A gradient is a sum of fp32 terms, at most 32 in turn and then the chunks' sums
with their rounding errors carried along (2u), times the factor, added to what was there,
and rounded to the table's type: within 36u of the sum of its terms' absolute values,
and half a step of the result."""
import math

import pytest
import torch

from test_training_ends_cpu import embed_grad_reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _df():
    import block_diffusion_drafter_dflash_gb300 as df
    return df


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rows_of(n, D, dtype, g, pad=0, offset=0, fill=math.nan):
    store = torch.full((n * (D + pad) + offset,), fill, dtype=dtype, device="cuda")
    return store, store[offset:].view(n, D + pad)[:, :D]


def make_tokens(n, V, g, mask=0.0, ignored=0.0):
    t = (V * torch.rand(n, generator=g, device="cuda") ** 3).long().clamp(max=V - 1)
    t = torch.where(torch.rand(n, generator=g, device="cuda") < mask, V - 1, t)
    bad = torch.tensor([-1, V, -(2 ** 31), 2 ** 31 - 1], device="cuda")[torch.randint(0, 4, (n,), generator=g, device="cuda")]
    return torch.where(torch.rand(n, generator=g, device="cuda") < ignored, bad, t).to(torch.int32)


def backward(d_out, t, V, dtype, scale=1.0, into=None, ws=None, stream=None):
    df = _df()
    n, D = d_out.shape
    d = torch.full((V, D), 777.0, dtype=dtype, device="cuda") if into is None else into
    ws = df.dflash_embed_tokens_backward_workspace(n, D, V) if ws is None else ws
    df.dflash_embed_tokens_backward(d_out, t, d, ws, scale=scale, accumulate=into is not None, stream=stream)
    return d


def check(d, d_out, t, V, scale, before=None):
    want, terms = embed_grad_reference(d_out, t, V, scale)
    if before is not None:
        want = want + before.double()
    tol = 36 * U * terms + U * want.abs()
    tol = tol + _half_step(d.dtype) * (want.abs() + tol) + 1e-44
    off = (d.double() - want).abs()
    assert bool((off <= tol).all()), f"{float((off / tol).max()):.3g} times the tolerance"


@pytest.mark.parametrize("table_dtype", [F32, BF16])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("n,D,V,pad,offset", [(1, 1, 1, 0, 0), (16, 4096, 1000, 0, 0), (33, 250, 77, 0, 0), (100, 12, 5, 4, 4),
                                              (65, 1001, 300, 3, 1), (7, 64, 100000, 8, 8), (3000, 40, 2000, 0, 2)])
def test_lookup(n, D, V, pad, offset, out_dtype, table_dtype):
    df = _df()
    g = torch.Generator(device="cuda").manual_seed(n + D)
    table = torch.randn((V, D), generator=g, device="cuda").to(table_dtype)
    t = make_tokens(n, V, g, ignored=0.2)
    inside = (t >= 0) & (t < V)
    for scale in (1.0, 0.3, 0.0):
        store, out = rows_of(n, D, out_dtype, g, pad, offset, fill=555.0)
        df.dflash_embed_tokens(table, t, out, scale=scale)
        want = torch.where(inside[:, None], table[torch.where(inside, t, 0).long()].double() * scale, 0.0)
        assert bool(((out.double() - want).abs() <= (2 * U + _half_step(out_dtype)) * want.abs()).all())
        if scale == 1.0 and out_dtype == F32:
            assert torch.equal(out.double(), want)
        assert bool((store[:offset] == 555.0).all()) and bool((store[offset:].view(n, D + pad)[:, D:] == 555.0).all())


SHAPES = [(1, 1, 1), (1, 8, 5), (31, 16, 3), (32, 16, 2), (33, 64, 1), (64, 32, 1), (65, 33, 2), (500, 250, 40),
          (1000, 3, 100000), (5000, 24, 511), (5000, 24, 512), (4097, 100, 262143), (9000, 136, 262144), (70000, 20, 1003)]


@pytest.mark.parametrize("mask", [0.0, 0.9])
@pytest.mark.parametrize("n,D,V", SHAPES)
def test_gradient(n, D, V, mask):
    g = torch.Generator(device="cuda").manual_seed(n + D + V)
    t = make_tokens(n, V, g, mask=mask, ignored=0.1)
    d_out = torch.randn((n, D), generator=g, device="cuda")
    check(backward(d_out, t, V, F32, 1.0), d_out, t, V, 1.0)
    check(backward(d_out.to(BF16), t, V, BF16, 0.7), d_out.to(BF16), t, V, 0.7)


@pytest.mark.parametrize("out_dtype,table_dtype", [(F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (4, 0), (2, 2), (1, 3)])
def test_gradient_types_strides_and_accumulation(out_dtype, table_dtype, pad, offset):
    n, D, V, scale = 777, 48, 90, 2.5
    g = torch.Generator(device="cuda").manual_seed(pad + offset)
    t = make_tokens(n, V, g, mask=0.5, ignored=0.1)
    t[t == 13] = 14                                   # a row that stays as it is
    _, d_out = rows_of(n, D, out_dtype, g, pad, offset)
    d_out.copy_(torch.randn((n, D), generator=g, device="cuda"))
    check(backward(d_out, t, V, table_dtype, scale), d_out, t, V, scale)
    before = torch.randn((V, D), generator=g, device="cuda").to(table_dtype)
    d = backward(d_out, t, V, table_dtype, scale, into=before.clone())
    check(d, d_out, t, V, scale, before)
    assert torch.equal(d[13], before[13])


@pytest.mark.parametrize("lengths", [(32, 32, 32), (31, 1, 32, 33, 64, 65, 1), (96, 1, 95), (1, 127, 128), (200,), (16, 48, 16)])
def test_tokens_that_end_at_the_chunks_borders(lengths):
    """Runs of one token after sorting that fill, begin and end chunks of 32 in every way."""
    g = torch.Generator(device="cuda").manual_seed(len(lengths))
    t = torch.cat([torch.full((m,), 2 * i + 1) for i, m in enumerate(lengths)]).to(torch.int32).cuda()
    t = t[torch.randperm(len(t), generator=g, device="cuda")]
    d_out = torch.randn((len(t), 40), generator=g, device="cuda")
    V = 2 * len(lengths) + 2
    check(backward(d_out, t, V, F32), d_out, t, V, 1.0)


def test_ignored_tokens_reach_nothing():
    n, D, V = 300, 64, 50
    g = torch.Generator(device="cuda").manual_seed(3)
    t = make_tokens(n, V, g, ignored=0.4)
    d_out = torch.randn((n, D), generator=g, device="cuda")
    want = backward(d_out, t, V, F32)
    d_out[(t < 0) | (t >= V)] = math.nan
    assert torch.equal(backward(d_out, t, V, F32), want) and not bool(want.isnan().any())
    t.fill_(-1)
    assert bool((backward(d_out, t, V, F32) == 0).all())
    before = torch.randn((V, D), generator=g, device="cuda")
    assert torch.equal(backward(d_out, t, V, F32, into=before.clone()), before)


def test_no_tokens():
    none, V = torch.empty((0, 24), device="cuda"), 30
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    _df().dflash_embed_tokens(torch.ones((V, 24), device="cuda"), t, none)
    assert bool((backward(none, t, V, BF16) == 0).all())
    before = torch.ones((V, 24), device="cuda")
    assert torch.equal(backward(none, t, V, F32, into=before.clone()), before)


def test_infinities_and_nan_stay_in_their_row():
    n, D, V = 200, 32, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    t = make_tokens(n, V, g)
    t[:3] = torch.tensor([0, 1, 1])
    d_out = torch.randn((n, D), generator=g, device="cuda")
    d_out[0, 5], d_out[1, 6], d_out[2, 6] = math.inf, math.inf, -math.inf
    d = backward(d_out, t, V, F32)
    assert float(d[0, 5]) == math.inf and bool(d[1, 6].isnan())
    d[0, 5] = d[1, 6] = 0.0
    d_out[0, 5] = d_out[1, 6] = d_out[2, 6] = 0.0
    assert bool(d.isfinite().all())


def test_a_table_past_32_bits():
    """2.4 G values: a lookup and a gradient in rows behind 2^31, among them the last; rows of zeros everywhere else."""
    V, D, n = 590_000, 4096, 700
    g = torch.Generator(device="cuda").manual_seed(8)
    t = torch.randint(V - 3000, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    t[:3] = torch.tensor([V - 1, 0, V - 1])
    table = torch.zeros((V, D), dtype=BF16, device="cuda")
    table[t.long()] = torch.randn((n, D), generator=g, device="cuda").to(BF16)
    out = torch.empty((n, D), dtype=BF16, device="cuda")
    _df().dflash_embed_tokens(table, t, out)
    assert torch.equal(out, table[t.long()])
    d_out = torch.randn((n, D), generator=g, device="cuda")
    for k in (n, 200):                                    # the sorted form, and the one launch of few tokens
        table.fill_(7.0)
        d = backward(d_out[:k], t[:k], V, BF16, ws=_df().dflash_embed_tokens_backward_workspace(k, D, V))
        low, high = d[:1], d[V - 3000:]
        check(low, d_out[1:2], torch.zeros(1, dtype=torch.int32, device="cuda"), 1, 1.0)
        rest = torch.where(t[:k] >= V - 3000, t[:k] - (V - 3000), -1)
        check(high, d_out[:k], rest, 3000, 1.0)
        assert not bool(d[1:V - 3000].any())
        del d


def test_long_runs_keep_fp32():
    """120,000 terms of one token whose sum is a thousandth of their absolute values' root of squares."""
    n, D = 120000, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    d_out = torch.randn((n, D), generator=g, device="cuda") + 1.0
    t = torch.zeros(n, dtype=torch.int32, device="cuda")
    check(backward(d_out, t, 1, F32), d_out, t, 1, 1.0)


def test_same_bits_streams_and_capture():
    df = _df()
    n, D, V = 6000, 264, 5000
    sets = []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(20 + i)
        sets.append((torch.randn((n, D), generator=g, device="cuda"), make_tokens(n, V, g, mask=0.5 * i, ignored=0.1)))
    want = [backward(d, t, V, BF16) for d, t in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [df.dflash_embed_tokens_backward_workspace(n, D, V) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (d, t), st, x in zip(sets, streams, ws):
            with torch.cuda.stream(st):
                got.append(backward(d, t, V, BF16, ws=x, stream=st))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    d_out, t = sets[0][0].clone(), sets[0][1].clone()
    table, out = torch.randn((V, D), device="cuda"), torch.empty((n, D), dtype=BF16, device="cuda")
    d = torch.empty((V, D), dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df.dflash_embed_tokens(table, t, out)
        df.dflash_embed_tokens_backward(d_out, t, d, ws[0])
    for i in (1, 0):
        d_out.copy_(sets[i][0]), t.copy_(sets[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want[i])
        inside = (t >= 0) & (t < V)
        assert torch.equal(out, torch.where(inside[:, None], table[torch.where(inside, t, 0).long()].to(BF16), 0.0))


def test_binding_refusals():
    df = _df()
    f = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    t = torch.zeros(6, dtype=torch.int32, device="cuda")
    ok = [f(10, 8), t, f(6, 8)]
    for i, bad in ((0, f(10, 7)), (0, f(80)), (0, f(8, 10).t()), (0, f(10, 8).half()), (0, f(10, 8).cpu()), (1, t.long()),
                   (1, t[:5]), (2, f(6, 8).half()), (2, f(8, 6).t()), (2, f(6, 8).cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            df.dflash_embed_tokens(*args)
    ws = df.dflash_embed_tokens_backward_workspace(6, 8, 10)
    for bad in (f(10, 7), f(10, 8).half(), f(10, 8).cpu()):
        with pytest.raises(ValueError):
            df.dflash_embed_tokens_backward(f(6, 8), t, bad, ws)
    with pytest.raises(df.DFlashError):
        df.dflash_embed_tokens_backward(f(6, 8), t, f(10, 8), ws[:512])
    with pytest.raises(df.DFlashError):
        df.dflash_embed_tokens(f(10, 8), t, f(6, 8), scale=math.inf)


@pytest.mark.parametrize("table_dtype,out_dtype,D", [(F32, F32, 40), (BF16, BF16, 40), (F32, BF16, 33), (BF16, F32, 1300)])
def test_runs_over_chunks(table_dtype, out_dtype, D):
    """Runs of one token that begin and end at, before and behind every 32nd sorted token."""
    g = torch.Generator(device="cuda").manual_seed(D)
    for i, choice in enumerate([(1, 31, 32, 33), (32,), (64,), (31, 33), (63, 65), (96, 1), (32, 64, 96, 128), (1, 2, 62, 63, 64, 65, 66),
                                (400, 31), (500,)]):
        lengths = [choice[int(k)] for k in torch.randint(0, len(choice), (24,), generator=torch.Generator().manual_seed(i))]
        t = torch.cat([torch.full((n,), 3 * v + 1) for v, n in enumerate(lengths)] + [torch.tensor([-1] * (i * 7))])
        n, V = t.numel(), 3 * len(lengths)
        t = t.to("cuda", torch.int32)[torch.randperm(n, generator=g, device="cuda")]
        _, d_out = rows_of(n, D, out_dtype, g, 3)
        d_out.copy_(torch.randn((n, D), generator=g, device="cuda"))
        check(backward(d_out, t, V, table_dtype, 0.7), d_out, t, V, 0.7)
        before = torch.randn((V, D), generator=g, device="cuda").to(table_dtype)
        check(backward(d_out, t, V, table_dtype, 0.7, into=before.clone()), d_out, t, V, 0.7, before)


@pytest.mark.parametrize("table_dtype,out_dtype", [(F32, BF16), (BF16, F32), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("D,pad,offset", [(64, 4, 4), (64, 8, 8), (64, 4, 8), (72, 8, 4), (1032, 12, 4), (60, 4, 4), (64, 2, 4)])
def test_rows_at_sixteen_bytes(D, pad, offset, table_dtype, out_dtype):
    """Rows that allow 16 bytes of both types, of the wider one alone, or of neither, by their start, step or length."""
    df = _df()
    g = torch.Generator(device="cuda").manual_seed(D + pad)
    for n in (7, 300):
        V = 50
        t = make_tokens(n, V, g, mask=0.3, ignored=0.1)
        _, d_out = rows_of(n, D, out_dtype, g, pad, offset)
        d_out.copy_(torch.randn((n, D), generator=g, device="cuda"))
        check(backward(d_out, t, V, table_dtype, 1.3), d_out, t, V, 1.3)
        whole = torch.randn(V * D + offset, generator=g, device="cuda").to(table_dtype)
        table = whole[offset:].view(V, D)
        store, out = rows_of(n, D, out_dtype, g, pad, offset, fill=555.0)
        df.dflash_embed_tokens(table, t, out)
        inside = (t >= 0) & (t < V)
        want = torch.where(inside[:, None], table[torch.where(inside, t, 0).long()].float(), 0.0).to(out_dtype)
        assert torch.equal(out, want)
        assert bool((store[:offset] == 555.0).all()) and bool((store[offset:].view(n, D + pad)[:, D:] == 555.0).all())


@pytest.mark.parametrize("table_dtype,out_dtype", [(F32, BF16), (BF16, F32), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("D,pad", [(1032, 0), (1031, 2), (1028, 4)])
def test_many_rows(D, pad, table_dtype, out_dtype):
    """Enough rows for the lookup's accesses in pairs and for the joins of eight columns a lane."""
    df = _df()
    n, V = 20011, 500
    g = torch.Generator(device="cuda").manual_seed(D)
    t = make_tokens(n, V, g, mask=0.2, ignored=0.05)
    _, d_out = rows_of(n, D, out_dtype, g, pad)
    d_out.copy_(torch.randn((n, D), generator=g, device="cuda"))
    check(backward(d_out, t, V, table_dtype, 0.9), d_out, t, V, 0.9)
    table = torch.randn((V, D), generator=g, device="cuda").to(table_dtype)
    store, out = rows_of(n, D, out_dtype, g, pad, fill=555.0)
    df.dflash_embed_tokens(table, t, out)
    inside = (t >= 0) & (t < V)
    want = torch.where(inside[:, None], table[torch.where(inside, t, 0).long()].float(), 0.0).to(out_dtype)
    assert torch.equal(out, want)
    assert bool((store.view(n, D + pad)[:, D:] == 555.0).all())
