"""dflash_clip_grad_norm against sums in 64 bits.

A thread adds up to 64 fp32 squares before it goes on in double: the sum is
within 65 u (u = 2^-24) of its value, the norm within 33 u with its own
rounding, the factor within 34 u, a clipped value within 35 u (bf16: and its
rounding, 2^-8)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = [1, 3, 0, 4096, 8191, 65537, 70001, 5, 300000]


def _df():
    import block_diffusion_drafter_dflash_gb300 as df
    return df


def _grads(sizes, seed, dtypes=(torch.float32, torch.bfloat16), scale=1.0, shift=0):
    """Tensors of the sizes, types in turn, each `shift` elements into its storage."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + shift, generator=g, device="cuda") * scale * (1 + i)
        out.append(t.to(dtypes[i % len(dtypes)])[shift:])
    return out


def _norm(grads):
    return float(torch.sqrt(sum(g.double().square().sum() for g in grads)))


def _clip(grads, max_norm, out=None, **kw):
    norm = torch.full((1,), 777.0, device="cuda")
    _df().dflash_clip_grad_norm(grads, max_norm, norm, out=out, **kw)
    return norm


def _check(before, after, norm, max_norm):
    want = _norm(before)
    assert abs(float(norm) - want) <= 34 * U * want
    if want > max_norm:
        for b, a in zip(before, after):
            w = b.double() * (max_norm / want)
            assert bool(((a.double() - w).abs() <= w.abs() * (36 * U + (2.0 ** -8 * 1.01 if a.dtype == torch.bfloat16 else 0))
                         + 1e-40).all())
    else:
        assert all(torch.equal(a, b) for a, b in zip(after, before))


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("max_norm", [1.0, 1e9])
def test_in_place_and_out_of_place(shift, max_norm):
    grads = _grads(SIZES, 1, shift=shift)
    before = [g.clone() for g in grads]
    out = [torch.full((g.numel() + 2,), 9.0, dtype=g.dtype, device="cuda")[2:] for g in grads]   # another alignment
    same = [torch.empty_like(b) for b in before]
    norm = _clip(grads, max_norm, out=out)
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    _check(before, out, norm, max_norm)
    _clip(grads, max_norm, out=same)
    n2 = _clip(grads, max_norm)
    assert torch.equal(n2, norm)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(grads, out, same))


def test_neighbours_are_left_alone():
    for dtype in (torch.float32, torch.bfloat16):
        store = torch.full((20000,), 3.0, dtype=dtype, device="cuda")
        _clip([store[5:7007], store[7009:19001]], 1.0)
        assert bool((store[:5] == 3).all()) and bool((store[7007:7009] == 3).all()) and bool((store[19001:] == 3).all())
        assert bool((store[5:7007] < 1).all())


@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e-41])
def test_squares_outside_fp32(scale):
    """Gradients whose squares overflow or vanish in fp32 (1e-41: denormal values)."""
    grads = _grads([5000, 3, 4000], 2, dtypes=(torch.float32,), scale=scale)
    before = [g.clone() for g in grads]
    want = _norm(before)
    norm = _clip(grads, want / 4)
    # the double path has no fp32 roundings; fp32's smallest step bounds what denormals lose
    assert abs(float(norm) - want) <= 2 * U * want + 2.0 ** -149
    for b, a in zip(before, grads):
        w = b.double() / 4
        assert bool(((a.double() - w).abs() <= w.abs() * 4 * U + 2.0 ** -149).all())


def test_norm_that_is_not_finite_changes_nothing():
    for bad in (float("inf"), float("nan")):
        grads = _grads([1000, 5000], 3)
        grads[1][17] = bad
        before = [g.clone() for g in grads]
        norm = _clip(grads, 1.0)
        assert not bool(norm.isfinite().all())
        assert all(torch.equal(g.nan_to_num(7.0, 8.0), b.nan_to_num(7.0, 8.0)) for g, b in zip(grads, before))
        out = [torch.zeros_like(g) for g in grads]
        _clip(grads, 1.0, out=out)
        assert all(torch.equal(g.nan_to_num(7.0, 8.0), b.nan_to_num(7.0, 8.0)) for g, b in zip(out, before))


def test_no_tensors_zero_gradients_and_limits():
    assert float(_clip([], 1.0)) == 0.0
    z = [torch.zeros(1000, device="cuda"), torch.zeros(7, device="cuda", dtype=torch.bfloat16)]
    assert float(_clip(z, 1.0)) == 0.0
    grads = _grads([1000, 2000], 4)
    before = [g.clone() for g in grads]
    norm = _clip(grads, float("inf"))                       # the norm alone
    _check(before, grads, norm, float("inf"))
    _clip(grads, 0.0)                                       # a limit of 0 clips to nothing
    assert all(bool((g == 0).all()) for g in grads)


def test_more_tensors_than_one_launch_holds():
    grads = _grads([17 + 31 * (i % 90) for i in range(1100)], 5)
    before = [g.clone() for g in grads]
    norm = _clip(grads, 2.0)
    _check(before, grads, norm, 2.0)


def test_same_bits_every_time_and_under_a_graph():
    df = _df()
    grads = _grads([2_000_000, 999, 123457], 6)
    out = [torch.empty_like(g) for g in grads]
    norm, ws = torch.empty(1, device="cuda"), df.dflash_clip_workspace()
    first = _clip(grads, 1.0, out=out).clone()
    kept = [o.clone() for o in out]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        df.dflash_clip_grad_norm(grads, 1.0, norm, out=out, stream=side)
    side.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(a, b) for a, b in zip(out, kept))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df.dflash_clip_grad_norm(grads, 1.0, norm, out=out, workspace=ws)
    for g in grads:
        g.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm) == 2 * float(first)
    assert all(torch.equal(a, b) for a, b in zip(out, kept))   # half of twice: the same values


def test_wrapper_refusals():
    df = _df()
    g = torch.ones(8, device="cuda")
    norm = torch.empty(1, device="cuda")
    for grads, kw in (([g.double()], {}), ([g.view(2, 4).t()], {}), ([g.cpu()], {}), ([g], dict(out=[])),
                      ([g], dict(out=[torch.ones(7, device="cuda")])), ([g], dict(out=[g.bfloat16()]))):
        with pytest.raises(ValueError):
            df.dflash_clip_grad_norm(grads, 1.0, norm, **kw)
    for grads, most in (([g, g], 1.0), ([g], -1.0), ([g[:5], g[4:]], 1.0)):
        with pytest.raises(df.DFlashError):
            df.dflash_clip_grad_norm(grads, most, norm)
    with pytest.raises(df.DFlashError):
        df.dflash_clip_grad_norm([g], 1.0, norm, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_offsets_past_32_bits():
    """A tensor of more than 2^31 values, a short one before and behind it."""
    n, reps = 1 << 20, 2049
    base = _grads([n], 3, dtypes=(torch.bfloat16,))[0]
    big, ends = base.repeat(reps), _grads([77, 300], 4)
    assert big.numel() > 2 ** 31
    grads = [ends[0], big, ends[1]]
    before = [ends[0].clone(), ends[1].clone()]
    want = float(torch.sqrt(reps * base.double().square().sum() + sum(g.double().square().sum() for g in before)))
    norm = _clip(grads, 1.0)
    assert abs(float(norm) - want) <= 34 * U * want
    first = big[:n].clone()
    assert bool((big.view(reps, n) == first).all())
    for b, a in zip((base, *before), (first, ends[0], ends[1])):
        w = b.double() / want
        assert bool(((a.double() - w).abs() <= w.abs() * (36 * U + (2.0 ** -8 * 1.01 if a.dtype == torch.bfloat16 else 0))
                     + 1e-40).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e-6])
def test_factor_outside_fp32(max_norm, dtype):
    """Gradients near fp32's largest: norm_dev is infinite, the norm finite in double, and max_norm / norm below
    fp32's normal range (2.5e-46 in the last case, which no fp32 holds)."""
    grads = _grads([5000, 3, 4000], 2, dtypes=(dtype,), scale=2e37)
    before = [g.clone() for g in grads]
    want = _norm(before)
    assert 3.5e38 < want < 1e40 and all(bool(g.isfinite().all()) for g in grads)
    norm = _clip(grads, max_norm)
    assert float(norm) == float("inf")
    own = 36 * U + (2.0 ** -8 * 1.01 if dtype == torch.bfloat16 else 0)
    for b, a in zip(before, grads):
        w = b.double() * (float(torch.tensor(max_norm)) / want)
        assert bool(((a.double() - w).abs() <= w.abs() * own + 1e-40).all())
