"""Host-side checks of the cross-entropy at the LM head and of the token embedding
that need no GPU: every refusal happens before a launch, and the reference
formulas that the GPU tests hold the kernels to agree with differences of the
definitions."""
import numpy as np
import pytest
import torch

from test_abi_cpu import L  # noqa: F401  (the built library)

P = 1 << 32      # an address that no check dereferences
INF = float("inf")


def _loss(L, hidden=P, dtype=0, stride=16, weight=2 * P, targets=3 * P, rows=2, dim=16, vocab=8, temp=1.0, loss=4 * P,
          lse=5 * P, ws=6 * P, ws_bytes=1 << 40):
    return L.dflash_linear_cross_entropy(hidden, dtype, stride, weight, targets, rows, dim, vocab, temp, loss, lse, ws,
                                         ws_bytes, None)


SHARED = [
    (dict(rows=-1), -1), (dict(rows=(1 << 20) + 1), -2), (dict(dim=0), -2), (dict(dim=12), -2), (dict(dim=65544), -2),
    (dict(vocab=0), -2), (dict(vocab=(1 << 24) + 1), -2), (dict(dtype=2), -1), (dict(temp=0.0), -1),
    (dict(temp=-1.0), -1), (dict(temp=INF), -1), (dict(temp=float("nan")), -1), (dict(temp=4.2e-39), -1),
    (dict(stride=15), -1), (dict(hidden=None), -1), (dict(weight=None), -1), (dict(targets=None), -1),
    (dict(hidden=P + 2), -1), (dict(hidden=P + 1, dtype=1), -1), (dict(targets=3 * P + 2), -1), (dict(weight=2 * P + 8), -1), (dict(ws=None), -1),
    (dict(ws=6 * P + 128), -1),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(loss=None), -1), (dict(lse=None), -1), (dict(loss=4 * P + 2), -1),
    (dict(loss=5 * P + 4), -1), (dict(loss=P + 64), -1), (dict(lse=2 * P), -1), (dict(lse=3 * P + 4), -1),   # one over another
])
def test_loss_refusals(L, kw, code):  # noqa: F811
    assert _loss(L, **kw) == code
    assert len(L.dflash_last_error()) > 0


def _loss_grad(L, hidden=P, dtype=0, stride=16, weight=2 * P, targets=3 * P, rows=2, dim=16, vocab=8, temp=1.0, lse=4 * P,
               d_loss=5 * P, d_hidden=7 * P, d_stride=16, d_weight=8 * P, ws=6 * P, ws_bytes=1 << 40):
    return L.dflash_linear_cross_entropy_backward(hidden, dtype, stride, weight, targets, rows, dim, vocab, temp, lse,
                                                  d_loss, d_hidden, d_stride, d_weight, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(lse=None), -1), (dict(d_loss=None), -1), (dict(lse=4 * P + 1), -1), (dict(d_loss=5 * P + 2), -1), (dict(d_hidden=None, d_weight=None), -1), (dict(d_stride=15), -1),
    (dict(d_hidden=7 * P + 2), -1), (dict(d_weight=8 * P + 4), -1),
    (dict(d_hidden=P + 4), -1), (dict(d_hidden=P, d_stride=17), -1),     # the hidden states' place, but not their rows
    (dict(d_hidden=2 * P + 64), -1), (dict(d_weight=2 * P), -1), (dict(d_weight=P + 16), -1),
    (dict(d_hidden=8 * P + 16), -1),                                     # the other gradient
    (dict(d_hidden=4 * P), -1), (dict(d_weight=5 * P), -1), (dict(d_hidden=3 * P + 4), -1),     # lse, d_loss, targets
])
def test_loss_gradient_refusals(L, kw, code):  # noqa: F811
    assert _loss_grad(L, **kw) == code
    assert len(L.dflash_last_error()) > 0


def test_workspace_sizes_of_bad_shapes_are_zero(L):  # noqa: F811
    for f in (L.dflash_linear_cross_entropy_workspace_bytes, L.dflash_linear_cross_entropy_backward_workspace_bytes):
        assert f(-1, 16, 8, 0) == f(2, 12, 8, 0) == f(2, 16, 0, 0) == f(2, 16, 8, 3) == 0
    f = L.dflash_embed_tokens_backward_workspace_bytes
    assert f(-1, 16, 8) == f(2, 0, 8) == f(2, 16, 0) == f((1 << 24) + 1, 16, 8) == 0
    assert f(0, 16, 8) > 0


def _embed(L, table=P, table_dtype=0, vocab=8, dim=5, tokens=2 * P, n=3, scale=1.0, out=3 * P, out_dtype=0, stride=5):
    return L.dflash_embed_tokens(table, table_dtype, vocab, dim, tokens, n, scale, out, out_dtype, stride, None)


def _embed_grad(L, table=P, table_dtype=0, vocab=8, dim=5, tokens=2 * P, n=3, scale=1.0, out=3 * P, out_dtype=0, stride=5,
                accumulate=0, ws=6 * P, ws_bytes=1 << 40):
    return L.dflash_embed_tokens_backward(out, out_dtype, stride, tokens, n, vocab, dim, scale, table, table_dtype,
                                          accumulate, ws, ws_bytes, None)


EMBED = [
    (dict(n=-1), -1), (dict(n=(1 << 24) + 1), -2), (dict(dim=0), -2), (dict(dim=65537, stride=65537), -2),
    (dict(vocab=0), -2), (dict(vocab=(1 << 24) + 1), -2), (dict(table_dtype=4), -1), (dict(out_dtype=-1), -1),
    (dict(scale=INF), -1), (dict(scale=float("nan")), -1), (dict(table=None), -1), (dict(tokens=None), -1),
    (dict(out=None), -1), (dict(stride=4), -1), (dict(table=P + 2), -1), (dict(out=3 * P + 1, out_dtype=1), -1), (dict(tokens=2 * P + 2), -1),
    (dict(out=P + 8), -1), (dict(out=2 * P + 4), -1), (dict(tokens=P + 16), -1),      # one tensor over another
]


@pytest.mark.parametrize("kw,code", EMBED)
def test_embed_refusals(L, kw, code):  # noqa: F811
    assert _embed(L, **kw) == code
    assert len(L.dflash_last_error()) > 0


@pytest.mark.parametrize("kw,code", EMBED + [
    (dict(accumulate=2), -1), (dict(ws=None), -1), (dict(ws=6 * P + 16), -1), (dict(ws_bytes=100), -7)])
def test_embed_gradient_refusals(L, kw, code):  # noqa: F811
    assert _embed_grad(L, **kw) == code
    assert len(L.dflash_last_error()) > 0


def test_no_tokens_is_no_launch(L):  # noqa: F811
    assert _embed(L, n=0, table=None, tokens=None, out=None) == 0


# ---------------------------------------------------------------- reference formulas (64 bits)
def loss_reference(h, w, targets, temp):
    """(loss, lse) of fp64 tensors by the definition; 0 in ignored rows, whatever they hold."""
    V = w.shape[0]
    inside = (targets >= 0) & (targets < V)
    z = torch.where(inside[:, None], h, 0.0) @ w.t() / temp
    lse = torch.logsumexp(z, dim=1)
    picked = z.gather(1, torch.where(inside, targets, 0).long()[:, None])[:, 0]
    return torch.where(inside, lse - picked, 0.0), torch.where(inside, lse, 0.0)


def loss_grad_reference(h, w, targets, temp, d_loss):
    """(d_hidden, d_weight, G) by the formula."""
    V = w.shape[0]
    inside = (targets >= 0) & (targets < V)
    h = torch.where(inside[:, None], h, 0.0)
    p = torch.softmax(h @ w.t() / temp, dim=1)
    p[torch.arange(len(targets)), torch.where(inside, targets, 0).long()] -= 1.0
    g = p * torch.where(inside, d_loss, 0.0)[:, None] / temp
    return g @ w, g.t() @ h, g


def test_reference_gradient_is_the_difference_of_the_definition():
    rng = np.random.default_rng(0)
    h, w = torch.tensor(rng.normal(size=(4, 6))), torch.tensor(rng.normal(size=(5, 6)))
    targets, temp = torch.tensor([3, 0, -1, 5]), 0.7          # the last two are ignored
    d_loss = torch.tensor(rng.normal(size=4))
    d_h, d_w, _ = loss_grad_reference(h, w, targets, temp, d_loss)
    f = lambda a, b: float((loss_reference(a, b, targets, temp)[0] * d_loss).sum())  # noqa: E731
    eps = 1e-6
    for x, g, other in ((h, d_h, "h"), (w, d_w, "w")):
        for i in range(x.shape[0]):
            for j in range(x.shape[1]):
                a, b = x.clone(), x.clone()
                a[i, j] += eps
                b[i, j] -= eps
                up, down = (f(a, w), f(b, w)) if other == "h" else (f(h, a), f(h, b))
                # central differences: O(eps^2) truncation and 2^-52 |f| / eps rounding, both under 1e-8 here
                assert abs((up - down) / (2 * eps) - float(g[i, j])) < 1e-8


def embed_grad_reference(d_out, tokens, vocab, scale):
    """(gradient, sums of the absolute values) in 64 bits."""
    inside = (tokens >= 0) & (tokens < vocab)
    at = tokens[inside].long()
    d = d_out[inside].double() * scale
    zero = lambda: torch.zeros((vocab, d_out.shape[1]), dtype=torch.float64, device=d_out.device)  # noqa: E731
    return zero().index_add_(0, at, d), zero().index_add_(0, at, d.abs())


def test_embed_reference_gradient_is_the_difference_of_the_definition():
    rng = np.random.default_rng(1)
    table, d_out = torch.tensor(rng.normal(size=(4, 3))), torch.tensor(rng.normal(size=(6, 3)))
    tokens, scale = torch.tensor([1, 3, 1, -1, 4, 1]), 1.5

    def f(t):
        inside = (tokens >= 0) & (tokens < 4)
        out = torch.where(inside[:, None], t[torch.where(inside, tokens, 0)] * scale, 0.0)
        return float((out * d_out).sum())

    g = embed_grad_reference(d_out, tokens, 4, scale)[0]
    for v in range(4):
        for j in range(3):
            a, b = table.clone(), table.clone()
            a[v, j] += 0.5
            b[v, j] -= 0.5
            assert abs(f(a) - f(b) - float(g[v, j])) < 1e-12      # linear: the difference is exact
