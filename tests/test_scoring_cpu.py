"""Host-side checks of the scoring and clipping entry points that need no GPU:
every refusal happens before a launch, and the reference formulas that the GPU
tests hold the kernels to agree with differences of the definitions."""
import ctypes

import numpy as np
import pytest

from test_abi_cpu import L  # noqa: F401  (the built library)

P = 1 << 20      # an address that no check dereferences
INF = float("inf")


def _logprobs(L, logits=P, dtype=0, stride=8, tokens=P, rows=2, vocab=8, temp=1.0, k=0, logprob=P, entropy=None,
              lse=None, ids=None, top=None):
    return L.dflash_token_logprobs(logits, dtype, stride, tokens, rows, vocab, temp, k, logprob, entropy, lse, ids, top,
                                   None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(rows=65536), -2), (dict(vocab=0), -2), (dict(vocab=(1 << 24) + 1), -2),
    (dict(temp=0.0), -1), (dict(temp=-1.0), -1), (dict(temp=INF), -1), (dict(temp=float("nan")), -1),
    (dict(temp=1e-45), -1),                                    # its reciprocal overflows
    (dict(dtype=2), -1), (dict(stride=7), -1), (dict(logits=P + 2), -1), (dict(logits=P + 1, dtype=1), -1),
    (dict(logits=None), -1), (dict(tokens=None), -1), (dict(logprob=None), -1),
    (dict(tokens=None, logprob=None), -1),                     # nothing asked for
    (dict(k=-1), -2), (dict(k=33, vocab=100, stride=100), -2), (dict(k=9), -2), (dict(k=4), -1),
    (dict(k=4, ids=P), -1),
])
def test_logprob_refusals(L, kw, code):  # noqa: F811
    assert _logprobs(L, **kw) == code
    assert len(L.dflash_last_error()) > 0


def test_no_rows_is_no_launch(L):  # noqa: F811
    assert _logprobs(L, rows=0, logits=None, tokens=None, logprob=None) == 0
    assert _backward(L, rows=0, logits=None, lse=None, d_logits=None) == 0


def _backward(L, logits=P, dtype=0, stride=8, tokens=P, rows=2, vocab=8, temp=1.0, lse=P, entropy=None, d_logprob=P,
              d_entropy=None, d_logits=2 * P, d_stride=8):
    return L.dflash_token_logprobs_backward(logits, dtype, stride, tokens, rows, vocab, temp, lse, entropy, d_logprob,
                                            d_entropy, d_logits, d_stride, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(vocab=0), -2), (dict(temp=0.0), -1), (dict(dtype=7), -1), (dict(stride=7), -1),
    (dict(d_stride=7), -1), (dict(lse=None), -1), (dict(d_logits=None), -1), (dict(tokens=None), -1),
    (dict(d_logprob=None), -1), (dict(d_entropy=P), -1), (dict(d_logits=2 * P + 1), -1),
    (dict(d_logits=P + 4), -1),                                # shifted by one element: read after written
    (dict(d_logits=P, d_stride=9), -1), (dict(d_logits=P + 4 * 15), -1),
])
def test_logprob_gradient_refusals(L, kw, code):  # noqa: F811
    assert _backward(L, **kw) == code


def _clip(L, tensors, out=None, max_norm=1.0, norm=P + 4096, ws=P, ws_bytes=1 << 20, n=None):
    """tensors: (address, numel, dtype)"""
    k = len(tensors)
    ptrs = (ctypes.c_void_p * k)(*[t[0] for t in tensors])
    outs = None if out is None else (ctypes.c_void_p * k)(*out)
    return L.dflash_clip_grad_norm(ptrs, outs, (ctypes.c_int64 * k)(*[t[1] for t in tensors]),
                                   (ctypes.c_int32 * k)(*[t[2] for t in tensors]), k if n is None else n, max_norm,
                                   norm, ws, ws_bytes, None)


@pytest.mark.parametrize("tensors,kw,code", [
    ([(P, 4, 0)], dict(n=-1), -1), ([(P, 4, 0)], dict(max_norm=-1.0), -1), ([(P, 4, 0)], dict(max_norm=float("nan")), -1),
    ([(P, 4, 0)], dict(norm=None), -1), ([(P, 4, 0)], dict(ws=None), -1), ([(P, 4, 0)], dict(ws=P + 4), -1),
    ([(None, 4, 0)], {}, -1), ([(P, -1, 0)], {}, -2), ([(P, 4, 3)], {}, -1), ([(P + 2, 4, 0)], {}, -1),
    ([(P + 1, 4, 1)], {}, -1),
    ([(P, 4, 0), (P, 4, 0)], {}, -1),                          # one tensor twice, in place
    ([(P, 4, 0), (P + 12, 4, 0)], {}, -1),                     # two that overlap
    ([(P, 4, 0), (P + 64, 4, 0)], dict(out=[P + 256, P + 264]), -1),
    ([(P, 4, 0), (P + 64, 4, 0)], dict(out=[P + 72, P + 256]), -1),     # an output over another's input
    ([(P, 4, 0)], dict(out=[P + 4]), -1),                      # an output over its own input, shifted
    ([(P, 4, 0)], dict(out=[None]), -1),
    ([(P, 4, 0)], dict(norm=P + 12), -1),                      # the norm inside a gradient
    ([(P, 4, 0)], dict(out=[P + 64], norm=P + 4), -1),
])
def test_clip_refusals(L, tensors, kw, code):  # noqa: F811
    assert _clip(L, tensors, **kw) == code
    assert len(L.dflash_last_error()) > 0


# ---------------------------------------------------------------- reference formulas (64 bits)
def logprob_reference(x, tokens, temp):
    """(logprob, entropy, lse) of fp64 rows by the definition."""
    z = np.asarray(x, np.float64) / temp
    m = z.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        ln_s = np.log(np.exp(z - m).sum(axis=1))
        lse = m[:, 0] + ln_s
        logp = (z - m) - ln_s[:, None]      # not z - lse: a maximum at fp32's lowest value swallows ln S
        plogp = np.where(logp == -INF, 0.0, np.exp(logp) * np.where(logp == -INF, 0.0, logp))
    lp = np.array([logp[r, t] if 0 <= t < z.shape[1] else 0.0 for r, t in enumerate(tokens)])
    return lp, -plogp.sum(axis=1), lse


def logprob_grad_reference(x, tokens, temp, d_lp, d_h):
    z = np.asarray(x, np.float64) / temp
    _, h, lse = logprob_reference(x, tokens, temp)
    logp = z - lse[:, None]
    p = np.exp(logp)
    g = np.array([d if 0 <= t < z.shape[1] else 0.0 for t, d in zip(tokens, d_lp)])
    out = -g[:, None] * p
    for r, t in enumerate(tokens):
        if 0 <= t < z.shape[1]:
            out[r, t] += g[r]
    if d_h is not None:
        out -= np.asarray(d_h)[:, None] * np.where(p > 0, p * (np.where(p > 0, logp, 0.0) + h[:, None]), 0.0)
    return out / temp


def test_reference_gradient_is_the_difference_of_the_definition():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 7)) * 2
    x[1, 2] = -INF
    tokens, temp = [3, 0, -1], 0.7
    d_lp, d_h = rng.normal(size=3), rng.normal(size=3)

    def f(y):
        lp, h, _ = logprob_reference(y, tokens, temp)
        return float((lp * d_lp).sum() + (h * d_h).sum())

    g, eps = logprob_grad_reference(x, tokens, temp, d_lp, d_h), 1e-6
    for r in range(3):
        for v in range(7):
            if x[r, v] == -INF:
                assert g[r, v] == 0.0
                continue
            a, b = x.copy(), x.copy()
            a[r, v] += eps
            b[r, v] -= eps
            # central differences: O(eps^2) truncation and 2^-52 |f| / eps rounding, both under 1e-8 here
            assert abs((f(a) - f(b)) / (2 * eps) - g[r, v]) < 1e-8


@pytest.mark.parametrize("temp", [2.95e-39, 4.2e-39])
def test_temperature_whose_exponent_scale_overflows_is_refused(L, temp):  # noqa: F811
    """1 / T is finite, log2(e) / T is not."""
    assert np.isfinite(np.float32(1) / np.float32(temp))
    assert _logprobs(L, temp=temp) == -1
    assert _backward(L, temp=temp) == -1
    assert _logprobs(L, rows=0, temp=4.3e-39) == 0      # both are finite


def test_workspace_on_another_device_is_refused():
    """By the device's number alone: stand-ins for tensors of two devices."""
    import block_diffusion_drafter_dflash_gb300 as df

    class OnDevice:
        is_cuda = True

        def __init__(self, device):
            self.index, self.device = device, f"cuda:{device}"

        get_device = lambda self: self.index  # noqa: E731
        is_contiguous = lambda self: True  # noqa: E731
        data_ptr = lambda self: P  # noqa: E731
        numel = lambda self: 100  # noqa: E731
        element_size = lambda self: 2  # noqa: E731

    assert df._workspace(OnDevice(1), OnDevice(1)) == (P, 200)
    with pytest.raises(ValueError):
        df._workspace(OnDevice(1), OnDevice(0))
