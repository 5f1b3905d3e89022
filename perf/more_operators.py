"""Timed cases of the two ends of a drafter's training step: the token embedding
and the loss at the LM head.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and as the calls a user makes of the package:

  loss / loss_grad     softmax cross-entropy of hidden states against an LM head, in
                       pieces of the vocabulary, without keeping the logits; its
                       gradient for the hidden states and, where the head is trained,
                       for the head
  embed / embed_grad   embedding lookup with a factor, and its gradient summed token
                       by token

``own`` selects the package's calls.  Inputs come from the seed alone.
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16


def _dt(name):
    return F32 if name == "fp32" else BF16


def _es(name):
    return 4 if name == "fp32" else 2


def listed():
    return [
        # the tiny fp32 drafter's loss over a few blocks (latency)
        dict(name="loss tiny", op="loss", dtype="fp32", rows=48, dim=256, vocab=1024, pad=0, ignored=0.25, temp=1.0),
        # one block of the 8B-shaped drafter scored against its own head: the head is read once
        dict(name="loss one block", op="loss", dtype="bf16", rows=15, dim=4096, vocab=151936, pad=0, ignored=0.0,
             temp=1.0),
        # a full training sequence: 512 blocks of 16 whose anchors carry no loss
        dict(name="loss training", op="loss", dtype="bf16", rows=8192, dim=4096, vocab=151936, pad=0,
             ignored=0.0625, temp=1.0),
        # an odd vocabulary, hidden states with a pad behind each row, a third of the rows ignored
        dict(name="loss odd", op="loss", dtype="bf16", rows=777, dim=2560, vocab=32003, pad=8, ignored=0.3, temp=0.7),
        # the gradient for the hidden states alone: the drafter's head is the target's, and frozen
        dict(name="loss gradient frozen head", op="loss_grad", dtype="bf16", rows=4096, dim=4096, vocab=151936, pad=0,
             ignored=0.0625, temp=1.0, weight=False),
        # the 4B-shaped drafter with a head that is trained too
        dict(name="loss gradient trained head", op="loss_grad", dtype="bf16", rows=2048, dim=2560, vocab=151936,
             pad=0, ignored=0.0625, temp=1.0, weight=True),
        # both gradients in fp32, an odd vocabulary, few rows
        dict(name="loss gradient fp32", op="loss_grad", dtype="fp32", rows=333, dim=256, vocab=8705, pad=3,
             ignored=0.1, temp=1.3, weight=True),
        # one block's tokens at serving time, bf16 table to the fp32 residual stream (latency)
        dict(name="embed one block", op="embed", dtype="bf16", act="fp32", tokens=16, dim=4096, vocab=151936,
             mask=0.9375, ignored=0.0, scale=1.0),
        # the training sequence's blocks: anchors and, fifteen times as many, the mask token
        dict(name="embed training", op="embed", dtype="bf16", act="fp32", tokens=8192, dim=4096, vocab=151936,
             mask=0.9375, ignored=0.0, scale=1.0),
        # its gradient: one row of the table collects fifteen sixteenths of it
        dict(name="embed gradient training", op="embed_grad", dtype="bf16", act="fp32", tokens=8192, dim=4096,
             vocab=151936, mask=0.9375, ignored=0.0, scale=1.0),
        # text with a long tail of words, padding among it, a factor of sqrt(dim)
        dict(name="embed gradient text", op="embed_grad", dtype="fp32", act="bf16", tokens=50001, dim=1000, vocab=32003,
             mask=0.0, ignored=0.1, scale=31.6),
        # a handful of tokens of the tiny drafter (latency)
        dict(name="embed gradient tiny", op="embed_grad", dtype="fp32", act="fp32", tokens=48, dim=256, vocab=1024,
             mask=0.75, ignored=0.0, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("loss", "loss", "loss_grad", "loss_grad", "embed", "embed_grad", "embed_grad"))
    if kind in ("loss", "loss_grad"):
        fp32 = rng.random() < 0.25
        dim = 8 * _log_int(rng, 8, 640)
        vocab = _log_int(rng, 300, 152000)
        weight = kind == "loss_grad" and rng.random() < 0.5
        most = 1e11 if fp32 else 4e12 if kind == "loss" else 1.2e12 if weight else 2e12   # rows x dim x vocab
        rows = _log_int(rng, 1, max(1, min(8192, int(most / (dim * vocab)))))
        case = dict(op=kind, dtype="fp32" if fp32 else "bf16", rows=rows, dim=dim, vocab=vocab,
                    pad=rng.choice((0, 0, 1, 8, 61)), ignored=rng.choice((0.0, 0.0625, 0.5)),
                    temp=rng.choice((1.0, 0.6, 1.5)))
        if kind == "loss_grad":
            case["weight"] = weight
        return case
    dim = _log_int(rng, 32, 5120)
    vocab = _log_int(rng, 300, 152000)
    return dict(op=kind, dtype=rng.choice(("fp32", "bf16")), act=rng.choice(("fp32", "bf16")),
                tokens=_log_int(rng, 1, max(1, min(60000, int(1.5e8 / dim)))), dim=dim, vocab=vocab,
                mask=rng.choice((0.0, 0.9, 0.9375)), ignored=rng.choice((0.0, 0.0, 0.1)),
                scale=rng.choice((1.0, 0.5, 11.3)))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    uni = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    if case["op"] in ("loss", "loss_grad"):
        return _prepare_loss(case, g, rnd, uni)
    n, D, V = case["tokens"], case["dim"], case["vocab"]
    # a long-tailed choice of words, the mask token (the last id) and padding (-1)
    tokens = (V * uni(n) ** 3).long().clamp(max=V - 1)
    tokens = torch.where(uni(n) < case["mask"], V - 1, tokens)
    tokens = torch.where(uni(n) < case["ignored"], -1, tokens).to(torch.int32)
    s = dict(op=case["op"], tokens=tokens, scale=case["scale"], vocab=V, ws=[])
    if case["op"] == "embed":
        s.update(table=(rnd(V, D) * 0.02).to(_dt(case["dtype"])),
                 out=torch.empty((n, D), dtype=_dt(case["act"]), device="cuda"))
    else:
        s.update(d_out=(rnd(n, D) / n).to(_dt(case["act"])),
                 d_table=torch.empty((V, D), dtype=_dt(case["dtype"]), device="cuda"))
    return s


def _prepare_loss(case, g, rnd, uni):
    """Normed hidden states that lean towards their target's row of the head by an amount of their own: targets of
    all probabilities; ignored rows have the target -1."""
    R, D, V, dt = case["rows"], case["dim"], case["vocab"], _dt(case["dtype"])
    head = torch.empty((V, D), dtype=dt, device="cuda")
    for v in range(0, V, 32768):
        head[v:v + 32768] = rnd(min(32768, V - v), D) * 0.02
    targets = torch.randint(0, V, (R,), generator=g, device="cuda")
    lean = 16.0 * uni(R, 1) / (0.0004 * D)
    store = torch.zeros((R, D + case["pad"]), dtype=dt, device="cuda")
    hidden = store[:, :D]
    hidden.copy_(rnd(R, D) + lean * head[targets].float())
    targets = torch.where(uni(R) < case["ignored"], -1, targets).to(torch.int32)
    new = lambda *sh, dtype=F32: torch.empty(sh, dtype=dtype, device="cuda")  # noqa: E731
    s = dict(op=case["op"], hidden=hidden, head=head, targets=targets, temp=case["temp"], ws=[])
    if case["op"] == "loss":
        s.update(loss=new(R), lse=new(R))
    else:
        _, lse = _loss_plain(s)
        s.update(lse=lse, d_loss=(0.1 + uni(R)) / R, d_hidden=new(R, D, dtype=dt),
                 d_head=new(V, D, dtype=dt) if case["weight"] else None)
    return s


# ---------------------------------------------------------------- plain forms
def _loss_plain(s):
    """Per row ln sum_v e^(z_v) - z_target with z = hidden head' / T; 0 for ignored rows."""
    z = torch.matmul(s["hidden"].float(), s["head"].float().t()).div_(s["temp"])
    inside = (s["targets"] >= 0) & (s["targets"] < z.shape[1])
    picked = z.gather(1, torch.where(inside, s["targets"], 0).long()[:, None])[:, 0]
    m = z.max(dim=1, keepdim=True).values
    lse = m[:, 0] + z.sub_(m).exp_().sum(dim=1, dtype=torch.float64).log().float()
    return torch.where(inside, lse - picked, 0.0), torch.where(inside, lse, 0.0)


def _loss_grad_plain(s):
    """G = d_loss / T (softmax(z) - 1[target]); G head and G' hidden."""
    h, w = s["hidden"].float(), s["head"].float()
    inside = (s["targets"] >= 0) & (s["targets"] < w.shape[0])
    g = torch.where(inside, s["d_loss"], 0.0)[:, None] / s["temp"]
    p = torch.matmul(h, w.t()).div_(s["temp"]).sub_(s["lse"][:, None]).exp_().mul_(g)
    p.scatter_add_(1, torch.where(inside, s["targets"], 0).long()[:, None], -g)
    d_hidden = torch.matmul(p, w).to(s["hidden"].dtype)
    if s["d_head"] is None:
        return dict(d_hidden=d_hidden)
    return dict(d_hidden=d_hidden, d_head=torch.matmul(p.t(), h).to(s["head"].dtype))


def _embed_plain(s):
    inside = (s["tokens"] >= 0) & (s["tokens"] < s["vocab"])
    rows = s["table"][torch.where(inside, s["tokens"], 0).long()].float() * s["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(s["out"].dtype)


def _embed_grad_plain(s):
    inside = (s["tokens"] >= 0) & (s["tokens"] < s["vocab"])
    d = torch.zeros(s["d_table"].shape, dtype=F32, device="cuda")
    d.index_add_(0, torch.where(inside, s["tokens"], 0).long(), torch.where(inside[:, None], s["d_out"].float(), 0.0))
    return d.mul_(s["scale"]).to(s["d_table"].dtype)


# ---------------------------------------------------------------- one pass
def run(s):
    if s["op"] == "loss":
        if own:
            import block_diffusion_drafter_dflash_gb300 as df
            (R, D), V = s["hidden"].shape, s["head"].shape[0]
            if not s["ws"]:
                s["ws"].append(df.dflash_linear_cross_entropy_workspace(R, D, V, s["head"].dtype))
            df.dflash_linear_cross_entropy(s["hidden"], s["head"], s["targets"], s["loss"], s["lse"], s["ws"][0],
                                           temperature=s["temp"])
            return dict(loss=s["loss"], lse=s["lse"])
        return dict(zip(("loss", "lse"), _loss_plain(s)))
    if s["op"] == "loss_grad":
        if own:
            import block_diffusion_drafter_dflash_gb300 as df
            (R, D), V = s["hidden"].shape, s["head"].shape[0]
            if not s["ws"]:
                s["ws"].append(df.dflash_linear_cross_entropy_backward_workspace(R, D, V, s["head"].dtype))
            df.dflash_linear_cross_entropy_backward(s["hidden"], s["head"], s["targets"], s["lse"], s["d_loss"],
                                                    s["d_hidden"], s["d_head"], s["ws"][0], temperature=s["temp"])
            r = dict(d_hidden=s["d_hidden"])
            return r if s["d_head"] is None else dict(r, d_head=s["d_head"])
        return _loss_grad_plain(s)
    if s["op"] == "embed":
        if own:
            import block_diffusion_drafter_dflash_gb300 as df
            df.dflash_embed_tokens(s["table"], s["tokens"], s["out"], scale=s["scale"])
            return s["out"]
        return _embed_plain(s)
    if own:
        import block_diffusion_drafter_dflash_gb300 as df
        if not s["ws"]:
            n, D = s["d_out"].shape
            s["ws"].append(df.dflash_embed_tokens_backward_workspace(n, D, s["vocab"]))
        df.dflash_embed_tokens_backward(s["d_out"], s["tokens"], s["d_table"], s["ws"][0], scale=s["scale"])
        return s["d_table"]
    return _embed_grad_plain(s)


def work(case):
    if case["op"] in ("loss", "loss_grad"):
        R, D, V, es = case["rows"], case["dim"], case["vocab"], _es(case["dtype"])
        kept = R * (1.0 - case["ignored"])          # ignored rows need no logits
        product = 2.0 * kept * D * V
        if case["op"] == "loss":
            return dict(bytes=V * D * es + kept * D * es + 12 * R, flops=product)
        # the logits once more, then one product for each gradient
        weight = case["weight"]
        return dict(bytes=V * D * es * (2 if weight else 1) + (kept + R) * D * es + 12 * R,
                    flops=product * (3 if weight else 2))
    n, D, V = case["tokens"], case["dim"], case["vocab"]
    kept = n * (1.0 - case["ignored"])
    if case["op"] == "embed":
        read = min(V, kept * (1.0 - case["mask"]) + 1)   # the mask token's row counts once
        return dict(bytes=read * D * _es(case["dtype"]) + n * D * _es(case["act"]) + 4 * n, flops=n * D)
    return dict(bytes=kept * D * _es(case["act"]) + V * D * _es(case["dtype"]) + 4 * n, flops=kept * D)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("loss", "loss_grad"):
        return _exact_loss(s)
    tok = s["tokens"].long()
    at = ((tok >= 0) & (tok < s["vocab"])).nonzero()[:, 0]
    if s["op"] == "embed":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        out[at] = s["table"].double()[tok[at]] * s["scale"]
        return out
    # tokens in order, a running sum over their rows, and its differences at the tokens' borders
    order = at[torch.argsort(tok[at], stable=True)]
    d = torch.zeros(s["d_table"].shape, dtype=torch.float64, device="cuda")
    if len(order):
        ids, counts = torch.unique_consecutive(tok[order], return_counts=True)
        ends = counts.cumsum(0)
        for c in range(0, d.shape[1], 512):
            sums = s["d_out"][order, c:c + 512].double().cumsum(0)[ends - 1]
            d[ids, c:c + 512] = torch.diff(sums, dim=0, prepend=torch.zeros_like(sums[:1])) * s["scale"]
    return d


def _exact_loss(s):
    """Through the derivative of the definition, a slice of rows at a time."""
    tok, V = s["targets"].long(), s["head"].shape[0]
    at = ((tok >= 0) & (tok < V)).nonzero()[:, 0]
    w = s["head"].double()
    R, D = s["hidden"].shape
    new = lambda *sh: torch.zeros(sh, dtype=torch.float64, device="cuda")  # noqa: E731
    if s["op"] == "loss":
        r = dict(loss=new(R), lse=new(R))
        for i in range(0, len(at), 1024):
            rows = at[i:i + 1024]
            z = torch.nn.functional.linear(s["hidden"][rows].double(), w) / s["temp"]
            r["lse"][rows] = torch.logsumexp(z, dim=1)
            r["loss"][rows] = torch.nn.functional.cross_entropy(z, tok[rows], reduction="none")
        return r
    if s["d_head"] is not None:
        w.requires_grad_()
    r = dict(d_hidden=new(R, D))
    for i in range(0, len(at), 1024):
        rows = at[i:i + 1024]
        h = s["hidden"][rows].double().requires_grad_()
        z = torch.nn.functional.linear(h, w) / s["temp"]
        loss = torch.nn.functional.cross_entropy(z, tok[rows], reduction="none")
        (loss * s["d_loss"][rows].double()).sum().backward()
        r["d_hidden"][rows] = h.grad
    if s["d_head"] is not None:
        r["d_head"] = new(V, D) if w.grad is None else w.grad
    return r
