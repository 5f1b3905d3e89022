"""Timed cases of the drafter's training and scoring operators.

Three operators, each in a plain form (elementary torch operations in 32 bits,
64 where 32 lose what matters) and as the calls a user makes of the package:

  logprobs / logprobs_grad   log probabilities of given tokens with entropy and
                             top alternatives, and their gradient
  attn_grad                  gradients of the packed training attention
  clip                       global gradient norm over many tensors, and clipping

``own`` selects the package's calls.  Inputs come from the seed alone.
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16


def _dt(case):
    return F32 if case["dtype"] == "fp32" else BF16


def _es(case):
    return 4 if case["dtype"] == "fp32" else 2


def listed():
    return [
        # one token being served: its log probability, entropy and 20 alternatives (latency)
        dict(name="logprobs 1 row", op="logprobs", dtype="fp32", rows=1, vocab=151936, pad=0, top_k=20, temp=1.0,
             masked=0.0),
        # a batch-32 cycle's 15 mask rows scored from the drafter's own fp32 logits
        dict(name="logprobs cycle batch 32", op="logprobs", dtype="fp32", rows=480, vocab=151936, pad=0, top_k=5,
             temp=0.8, masked=0.0),
        # a training step's bf16 logits: log probabilities and entropy only
        dict(name="logprobs training bf16", op="logprobs", dtype="bf16", rows=2048, vocab=151936, pad=0, top_k=0,
             temp=1.0, masked=0.0),
        # an odd vocabulary in padded rows, half of it masked by a grammar, as many alternatives as there may be
        dict(name="logprobs odd masked", op="logprobs", dtype="fp32", rows=77, vocab=32003, pad=13, top_k=32, temp=1.3,
             masked=0.5),
        # the gradient of the training step's loss (log probabilities alone)
        dict(name="logprobs gradient bf16", op="logprobs_grad", dtype="bf16", rows=2048, vocab=151936, pad=0,
             temp=1.0, entropy=False, masked=0.0),
        # a few rows of a small odd vocabulary with an entropy term
        dict(name="logprobs gradient odd", op="logprobs_grad", dtype="fp32", rows=45, vocab=8705, pad=3, temp=0.7,
             entropy=True, masked=0.2),
        # a short sequence with few blocks (latency)
        dict(name="attention gradient short", op="attn_grad", dtype="bf16", blocks=12, block=8, seq=500, kv_heads=2,
             group=4, head_dim=64),
        # blocks of 10 in a sequence whose length ends inside a tile
        dict(name="attention gradient ragged", op="attn_grad", dtype="bf16", blocks=100, block=10, seq=1999,
             kv_heads=8, group=4, head_dim=128),
        # a full training sequence of the 8B-shaped drafter: 512 blocks of 16
        dict(name="attention gradient training", op="attn_grad", dtype="bf16", blocks=512, block=16, seq=4096,
             kv_heads=8, group=4, head_dim=128),
        # the tiny fp32 drafter's heads
        dict(name="attention gradient fp32", op="attn_grad", dtype="fp32", blocks=96, block=7, seq=1000, kv_heads=2,
             group=2, head_dim=64),
        # the tiny fp32 drafter's gradients (latency)
        dict(name="clip tiny", op="clip", dtype="fp32", hidden=256, layers=2, q_heads=4, kv_heads=2, head_dim=64,
             ffn=768, over=3.0),
        # the 8B-shaped drafter's gradients (embedding and LM head are frozen)
        dict(name="clip 8b", op="clip", dtype="bf16", hidden=4096, layers=5, q_heads=32, kv_heads=8, head_dim=128,
             ffn=12288, over=3.0),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("logprobs", "logprobs", "logprobs_grad", "attn_grad", "attn_grad", "clip"))
    if kind in ("logprobs", "logprobs_grad"):
        vocab = _log_int(rng, 300, 152000)
        rows = _log_int(rng, 1, min(4096, max(1, 300_000_000 // vocab)))
        case = dict(op=kind, dtype=rng.choice(("fp32", "bf16")), rows=rows, vocab=vocab,
                    pad=rng.choice((0, 0, 1, 8, 61)), temp=rng.choice((1.0, 0.6, 1.5)),
                    masked=rng.choice((0.0, 0.0, 0.3, 0.9)))
        if kind == "logprobs":
            case["top_k"] = rng.choice((0, 1, 5, 20, 32))
        else:
            case["entropy"] = rng.random() < 0.5
        return case
    if kind == "attn_grad":
        fp32 = rng.random() < 0.25
        kv, group, hd = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8)), rng.choice((64, 128))
        block = rng.randint(1, 32)
        seq = _log_int(rng, 1, 4096)
        most = int((1e8 if fp32 else 1e9) / (kv * group * block * (seq + block)))   # query rows x keys
        return dict(op="attn_grad", dtype="fp32" if fp32 else "bf16", blocks=_log_int(rng, 1, max(1, min(512, most))),
                    block=block, seq=seq, kv_heads=kv, group=group, head_dim=hd)
    hidden = 64 * rng.randint(2, 40)
    return dict(op="clip", dtype=rng.choice(("fp32", "bf16")), hidden=hidden, layers=rng.randint(1, 5),
                q_heads=rng.randint(1, 6) * 4, kv_heads=4, head_dim=rng.choice((64, 128)),
                ffn=64 * rng.randint(4, 96) + rng.choice((0, 1)), over=rng.choice((0.5, 3.0, 40.0)))


def _grad_shapes(case):
    """The shapes of a drafter's trained tensors: fusion, its gain, the layers, the final gain."""
    D, F = case["hidden"], case["ffn"]
    hq, hk = case["q_heads"] * case["head_dim"], case["kv_heads"] * case["head_dim"]
    layer = [(D,), (hq, D), (hk, D), (hk, D), (D, hq), (D,), (F, D), (F, D), (D, F)]
    return [(D, 5 * D), (D,)] + layer * case["layers"] + [(D,)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if case["op"] in ("logprobs", "logprobs_grad"):
        return _prepare_logprobs(case, g, rnd)
    if case["op"] == "attn_grad":
        return _prepare_attention(case, g, rnd)
    shapes = _grad_shapes(case)
    scales = torch.exp(torch.rand(len(shapes), generator=g, device="cuda") * 6.0 - 6.0).tolist()
    n = sum(math.prod(s) * w * w for s, w in zip(shapes, scales))
    unit = case["over"] / math.sqrt(n)             # the global norm comes out near `over`
    grads = [(rnd(*s) * (w * unit)).to(_dt(case)) for s, w in zip(shapes, scales)]
    return dict(op="clip", grads=grads, out=[torch.empty_like(t) for t in grads], max_norm=1.0,
                norm=torch.empty(1, device="cuda"), ws=[])


def _prepare_logprobs(case, g, rnd):
    """A language model's logits: a wide background, eight likely tokens a row, a share of the vocabulary masked;
    one token in eight of a longer batch is padding (-1)."""
    R, V = case["rows"], case["vocab"]
    store = torch.zeros((R, V + case["pad"]), dtype=_dt(case), device="cuda")
    logits = store[:, :V]
    ids = torch.randint(0, V, (R, 8), generator=g, device="cuda")
    x = rnd(R, V) * 2.0
    if case["masked"]:
        x.masked_fill_(torch.rand(x.shape, generator=g, device="cuda") < case["masked"], -math.inf)
    likely = 6.0 + 8.0 * torch.rand(ids.shape, generator=g, device="cuda")
    logits.copy_(x.scatter_reduce_(1, ids, likely, "amax"))   # the larger where an id comes twice
    tokens = torch.where(torch.rand(R, generator=g, device="cuda") < 0.7, ids[:, 0],
                         torch.randint(0, V, (R,), generator=g, device="cuda"))
    if case["masked"]:
        tokens = ids[:, 0]
    if R >= 16:
        tokens = torch.where(torch.rand(R, generator=g, device="cuda") < 0.125, -1, tokens)
    s = dict(op=case["op"], logits=logits, tokens=tokens.to(torch.int32), temp=case["temp"])
    new = lambda *sh, dtype=F32: torch.empty(sh, dtype=dtype, device="cuda")  # noqa: E731
    if case["op"] == "logprobs":
        k = case["top_k"]
        s.update(k=k, logprob=new(R), entropy=new(R), lse=new(R), ids=new(R, k, dtype=torch.int32), top=new(R, k))
    else:
        _, ent, lse, _, _ = _logprobs_plain(logits, s["tokens"], case["temp"], 0)
        s.update(lse=lse, entropy=ent if case["entropy"] else None, d_logprob=rnd(R) / R,
                 d_entropy=rnd(R) / R if case["entropy"] else None, d_logits=new(R, V, dtype=_dt(case)))
    return s


def _prepare_attention(case, g, rnd):
    N, b, S, nkv, hd, dt = (case[k] for k in ("blocks", "block", "seq", "kv_heads", "head_dim", "dtype"))
    dt, nq = _dt(case), nkv * case["group"]
    q, kc, vc = rnd(N, b, nq, hd).to(dt), rnd(S, nkv, hd).to(dt), rnd(S, nkv, hd).to(dt)
    kb, vb, d_out = rnd(N, b, nkv, hd).to(dt), rnd(N, b, nkv, hd).to(dt), rnd(N, b, nq, hd)
    anchors = torch.randint(0, S + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    out, lse = _attention_plain(q, kc, vc, kb, vb, anchors)
    new = torch.empty_like
    return dict(op="attn_grad", q=q, kc=kc, vc=vc, kb=kb, vb=vb, anchors=anchors, out=out, lse=lse, d_out=d_out,
                grads=[new(q), new(kc), new(vc), new(kb), new(vb)], ws=[])


# ---------------------------------------------------------------- plain forms
def _logprobs_plain(logits, tokens, temp, k):
    z = logits.float() / temp
    m = z.max(dim=1, keepdim=True).values
    w = z - m
    e = w.exp()
    total = e.sum(dim=1, dtype=torch.float64)
    log_total = total.log()
    lse = (m[:, 0] + log_total).float()
    inside = (tokens >= 0) & (tokens < z.shape[1])
    at = torch.where(inside, tokens, 0).long()[:, None]
    logprob = torch.where(inside, (w.gather(1, at)[:, 0] - log_total).float(), 0.0)
    mean = torch.where(e > 0, e * w, 0.0).sum(dim=1, dtype=torch.float64) / total
    entropy = (log_total - mean).float()
    if k == 0:
        return logprob, entropy, lse, None, None
    x, order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = order[:, :k]
    return logprob, entropy, lse, ids.to(torch.int32), (w.gather(1, ids) - log_total[:, None]).float()


def _logprobs_grad_plain(s):
    z = s["logits"].float() / s["temp"]
    logp = z - s["lse"][:, None]
    p = logp.exp()
    inside = (s["tokens"] >= 0) & (s["tokens"] < z.shape[1])
    g = torch.where(inside, s["d_logprob"], 0.0)
    d = -g[:, None] * p
    d.scatter_add_(1, torch.where(inside, s["tokens"], 0).long()[:, None], g[:, None])
    if s["d_entropy"] is not None:
        d -= s["d_entropy"][:, None] * torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0)
    return (d / s["temp"]).to(s["logits"].dtype)


def _scores(q, kc, kb, anchors):
    """Masked scores against the context, [kv head, block * position * group, S], and against the own block."""
    N, b, nq, hd = q.shape
    S, nkv = kc.shape[0], kc.shape[1]
    G = nq // nkv
    qh = q.float().view(N, b, nkv, G, hd).permute(2, 0, 1, 3, 4)                  # [nkv, N, b, G, hd]
    sc = torch.matmul(qh.reshape(nkv, N * b * G, hd), kc.float().permute(1, 2, 0)) / math.sqrt(hd)
    seen = torch.arange(S, device=q.device)[None, :] < anchors[:, None]           # [N, S]
    sc = sc.view(nkv, N, b * G, S).masked_fill_(~seen[None, :, None, :], -math.inf)
    sb = torch.matmul(qh.reshape(nkv, N, b * G, hd), kb.float().permute(2, 0, 3, 1)) / math.sqrt(hd)
    return qh.reshape(nkv, N, b * G, hd), sc, sb


def _heads(x, nkv):
    """[N, b, nq, ...] as [nkv, N, b * G, ...]."""
    N, b, nq = x.shape[:3]
    x = x.float().view(N, b, nkv, nq // nkv, -1).permute(2, 0, 1, 3, 4)
    return x.reshape(nkv, N, b * (nq // nkv), -1)


def _rows(x, b):
    """[nkv, N, b * G, d] as [N, b, nkv * G, d]."""
    nkv, N, bG, d = x.shape
    return x.view(nkv, N, b, bG // b, d).permute(1, 2, 0, 3, 4).reshape(N, b, nkv * (bG // b), d)


def _attention_plain(q, kc, vc, kb, vb, anchors):
    b, nkv = q.shape[1], kb.shape[2]
    _, sc, sb = _scores(q, kc, kb, anchors)
    m = torch.maximum(sc.max(dim=-1, keepdim=True).values, sb.max(dim=-1, keepdim=True).values)
    pc, pb = (sc - m).exp(), (sb - m).exp()
    total = pc.sum(-1, keepdim=True) + pb.sum(-1, keepdim=True)
    shape = pc.shape
    o = torch.matmul(pc.view(nkv, -1, shape[3]), vc.float().permute(1, 0, 2)).view(*shape[:3], -1)
    o = (o + torch.matmul(pb, vb.float().permute(2, 0, 1, 3))) / total
    return _rows(o, b).contiguous(), _rows(m + total.log(), b)[..., 0].contiguous()


def _attention_grad_plain(s):
    q, kc, vc, kb, vb = (s[k] for k in ("q", "kc", "vc", "kb", "vb"))
    b, nkv, hd = q.shape[1], kb.shape[2], q.shape[3]
    qh, pc, pb = _scores(q, kc, kb, s["anchors"])
    lse, do = _heads(s["lse"], nkv), _heads(s["d_out"], nkv)
    delta = (do * _heads(s["out"], nkv)).sum(-1, keepdim=True)
    pc.sub_(lse).exp_()
    pb.sub_(lse).exp_()
    shape = pc.shape
    flat = lambda x: x.reshape(nkv, -1, x.shape[-1])  # noqa: E731
    dvc = torch.matmul(flat(pc).transpose(1, 2), flat(do))
    dvb = torch.matmul(pb.transpose(2, 3), do)
    dsc = torch.matmul(flat(do), vc.float().permute(1, 2, 0)).view(shape).sub_(delta).mul_(pc).div_(math.sqrt(hd))
    dsb = torch.matmul(do, vb.float().permute(2, 0, 3, 1)).sub_(delta).mul_(pb).div_(math.sqrt(hd))
    dq = torch.matmul(flat(dsc), kc.float().permute(1, 0, 2)).view(qh.shape)
    dq = dq + torch.matmul(dsb, kb.float().permute(2, 0, 1, 3))
    dkc = torch.matmul(flat(dsc).transpose(1, 2), flat(qh))
    dkb = torch.matmul(dsb.transpose(2, 3), qh)
    t = q.dtype
    ctx, blk = (lambda x: x.permute(1, 0, 2).to(t)), (lambda x: x.permute(1, 2, 0, 3).to(t))  # noqa: E731
    return dict(d_q=_rows(dq, b).to(t), d_k_ctx=ctx(dkc), d_v_ctx=ctx(dvc), d_k_blk=blk(dkb), d_v_blk=blk(dvb))


def _clip_plain(s):
    grads, most = s["grads"], s["max_norm"]
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()
    scale = torch.where(norm.isfinite() & (norm > most), most / norm, 1.0).float()
    return dict(norm=norm.float().view(1), out=[(g.float() * scale).to(g.dtype) for g in grads])


# ---------------------------------------------------------------- one pass
def run(s):
    if s["op"] == "logprobs":
        if own:
            import block_diffusion_drafter_dflash_gb300 as df
            top = dict(top_ids=s["ids"], top_logprobs=s["top"]) if s["k"] else {}
            df.dflash_token_logprobs(s["logits"], s["tokens"], s["temp"], s["logprob"], entropy=s["entropy"],
                                     lse=s["lse"], **top)
            r = s["logprob"], s["entropy"], s["lse"], s["ids"], s["top"]
        else:
            r = _logprobs_plain(s["logits"], s["tokens"], s["temp"], s["k"])
        r = dict(zip(("logprob", "entropy", "lse", "top_ids", "top_logprobs"), r))
        return r if s["k"] else {k: r[k] for k in ("logprob", "entropy", "lse")}
    if s["op"] == "logprobs_grad":
        if own:
            import block_diffusion_drafter_dflash_gb300 as df
            df.dflash_token_logprobs_backward(s["logits"], s["tokens"], s["temp"], s["lse"], s["d_logits"],
                                              d_logprob=s["d_logprob"], entropy=s["entropy"],
                                              d_entropy=s["d_entropy"])
            return s["d_logits"]
        return _logprobs_grad_plain(s)
    if s["op"] == "attn_grad":
        if own:
            import block_diffusion_drafter_dflash_gb300 as df
            if not s["ws"]:
                N, b, nq, hd = s["q"].shape
                s["ws"].append(df.dflash_packed_attention_backward_workspace(N, b, s["kc"].shape[0], nq,
                                                                             s["kb"].shape[2], hd, s["q"].dtype))
            d_q, d_kc, d_vc, d_kb, d_vb = s["grads"]
            df.dflash_packed_block_attention_backward(s["q"], s["kc"], s["vc"], s["kb"], s["vb"], s["anchors"],
                                                      s["out"], s["lse"], s["d_out"], d_q, d_kc, d_vc, d_kb, d_vb,
                                                      s["ws"][0])
            return dict(d_q=d_q, d_k_ctx=d_kc, d_v_ctx=d_vc, d_k_blk=d_kb, d_v_blk=d_vb)
        return _attention_grad_plain(s)
    if own:
        import block_diffusion_drafter_dflash_gb300 as df
        if not s["ws"]:
            s["ws"].append(df.dflash_clip_workspace())
        df.dflash_clip_grad_norm(s["grads"], s["max_norm"], s["norm"], out=s["out"], workspace=s["ws"][0])
        return dict(norm=s["norm"], out=s["out"])
    return _clip_plain(s)


def work(case):
    op = case["op"]
    if op == "logprobs":
        n = case["rows"] * case["vocab"]
        return dict(bytes=n * _es(case) + case["rows"] * (16 + 8 * case["top_k"]), flops=5 * n)
    if op == "logprobs_grad":
        n = case["rows"] * case["vocab"]
        return dict(bytes=2 * n * _es(case) + 20 * case["rows"], flops=5 * n)
    if op == "attn_grad":
        N, b, S, nkv, hd = (case[k] for k in ("blocks", "block", "seq", "kv_heads", "head_dim"))
        nq, es = nkv * case["group"], _es(case)
        rows = N * b * nq
        ios = rows * hd * (2 * es + 8) + 4 * rows + 4 * es * nkv * hd * (S + N * b)
        return dict(bytes=ios, flops=10.0 * hd * rows * (S / 2 + b))     # anchors lie at S / 2 in the mean
    n = sum(math.prod(s) for s in _grad_shapes(case))
    return dict(bytes=2 * n * _es(case) + 4, flops=3 * n)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "logprobs":
        return _exact_logprobs(s)
    if s["op"] == "logprobs_grad":
        # through the derivative of the definition, a slice of rows at a time
        parts = []
        for r in range(0, s["logits"].shape[0], 256):
            cut = slice(r, r + 256)
            x = s["logits"][cut].double().requires_grad_()
            logp = torch.log_softmax(x / s["temp"], dim=1)
            tok = s["tokens"][cut].long()
            inside = (tok >= 0) & (tok < x.shape[1])
            lp = logp.gather(1, tok.clamp(0, x.shape[1] - 1)[:, None])[:, 0]
            loss = (lp[inside] * s["d_logprob"][cut].double()[inside]).sum()
            if s["d_entropy"] is not None:
                finite = torch.where(logp.isinf(), 0.0, logp)
                loss = loss + (-(logp.exp() * finite).sum(1) * s["d_entropy"][cut].double()).sum()
            parts.append(torch.autograd.grad(loss, x)[0])
        return torch.cat(parts)
    if s["op"] == "attn_grad":
        return _exact_attention(s)
    norm = torch.sqrt(sum(torch.linalg.vector_norm(g, dtype=torch.float64) ** 2 for g in s["grads"]))
    ratio = min(1.0, s["max_norm"] / float(norm))
    return dict(norm=norm.view(1), out=[g.double() * ratio for g in s["grads"]])


def _exact_logprobs(s):
    logp = torch.log_softmax(s["logits"].double() / s["temp"], dim=1)
    tok = s["tokens"].long()
    picked = logp[torch.arange(len(tok), device="cuda"), tok.clamp(0, logp.shape[1] - 1)]
    r = dict(logprob=torch.where((tok >= 0) & (tok < logp.shape[1]), picked, 0.0),
             entropy=-(logp.exp() * torch.where(logp.isinf(), 0.0, logp)).sum(1),
             lse=torch.logsumexp(s["logits"].double() / s["temp"], dim=1))
    return r if not s["k"] else dict(r, top_ids=None, top_logprobs=torch.topk(logp, s["k"], dim=1).values)


def _exact_attention(s):
    """Derivative of the masked softmax in 64 bits, a kv head at a time (None where 64 bits take too long)."""
    N, b, nq, hd = s["q"].shape
    S, nkv = s["kc"].shape[0], s["kb"].shape[2]
    G = nq // nkv
    if 10.0 * hd * N * b * nq * (S + b) > 6e12:
        return None
    seen = (torch.arange(S, device="cuda")[None, :] < s["anchors"][:, None])[:, None, None, :]
    got = {k: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
           for k, n in (("d_q", "q"), ("d_k_ctx", "kc"), ("d_v_ctx", "vc"), ("d_k_blk", "kb"), ("d_v_blk", "vb"))}
    for h in range(nkv):
        hs = slice(h * G, h * G + G)
        leaf = [t.double().requires_grad_() for t in (s["q"][:, :, hs], s["kc"][:, h], s["vc"][:, h], s["kb"][:, :, h],
                                                      s["vb"][:, :, h])]
        q, kc, vc, kb, vb = leaf
        ctx = torch.einsum("nigd,sd->nigs", q, kc).masked_fill(~seen, -math.inf)
        blk = torch.einsum("nigd,njd->nigj", q, kb)
        p = torch.softmax(torch.cat([ctx, blk], dim=-1) / math.sqrt(hd), dim=-1)
        o = torch.einsum("nigs,sd->nigd", p[..., :S], vc) + torch.einsum("nigj,njd->nigd", p[..., S:], vb)
        grads = torch.autograd.grad(o, leaf, s["d_out"][:, :, hs].double())
        got["d_q"][:, :, hs], got["d_k_ctx"][:, h], got["d_v_ctx"][:, h] = grads[:3]
        got["d_k_blk"][:, :, h], got["d_v_blk"][:, :, h] = grads[3:]
    return got
