"""Measured cases of the operators on either side of the logits: the last norm
with the residual's addition and 8-bit codes, log probabilities of given tokens
with entropy and top alternatives (and their gradient), and the distillation of
a draft model from a target's top tokens (loss and gradient).

``run`` computes each operator in elementary torch operations, or, where
``own`` is true, by the calls a user of the library makes. Sizes come from the
library's own workloads (vocabularies 8192, 32000, 128256, 151936; 64
sequences of 4 drafts; 256 and 1024 rows) and generic hidden widths.
"""
import torch

own = False
_sampler = None


def sampler():
    """The handle a program creates once and keeps."""
    global _sampler
    if _sampler is None:
        import token_sampling_row_amd as tsr
        _sampler = tsr.Sampler(0, max_rows=4096, max_vocab=1 << 18, max_k=8, seed=1)
    return _sampler


DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
REST_MIN = 2.0 ** -20   # a teacher's remainder below this is rounding of its log probabilities


def listed():
    return [
        # one sequence's single-token step, before the 8-bit projection
        dict(name="norm 1x4096", op="norm", rows=1, width=4096, dtype="bf16", wtype="bf16",
             residual=True),
        # odd sizes in float32: a batch cut short, a width that splits into no whole chunks
        dict(name="norm 333x5003 f32", op="norm", rows=333, width=5003, dtype="f32", wtype="f32",
             residual=False),
        # every position of a batch of prompts; weights kept in float32
        dict(name="norm 16384x4096", op="norm", rows=16384, width=4096, dtype="bf16",
             wtype="f32", residual=True),
        # single-token decoding that returns its alternatives
        dict(name="logprobs 1x128256 top20", op="logprobs", rows=1, vocab=128256, dtype="bf16",
             tokens=1, top=20, temperature=1.0, masked=False),
        # choices scored against odd float32 rows with tokens masked out
        dict(name="logprobs 333x50001 f32 n4 top5", op="logprobs", rows=333, vocab=50001,
             dtype="f32", tokens=4, top=5, temperature=0.7, masked=True),
        # the verify rows of 64 sequences with 4 drafts each, scored with entropy only
        dict(name="logprobs 320x32000 f32", op="logprobs", rows=320, vocab=32000, dtype="f32",
             tokens=1, top=0, temperature=1.0, masked=False),
        # a teacher's pass over the largest batch: its 64 likeliest tokens per position
        dict(name="logprobs 1024x151936 top64", op="logprobs", rows=1024, vocab=151936,
             dtype="bf16", tokens=1, top=64, temperature=1.0, masked=False),
        # policy gradients: a small float32 batch, no entropy term
        dict(name="logprobs grad 64x32000 f32", op="grad", rows=64, vocab=32000, dtype="f32",
             tokens=1, entropy=False, temperature=1.0, masked=False),
        # the same over a large batch, with an entropy bonus and a temperature
        dict(name="logprobs grad 1024x128256", op="grad", rows=1024, vocab=128256, dtype="bf16",
             tokens=1, entropy=True, temperature=0.8, masked=False),
        # a small draft model's step on 8 teacher entries a position; odd sizes
        dict(name="distill 33x8191 f32 k8", op="distill", rows=33, vocab=8191, dtype="f32", k=8,
             tail=True, temperature=1.0),
        # an ordinary batch, teacher's probabilities renormalised over its entries
        dict(name="distill 256x128256 k20", op="distill", rows=256, vocab=128256, dtype="bf16",
             k=20, tail=False, temperature=2.0),
        # the largest batch on the widest vocabulary, the rest of the ids as one bucket
        dict(name="distill 1024x151936 k64 tail", op="distill", rows=1024, vocab=151936,
             dtype="bf16", k=64, tail=True, temperature=1.0),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, int(lo * (hi / lo) ** rng.random() + 0.5))


def draw(rng):
    op = rng.choice(["norm", "logprobs", "logprobs", "grad", "distill", "distill"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "norm":
        width = _between(rng, 256, 8192)
        if rng.random() < 0.5:   # the widths of most models
            width = max(256, width // 256 * 256)
        most = min(32768, 16384 * 4096 // width) // (2 if dtype == "f32" else 1)
        return dict(op=op, rows=_between(rng, 1, most), width=width, dtype=dtype,
                    wtype=rng.choice(["f32", "bf16"]), residual=rng.random() < 0.7)
    vocab = _between(rng, 8192, 151936)
    most = 1024 * 151936 // vocab // (2 if dtype == "f32" else 1)
    case = dict(op=op, rows=_between(rng, 1, min(4096, most)), vocab=vocab, dtype=dtype,
                temperature=rng.choice([1.0, 1.0, 0.7, 1.5]))
    if op == "logprobs":
        return dict(case, tokens=_between(rng, 1, 8), masked=rng.random() < 0.3,
                    top=0 if rng.random() < 0.3 else _between(rng, 1, 64))
    if op == "grad":
        return dict(case, tokens=_between(rng, 1, 8), masked=rng.random() < 0.3,
                    entropy=rng.random() < 0.5)
    return dict(case, k=_between(rng, 1, 64), tail=rng.random() < 0.5)


def _logits(rows, vocab, g, noise=0.5):
    """The workloads' head and long tail: -1.0 ln(rank) + noise, ranks at random."""
    z = torch.rand(rows, vocab, device="cuda", generator=g).mul_(vocab).add_(1.0).log_().neg_()
    return z.add_(noise * torch.randn(rows, vocab, device="cuda", generator=g)).add_(8.0)


def _tokens(z, n, g):
    """Ids that were drawn from the rows (the largest of z plus Gumbel noise among a few
    hundred random ids), and others at random."""
    rows, vocab = z.shape
    some = torch.randint(0, vocab, (rows, 512), device="cuda", generator=g)
    u = torch.rand(rows, 512, device="cuda", generator=g).clamp_(1e-9, 1.0 - 1e-7)
    best = (z.gather(1, some) - (-u.log()).log()).argmax(1, keepdim=True)
    rest = torch.randint(0, vocab, (rows, n - 1), device="cuda", generator=g)
    return torch.cat([some.gather(1, best), rest], 1).to(torch.int32)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rows = case["rows"]
    st = dict(case=case)
    if case["op"] == "norm":
        # a block's output and the residual stream: a few channels far larger than the rest
        W = case["width"]
        big = torch.randint(0, W, (max(1, W // 512),), device=dev, generator=g)
        x = torch.randn(rows, W, device=dev, generator=g)
        x *= torch.exp(0.5 * torch.randn(rows, 1, device=dev, generator=g))
        x[:, big] *= 8.0
        st["x"] = x.to(dt)
        st["residual"] = None
        if case["residual"]:
            r = 4.0 * torch.randn(rows, W, device=dev, generator=g)
            r[:, big] *= 8.0
            st["residual"] = r.to(dt)
        w = torch.exp(0.2 * torch.randn(W, device=dev, generator=g))
        st["w"] = w.to(DTYPES[case["wtype"]])
        return st
    V, T = case["vocab"], case["temperature"]
    z = _logits(rows, V, g)
    if case["op"] == "distill":
        k = case["k"]
        # the target's logits, near the draft's; its top entries at the same temperature
        t = (z + 0.8 * torch.randn(rows, V, device=dev, generator=g)) / T
        top, ids = t.topk(k, 1)
        st["teacher"] = top - torch.logsumexp(t, 1, keepdim=True)
        st["ids"] = ids.to(torch.int32)
        del t, top, ids
        # the mean over the batch's positions, of which a few are padding
        real = torch.rand(rows, device=dev, generator=g) >= 0.05
        real[0] = True
        st["weight"] = real.float() / real.sum()
        st["z"] = z.to(dt)
        return st
    if case["masked"]:   # a tenth of the ids is not allowed
        z.masked_fill_(torch.rand(rows, V, device=dev, generator=g) < 0.1, float("-inf"))
        z[:, 0] = 0.0
    st["z"] = z.to(dt)
    st["tokens"] = _tokens(z, case["tokens"], g)
    if case["op"] == "grad":
        # what the forward pass has left, and the gradients that come back
        M = st["z"].float().amax(1)
        x = (st["z"].float() - M[:, None]).div_(T)
        e = x.exp()
        Z = e.sum(1)
        st["norm"] = torch.stack([M, Z], 1)
        st["g"] = torch.randn(rows, case["tokens"], device=dev, generator=g) / rows
        st["entropy"] = st["ge"] = None
        if case["entropy"]:
            x = torch.where(e > 0, x, 0.0)
            st["entropy"] = Z.log() - (e * x).sum(1) / Z
            st["ge"] = torch.full((rows,), 0.01 / rows, device=dev)
    return st


def _norm(st):
    x, w = st["x"], st["w"].float()
    h = x if st["residual"] is None else (x.float() + st["residual"].float()).to(x.dtype)
    hf = h.float()
    factor = 1.0 / (hf.square().mean(1) + EPS).sqrt()
    # the row's factor cancels in the codes; in 64 bits: a quotient next to a half decides
    t = hf.double() * w.double()
    most = t.abs().amax(1)
    q = (127.0 * t / torch.where(most > 0, most, 1.0)[:, None]).round()
    scale = most.float() * factor / 127.0
    out = (q.float() * scale[:, None], scale)
    return out if st["residual"] is None else out + (h,)


def _top(z, k):
    """The k largest of each row in order, equal ones by their ids: whole numbers that
    order as (value, then -id) do."""
    V = z.shape[1]
    bits = (z + 0.0).view(torch.int32)
    key = bits ^ ((bits >> 31) & 0x7FFFFFFF)
    key = (key.long() << 32) + torch.arange(V - 1, -1, -1, device=z.device)
    return V - 1 - (key.topk(k, 1).values & 0xFFFFFFFF)


def _logprobs(st):
    z, T, k = st["z"].float(), st["case"]["temperature"], st["case"]["top"]
    M = z.amax(1, keepdim=True)
    x = (z - M) / T
    e = x.exp()
    Z = e.sum(1, keepdim=True)
    logZ = Z.log()
    out = dict(logprob=x.gather(1, st["tokens"].long()) - logZ, norm=torch.cat([M, Z], 1))
    out["entropy"] = (logZ - (e * torch.where(e > 0, x, 0.0)).sum(1, keepdim=True) / Z)[:, 0]
    if k:
        ids = _top(z, k)
        out["top_logprob"] = x.gather(1, ids) - logZ
        out["top_ids"] = ids.int()
    return out


def _grad(st):
    z, T = st["z"].float(), st["case"]["temperature"]
    M, Z = st["norm"][:, :1], st["norm"][:, 1:]
    x = (z - M) / T
    p = x.exp() / Z
    factor = st["g"].sum(1, keepdim=True)
    if st["entropy"] is not None:
        logp = torch.where(p > 0, x - Z.log(), 0.0)
        factor = factor + st["ge"][:, None] * (logp + st["entropy"][:, None])
    out = -p * factor
    out.scatter_add_(1, st["tokens"].long(), st["g"])
    return (out / T).to(st["z"].dtype)


def _distill(st):
    case = st["case"]
    z, T = st["z"].float(), case["temperature"]
    ids, weight = st["ids"].long(), st["weight"][:, None]
    logq = st["teacher"]
    q = logq.exp()
    if case["tail"]:
        # in 64 bits: what the entries leave over, and the share of the other ids
        rest = (1.0 - q.double().sum(1, keepdim=True)).float()
        rest = torch.where(rest > REST_MIN, rest, 0.0)
    else:
        total = q.sum(1, keepdim=True)
        q, logq, rest = q / total, logq - total.log(), torch.zeros_like(total)
    x = (z - z.amax(1, keepdim=True)) / T
    e = x.exp()
    Z = e.sum(1, keepdim=True)
    logp = x.gather(1, ids) - Z.log()
    p_rest = e.scatter(1, ids, 0.0).sum(1, keepdim=True) / Z
    loss = (q * (logq - logp)).sum(1, keepdim=True)
    loss = loss + torch.where(rest > 0, rest * (rest / p_rest).log(), 0.0)
    whole = q.sum(1, keepdim=True) + rest
    p = e / Z
    grad = p * (whole - torch.where(rest > 0, rest / p_rest, 0.0))
    grad.scatter_(1, ids, p.gather(1, ids) * whole - q)
    return (weight * loss)[:, 0], (grad * (weight / T)).to(st["z"].dtype)


def run(st):
    case = st["case"]
    if case["op"] == "norm":
        if own:
            got = sampler().norm_quantize_rows(st["x"], st["w"], eps=EPS,
                                               residual=st["residual"])
            return (got[0] * got[1][:, None],) + got[1:]   # the values that the codes stand for
        return _norm(st)
    if case["op"] == "logprobs":
        if own:
            got = sampler().token_logprobs(st["z"], st["tokens"], top_k=case["top"],
                                           temperature=case["temperature"])
            out = dict(logprob=got.logprob, norm=got.norm, entropy=got.entropy)
            if case["top"]:
                out["top_logprob"], out["top_ids"] = got.top_logprob, got.top_ids
            return out
        return _logprobs(st)
    if case["op"] == "grad":
        if own:
            return sampler().token_logprobs_grad(
                st["z"], st["tokens"], st["norm"], st["g"], entropy=st["entropy"],
                grad_entropy=st["ge"], temperature=case["temperature"])
        return _grad(st)
    if own:
        return sampler().distill_topk(st["z"], st["ids"], st["teacher"],
                                      temperature=case["temperature"], tail=case["tail"],
                                      row_weight=st["weight"])
    return _distill(st)


def work(case):
    rows = case["rows"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = rows * case["width"]
        moved = 3 * size if case["residual"] else size
        return dict(bytes=n * (moved + 1) + 4 * rows
                    + case["width"] * (4 if case["wtype"] == "f32" else 2), flops=6 * n)
    n = rows * case["vocab"]
    if case["op"] == "logprobs":
        return dict(bytes=n * size + rows * (8 * case["tokens"] + 8 * case["top"] + 12),
                    flops=6 * n)
    if case["op"] == "grad":
        return dict(bytes=2 * n * size + rows * (8 * case["tokens"] + 16), flops=6 * n)
    return dict(bytes=2 * n * size + rows * (8 * case["k"] + 8), flops=8 * n)


def exact(case, seed):
    """The outputs from the definitions, in 64 bits, a few rows at a time."""
    st = prepare(case, seed)
    if case["op"] == "norm":
        h = st["x"].double()
        if st["residual"] is not None:
            # the sum is held in the rows' type: that value is normed
            h = (h + st["residual"].double()).to(st["x"].dtype).double()
        # a code is its value's share of the row's largest: without the row's factor, which
        # would decide halves by its own rounding
        t = h * st["w"].double()
        most = torch.maximum(t.amax(1), -t.amin(1))
        scale = most * torch.rsqrt(torch.mean(h * h, dim=1) + EPS) / 127
        values = torch.round(t * 127 / most[:, None]).clamp_(-127, 127) * scale[:, None]
        return (values, scale) if st["residual"] is None else (values, scale, h)
    T, parts = case["temperature"], []
    for a in range(0, case["rows"], 64):
        z = st["z"][a:a + 64].double() / T
        lse = torch.logsumexp(z, 1, keepdim=True)
        logp = z - lse
        if case["op"] == "logprobs":
            ids = st["tokens"][a:a + 64].long()
            p = logp.exp()
            most = z.amax(1, keepdim=True)
            part = dict(logprob=logp.gather(1, ids),
                        entropy=-torch.nan_to_num(p * logp, nan=0.0).sum(1),
                        norm=torch.cat([most * T, (lse - most).exp()], 1))
            if case["top"]:
                value, order = torch.sort(logp, dim=1, descending=True, stable=True)
                part["top_logprob"] = value[:, :case["top"]].clone()
                part["top_ids"] = order[:, :case["top"]].int()
            parts.append(part)
        elif case["op"] == "grad":
            p = logp.exp()
            g = st["g"][a:a + 64].double()
            grad = torch.zeros_like(p)
            for i in range(case["tokens"]):
                grad.scatter_add_(1, st["tokens"][a:a + 64, i:i + 1].long(), g[:, i:i + 1])
            grad = grad - p * g.sum(1, keepdim=True)
            if case["entropy"]:
                plogp = torch.nan_to_num(p * logp, nan=0.0)
                H = -plogp.sum(1, keepdim=True)
                grad = grad - st["ge"][a:a + 64, None].double() * (plogp + p * H)
            parts.append(grad / T)
        else:
            ids = st["ids"][a:a + 64].long()
            t = st["teacher"][a:a + 64].double()
            inside = torch.zeros_like(logp, dtype=torch.bool).scatter_(1, ids, True)
            q = torch.zeros_like(logp).scatter_(1, ids, t.exp())
            p = logp.exp()
            if case["tail"]:
                # spread over the other ids as the draft spreads it: the same loss
                rest = 1.0 - q.sum(1, keepdim=True)
                rest = torch.where(rest > REST_MIN, rest, 0.0)
                other = torch.where(inside, 0.0, p)
                q = q + rest * other / other.sum(1, keepdim=True)
            else:
                q = q / q.sum(1, keepdim=True)
            weight = st["weight"][a:a + 64, None].double()
            kl = torch.where(q > 0, q * (q.clamp(min=1e-300).log() - logp), 0.0)
            grad = q.sum(1, keepdim=True) * p - q
            parts.append(((weight * kl.sum(1, keepdim=True))[:, 0], grad * weight / T))
    if case["op"] == "logprobs":
        return {k: torch.cat([part[k] for part in parts]) for k in parts[0]}
    if case["op"] == "grad":
        return torch.cat(parts)
    return tuple(torch.cat([part[i] for part in parts]) for i in range(2))
