"""Measured cases of the operators around the sampler: per-row 8-bit
quantisation, the 8-bit output projection, and the verification of drafted
tokens from probabilities and given random numbers.

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


def listed():
    return [
        # one sequence's K + 1 hidden states of a verify step
        dict(name="quantize 5x4096", op="quantize", rows=5, width=4096, dtype="bf16"),
        # odd sizes in float32: a batch cut short, a width that splits into no whole chunks
        dict(name="quantize 333x5003 f32", op="quantize", rows=333, width=5003, dtype="f32"),
        # the weight of a 32000-token head, quantised once per channel when it is loaded
        dict(name="quantize 32000x4096", op="quantize", rows=32000, width=4096, dtype="bf16"),
        # single-token decoding of one sequence with a 128k-token head
        dict(name="logits 1x128256x4096", op="logits", rows=1, vocab=128256, width=4096,
             dtype="bf16", bias=False),
        # one verify step of a small model; odd sizes, float32 logits and a bias
        dict(name="logits 5x8191x1003 f32", op="logits", rows=5, vocab=8191, width=1003,
             dtype="f32", bias=True),
        # a decode batch of 64 sequences
        dict(name="logits 64x128256x4096", op="logits", rows=64, vocab=128256, width=4096,
             dtype="bf16", bias=False),
        # the verify rows of 64 sequences with 4 drafts each
        dict(name="logits 320x32000x4096 f32", op="logits", rows=320, vocab=32000, width=4096,
             dtype="f32", bias=False),
        # the largest batch on the widest vocabulary
        dict(name="logits 1024x151936x4096", op="logits", rows=1024, vocab=151936, width=4096,
             dtype="bf16", bias=False),
        # one sequence: latency
        dict(name="verify 1xK4x32000", op="verify", rows=1, drafts=4, vocab=32000, dtype="f32",
             draft="model", min_p=0.0, ragged=False),
        # the library's verify workload
        dict(name="verify 64xK4x32000", op="verify", rows=64, drafts=4, vocab=32000,
             dtype="f32", draft="model", min_p=0.0, ragged=False),
        # proposals looked up in the text (no draft distribution), filtered target
        # probabilities, drafts of unequal length, odd vocabulary, bf16
        dict(name="verify 33xK7x151935 lookup", op="verify", rows=33, drafts=7, vocab=151935,
             dtype="bf16", draft="lookup", min_p=0.05, ragged=True),
        # a large batch on a 128k-token vocabulary, drafts of unequal length
        dict(name="verify 128xK4x128256", op="verify", rows=128, drafts=4, vocab=128256,
             dtype="f32", draft="model", min_p=0.0, ragged=True),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm."""
    return min(hi, int(lo * (hi / lo) ** rng.random() + 0.5))


def draw(rng):
    op = rng.choice(["quantize", "logits", "logits", "verify", "verify"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "quantize":
        width = _between(rng, 256, 8192)
        rows = _between(rng, 1, min(32000, 32000 * 4096 // width) // (2 if dtype == "f32" else 1))
        return dict(op=op, rows=rows, width=width, dtype=dtype)
    if op == "logits":
        vocab = _between(rng, 8192, 151936)
        width = _between(rng, 512, min(8192, 151936 * 4096 // vocab))
        if rng.random() < 0.5:   # the widths of most models
            width = max(512, width // 256 * 256)
        rows = _between(rng, 1, 1024)
        # f32 logits cost twice the output bytes
        rows = rows // 2 + 1 if dtype == "f32" else rows
        return dict(op=op, rows=rows, vocab=vocab, width=width, dtype=dtype,
                    bias=rng.random() < 0.3)
    drafts = _between(rng, 1, 8)
    vocab = _between(rng, 8192, 151936)
    rows = _between(rng, 1, max(1, min(256, 128 * 5 * 128256 // ((drafts + 1) * vocab))))
    return dict(op=op, rows=rows, drafts=drafts, vocab=vocab, dtype=dtype,
                draft=rng.choice(["model", "model", "lookup"]), min_p=rng.choice([0.0, 0.05]),
                ragged=rng.random() < 0.5)


def _codes(x):
    """Absmax codes and scales of each row (inputs of the product)."""
    s = x.abs().amax(1) / 127.0
    return (x / s[:, None]).round_().clamp_(-127, 127).to(torch.int8), s


def _probs(z, min_p):
    p = torch.softmax(z, -1)
    if min_p:
        p = p * (p >= min_p * p.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    return p


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rows = case["rows"]
    st = dict(case=case)
    if case["op"] == "quantize":
        # hidden states: rows of unequal size, a few channels far larger than the rest
        x = torch.randn(rows, case["width"], device=dev, generator=g)
        x *= torch.exp(0.5 * torch.randn(rows, 1, device=dev, generator=g))
        big = torch.randint(0, case["width"], (max(1, case["width"] // 512),), device=dev,
                            generator=g)
        x[:, big] *= 8.0
        st["x"] = x.to(dt)
    elif case["op"] == "logits":
        hidden = torch.randn(rows, case["width"], device=dev, generator=g)
        st["x"], st["xs"] = _codes(hidden)
        weight = torch.randn(case["vocab"], case["width"], device=dev, generator=g)
        weight *= 0.02 * torch.exp(0.3 * torch.randn(case["vocab"], 1, device=dev, generator=g))
        st["w"], st["ws"] = _codes(weight)
        st["bias"] = (torch.randn(case["vocab"], device=dev, generator=g) if case["bias"]
                      else None)
    else:
        K, V = case["drafts"], case["vocab"]
        # the workloads' head and long tail: -1.0 ln(rank) + N(0, 0.5), ranks permuted
        order = torch.rand(rows, 1, V, device=dev, generator=g).argsort(-1)
        z = -torch.log(order.float() + 1.0)
        z = z + 0.5 * torch.randn(rows, K + 1, V, device=dev, generator=g)
        st["p"] = _probs(z, case["min_p"]).to(dt)
        if case["draft"] == "model":
            z = z[:, :K] + 0.8 * torch.randn(rows, K, V, device=dev, generator=g)
            st["q"] = _probs(z, case["min_p"]).to(dt)
            guess = st["q"].float()
        else:   # looked up: often the target's likeliest token
            st["q"] = None
            guess = st["p"][:, :K].float() ** 2
        st["x"] = torch.multinomial(guess.reshape(rows * K, V), 1, generator=g).reshape(
            rows, K).to(torch.int32)
        st["lens"] = (torch.randint(0, K + 1, (rows,), device=dev, generator=g).to(torch.int32)
                      if case["ragged"] else None)
        st["u"] = torch.rand(rows, K, device=dev, generator=g)
        st["v"] = torch.rand(rows, device=dev, generator=g)
    return st


def _quantize(x):
    x = x.float()
    scale = x.abs().amax(1) / 127.0
    unit = torch.where(scale > 0, scale, 1.0)
    # in 64 bits: a quotient next to a half decides the code
    q = (x.double() / unit[:, None].double()).round().clamp(-127, 127)
    return (q * scale[:, None]).float(), scale


def _logits(st):
    out = st["x"].float() @ st["w"].float().t()
    out = out * st["xs"][:, None] * st["ws"]
    if st["bias"] is not None:
        out = out + st["bias"]
    return out.to(DTYPES[st["case"]["dtype"]])


def _verify(st):
    p, q, x = st["p"], st["q"], st["x"].long()
    rows, K = x.shape
    V = p.shape[2]
    at = torch.arange(rows, device=p.device)
    step = torch.arange(K, device=p.device)
    lens = torch.full_like(at, K) if st["lens"] is None else st["lens"].long()
    # draft j is kept while u_j < min(1, p(x_j) / q(x_j)); compared in 64 bits
    px = p[:, :K].gather(2, x[:, :, None])[:, :, 0].double()
    qx = 1.0 if q is None else q.gather(2, x[:, :, None])[:, :, 0].double()
    kept = (st["u"].double() * qx < px) & (step < lens[:, None])
    n = kept.int().cumprod(1).sum(1)
    # the row drawn from, less the draft's where a draft was rejected
    w0 = p[at, n].double()
    refused = n < lens
    j = n.clamp(max=K - 1)
    if q is None:
        less = torch.zeros_like(w0)
        less[at, x[at, j]] = 1.0
    else:
        less = q[at, j].double()
    w = torch.where(refused[:, None], (w0 - less).clamp(min=0.0), w0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, w0)
    # the draw: the first id whose running total exceeds v of the whole (sums in 64 bits)
    total = w.cumsum(1)
    token = (total <= st["v"].double()[:, None] * total[:, -1:]).sum(1)
    last = torch.where(w > 0, torch.arange(V, device=p.device), 0).amax(1)
    token = torch.minimum(token, last)
    slot = torch.arange(K + 1, device=p.device)
    out = torch.cat([x, torch.full_like(x[:, :1], -1)], 1)
    out = torch.where(slot < n[:, None], out, -1)
    out = torch.where(slot == n[:, None], token[:, None], out)
    return out.int(), n.int()


def run(st):
    op = st["case"]["op"]
    if op == "quantize":
        if own:
            q, scale = sampler().quantize_rows(st["x"])
            return q * scale[:, None], scale   # the values that the codes stand for
        return _quantize(st["x"])
    if op == "logits":
        if own:
            return sampler().int8_logits(st["x"], st["xs"], st["w"], st["ws"], bias=st["bias"],
                                         dtype=DTYPES[st["case"]["dtype"]])
        return _logits(st)
    if own:
        return sampler().verify_probs(st["p"], st["q"], st["x"], st["u"], st["v"],
                                      draft_lens=st["lens"])
    return _verify(st)


def work(case):
    rows = case["rows"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "quantize":
        n = rows * case["width"]
        return dict(bytes=n * (size + 1) + 4 * rows, flops=3 * n)
    if case["op"] == "logits":
        V, W = case["vocab"], case["width"]
        return dict(bytes=rows * W + V * W + 4 * (rows + V) + rows * V * size
                    + (4 * V if case["bias"] else 0), flops=2 * rows * V * W)
    K, V = case["drafts"], case["vocab"]
    # a sequence draws from one target row; the draft's row is read as well where a
    # draft was refused (counted for every second sequence: the share goes by the data)
    read = rows * V * size * (1.5 if case["draft"] == "model" else 1.0)
    return dict(bytes=read + rows * K * (8 + 2 * size) + rows * (4 * (K + 1) + 8),
                flops=3 * rows * V)


def exact(case, seed):
    """The outputs from the definitions, in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "quantize":
        x = st["x"].double()
        # the scale is held in 32 bits: the codes are formed against that value
        scale = (torch.maximum(x.amax(1), -x.amin(1)) / 127).float().double()
        q = torch.round(x / scale[:, None])
        return torch.clip(q, -127, 127) * scale[:, None], scale
    if case["op"] == "logits":
        # channels in slices of a bounded size, each a sum of products of whole numbers
        out = torch.empty(case["rows"], case["vocab"], dtype=torch.float64, device="cuda")
        x = st["x"].double().t().contiguous() * st["xs"].double()
        for a in range(0, case["vocab"], 16384):
            part = torch.mm(st["w"][a:a + 16384].double(), x)
            part *= st["ws"][a:a + 16384, None].double()
            if st["bias"] is not None:
                part += st["bias"][a:a + 16384, None].double()
            out[:, a:a + 16384] = part.t()
        return out
    tokens = torch.full((case["rows"], case["drafts"] + 1), -1, dtype=torch.int32)
    counts = torch.zeros(case["rows"], dtype=torch.int32)
    x, u, v = st["x"].tolist(), st["u"].tolist(), st["v"].tolist()
    lens = [case["drafts"]] * case["rows"] if st["lens"] is None else st["lens"].tolist()
    for b in range(case["rows"]):
        n = 0
        weight = None
        while n < lens[b] and weight is None:
            row, t = st["p"][b, n], x[b][n]
            q_t = 1.0 if st["q"] is None else float(st["q"][b, n, t])
            if u[b][n] * q_t < float(row[t]):
                n += 1
                continue
            weight = row.double()
            if st["q"] is None:
                weight[t] -= 1.0
            else:
                weight = weight - st["q"][b, n].double()
            weight = torch.relu(weight)
        if weight is None or float(weight.sum()) == 0.0:
            weight = st["p"][b, n].double()
        c = torch.cumsum(weight, 0)
        aim = torch.tensor([v[b]], dtype=torch.float64, device="cuda") * c[-1]
        pick = int(torch.searchsorted(c, aim, right=True)[0])
        pick = min(pick, int(torch.nonzero(weight)[-1, 0]))
        tokens[b, :n] = torch.tensor(x[b][:n], dtype=torch.int32)
        tokens[b, n] = pick
        counts[b] = n
    return tokens, counts
