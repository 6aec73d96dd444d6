"""token_logprobs and token_logprobs_grad against the references in 64 bits
(oracle/scores.py, which derives the bounds)."""
import numpy as np
import pytest

from tests.gpu_common import device, gpu_available, torch

import token_sampling_row_amd as tsr
from oracle import scores as sc

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

TD = {"f32": torch.float32, "bf16": torch.bfloat16}
NP = {torch.float32: "f32", torch.bfloat16: "bf16"}
VOCABS = [1, 2, 7, 8, 63, 255, 1003, 4096, 8191, 16384, 16387, 32768, 32771, 50001, 65536, 65541,
          128256, 151935, 262145]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=8, max_vocab=1000, max_k=1, seed=3) as h:
        yield h


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device())


def logits(rng, rows, V, dtype, scale=2.0):
    return dev(rng.normal(0, scale, (rows, V)).astype(np.float32)).to(TD[dtype])


def tokens_of(rng, rows, V, n):
    t = rng.integers(0, V, (rows, n)).astype(np.int32)
    if n > 2:
        t[:, 1] = -1
        t[:, 2] = t[:, 0]
    return t


def within(got, want, off):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    d = np.abs(got[fin] - want[fin])
    lim = np.broadcast_to(off, want.shape)[fin]
    assert (d <= lim).all(), (d.max(), lim[d.argmax()])


def check(got, z, tok, k, T, rows=None):
    zv = z.float().cpu().numpy()
    for r in range(len(zv)) if rows is None else rows:
        w = sc.logprobs(zv[r], tok[r] if tok is not None else [], k, T)
        off = w["off"]
        if tok is not None:
            within(got.logprob[r].cpu().numpy().reshape(-1), w["logprob"], off["logprob"])
        if got.entropy is not None:
            within(got.entropy[r].item(), w["entropy"], off["entropy"])
        if got.norm is not None:
            within(got.norm[r].cpu().numpy(), w["norm"], off["norm"])
        if k:
            assert got.top_ids[r].tolist() == w["top_ids"].tolist()
            within(got.top_logprob[r].cpu().numpy(), w["top_logprob"], off["top_logprob"])
        if got.status is not None:
            assert got.status[r].item() == w["status"]


def new_status(rows):
    return torch.full((rows,), -7, dtype=torch.int32, device=device())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("rows", [1, 5])
@pytest.mark.parametrize("n,k", [(0, 3), (1, 0), (3, 20), (1, 64)])
def test_matches(s, dtype, V, rows, n, k):
    rng = np.random.default_rng([V, rows, n])
    z = logits(rng, rows, V, dtype)
    tok = tokens_of(rng, rows, V, n) if n else None
    for T in (1.0, 0.7):
        got = s.token_logprobs(z, None if tok is None else dev(tok), top_k=k, temperature=T,
                               status=new_status(rows))
        check(got, z, tok, k, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(40, 32771), (130, 16390), (300, 70001), (700, 5003),
                                    (1100, 33001), (2500, 20001)])
@pytest.mark.parametrize("k", [0, 7, 64])
def test_many_rows(s, dtype, rows, V, k):
    """However rows are divided: some against the reference, all as in small batches (to the
    bounds: the sums may be divided otherwise)."""
    g = torch.Generator(device()).manual_seed(V + k)
    z = (2 * torch.randn(rows, V, device=device(), generator=g)).to(TD[dtype])
    tok = torch.randint(0, V, (rows,), device=device(), generator=g).int()
    got = s.token_logprobs(z, tok, top_k=k, status=new_status(rows))
    some = [0, 1, rows // 2, rows - 1]
    check(got, z, tok.cpu().numpy()[:, None], k, 1.0, some)
    part = [s.token_logprobs(z[a:a + 3], tok[a:a + 3].contiguous(), top_k=k)
            for a in range(0, rows, 3)]
    lse = torch.logsumexp(z[some].double(), 1)
    assert bool(((got.norm[some, 0].double() + got.norm[some, 1].double().log()) - lse).abs().max()
                < 1e-5)
    for name in ("logprob", "entropy", "norm", "top_logprob", "top_ids"):
        a = getattr(got, name)
        if a is None:
            continue
        b = torch.cat([getattr(p, name) for p in part])
        if name == "top_ids":
            assert torch.equal(a, b)
        else:   # twice the largest weight_error of these rows: m below 12
            assert bool(((a - b).abs() <= 2 * 45 * sc.U * (1 + b.abs())).all()), name


@pytest.mark.parametrize("dtype,rows,V,k", [("bf16", 1100, 70001, 20), ("bf16", 1100, 70001, 0),
                                            ("bf16", 9000, 8190, 5), ("f32", 9000, 4101, 64),
                                            ("f32", 20000, 1001, 3), ("bf16", 17000, 33001, 50),
                                            ("f32", 8195, 20011, 0), ("bf16", 35000, 2500, 0)])
def test_batches_past_the_caches_and_the_workspace(s, dtype, rows, V, k):
    """More than 128 MB of logits, more than 8192 rows: rows on either side of each limit
    against the reference, forward and backward."""
    g = torch.Generator(device()).manual_seed(V)
    z = torch.empty(rows, V, dtype=TD[dtype], device=device()).normal_(generator=g)
    tok = torch.randint(0, V, (rows, 2), device=device(), generator=g).int()
    st = new_status(rows)
    z[rows - 2] = float("nan")
    z[rows - 3, 5] = float("inf")
    got = s.token_logprobs(z, tok, top_k=k, status=st)
    some = sorted({0, 1, 8191 % rows, 8192 % rows, 16383 % rows, 16384 % rows, rows // 2, rows - 3,
                   rows - 2, rows - 1})
    part = tsr.TokenLogprobs(*(None if t is None else t[some] for t in got))
    check(part, z[some], tok[some].cpu().numpy(), k, 1.0)
    up = torch.randn(rows, 2, device=device(), generator=g)
    grad = s.token_logprobs_grad(z, tok, got.norm, up)
    check_grad(grad[some], z[some], tok[some].cpu().numpy(), got.norm[some], up[some])
    assert int((st != 0).sum()) == 2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_special_rows(s, dtype):
    V = 40003
    rng = np.random.default_rng(5)
    z = rng.normal(0, 3, (14, V)).astype(np.float32)
    z[0, 17] = np.nan
    z[1, V - 1] = np.inf
    z[2] = -np.inf
    z[3] = -np.inf
    z[3, 39999] = -2.0                     # one id is left
    z[4] = -np.inf
    z[4, [5, 30000, 40002]] = [1.0, 1.0, 3.0]
    z[5] = 0.0                             # all equal
    z[5, ::2] = -0.0
    z[6, 20000] = 80.0                     # nearly certain
    z[7] *= 1e30
    z[8] += 3e4
    z[9] = np.sort(z[9])
    z[10] = -np.sort(-z[10])
    z[11] = np.round(z[11])                # many ties
    z[12, 0], z[12, 1:] = np.nan, -np.inf
    z[13] = -3e38
    z[13, 7] = 3e38                        # differences past float32
    t = dev(z).to(TD[dtype])
    tok = np.stack([np.array([0, 17, 39999, -1, V, -5, 40002, 5], dtype=np.int32)] * 14)
    for T in (1.0, 0.3, 5.0):
        for k in (0, 1, 5, 64):
            got = s.token_logprobs(t, dev(tok), top_k=k, temperature=T, status=new_status(14))
            check(got, t, tok, k, T)
    got = s.token_logprobs(t, dev(tok[:, :4]), status=new_status(14))
    assert got.status.tolist() == [1, 1, 2, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1, 0]


def hard_rows(rng, V):
    """Rows whose likeliest ids lie where a search by samples looks last."""
    base = rng.normal(0, 1, V).astype(np.float32)
    rows = []
    for start, step, count in ((0, 1, 200), (V - 200, 1, 200), (0, 256, 100), (3, 64, 300),
                               (5, 2048, 70), (0, 8, 2000), (1, 1024, 100)):
        row = base.copy()
        at = (start + step * np.arange(count)) % V
        row[at] = 10 + rng.permutation(len(at)).astype(np.float32) / 64
        rows.append(row)
        row = base.copy()
        row[at] = 10.0                     # the same, all equal
        rows.append(row)
    rows.append(np.full(V, -1.5, dtype=np.float32))
    rows.append(np.arange(V, dtype=np.float32) / 1024)
    rows.append(-np.arange(V, dtype=np.float32) / 1024)
    rows.append((np.arange(V) % 7).astype(np.float32))
    row = np.full(V, -np.inf, dtype=np.float32)
    row[rng.permutation(V)[:30]] = rng.normal(0, 1, 30)
    rows.append(row)
    return np.stack(rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 5000, 33000, 100003])
@pytest.mark.parametrize("k", [1, 2, 20, 63, 64])
def test_the_likeliest_wherever_they_are(s, dtype, V, k):
    t = dev(hard_rows(np.random.default_rng(V), V)).to(TD[dtype])
    got = s.token_logprobs(t, top_k=k)
    check(got, t, None, k, 1.0)
    alone = s.token_logprobs(t[4:5], top_k=k)
    assert torch.equal(alone.top_ids, got.top_ids[4:5])


# a mask's finite fill and flat rows: the k-th largest is one of many equal values
FILLS = [-1.5, -1e4, float(torch.finfo(torch.bfloat16).min), 0.0, 2.5]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [100003, 128256])
@pytest.mark.parametrize("k", [20, 41, 64])
@pytest.mark.parametrize("fill", FILLS)
def test_ties_of_a_fill(s, dtype, V, k, fill):
    """A few larger logits, the last slices' among them, over a fill: in a row alone and in
    several whose neighbours are ordinary."""
    rng = np.random.default_rng(13)
    z = rng.normal(0, 2, (9, V)).astype(np.float32)
    z[2:5] = z[7:] = fill
    for r in (2, 4, 7, 8):
        z[r, [50, 70000, V - 3001, V - 1]] = [fill / 2 + 0.5, fill / 4 + 1, 3.5, 3.25]
    z[8, rng.permutation(V)[:30]] = rng.normal(4, 1, 30)
    t = dev(z).to(TD[dtype])
    check(s.token_logprobs(t, top_k=k, status=new_status(9)), t, None, k, 1.0)
    for r in (2, 3, 8):
        check(s.token_logprobs(t[r:r + 1], top_k=k), t[r:r + 1], None, k, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(300, 33001), (700, 70001)])
@pytest.mark.parametrize("k", [20, 64])
@pytest.mark.parametrize("fill", FILLS)
def test_ties_of_a_fill_in_large_batches(s, dtype, rows, V, k, fill):
    """Every other row a fill with larger logits at its ends."""
    g = torch.Generator(device()).manual_seed(V)
    z = (2 * torch.randn(rows, V, device=device(), generator=g)).to(TD[dtype])
    z[::2] = fill
    z[::2, 7], z[::2, V - 5] = 3.0, 3.5
    got = s.token_logprobs(z, top_k=k)
    want = torch.sort(z.float(), dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(got.top_ids.long(), want)
    check(got, z, None, k, 1.0, [0, 1, rows // 2, rows - 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 5])
@pytest.mark.parametrize("V", [13, 9001, 70003])
def test_strided_rows(s, dtype, off, V):
    rng = np.random.default_rng(off)
    z = logits(rng, 6, V + 37, dtype)[:, off:off + V]
    tok = tokens_of(rng, 6, V, 4)
    check(s.token_logprobs(z, dev(tok), top_k=5), z, tok, 5, 1.0)
    got = s.token_logprobs(z, dev(tok))
    g = dev(rng.normal(0, 1, (6, 4)).astype(np.float32))
    out = torch.full((6, V + 29), 77.0, dtype=TD[dtype], device=device())
    grad = s.token_logprobs_grad(z, dev(tok), got.norm, g, out=out[:, off:off + V])
    check_grad(grad, z, tok, got.norm, g)
    assert bool((out[:, :off] == 77).all()) and bool((out[:, off + V:] == 77).all())


def check_grad(grad, z, tok, norm, g, T=1.0, H=None, ge=None, rows=None):
    zv, nv = z.float().cpu().numpy(), norm.cpu().numpy()
    gv = None if g is None else g.cpu().numpy().reshape(len(zv), -1)
    for r in range(len(zv)) if rows is None else rows:
        want, off = sc.logprobs_grad(zv[r], [] if tok is None else tok[r], nv[r],
                                     [] if g is None else gv[r], T,
                                     0.0 if H is None else H[r].item(),
                                     0.0 if ge is None else ge[r].item(), NP[z.dtype])
        within(grad[r].float().cpu().numpy(), want, off)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("n,entropy", [(1, False), (4, True), (0, True)])
def test_gradient_matches(s, dtype, V, n, entropy):
    rng = np.random.default_rng([V, n])
    rows, T = 4, 0.8
    z = logits(rng, rows, V, dtype)
    tok = tokens_of(rng, rows, V, n) if n else None
    fwd = s.token_logprobs(z, None if tok is None else dev(tok), temperature=T)
    g = dev(rng.normal(0, 1, (rows, n)).astype(np.float32)) if n else None
    ge = dev(rng.normal(0, 1, rows).astype(np.float32)) if entropy else None
    grad = s.token_logprobs_grad(z, None if tok is None else dev(tok), fwd.norm, g, fwd.entropy,
                                 ge, temperature=T)
    check_grad(grad, z, tok, fwd.norm, g, T, fwd.entropy, ge)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(300, 9001), (1030, 40001)])
def test_gradient_of_many_rows(s, dtype, rows, V):
    g = torch.Generator(device()).manual_seed(V)
    z = (2 * torch.randn(rows, V, device=device(), generator=g)).to(TD[dtype])
    tok = torch.randint(0, V, (rows,), device=device(), generator=g).int()
    up = torch.randn(rows, device=device(), generator=g)
    up[3] = 0.0
    fwd = s.token_logprobs(z, tok)
    grad = s.token_logprobs_grad(z, tok, fwd.norm, up)
    check_grad(grad, z, tok.cpu().numpy()[:, None], fwd.norm, up, rows=[0, 3, rows // 2, rows - 1])
    for a in range(0, rows, 100):
        part = s.token_logprobs_grad(z[a:a + 100], tok[a:a + 100], fwd.norm[a:a + 100],
                                     up[a:a + 100])
        assert torch.equal(part, grad[a:a + 100])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_special_rows(s, dtype):
    """Masked logits, ids given twice, padding, rows to which nothing comes back, bad ids,
    rows without a norm."""
    V = 20011
    rng = np.random.default_rng(6)
    z = rng.normal(0, 3, (8, V)).astype(np.float32)
    z[0, ::3] = -np.inf
    z[1] = np.nan
    z[2] = np.nan                              # nothing comes back to it
    z[4] = -np.inf
    z[5] = -np.inf
    z[5, 77] = 2.0
    z[6, 5] = 90.0
    t = dev(z).to(TD[dtype])
    tok = np.tile(np.array([3, 20010, 3, -1, 3], dtype=np.int32), (8, 1))
    tok[3, 1] = V
    tok[2] = -1
    g = rng.normal(0, 1, (8, 5)).astype(np.float32)
    g[:, 3] = np.nan                           # the padding's does not count
    ge = rng.normal(0, 1, 8).astype(np.float32)
    ge[2] = 0.0
    fwd = s.token_logprobs(t, dev(tok), status=new_status(8))
    assert fwd.status.tolist() == [0, 1, 1, 3, 2, 0, 0, 0]
    for e in (None, dev(ge)):
        grad = s.token_logprobs_grad(t, dev(tok), fwd.norm, dev(g), fwd.entropy, e)
        check_grad(grad, t, tok, fwd.norm, dev(g), 1.0, fwd.entropy, e)
        assert not bool(grad[2].any()) and bool(grad[[1, 3, 4]].isnan().all())
        # logits of -inf get nothing, where they are no given token (3 and 20010 are)
        assert not bool(grad[0, torch.arange(6, 20010, 3, device=device())].any())


def test_gradient_against_differences(s):
    """Along random directions d in [-1, 1]: the forward call's own values at z +- h d. The
    third derivative along d of log p and of H stays below 8 and 8 (1 + log V) for
    |d| <= 1 (cumulants of a variable within [-1, 1], times log p for H), so h^2 / 6 of
    that, and the values' own errors over h."""
    V, h = 3001, 2.0 ** -6
    rng = np.random.default_rng(7)
    z = logits(rng, 1, V, "f32")
    tok = dev(np.array([[5, 900, 5]], dtype=np.int32))
    g, ge = torch.tensor([[0.7, -1.1, 0.4]], device=device()), torch.tensor([0.9], device=device())
    fwd = s.token_logprobs(z, tok)
    grad = s.token_logprobs_grad(z, tok, fwd.norm, g, fwd.entropy, ge)[0].double()
    for _ in range(10):
        d = dev(rng.uniform(-1, 1, (1, V)).astype(np.float32))

        def value(zz):
            r = s.token_logprobs(zz, tok)
            return float((r.logprob.double() * g).sum() + (r.entropy.double() * ge).sum())

        diff = (value(z + h * d) - value(z - h * d)) / (2 * h)
        bound = h * h / 6 * 8 * (2.2 + 0.9 * (1 + np.log(V))) + 6 * 60 * sc.U * 8 / h
        assert abs(diff - float(grad @ d[0].double())) < bound


def test_many_tokens(s):
    rng = np.random.default_rng(8)
    z = logits(rng, 2, 5000, "bf16")
    tok = rng.integers(0, 300, (2, 1024)).astype(np.int32)
    fwd = s.token_logprobs(z, dev(tok))
    check(fwd, z, tok, 0, 1.0)
    g = dev(rng.normal(0, 1, (2, 1024)).astype(np.float32))
    check_grad(s.token_logprobs_grad(z, dev(tok), fwd.norm, g), z, tok, fwd.norm, g)
    for call in (lambda t: s.token_logprobs(z, t),
                 lambda t: s.token_logprobs_grad(z, t, fwd.norm, torch.zeros(t.shape, device=device()))):
        with pytest.raises(tsr.TsrError):
            call(torch.zeros(2, 1025, dtype=torch.int32, device=device()))
    with pytest.raises(tsr.TsrError):
        s.token_logprobs(z, top_k=65)
    with pytest.raises(tsr.TsrError):
        s.token_logprobs(z, temperature=0.0)
    with pytest.raises(tsr.TsrError):   # the gradient in the logits' place
        s.token_logprobs_grad(z, dev(tok), fwd.norm, g, out=z)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ids", [[77], [0, 77, 4095, 4999]])
@pytest.mark.parametrize("entropy", [False, True])
def test_gradients_of_one_token_that_cancel(s, dtype, ids, entropy):
    """1024 tokens of few ids, whose gradients of some 10^4 leave a sum of some 10 to each id:
    as one token of each with the sum. Sums in 64 bits are off by 1024 * 2^-53 of their
    terms' sizes, in the id's own sum and in the row's."""
    rng = np.random.default_rng(len(ids))
    T, n = 0.7, 1024 // len(ids)
    z = logits(rng, 2, 5000, dtype)
    g = rng.normal(0, 1e4, (2, len(ids), n)).astype(np.float32)
    g[:, :, n // 2:] = -g[:, :, :n // 2]
    g[:, :, 0] += rng.normal(0, 10, g.shape[:2]).astype(np.float32)
    order = rng.permutation(1024)
    tok = np.tile(np.repeat(np.array(ids, dtype=np.int32), n)[order], (2, 1))
    fwd = s.token_logprobs(z, dev(tok), temperature=T)
    ge = dev(rng.normal(0, 1, 2).astype(np.float32)) if entropy else None
    grad = s.token_logprobs_grad(z, dev(tok), fwd.norm, dev(g.reshape(2, 1024)[:, order]),
                                 fwd.entropy, ge, temperature=T).float().cpu().numpy()
    zv, norm, size = z.float().cpu().numpy(), fwd.norm.cpu().numpy(), np.abs(g).sum()
    for r in range(2):
        want, off = sc.logprobs_grad(zv[r], ids, norm[r], g[r].astype(np.float64).sum(1), T,
                                     fwd.entropy[r].item(), ge[r].item() if entropy else 0.0, dtype)
        within(grad[r], want, off + 2 * 1024 * 2.0 ** -53 * size / T)


@pytest.mark.parametrize("T", [1e-30, 1e-6, 1e6, 1e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_temperatures_far_from_one(s, dtype, T):
    """Down to the largest logit alone, up to all finite logits alike."""
    rng = np.random.default_rng(11)
    z = rng.normal(0, 3, (3, 33001)).astype(np.float32)
    z[1, ::5] = -np.inf
    z[2] *= 1e20
    t = dev(z).to(TD[dtype])
    tok = np.tile(np.array([[7, 5]], dtype=np.int32), (3, 1))
    tok[:, 1] = t.float().cpu().numpy().argmax(1)
    got = s.token_logprobs(t, dev(tok), top_k=4, temperature=T)
    check(got, t, tok, 4, T)
    g = dev(rng.normal(0, 1, (3, 2)).astype(np.float32))
    ge = dev(rng.normal(0, 1, 3).astype(np.float32))
    if T >= 1e-6:   # 1 / T times a gradient is a float32 number
        grad = s.token_logprobs_grad(t, dev(tok), got.norm, g, got.entropy, ge, temperature=T)
        check_grad(grad, t, tok, got.norm, g, T, got.entropy, ge)


def test_a_vocabulary_of_millions(s):
    V = 5_000_003
    g = torch.Generator(device()).manual_seed(2)
    z = torch.randn(2, V, device=device(), generator=g)
    tok = torch.tensor([V - 1, 12], device=device(), dtype=torch.int32)
    check(s.token_logprobs(z, tok, top_k=9), z, tok.cpu().numpy()[:, None], 9, 1.0)


@pytest.mark.parametrize("dtype,V,k", [("bf16", 524301, 64), ("bf16", 1048589, 20),
                                       ("f32", 262155, 64), ("f32", 524303, 20)])
def test_special_rows_of_wide_vocabularies(s, dtype, V, k):
    """Just past the widest rows that are cut into slices for so many alternatives."""
    rng = np.random.default_rng(V)
    z = rng.normal(0, 3, (12, V)).astype(np.float32)
    z[0, V - 1] = np.nan
    z[1, 17] = np.inf
    z[2] = -np.inf
    z[3] = -np.inf
    z[3, [5, V // 2, V - 1]] = [1.0, 1.0, 3.0]   # fewer than k are left
    z[4] = 0.0
    z[4, ::2] = -0.0
    z[5] = torch.finfo(torch.bfloat16).min
    z[5, [9, V - 2]] = [-1.0, 2.0]
    z[6] = np.round(z[6])
    z[7] = -1.5
    z[8] = np.sort(z[8])
    z[9] *= 1e30
    z[10, 0], z[10, 1:] = np.nan, -np.inf
    t = dev(z).to(TD[dtype])
    tok = np.tile(np.array([0, 17, V - 1, -1, V, -5, V // 2], dtype=np.int32), (12, 1))
    tok[11] = [0, 17, V - 1, -1, 3, 3, V // 2]
    for T in (1.0, 0.3):
        got = s.token_logprobs(t, dev(tok), top_k=k, temperature=T, status=new_status(12))
        check(got, t, tok, k, T)
    assert got.status.tolist() == [1, 1, 2] + [3] * 7 + [1, 0]


def test_rows_past_2_31_bytes(s):
    rows, stride, V = 4, (1 << 31) // 3, 9000
    big = torch.zeros(3 * stride + V, dtype=torch.float32, device=device())
    z = big.as_strided((rows, V), (stride, 1))
    z.copy_(torch.randn(rows, V, device=device()))
    tok = np.array([[1], [2], [8999], [4]], dtype=np.int32)
    fwd = s.token_logprobs(z, dev(tok), top_k=3)
    check(fwd, z, tok, 3, 1.0)
    g = torch.ones(rows, 1, device=device())
    out = torch.zeros_like(big).as_strided((rows, V), (stride, 1))
    check_grad(s.token_logprobs_grad(z, dev(tok), fwd.norm, g, out=out), z, tok, fwd.norm, g)


def test_no_rows(s):
    z = torch.zeros(0, 50, device=device())
    got = s.token_logprobs(z, torch.zeros(0, 2, dtype=torch.int32, device=device()), top_k=3)
    assert got.logprob.shape == (0, 2) and got.top_ids.shape == (0, 3)
    assert s.token_logprobs_grad(z, None, got.norm, None, got.entropy, got.entropy).shape == (0, 50)
