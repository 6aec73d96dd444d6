"""verify_probs against the plain reference in 64 bits (oracle/vprobs.py):
tokens, counts and statuses are equal. The kernels and the reference add the
same float64 weights in different orders, so a draw could differ only where it
comes within the sums' rounding (V * 2^-53 relative) of a neighbouring token;
each comparison asserts that it does not come that near."""
import numpy as np
import pytest

from tests.gpu_common import device, gpu_available, to_dev, torch

import token_sampling_row_amd as tsr
from oracle import vprobs as ov
from token_sampling_row_amd import workloads as wl

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=4096, max_vocab=1 << 21, max_k=32, seed=3) as h:
        yield h


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device())


def stored(p, dtype):
    """float values [..., V] -> (device tensor, float64 values)."""
    p = np.ascontiguousarray(p, dtype=np.float32)
    if dtype == "f32":
        return dev(p), p.astype(np.float64)
    bits = wl.f32_to_bf16_bits(p)
    t = dev(bits.view(np.int16)).view(torch.bfloat16)
    return t, wl.bf16_bits_to_f32(bits).astype(np.float64)


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def batch(rng, rows, K, V, sharp=1.5, noise=0.8):
    z = rng.normal(0, sharp, (rows, K + 1, V))
    return softmax(z), softmax(z[:, :K] + rng.normal(0, noise, (rows, K, V)))


def drafts_from(rng, q):
    """Draft tokens drawn from q [rows, K, V]."""
    c = np.cumsum(q, -1)
    u = rng.random(q.shape[:2])[..., None] * c[..., -1:]
    return np.minimum((c <= u).sum(-1), q.shape[-1] - 1).astype(np.int32)


def check(got, p, q, x, lens, u, v, status=None):
    tokens, accepted = got[0].cpu().numpy(), got[1].cpu().numpy()
    V = p.shape[-1]
    seen = set()
    for b in range(len(x)):
        r = ov.verify_probs_row(p[b], None if q is None else q[b], x[b],
                                x.shape[1] if lens is None else int(lens[b]), u[b], v[b])
        if r.status == 0 and np.isfinite(r.margin):
            exact_edge = r.margin == 0.0
            assert exact_edge or r.margin > V * 2.0 ** -53
        assert list(tokens[b]) == list(r.tokens), (b, tokens[b], r)
        assert accepted[b] == r.accepted
        if status is not None:
            assert int(status[b]) == r.status, (b, int(status[b]), r)
        seen.add((r.status, r.accepted))
    return seen


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,K,V", [
    (3, 1, 1), (5, 2, 2), (7, 3, 7), (4, 4, 63), (9, 4, 64), (8, 1, 255), (6, 5, 256),
    (6, 5, 257), (5, 2, 511), (5, 2, 512), (5, 3, 513), (33, 8, 1000), (3, 32, 700),
    (64, 4, 4099), (17, 7, 8191), (1, 4, 32000), (2, 3, 65537), (40, 2, 32003), (3, 2, 151935),
    (300, 3, 5000), (2, 1, 300007)])
def test_batches_match(s, dtype, rows, K, V):
    rng = np.random.default_rng([rows, K, V])
    p, q = batch(rng, rows, K, V)
    (pt, p), (qt, q) = stored(p, dtype), stored(q, dtype)
    x = drafts_from(rng, q)
    u, v = rng.random((rows, K), dtype=np.float32), rng.random(rows, dtype=np.float32)
    lens = rng.integers(0, K + 1, rows).astype(np.int32)
    lens[0] = K
    st = torch.full((rows,), -7, dtype=torch.int32, device=device())
    for ln in (None, lens):
        for with_q in (True, False):
            got = s.verify_probs(pt, qt if with_q else None, dev(x), dev(u), dev(v),
                                 draft_lens=None if ln is None else dev(ln), out_status=st)
            check(got, p, q if with_q else None, x, ln, u, v, st)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1 << 18, 600001, (1 << 20) + 3])
def test_wide_vocabularies(s, dtype, V):
    """Rows cut into more spans than a workgroup keeps sums for."""
    rng = np.random.default_rng(V)
    p, q = batch(rng, 3, 2, V)
    (pt, p), (qt, q) = stored(p, dtype), stored(q, dtype)
    x = drafts_from(rng, q)
    u, v = rng.random((3, 2), dtype=np.float32), rng.random(3, dtype=np.float32)
    u[1] = 0.0
    check(s.verify_probs(pt, qt, dev(x), dev(u), dev(v)), p, q, x, None, u, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [2, 70])
def test_filtered_probabilities(s, dtype, rows):
    """Rows that are zero outside a few tokens, in one row at either end only;
    draws of 0 and of the largest uniform below 1 land on kept tokens."""
    K, V = 3, 9001
    rng = np.random.default_rng(rows)
    p, q = batch(rng, rows, K, V, sharp=3.0)
    p = np.where(p >= 0.2 * p.max(-1, keepdims=True), p, 0)
    q = np.where(q >= 0.2 * q.max(-1, keepdims=True), q, 0)
    p[0, 0] = 0
    p[0, 0, V - 1] = 1.0
    p[1, 0] = 0
    p[1, 0, 0] = 1.0
    (pt, p), (qt, q) = stored(p, dtype), stored(q, dtype)
    x = drafts_from(rng, q)
    x[0, 0], x[1, 0] = 5, 6
    u = rng.random((rows, K), dtype=np.float32)
    for v0 in (0.0, float(np.float32(1) - np.float32(2.0 ** -24)), 0.5):
        v = np.full(rows, v0, dtype=np.float32)
        for qq, qn in ((qt, q), (None, None)):
            got = s.verify_probs(pt, qq, dev(x), dev(u), dev(v))
            check(got, p, qn, x, None, u, v)
            n = got[1].long()
            drawn = got[0].gather(1, n[:, None])[:, 0].long()
            assert bool((pt[torch.arange(rows), n, drawn] > 0).all())


def test_every_draft_kept_or_none(s):
    rows, K, V = 6, 5, 2000
    rng = np.random.default_rng(1)
    p, _ = batch(rng, rows, K, V)
    pt, p = stored(p, "f32")
    x = drafts_from(rng, p[:, :K])
    v = rng.random(rows, dtype=np.float32)
    u = np.full((rows, K), np.float32(1) - np.float32(2.0 ** -24), dtype=np.float32)
    got = s.verify_probs(pt, pt[:, :K], dev(x), dev(u), dev(v))     # p = q: always kept
    assert bool((got[1] == K).all())
    check(got, p, p[:, :K], x, None, u, v)
    none = p.copy()
    for b in range(rows):
        for j in range(K):
            none[b, j, x[b, j]] = 0.0
    nt, none = stored(none, "f32")
    u[:] = 0.0
    got = s.verify_probs(nt, pt[:, :K], dev(x), dev(u), dev(v))     # p(x) = 0: never kept
    assert bool((got[1] == 0).all())
    check(got, none, p[:, :K], x, None, u, v)


@pytest.mark.parametrize("rows", [3, 80])
def test_an_empty_residual_draws_from_the_target(s, rows):
    """q >= p everywhere (rows that need not sum to 1), and a certain proposal
    that the target gives all its weight but the uniform still refuses."""
    K, V = 2, 5003
    rng = np.random.default_rng(rows)
    p, _ = batch(rng, rows, K, V)
    q = p[:, :K] * 2.0
    (pt, p), (qt, q) = stored(p, "f32"), stored(q, "f32")
    x = drafts_from(rng, q)
    u = np.full((rows, K), 0.75, dtype=np.float32)
    v = rng.random(rows, dtype=np.float32)
    got = s.verify_probs(pt, qt, dev(x), dev(u), dev(v))
    assert bool((got[1] == 0).all())
    check(got, p, q, x, None, u, v)
    one = np.zeros((rows, K + 1, V))
    one[:, :, 17] = 0.5                                 # weight 0.5 on one token: u 0.75 refuses
    ot, one = stored(one, "f32")
    x[:] = 17
    got = s.verify_probs(ot, None, dev(x), dev(u), dev(v))
    assert bool((got[0][:, 0] == 17).all()) and bool((got[1] == 0).all())
    check(got, one, None, x, None, u, v)


@pytest.mark.parametrize("V", [300, 40000])
@pytest.mark.parametrize("rows_more", [0, 200])
def test_statuses(s, V, rows_more):
    K = 3
    rows = 16 + rows_more
    rng = np.random.default_rng(V)
    p, q = batch(rng, rows, K, V)
    x = drafts_from(rng, q)
    u, v = rng.random((rows, K), dtype=np.float32), rng.random(rows, dtype=np.float32)
    lens = np.full(rows, K, dtype=np.int32)
    u[:16] = 0.0                                        # drafts kept unless said otherwise
    x[0, 2] = V                                         # out of range
    x[1, 0] = -1
    x[2, 2], lens[2] = 1 << 30, 2                       # ... past the drafts: not read
    lens[3], lens[4] = -1, K + 1
    p[5, 1, x[5, 1]] = np.nan                           # a tested probability
    q[6, 0, x[6, 0]] = np.inf
    p[7, 0, x[7, 0]] = -0.25                            # (refused at once)
    u[8, 1] = 1.0
    u[9, 2] = np.nan
    v[10] = 1.0
    v[11] = np.nan
    p[12, K, V - 1] = np.nan                            # in the row drawn from
    p[13, K] = 0.0                                      # nothing to draw from
    u[14, 0], p[14, 0, x[14, 0]] = 0.5, 0.0             # refused at 0:
    p[14, 1] = np.nan                                   # ... later rows are not looked at
    x[14, 1] = x[14, 0]
    u[15, 0], p[15, 0, x[15, 0]] = 0.5, 0.0
    q[15, 0, (x[15, 0] + 1) % V] = -1e-6                # in the draft's row at a refusal
    (pt, p), (qt, q) = stored(p, "f32"), stored(q, "f32")
    st = torch.full((rows,), -7, dtype=torch.int32, device=device())
    got = s.verify_probs(pt, qt, dev(x), dev(u), dev(v), draft_lens=dev(lens), out_status=st)
    check(got, p, q, x, lens, u, v, st)
    assert st[:16].tolist() == [3, 3, 0, 4, 4, 1, 1, 1, 4, 4, 4, 4, 1, 2, 0, 1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_strided_rows(s, dtype, off):
    """Sequences and positions inside wider tensors at odd offsets, positions
    and sequences swapped in memory, and one row repeated for every sequence."""
    rows, K, V = 5, 3, 1501
    rng = np.random.default_rng(off)
    p, q = batch(rng, rows, K, V)
    x = drafts_from(rng, q)
    u, v = rng.random((rows, K), dtype=np.float32), rng.random(rows, dtype=np.float32)
    wide_p = np.full((K + 1, rows, V + 11), np.nan)
    wide_q = np.full((rows, K, V + 5), np.nan)
    wide_p[:, :, off:off + V] = p.transpose(1, 0, 2)
    wide_q[:, :, off:off + V] = q
    (wp, pv), (wq, qv) = stored(wide_p, dtype), stored(wide_q, dtype)
    pt = wp.transpose(0, 1)[:, :, off:off + V]
    qt = wq[:, :, off:off + V]
    p, q = pv.transpose(1, 0, 2)[:, :, off:off + V], qv[:, :, off:off + V]
    check(s.verify_probs(pt, qt, dev(x), dev(u), dev(v)), p, q, x, None, u, v)
    same_p, same_q = pt[:1, :1].expand(rows, K + 1, V), qt[:1, :1].expand(rows, K, V)
    check(s.verify_probs(same_p, same_q, dev(x), dev(u), dev(v)),
          np.broadcast_to(p[:1, :1], p.shape), np.broadcast_to(q[:1, :1], q.shape), x, None, u, v)


def test_positions_past_32_bit_offsets(s):
    """A target whose last sequences start past 2^32 bytes."""
    rows, K, V = 1700, 4, 151936
    t = torch.zeros(rows, K + 1, V, dtype=torch.float32, device=device())
    t[:, :, 5] = 0.25
    t[:, :, V - 1] = 0.75
    x = torch.full((rows, K), V - 1, dtype=torch.int32, device=device())
    u = torch.full((rows, K), 0.5, device=device())
    u[::2, 2] = 0.8
    v = torch.full((rows,), 0.1, device=device())
    tokens, accepted = s.verify_probs(t, None, x, u, v)
    want = torch.full((rows, K + 1), V - 1, dtype=torch.int32, device=device())
    want[:, K] = 5
    want[::2, 2] = 5
    want[::2, 3:] = -1
    assert torch.equal(tokens, want)
    assert torch.equal(accepted, (tokens >= 0).sum(1).int() - 1)


@pytest.mark.parametrize("rows", [1, 6, 90])
def test_captured_calls_replay(s, rows):
    rng = np.random.default_rng(rows)
    K, V = 4, 40001
    p, q = batch(rng, rows, K, V)
    (pt, _), (qt, qn) = stored(p, "f32"), stored(q, "f32")
    x = dev(drafts_from(rng, qn))
    u, v = torch.zeros(rows, K, device=device()), torch.zeros(rows, device=device())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.verify_probs(pt, qt, x, u, v)
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = s.verify_probs(pt, qt, x, u, v)
    for k in range(4):
        u.copy_(torch.from_numpy(rng.random((rows, K), dtype=np.float32)))
        v.copy_(torch.from_numpy(rng.random(rows, dtype=np.float32)))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = s.verify_probs(pt, qt, x, u, v)
        torch.cuda.synchronize()
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])


def test_the_whole_step_from_hidden_states(s):
    """As a serving loop runs it: hidden states of the draft and the target through
    an 8-bit projection, drafts drawn by the sampler, the distributions both
    were drawn from, and the verify step on the caller's uniforms."""
    B, K, V, W = 12, 3, 4001, 384
    rng = np.random.default_rng(2)
    w, ws = s.quantize_rows(dev(rng.normal(0, 0.06, (V, W)).astype(np.float32)))
    hidden = rng.normal(0, 1, (B, K + 1, W)).astype(np.float32)
    near = (hidden[:, :K] + rng.normal(0, 0.3, (B, K, W))).astype(np.float32)
    prm = {"temperature": 0.9, "top_k": 40}

    def distributions(hid, step):
        n = hid.shape[0] * hid.shape[1]
        probs = torch.empty(n, V, device=device())
        tok = s.sample_hidden(dev(hid.reshape(n, W)), w, ws, prm, step, dtype=torch.float32,
                              diag={"probs": probs})
        return probs.view(hid.shape[0], hid.shape[1], V), tok.view(hid.shape[0], hid.shape[1])

    q, x = distributions(near, 1)
    p, _ = distributions(hidden, 2)
    u, v = rng.random((B, K), dtype=np.float32), rng.random(B, dtype=np.float32)
    got = s.verify_probs(p, q, x, dev(u), dev(v))
    seen = check(got, p.double().cpu().numpy(), q.double().cpu().numpy(), x.cpu().numpy(), None,
                 u, v)
    assert len({a for _, a in seen}) > 1


def test_refusals(s):
    d = device()
    B, K, V = 4, 2, 50
    p = torch.full((B, K + 1, V), 1.0 / V, device=d)
    q = p[:, :K].contiguous()
    x = torch.zeros(B, K, dtype=torch.int32, device=d)
    u, v = torch.zeros(B, K, device=d), torch.zeros(B, device=d)
    for call in (
            lambda: s.verify_probs(p[0], q, x, u, v),
            lambda: s.verify_probs(p.transpose(1, 2), q, x, u, v),
            lambda: s.verify_probs(p[:, :1], None, x[:, :0], u[:, :0], v),
            lambda: s.verify_probs(p, q[:, :1], x, u, v),
            lambda: s.verify_probs(p, q.to(torch.bfloat16), x, u, v),
            lambda: s.verify_probs(p, q[:, :, :49], x, u, v),
            lambda: s.verify_probs(p, q, x.long(), u, v),
            lambda: s.verify_probs(p, q, x[:3], u, v),
            lambda: s.verify_probs(p, q, x, u.double(), v),
            lambda: s.verify_probs(p, q, x, u[:, :1], v),
            lambda: s.verify_probs(p, q, x, u, v[:3]),
            lambda: s.verify_probs(p, q, x, u, v.cpu()),
            lambda: s.verify_probs(p, q, x, u, v, draft_lens=x[:, 0]),
            lambda: s.verify_probs(p, q, x, u, v, out_tokens=x),
            lambda: s.verify_probs(p, q, x, u, v, out_status=torch.zeros(3, dtype=torch.int32,
                                                                         device=d))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        s.verify_probs(p.half(), q.half(), x, u, v)
    with tsr.Sampler(0, max_rows=3, max_vocab=50, max_k=2) as few:
        with pytest.raises(tsr.TsrError) as e:
            few.verify_probs(p, q, x, u, v)
        assert e.value.code == 1
    with tsr.Sampler(0, max_rows=4, max_vocab=50, max_k=1) as few:
        with pytest.raises(tsr.TsrError) as e:
            few.verify_probs(p, q, x, u, v)
        assert e.value.code == 1
    assert s.verify_probs(p[:0], q[:0], x[:0], u[:0], v[:0])[0].shape == (0, K + 1)


@pytest.mark.parametrize("groups,last", [(32, 31), (40, 32)])
def test_draw_where_sums_of_two_orders_straddle_the_aim(s, groups, last):
    """Weights 1, 2^-53, 2^-53, 1 in the first, second, fourth and last of runs of
    1024 ids: their running total is 1 in one order of addition and 1 + 2^-52 in
    another, and half of the total is 1. Runs without a weight lie where the
    orders part; the draw takes a token with a weight all the same."""
    ids = [0, 1024, 3 * 1024, last * 1024]
    p = np.zeros((1, 2, groups * 1024), np.float32)
    p[0, 0, ids] = [1.0, 2.0 ** -53, 2.0 ** -53, 1.0]
    status = torch.full((1,), -1, dtype=torch.int32, device=device())
    tokens, accepted = s.verify_probs(
        dev(p), None, dev(np.zeros((1, 1), np.int32)), dev(np.zeros((1, 1), np.float32)),
        dev(np.array([0.5], np.float32)), draft_lens=dev(np.zeros(1, np.int32)), out_status=status)
    assert int(status[0]) == 0 and int(accepted[0]) == 0
    assert int(tokens[0, 0]) in ids[2:] and int(tokens[0, 1]) == -1
