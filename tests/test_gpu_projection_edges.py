"""Calls that the documentation of quantize_rows, int8_logits, sample_hidden and
verify_probs allows and that lie off the usual path: operands of unlike
alignment, several handles at once, sizes of one, probabilities below the
normal range, outputs that the caller keeps, C-level refusals."""
import ctypes

import numpy as np
import pytest

from tests.gpu_common import device, gpu_available, torch
from tests.test_gpu_int8 import check_logits, dev, operands
from tests.test_gpu_verify_probs import batch, check, drafts_from, stored

import token_sampling_row_amd as tsr

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=2048, max_vocab=1 << 18, max_k=32, seed=3) as h:
        yield h


@pytest.mark.parametrize("rows", [3, 30, 60, 90, 140, 400])
@pytest.mark.parametrize("xs,ws", [(0, 1), (1, 0), (4, 2), (2, 4), (3, 3), (64, 128), (128, 128)])
def test_operands_of_unlike_alignment(s, rows, xs, ws):
    """codes and weight each at a byte offset of their own, in rows of 1152 or
    1151 bytes (odd offsets with odd strides)."""
    vocab, width = 700, 901
    rng = np.random.default_rng([rows, xs, ws])
    c, cs, w, wsc, b = operands(rng, rows, vocab, width)

    def inside(a, off):
        stride = 1151 if off % 2 else 1152
        big = torch.from_numpy(rng.integers(-128, 128, (a.shape[0], stride)).astype(np.int8))
        big[:, off:off + width] = torch.from_numpy(a)
        return big.to(device())[:, off:off + width]

    got = s.int8_logits(inside(c, xs), dev(cs), inside(w, ws), dev(wsc), bias=dev(b),
                        dtype=torch.float32)
    check_logits(got, "f32", c, cs, w, wsc, b)


@pytest.mark.parametrize("rows", [1, 17, 33, 65, 300])
@pytest.mark.parametrize("width", [127, 128, 129, 255, 256, 257, 383, 384, 512, 640, 768, 1024,
                                   1279])
def test_widths_about_the_stages(s, rows, width):
    """Every number of whole stages below a turn of the ring and above, with and
    without a partial one; rows a multiple of 128 bytes apart and not."""
    rng = np.random.default_rng([rows, width])
    c, cs, w, ws, _ = operands(rng, rows, 200, width)
    want = None
    for pad in (0, -width % 128, 4 - width % 4):
        cc = torch.zeros(rows, width + pad, dtype=torch.int8, device=device())
        ww = torch.zeros(200, width + pad, dtype=torch.int8, device=device())
        cc[:, :width], ww[:, :width] = dev(c), dev(w)
        got = s.int8_logits(cc[:, :width], dev(cs), ww[:, :width], dev(ws), dtype=torch.float32)
        if want is None:
            check_logits(got, "f32", c, cs, w, ws)
            want = got
        assert torch.equal(got, want)      # whole sums: the same bits by every path


def test_one_of_everything(s):
    one = torch.ones(1, 1, device=device())
    q, scale = s.quantize_rows(one)
    assert q.item() == 127
    y = s.int8_logits(q, scale, q, scale, dtype=torch.float32)
    assert abs(y.item() - 1.0) <= 4 * 2.0 ** -24
    assert s.sample_hidden(one, q, scale, {"temperature": 1.0}, 0).item() == 0
    p = torch.ones(1, 2, 1, device=device())
    x = torch.zeros(1, 1, dtype=torch.int32, device=device())
    half = torch.full((1, 1), 0.5, device=device())
    t, a = s.verify_probs(p, p[:, :1], x, half, half[0])
    assert t.tolist() == [[0, 0]] and a.tolist() == [1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [70, 50000])
def test_probabilities_below_the_normal_range(s, dtype, V):
    """Rows of subnormal weights (2^-133 and its multiples in bfloat16 as well)."""
    rows, K = 3, 2
    rng = np.random.default_rng(V)
    p = rng.integers(0, 5, (rows, K + 1, V)) * 2.0 ** -133
    q = rng.integers(1, 4, (rows, K, V)) * 2.0 ** -133
    (pt, p), (qt, q) = stored(p, dtype), stored(q, dtype)
    assert p.max() == 4 * 2.0 ** -133
    x = rng.integers(0, V, (rows, K)).astype(np.int32)
    u = rng.random((rows, K), dtype=np.float32)
    v = rng.random(rows, dtype=np.float32)
    check(s.verify_probs(pt, qt, dev(x), dev(u), dev(v)), p, q, x, None, u, v)


def test_negative_zero_is_a_probability(s):
    V = 600
    p = np.zeros((1, 2, V))
    p[0, :, 5], p[0, :, 500] = 0.25, 0.75
    pt, p = stored(p, "f32")
    pt[0, 0, 100:200] = -0.0
    x = np.array([[7]], dtype=np.int32)
    u, v = np.array([[0.0]], dtype=np.float32), np.array([0.3], dtype=np.float32)
    st = torch.full((1,), -7, dtype=torch.int32, device=device())
    check(s.verify_probs(pt, None, dev(x), dev(u), dev(v), out_status=st), p, None, x, None, u, v,
          st)


def test_handles_work_at_the_same_time(s):
    """Two handles on two streams: each has verify workspace of its own."""
    rng = np.random.default_rng(4)
    rows, K, V = 40, 3, 90001
    p, q = batch(rng, rows, K, V)
    (pt, p), (qt, q) = stored(p, "f32"), stored(q, "f32")
    x = drafts_from(rng, q)
    sets = [(rng.random((rows, K), dtype=np.float32), rng.random(rows, dtype=np.float32))
            for _ in range(2)]
    dsets = [(dev(u), dev(v)) for u, v in sets]
    dx = dev(x)
    torch.cuda.synchronize()
    with tsr.Sampler(0, max_rows=64, max_vocab=1 << 18, max_k=4) as other:
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        got = [None, None]
        for _ in range(5):
            for k, h in enumerate((s, other)):
                got[k] = h.verify_probs(pt, qt, dx, *dsets[k], stream=streams[k])
        torch.cuda.synchronize()
        for k in range(2):
            check(got[k], p, q, x, None, *sets[k])


def test_outputs_of_the_callers(s):
    """Preallocated outputs are the ones returned; rows of a larger buffer behind
    the batch stay as they were."""
    rng = np.random.default_rng(6)
    rows, K, V = 5, 2, 1000
    p, q = batch(rng, rows, K, V)
    (pt, p), (qt, q) = stored(p, "bf16"), stored(q, "bf16")
    x = drafts_from(rng, q)
    u, v = rng.random((rows, K), dtype=np.float32), rng.random(rows, dtype=np.float32)
    tokens = torch.full((rows + 3, K + 1), -9, dtype=torch.int32, device=device())
    counts = torch.full((rows + 3,), -9, dtype=torch.int32, device=device())
    got = s.verify_probs(pt, qt, dev(x), dev(u), dev(v), out_tokens=tokens[:rows],
                         out_accepted=counts[:rows])
    assert got[0].data_ptr() == tokens.data_ptr() and got[1].data_ptr() == counts.data_ptr()
    check(got, p, q, x, None, u, v)
    assert bool((tokens[rows:] == -9).all()) and bool((counts[rows:] == -9).all())
    for n in (5, 70, 260):
        c, cs, w, ws, _ = operands(rng, n, 300, 200)
        out = torch.full((n + 40, 300), 3.0, device=device())
        got = s.int8_logits(dev(c), dev(cs), dev(w), dev(ws), out=out[:n])
        check_logits(got, "f32", c, cs, w, ws)
        assert bool((out[n:] == 3).all())


def test_new_codes_lie_in_whole_lines(s):
    q, _ = s.quantize_rows(torch.randn(6, 1003, device=device()))
    assert q.shape == (6, 1003) and q.stride() == (1024, 1) and q.data_ptr() % 128 == 0


def test_refusals_through_the_c_interface(s):
    """Each class of invalid argument returns its code and leaves the outputs."""
    lib, h = tsr.load_library(), s._h
    d = device()
    f = torch.zeros(4, 64, device=d)
    b = torch.zeros(4, 64, dtype=torch.int8, device=d)
    sc = torch.ones(64, device=d)
    out = torch.full((4, 64), -7.0, device=d)
    tok = torch.full((64,), -7, dtype=torch.int32, device=d)

    def vp(t, off=0):
        return t.data_ptr() + off

    def quant(x=vp(f), dt=0, rows=4, width=64, stride=64, q=vp(b), qs=64, scale=vp(sc)):
        return lib.quantize_rows(h, x, dt, rows, width, stride, q, qs, scale, None)

    assert quant(rows=0) == 0
    for bad in (dict(x=None), dict(dt=2), dict(rows=-1), dict(width=0), dict(stride=63),
                dict(q=None), dict(qs=63), dict(scale=None), dict(x=vp(f, 2)),
                dict(scale=vp(sc, 2))):
        assert quant(**bad) == 1, bad
    assert quant(rows=1 << 24) == 4
    assert quant(width=(1 << 30) + 1, stride=1 << 31, qs=1 << 31) == 4

    def logits(c=vp(b), cst=64, cs=vp(sc), rows=4, w=vp(b), wst=64, ws=vp(sc), bias=None, vocab=4,
               width=64, o=vp(out), dt=0, ost=64, head=True):
        hd = tsr._Head(w, wst, ws, bias, vocab, width)
        return lib.int8_logits(h, c, cst, cs, rows, ctypes.byref(hd) if head else None, o, dt, ost,
                               None)

    assert logits(rows=0) == 0
    for bad in (dict(c=None), dict(cst=63), dict(cs=None), dict(cs=vp(sc, 1)), dict(rows=-1),
                dict(rows=2049), dict(w=None), dict(wst=63), dict(ws=None), dict(ws=vp(sc, 2)),
                dict(bias=vp(sc, 2)), dict(vocab=0), dict(vocab=(1 << 18) + 1, ost=1 << 19),
                dict(width=0), dict(o=None), dict(dt=2), dict(ost=3), dict(o=vp(out, 2)),
                dict(head=False)):
        assert logits(**bad) == 1, bad
    for bad in (dict(width=131072, cst=131072, wst=131072), dict(cst=1 << 22), dict(wst=1 << 22)):
        assert logits(**bad) == 4, bad

    # more channels than a launch takes, on a handle that allows them
    with tsr.Sampler(0, max_rows=1, max_vocab=1 << 30, max_k=1, seed=0) as big:
        n = (1 << 29) + 1
        hd = tsr._Head(vp(b), 64, vp(sc), None, n, 64)
        assert lib.int8_logits(big._h, vp(b), 64, vp(sc), 1, ctypes.byref(hd), vp(out), 0, n,
                               None) == 4

    prm = tsr._Params(1.0, 0, 1.0, 0.0, 0)

    def hidden(x=vp(f), dt=0, rows=4, stride=64, q=vp(b), qs=64, scale=vp(sc), lg=vp(out),
               params=prm, o=vp(tok), vocab=4):
        hd = tsr._Head(vp(b), 64, vp(sc), None, vocab, 64)
        return lib.sample_hidden(h, x, 0, rows, stride, ctypes.byref(hd), q, qs, scale, lg, dt,
                                 ctypes.byref(params) if params else None, 0, o, None, None)

    assert hidden(rows=0) == 0
    for bad in (dict(x=None), dict(stride=63), dict(q=None), dict(qs=63), dict(scale=None),
                dict(lg=None), dict(o=None), dict(params=None), dict(rows=2049), dict(dt=3),
                dict(params=tsr._Params(-1.0, 0, 1.0, 0.0, 0))):
        assert hidden(**bad) == 1, bad

    u = torch.zeros(64, device=d)

    def verify(t=vp(f), ts=2, tr=1, q=vp(f), qs=2, qr=1, dt=0, x=vp(tok), ln=None, au=vp(u),
               du=vp(u), rows=4, K=2, V=4, ot=vp(tok), oa=vp(tok), st=None):
        return lib.verify_probs(h, t, ts, tr, q, qs, qr, dt, x, ln, au, du, rows, K, V, ot, oa, st,
                                None)

    assert verify(rows=0) == 0
    for bad in (dict(t=None), dict(ts=-1), dict(tr=-1), dict(qs=-1), dict(qr=-1), dict(dt=2),
                dict(x=None), dict(au=None), dict(du=None), dict(rows=-1), dict(rows=2049),
                dict(K=0), dict(K=33), dict(V=0), dict(V=(1 << 18) + 1), dict(ot=None),
                dict(oa=None), dict(t=vp(f, 2)), dict(q=vp(f, 1)), dict(x=vp(tok, 2)),
                dict(ln=vp(tok, 1)), dict(au=vp(u, 2)), dict(du=vp(u, 3)), dict(ot=vp(tok, 1)),
                dict(oa=vp(tok, 2)), dict(st=vp(tok, 2))):
        assert verify(**bad) == 1, bad
    torch.cuda.synchronize()
    assert bool((out == -7).all()) and bool((tok == -7).all()) and not b.any()


def large_batch(s, dtype, rows, vocab, width, stride):
    """Logits of a batch that fills the card, held to the bound around float64
    products of whole numbers below 2^53."""
    from oracle import int8 as oi
    g = torch.Generator(device()).manual_seed(rows)

    def matrix(n):
        m = torch.randint(-128, 128, (n, stride), dtype=torch.int8, device=device(), generator=g)
        return m[:, :width]

    c, w = matrix(rows), matrix(vocab)
    cs = torch.rand(rows, device=device(), generator=g)
    ws = torch.rand(vocab, device=device(), generator=g)
    b = torch.randn(vocab, device=device(), generator=g) * 1000
    got = s.int8_logits(c, cs, w, ws, bias=b,
                        dtype={"f32": torch.float32, "bf16": torch.bfloat16}[dtype]).double()
    product = (c.double() @ w.double().t()) * cs.double()[:, None] * ws.double()
    want = product + b.double()
    half = 2.0 ** -23 * product.abs() + 2.0 ** -24 * want.abs()
    if dtype == "bf16":
        half = half + 2.0 ** -8 * (want.abs() + half)
    assert bool(((got - want).abs() <= half * (1 + 2.0 ** -20)).all())
    # the same bound as the reference's
    some = want[:2, :50].cpu().numpy(), product[:2, :50].abs().cpu().numpy()
    assert np.allclose(oi.logits_bound(*some, dtype),
                       (half * (1 + 2.0 ** -20))[:2, :50].cpu().numpy(), atol=1e-40)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(512, 32000), (384, 32003), (256, 32000), (320, 32001),
                                        (128, 32000), (200, 8960), (500, 31999), (1024, 33000),
                                        (310, 32003), (190, 40003), (60, 33001)])
def test_every_tile_shape(s, dtype, rows, vocab):
    """Batches where each tile shape is the one taken, with rows in whole lines, at
    words and at bytes, and with a partial stage."""
    for width in (384, 300, 641):
        large_batch(s, dtype, rows, vocab, width, width)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,width,stride", [
    (1000, 131072, 500, 512), (192, 131071, 500, 512), (320, 131072, 512, 512),
    (128, 131073, 500, 512), (100, 40000, 1400, 1408), (700, 50001, 1100, 1152),
    (90, 14000, 4000, 4096), (64, 40000, 1408, 1408), (63, 32768, 1600, 1664), (30, 40001, 1400, 1408),
    (9, 13000, 4100, 4224), (3, 13000, 4096, 4096)])
def test_large_weights(s, dtype, rows, vocab, width, stride):
    """Weights that outgrow the caches, in rows of whole lines; batches in one
    launch and in two."""
    large_batch(s, dtype, rows, vocab, width, stride)


@pytest.mark.parametrize("rows", [320, 200])
@pytest.mark.parametrize("width", [500, 501])
def test_the_widest_rows(s, rows, width):
    """Hidden rows nearly 2^22 bytes apart, the last of them past 2^30 bytes."""
    stride = (1 << 22) - 128 if width % 4 == 0 else (1 << 22) - 1
    g = torch.Generator(device()).manual_seed(width)
    c = torch.zeros(rows * stride, dtype=torch.int8, device=device()).view(rows, stride)[:, :width]
    c.copy_(torch.randint(-128, 128, (rows, width), dtype=torch.int8, device=device(), generator=g))
    w = torch.randint(-128, 128, (32000, width), dtype=torch.int8, device=device(), generator=g)
    one = torch.ones(rows, device=device()), torch.ones(32000, device=device())
    got = s.int8_logits(c, one[0], w, one[1], dtype=torch.float32)
    assert torch.equal(got.double(), c.double() @ w.double().t())   # sums below 2^24


@pytest.mark.parametrize("rows,vocab", [(512, 32000), (384, 32000), (320, 32000), (256, 32000),
                                        (64, 33000)])
def test_stages_of_large_tiles(s, rows, vocab):
    """One whole stage to more than two turns of the rings, without and with a
    partial one behind."""
    for stages in range(1, 15):
        large_batch(s, "bf16", rows, vocab, 128 * stages, 128 * stages)
        large_batch(s, "bf16", rows, vocab, 128 * stages + 60, 128 * stages + 64)


@pytest.mark.parametrize("rows", [1, 5, 70])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_empty_residual_of_many_ids(s, rows, dtype):
    """q = 2 p over rows that several workgroups sum: the draw is from p."""
    K, V = 2, 70001
    rng = np.random.default_rng(rows)
    p, _ = batch(rng, rows, K, V)
    pt, p = stored(p, dtype)
    qt, q = pt[:, :K] * 2, p[:, :K] * 2
    x = drafts_from(rng, q)
    u = np.full((rows, K), 0.75, dtype=np.float32)
    v = rng.random(rows, dtype=np.float32)
    got = s.verify_probs(pt, qt, dev(x), dev(u), dev(v))
    assert bool((got[1] == 0).all())
    check(got, p, q, x, None, u, v)
