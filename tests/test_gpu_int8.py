"""quantize_rows, int8_logits and sample_hidden against the plain references in
64 bits (oracle/int8.py, whose logits_bound derives the tolerance)."""
import numpy as np
import pytest

from tests.gpu_common import device, gpu_available, to_dev, torch

import token_sampling_row_amd as tsr
from oracle import int8 as oi
from token_sampling_row_amd import workloads as wl

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=2048, max_vocab=1 << 18, max_k=8, seed=3) as h:
        yield h


def stored(x, dtype):
    """float64 values -> (device tensor, its float32 values)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    if dtype == "f32":
        return to_dev(x, "f32"), x
    bits = wl.f32_to_bf16_bits(x)
    return to_dev(bits, "bf16"), wl.bf16_bits_to_f32(bits)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device())


def check_codes(got, x):
    codes, scale = got[0].cpu().numpy(), got[1].cpu().numpy()
    want, want_s = oi.quantize_rows(x)
    assert np.array_equal(scale.view(np.uint32) | (np.isnan(scale) * np.uint32(0xFFFFFFFF)),
                          want_s.view(np.uint32) | (np.isnan(want_s) * np.uint32(0xFFFFFFFF)))
    assert np.array_equal(codes, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 2), (1, 7), (5, 8), (2, 63), (7, 255),
                                        (4, 1003), (33, 2048), (1, 4096), (3, 4097), (2, 8191),
                                        (1500, 300), (1027, 4099), (2, 16384), (3, 16391),
                                        (1, 40000)])
def test_codes_match(s, dtype, rows, width):
    rng = np.random.default_rng([rows, width])
    x, v = stored(rng.normal(0, 1, (rows, width)) * np.exp(rng.normal(0, 2, (rows, 1))), dtype)
    check_codes(s.quantize_rows(x), v)


@pytest.mark.parametrize("dtype,epc", [("f32", 4), ("bf16", 8)])
@pytest.mark.parametrize("rows", [4095, 4097])
@pytest.mark.parametrize("chunks", [1, 64, 65, 128, 129, 192, 193, 256, 257, 384, 385, 512])
def test_codes_of_many_rows(s, dtype, epc, rows, chunks):
    """Rows of one, two and four wavefronts, on either side of each limit; a row
    number that does not fill the last workgroup; a partial chunk behind."""
    width = chunks * epc + chunks % 3 % epc
    g = torch.Generator(device()).manual_seed(chunks)
    x = torch.randn(rows, width, device=device(), generator=g)
    x = (x * torch.exp(torch.randn(rows, 1, device=device(), generator=g)))
    x[7, width - 1], x[rows - 1, 0], x[rows - 2] = float("nan"), 1e30, 0.0
    x = x.to({"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    codes, scale = s.quantize_rows(x)
    some = [0, 1, 7, rows // 2, rows - 3, rows - 2, rows - 1]
    check_codes((codes[some], scale[some]), x[some].float().cpu().numpy())
    for r0 in range(0, rows, 1000):   # the same rows, fewer at a time
        c, sc = s.quantize_rows(x[r0:r0 + 1000])
        assert torch.equal(c, codes[r0:r0 + 1000])
        assert torch.equal(sc.view(torch.int32), scale[r0:r0 + 1000].view(torch.int32))


@pytest.mark.parametrize("dtype,rows,width", [("bf16", 100001, 1007), ("bf16", 63001, 1601),
                                              ("bf16", 24581, 4097), ("f32", 9001, 5603),
                                              ("f32", 6301, 8000), ("f32", 66003, 763),
                                              ("f32", 36003, 1400)])
def test_codes_of_large_inputs(s, dtype, rows, width):
    """Inputs that outgrow the caches, against the same rows in small batches."""
    td = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x = torch.empty(rows, width, dtype=td, device=device()).normal_(
        generator=torch.Generator(device()).manual_seed(rows))
    codes, scale = s.quantize_rows(x)
    check_codes((codes[-3:], scale[-3:]), x[-3:].float().cpu().numpy())
    for r0 in range(0, rows, 4000):
        c, sc = s.quantize_rows(x[r0:r0 + 4000])
        assert torch.equal(c, codes[r0:r0 + 4000]) and torch.equal(sc, scale[r0:r0 + 4000])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_of_special_rows(s, dtype):
    """Zeros, negative zeros, halves, one value, NaN, infinities at either end,
    rows whose scale is below the smallest normal number or below any."""
    W = 515
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (12, W))
    x[0] = 0.0
    x[1] = -0.0
    x[2] = (rng.integers(-254, 255, W)) / 2.0
    x[2, 7] = 127.0                                   # scale 1: every odd entry is a half
    x[3] = 3.25
    x[4, 0] = np.nan
    x[5, W - 1] = np.inf
    x[6, 100] = -np.inf
    x[7] *= 1e-37
    x[8] *= 1e-39
    x[9] = 0.0
    x[9, 3] = 1e-45                                   # scale 0, though the row is not
    x[10] *= 3e37
    x[11] = -np.abs(x[11])
    t, v = stored(x, dtype)
    check_codes(s.quantize_rows(t), v)


def test_many_rows_beyond_the_handles(s):
    """A weight's rows are not bound by max_rows."""
    rng = np.random.default_rng(6)
    t, v = stored(rng.normal(0, 1, (5000, 70)), "bf16")
    check_codes(s.quantize_rows(t), v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_codes_of_strided_rows(s, dtype, off):
    """Rows inside a wider tensor, at odd element and byte offsets; the bytes
    between the output's rows stay as they were."""
    rng = np.random.default_rng(off)
    t, v = stored(rng.normal(0, 1, (9, 1100)), dtype)
    out = torch.full((9, 1111), 77, dtype=torch.int8, device=device())
    got = s.quantize_rows(t[:, off:off + 1001], out=out[:, off:off + 1001])
    check_codes(got, v[:, off:off + 1001])
    assert bool((out[:, :off] == 77).all()) and bool((out[:, off + 1001:] == 77).all())


def operands(rng, rows, vocab, width, extreme=False):
    if extreme:
        c = rng.choice(np.array([-128, 127], dtype=np.int8), (rows, width))
        w = rng.choice(np.array([-128, 127], dtype=np.int8), (vocab, width))
        c[0] = -128
        w[0] = -128
    else:
        c = rng.integers(-128, 128, (rows, width)).astype(np.int8)
        w = rng.integers(-128, 128, (vocab, width)).astype(np.int8)
    cs = np.exp(rng.normal(-4, 1, rows)).astype(np.float32)
    ws = np.exp(rng.normal(-4, 1, vocab)).astype(np.float32)
    b = rng.normal(0, 30, vocab).astype(np.float32)
    return c, cs, w, ws, b


def check_logits(got, dtype, c, cs, w, ws, b=None):
    want, product = oi.int8_logits(c, cs, w, ws, b)
    g = got.double().cpu().numpy()
    assert (np.abs(g - want) <= oi.logits_bound(want, product, dtype)).all(), \
        np.abs(g - want).max()


TD = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype,bias", [("f32", True), ("bf16", False)])
@pytest.mark.parametrize("rows,vocab,width", [
    (1, 1, 1), (1, 15, 15), (2, 64, 16), (1, 65, 17), (16, 63, 63), (17, 100, 64), (3, 1000, 65),
    (5, 8191, 1003), (31, 515, 127), (33, 300, 128), (48, 257, 129), (64, 512, 4096),
    (65, 130, 192), (100, 999, 1000), (127, 257, 320), (128, 256, 384), (129, 255, 512),
    (256, 512, 1024), (257, 513, 1029), (320, 700, 2048), (511, 300, 260), (1000, 1001, 640),
    (1, 32000, 512), (4, 32003, 1024), (1500, 260, 256)])
def test_logits_match(s, dtype, bias, rows, vocab, width):
    rng = np.random.default_rng([rows, vocab, width])
    c, cs, w, ws, b = operands(rng, rows, vocab, width)
    b = b if bias else None
    got = s.int8_logits(dev(c), dev(cs), dev(w), dev(ws), bias=None if b is None else dev(b),
                        dtype=TD[dtype])
    check_logits(got, dtype, c, cs, w, ws, b)


@pytest.mark.parametrize("rows,vocab,width", [(3, 70, 131071), (80, 130, 131071),
                                              (300, 300, 131071)])
def test_sums_near_the_edge_of_32_bits(s, rows, vocab, width):
    """The widest rows with codes of -128 and 127: the largest sum is 131071 * 2^14."""
    rng = np.random.default_rng(rows)
    c, cs, w, ws, _ = operands(rng, rows, vocab, width, extreme=True)
    got = s.int8_logits(dev(c), dev(cs), dev(w), dev(ws), dtype=torch.float32)
    check_logits(got, "f32", c, cs, w, ws)


@pytest.mark.parametrize("rows", [1, 5, 40, 70, 130, 300])
@pytest.mark.parametrize("off", [0, 1, 2, 13])
def test_strided_and_unaligned_operands(s, rows, off):
    """Every operand inside a wider tensor at an odd byte offset; what lies
    between the output's rows stays as it was."""
    vocab, width = 515, 643
    rng = np.random.default_rng([rows, off])
    c, cs, w, ws, b = operands(rng, rows, vocab, width)
    big_c = rng.integers(-128, 128, (rows, width + 29)).astype(np.int8)
    big_w = rng.integers(-128, 128, (vocab, width + 31)).astype(np.int8)
    big_c[:, off:off + width], big_w[:, off:off + width] = c, w
    for dtype in ("f32", "bf16"):
        out = torch.full((rows, vocab + 17), 5.0, dtype=TD[dtype], device=device())
        got = s.int8_logits(dev(big_c)[:, off:off + width], dev(cs),
                            dev(big_w)[:, off:off + width], dev(ws), bias=dev(b),
                            out=out[:, off:off + vocab])
        check_logits(got, dtype, c, cs, w, ws, b)
        assert bool((out[:, :off] == 5).all()) and bool((out[:, off + vocab:] == 5).all())


@pytest.mark.parametrize("rows", [2, 20, 200, 600])
def test_scales_of_nan_zero_and_infinity_stay_in_their_rows(s, rows):
    rng = np.random.default_rng(rows)
    c, cs, w, ws, _ = operands(rng, rows, 300, 256)
    cs[1], ws[7], ws[9] = np.nan, 0.0, np.inf
    got = s.int8_logits(dev(c), dev(cs), dev(w), dev(ws), dtype=torch.float32).cpu().numpy()
    assert np.isnan(got[1]).all()
    rest = np.delete(got, 1, 0)
    assert (rest[:, 7] == 0).all() and not np.isfinite(rest[:, 9]).any()
    keep = [i for i in range(300) if i not in (7, 9)]
    check_logits(torch.from_numpy(np.ascontiguousarray(rest[:, keep])), "f32", np.delete(c, 1, 0),
                 np.delete(cs, 1), w[keep], ws[keep])


def test_a_weight_beyond_32_bit_offsets(s):
    """Rows of a weight whose bytes pass 2^32: 151936 channels 28672 apart."""
    vocab, stride, width = 151936, 28672, 512
    big = torch.zeros(vocab, stride, dtype=torch.int8, device=device())
    rng = np.random.default_rng(1)
    for rows in (2, 70, 200):
        c, cs, w, ws, _ = operands(rng, rows, 64, width)
        scale = torch.ones(vocab, device=device())
        big[-64:, -width:] = dev(w)
        scale[-64:] = dev(ws)
        got = s.int8_logits(dev(c), dev(cs), big[:, -width:], scale, dtype=torch.float32)
        check_logits(got[:, -64:], "f32", c, cs, w, ws)
        assert bool((got[:, :-64] == 0).all())


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_captured_calls_replay(s, rows):
    """quantize_rows and int8_logits in a graph on another stream, replayed on new
    inputs with eager work between the replays."""
    rng = np.random.default_rng(rows)
    vocab, width = 1000, 512
    _, _, w, ws, b = operands(rng, rows, vocab, width)
    w, ws, b = dev(w), dev(ws), dev(b)
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device=device())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.int8_logits(*s.quantize_rows(x), w, ws, bias=b)
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = s.int8_logits(*s.quantize_rows(x), w, ws, bias=b)
    for k in range(4):
        x.copy_(torch.from_numpy(rng.normal(0, 1 + k, (rows, width)).astype(np.float32)))
        g.replay()
        eager = s.int8_logits(*s.quantize_rows(x), w, ws, bias=b)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_results_do_not_change_between_calls_or_streams(s):
    rng = np.random.default_rng(9)
    c, cs, w, ws, _ = (dev(a) for a in operands(rng, 320, 5000, 1000))
    first = s.int8_logits(c, cs, w, ws)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(3):
        a = s.int8_logits(c, cs, w, ws, stream=st)
        b = s.int8_logits(c, cs, w, ws)
        torch.cuda.synchronize()
        assert torch.equal(a, first) and torch.equal(b, first)


@pytest.mark.parametrize("rows", [1, 9, 130])
def test_hidden_states_to_tokens(s, rows):
    """sample_hidden equals its three steps, and its tokens the sampler's on the
    logits it hands out; a row of NaN is reported as such."""
    rng = np.random.default_rng(rows)
    vocab, width = 8191, 500
    weight, _ = stored(rng.normal(0, 0.05, (vocab, width)), "bf16")
    w, ws = s.quantize_rows(weight)
    hidden, _ = stored(rng.normal(0, 1, (rows, width)), "bf16")
    if rows > 1:
        hidden[3, 17] = float("nan")
    for prm in ({"temperature": 0.0}, {"temperature": 0.9, "top_k": 50, "top_p": 0.95}):
        logits = torch.empty(rows, vocab, dtype=torch.float32, device=device())
        status = torch.full((rows,), -7, dtype=torch.int32, device=device())
        got = s.sample_hidden(hidden, w, ws, prm, 11, logits=logits, diag={"status": status})
        codes, scale = s.quantize_rows(hidden)
        by_hand = s.int8_logits(codes, scale, w, ws, dtype=torch.float32)
        assert torch.equal(logits.nan_to_num(7.0), by_hand.nan_to_num(7.0))
        assert torch.equal(got, s.sample_rows(by_hand, prm, 11))
        if rows > 1:
            assert int(got[3]) == -1 and int(status[3]) == tsr.ROW_NONFINITE
            assert bool((status[torch.arange(rows) != 3] == 0).all())


def test_refusals(s):
    d = device()
    c = torch.zeros(4, 64, dtype=torch.int8, device=d)
    cs, ws = torch.ones(4, device=d), torch.ones(32, device=d)
    w = torch.zeros(32, 64, dtype=torch.int8, device=d)
    h = torch.zeros(4, 64, device=d)
    for bad in (h.half(), h.double()):
        with pytest.raises(TypeError):
            s.quantize_rows(bad)
    for call in (
            lambda: s.quantize_rows(h.t()),
            lambda: s.quantize_rows(h[:1].expand(4, 64)),
            lambda: s.quantize_rows(h.cpu()),
            lambda: s.quantize_rows(h, out=c[:3], scale=cs),
            lambda: s.quantize_rows(h, out=c.to(torch.uint8), scale=cs),
            lambda: s.quantize_rows(h, out=c, scale=cs[:3]),
            lambda: s.int8_logits(c, cs[:3], w, ws),
            lambda: s.int8_logits(c[:, :63], cs, w, ws),
            lambda: s.int8_logits(c[0], cs, w, ws),
            lambda: s.int8_logits(c[0, 0], cs, w, ws),
            lambda: s.int8_logits(c, cs, w.t(), ws),
            lambda: s.int8_logits(c, cs, w, ws[:31]),
            lambda: s.int8_logits(c, cs, w, ws.double()),
            lambda: s.int8_logits(c, cs, w, ws, bias=ws[:31]),
            lambda: s.int8_logits(c, cs, w.cpu(), ws),
            lambda: s.int8_logits(c, cs, w, ws, out=torch.zeros(4, 31, device=d)),
            lambda: s.int8_logits(c, cs, w, ws, out=torch.zeros(1, 32, device=d).expand(4, 32)),
            lambda: s.sample_hidden(h[:, :63], w, ws, {}, 0),
            lambda: s.sample_hidden(h, w, ws, {}, 0,
                                    out=torch.zeros(3, dtype=torch.int32, device=d)),
            lambda: s.sample_hidden(h, w, ws, {}, 0, logits=torch.zeros(4, 40, device=d)[:, :32])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: s.int8_logits(c, cs, w, ws, dtype=torch.float16),
                 lambda: s.int8_logits(c, cs, w, ws, out=torch.zeros(4, 32, device=d).half())):
        with pytest.raises(TypeError):
            call()
    wide = torch.zeros(2, 131072, dtype=torch.int8, device=d)
    with pytest.raises(tsr.TsrError) as e:
        s.int8_logits(wide, cs[:2], wide, ws[:2])
    assert e.value.code == 4
    many = torch.zeros(2049, 64, dtype=torch.int8, device=d)
    with pytest.raises(tsr.TsrError) as e:
        s.int8_logits(many, torch.ones(2049, device=d), w, ws)
    assert e.value.code == 1
    with pytest.raises(tsr.TsrError) as e:
        s.sample_hidden(h, w, ws, {"temperature": -1.0}, 0)
    assert e.value.code == 1
    # no rows: nothing to do
    assert s.int8_logits(c[:0], cs[:0], w, ws).shape == (0, 32)
    assert s.quantize_rows(h[:0])[0].shape == (0, 64)
