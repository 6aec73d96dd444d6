"""Refusals of the calls around the logits, without a GPU: the C ABI's (a handle that only
holds its limits; every call here is refused before the device is looked at, and one that
is not ends in TSR_EDEVICE) and the binding's."""
import ctypes
import types

import pytest

import token_sampling_row_amd as tsr
from tests.test_abi import lib  # noqa: F401

torch = pytest.importorskip("torch")

EINVAL, EUNSUPPORTED = 1, 4


@pytest.fixture(scope="module")
def handle():
    """device, max_rows, max_vocab, max_k, seed, and nothing behind them."""
    block = (ctypes.c_char * 512)()
    ctypes.memmove(block, (ctypes.c_int32 * 4)(0, 16, 1000, 4), 16)
    yield ctypes.addressof(block)
    del block


@pytest.fixture(scope="module")
def mem():
    block = ctypes.create_string_buffer(1 << 16)
    yield (ctypes.addressof(block) + 255) // 256 * 256
    del block


def refused(call, base, changes):
    """Each change of the arguments gives its code."""
    for change, code in changes:
        args = dict(base, **change)
        assert call(**args) == code, change


def test_norm_quantize_rows(lib, handle, mem):  # noqa: F811
    def call(h, x, xs, r, rs, dt, w, wdt, eps, rows, width, oh, hs, q, qs, sc):
        return lib.norm_quantize_rows(h, x, xs, r, rs, dt, w, wdt, eps, rows, width, oh, hs, q, qs,
                                      sc, None)

    base = dict(h=handle, x=mem, xs=64, r=mem + 4096, rs=64, dt=0, w=mem + 8192, wdt=0, eps=1e-6,
                rows=4, width=64, oh=mem + 12288, hs=64, q=mem + 16384, qs=64, sc=mem + 20480)
    assert call(**dict(base, rows=0)) == 0
    bad = [dict(h=None), dict(x=None), dict(q=None), dict(sc=None), dict(dt=2), dict(wdt=2),
           dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(rows=-1),
           dict(width=0), dict(xs=63), dict(rs=63), dict(hs=63), dict(qs=63), dict(x=mem + 2),
           dict(r=mem + 4098), dict(w=mem + 8193), dict(w=mem + 8193, wdt=1), dict(oh=mem + 12290),
           dict(sc=mem + 20482), dict(r=None),              # a sum to keep without a residual
           dict(oh=mem + 4), dict(oh=mem + 4096 - 256), dict(oh=mem, hs=65),   # shifted over inputs
           dict(oh=mem + 8192), dict(oh=mem + 20480), dict(q=mem), dict(q=mem + 4096),
           dict(q=mem + 8192 + 255), dict(q=mem + 12288), dict(q=mem + 20480), dict(sc=mem),
           dict(sc=mem + 4096), dict(sc=mem + 8192)]
    refused(call, base, [(c, EINVAL) for c in bad])
    refused(call, base, [(dict(rows=1 << 24), EUNSUPPORTED),
                         (dict(width=(1 << 30) + 1, xs=1 << 31, rs=1 << 31, hs=1 << 31, qs=1 << 31),
                          EUNSUPPORTED), (dict(xs=1 << 36), EUNSUPPORTED),
                         (dict(rs=1 << 36), EUNSUPPORTED), (dict(hs=1 << 36), EUNSUPPORTED),
                         (dict(qs=1 << 36), EUNSUPPORTED)])


def test_rows_between_each_others(lib, handle, mem):  # noqa: F811
    """Columns of one larger matrix do not overlap: such calls come as far as the device,
    which is not there (TSR_EDEVICE), or is (TSR_OK would run them: only without one)."""
    if torch.cuda.is_available():
        pytest.skip("would run on host memory")

    def norm(x, xs, r, rs, oh, hs, q, qs, rows=4, width=16, sc=mem + 20480):
        return lib.norm_quantize_rows(handle, x, xs, r, rs, 0, None, 0, 1e-6, rows, width, oh, hs, q,
                                      qs, sc, None)

    at, W = mem, 16
    # x | residual | sum | codes in rows of 64 floats, the codes in the last quarter
    assert norm(at, 64, at + 64, 64, at + 128, 64, at + 192, 256) == 3
    assert norm(at + 192, 64, at + 128, 64, at + 64, 64, at, 256) == 3
    # the last row's columns wrap into the next row's: still apart
    assert norm(at + 64, 64, at + 128, 64, at + 192, 64, at + 256, 256) == 3
    for bad in (at + 4, at + 60, at + 128 + 64 - 4):   # a column too many
        assert norm(at, 64, at + 128, 64, bad, 64, at + 8192, 64) == 1
    assert norm(at, 64, at + 128, 64, at + 64, 48, at + 8192, 64) == 1   # other strides
    # a single row in a gap, and one that is no gap
    assert norm(at, 64, None, 0, None, 0, at + 64, 64, rows=1, width=W) == 3
    assert norm(at, 64, None, 0, None, 0, at + 63, 64, rows=1, width=W) == 1

    def grad(z_at, out, zs=64, os=64):
        return lib.token_logprobs_grad(handle, z_at, 0, 4, 16, zs, 1.0, None, 0, mem + 9000 // 4 * 4,
                                       None, None, None, out, os, None)

    assert grad(at, at + 64) == 3 and grad(at + 64, at) == 3 and grad(at, at + 192) == 3
    assert grad(at, at + 60) == 1 and grad(at, at + 196) == 1 and grad(at, at) == 1
    assert grad(at, at + 64, 64, 32) == 1


def test_token_logprobs(lib, handle, mem):  # noqa: F811
    def call(h, z, dt, rows, V, stride, T, tok, n, k, out, ws=None, size=0):
        o = None if out is None else ctypes.byref(tsr._Logprobs(*out))
        return lib.token_logprobs(h, z, dt, rows, V, stride, T, tok, n, k, o, ws, size, None)

    good = (mem + 8192, mem + 8448, mem + 8704, mem + 8960, mem + 9216, mem + 9472)
    base = dict(h=handle, z=mem, dt=0, rows=4, V=64, stride=64, T=1.0, tok=mem + 4096, n=2, k=3,
                out=good)
    assert call(**dict(base, rows=0)) == 0

    def out(i, v):
        return dict(out=good[:i] + (v,) + good[i + 1:])

    bad = [dict(h=None), dict(z=None), dict(out=None), dict(dt=-1), dict(rows=-1), dict(V=0),
           dict(stride=63), dict(z=mem + 1), dict(z=mem + 2), dict(T=0.0), dict(T=-1.0),
           dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-31), dict(T=1e31), dict(tok=None), dict(n=-1),
           dict(k=-1), dict(tok=mem + 4098), out(0, None), out(2, None), out(3, None)]
    bad += [out(i, good[i] + 2) for i in range(6)]
    refused(call, base, [(c, EINVAL) for c in bad])
    refused(call, base, [(dict(n=1025), EUNSUPPORTED), (dict(k=65), EUNSUPPORTED),
                         (dict(rows=1 << 22), EUNSUPPORTED),
                         (dict(V=(1 << 30) + 1, stride=1 << 31), EUNSUPPORTED),
                         (dict(stride=1 << 36), EUNSUPPORTED)])


def test_token_logprobs_grad(lib, handle, mem):  # noqa: F811
    def call(h, z, dt, rows, V, stride, T, tok, n, norm, g, H, ge, out, os):
        return lib.token_logprobs_grad(h, z, dt, rows, V, stride, T, tok, n, norm, g, H, ge, out,
                                       os, None)

    base = dict(h=handle, z=mem, dt=1, rows=4, V=64, stride=64, T=1.0, tok=mem + 4096, n=2,
                norm=mem + 4352, g=mem + 4608, H=mem + 4864, ge=mem + 5120, out=mem + 8192, os=64)
    assert call(**dict(base, rows=0)) == 0
    bad = [dict(h=None), dict(z=None), dict(norm=None), dict(out=None), dict(tok=None),
           dict(g=None), dict(H=None), dict(n=-1), dict(os=63), dict(dt=3), dict(T=0.0),
           dict(out=mem + 8193), dict(out=mem), dict(out=mem + 64), dict(tok=mem + 4097),
           dict(norm=mem + 4353), dict(g=mem + 4609), dict(H=mem + 4865), dict(ge=mem + 5121)]
    refused(call, base, [(c, EINVAL) for c in bad])
    refused(call, base, [(dict(n=1025), EUNSUPPORTED), (dict(os=1 << 36), EUNSUPPORTED),
                         (dict(rows=1 << 22), EUNSUPPORTED)])


def test_distill_topk(lib, handle, mem):  # noqa: F811
    def call(h, z, dt, rows, V, stride, T, ids, lp, k, tail, w, loss, grad, gs, status, ws=None,
             size=0):
        return lib.distill_topk(h, z, dt, rows, V, stride, T, ids, lp, k, tail, w, loss, grad, gs,
                                status, ws, size, None)

    base = dict(h=handle, z=mem, dt=0, rows=4, V=64, stride=64, T=1.0, ids=mem + 4096,
                lp=mem + 4352, k=3, tail=1, w=mem + 4608, loss=mem + 4864, grad=mem + 8192, gs=64,
                status=mem + 5120)
    assert call(**dict(base, rows=0)) == 0
    bad = [dict(h=None), dict(z=None), dict(ids=None), dict(lp=None), dict(loss=None), dict(k=0),
           dict(k=-2), dict(tail=2), dict(tail=-1), dict(gs=63), dict(T=0.0), dict(grad=mem),
           dict(grad=mem + 512), dict(grad=mem + 8194), dict(ids=mem + 4097), dict(lp=mem + 4354),
           dict(w=mem + 4610), dict(loss=mem + 4866), dict(status=mem + 5122)]
    refused(call, base, [(c, EINVAL) for c in bad])
    refused(call, base, [(dict(k=65), EUNSUPPORTED), (dict(gs=1 << 36), EUNSUPPORTED),
                         (dict(stride=1 << 36), EUNSUPPORTED), (dict(rows=1 << 22), EUNSUPPORTED)])


def test_outputs_over_inputs_or_each_other(lib, handle, mem):  # noqa: F811
    """Every output over every input, by its last or first word, and over each other output;
    side by side they come as far as the device (only where there is none)."""
    R, V, n, k = 4, 64, 2, 3
    apart = 3 if not torch.cuda.is_available() else None

    def pairs(call, outs, ins):
        """outs, ins: name -> bytes. Each lies 4096 bytes from the next but for one pair."""
        at = {name: mem + 4096 * i for i, name in enumerate((*outs, *ins))}
        if apart is not None:
            assert call(at) == apart
        for o in outs:
            for other in (*outs, *ins):
                if other == o:
                    continue
                size = {**outs, **ins}[other]
                for where in (at[other], at[other] + size - 4, at[other] - outs[o] + 4):
                    if where >= mem:
                        assert call(dict(at, **{o: where})) == EINVAL, (o, other, where - at[other])
                if apart is not None and at[other] >= mem + 4096:
                    assert call(dict(at, **{o: at[other] + size})) == apart, (o, other)
                    assert call(dict(at, **{o: at[other] - outs[o]})) == apart, (o, other)

    def logprobs(p):
        o = tsr._Logprobs(p["lp"], p["H"], p["ids"], p["top"], p["norm"], p["status"])
        return lib.token_logprobs(handle, p["z"], 0, R, V, V, 1.0, p["tok"], n, k, ctypes.byref(o),
                                  None, 0, None)

    pairs(logprobs, dict(lp=4 * R * n, H=4 * R, ids=4 * R * k, top=4 * R * k, norm=8 * R,
                         status=4 * R), dict(z=4 * R * V, tok=4 * R * n))

    def grad(p):
        return lib.token_logprobs_grad(handle, p["z"], 0, R, V, V, 1.0, p["tok"], n, p["norm"],
                                       p["g"], p["H"], p["ge"], p["out"], V, None)

    pairs(grad, dict(out=4 * R * V), dict(z=4 * R * V, tok=4 * R * n, norm=8 * R, g=4 * R * n,
                                          H=4 * R, ge=4 * R))

    def distill(p):
        return lib.distill_topk(handle, p["z"], 0, R, V, V, 1.0, p["ids"], p["t"], k, 1, p["w"],
                                p["loss"], p["grad"], V, p["status"], None, 0, None)

    pairs(distill, dict(grad=4 * R * V, loss=4 * R, status=4 * R),
          dict(z=4 * R * V, ids=4 * R * k, t=4 * R * k, w=4 * R))


def test_a_workspace_over_other_memory(lib, handle, mem):  # noqa: F811
    """Large rows of one id each other: the workspace lies over an output, then an input.
    Nothing is read: the calls are refused."""
    rows, V = 3, 1 << 20
    far = 1 << 40   # addresses that no call gets as far as to use
    need = lib.token_logprobs_workspace(0, rows, V, 4)
    good = [far + (i << 30) for i in range(1, 7)]
    if need:
        for ws in (good[0], (good[5] - need) // 16 * 16 + 16, far, far + 4 * rows * V - 16, 2 * far):
            assert lib.token_logprobs(handle, far, 0, rows, V, V, 1.0, 2 * far, 1, 4,
                                      ctypes.byref(tsr._Logprobs(*good)), ws, need, None) == EINVAL
    need = lib.distill_topk_workspace(0, rows, V, 0)
    if need:
        for ws in (good[0], good[1], (good[2] - need) // 16 * 16 + 16, good[3], far):
            assert lib.distill_topk(handle, far, 0, rows, V, V, 1.0, good[0], good[1], 1, 0, good[2],
                                    good[3], None, 0, None, ws, need, None) == EINVAL


def test_a_workspace_that_does_not_do(lib, handle, mem):  # noqa: F811
    """Where a call takes one: none, too small, not aligned."""
    rows, V = 3, 1 << 20
    good = (mem + 8192, mem + 8448, mem + 8704, mem + 8960, mem + 9216, mem + 9472)
    o = ctypes.byref(tsr._Logprobs(*good))
    need = lib.token_logprobs_workspace(0, rows, V, 4)
    if need:
        for ws, size in ((None, 0), (None, need), (mem, need - 1), (mem + 8, need + 8)):
            assert lib.token_logprobs(handle, mem, 0, rows, V, V, 1.0, mem, 1, 4, o, ws, size,
                                      None) == EINVAL
    need = lib.distill_topk_workspace(0, rows, V, 0)
    if need:
        for ws, size in ((None, 0), (None, need), (mem, need - 1), (mem + 8, need + 8)):
            assert lib.distill_topk(handle, mem, 0, rows, V, V, 1.0, mem, mem, 1, 0, None, mem,
                                    None, 0, None, ws, size, None) == EINVAL


@pytest.mark.parametrize("size", ["token_logprobs_workspace", "distill_topk_workspace"])
def test_workspace_sizes(lib, size):  # noqa: F811
    """None for sizes that are refused; never past what an int holds, and never less for
    more rows."""
    f = getattr(lib, size)
    assert f(2, 4, 1000, 1) == 0 and f(0, 0, 1000, 1) == 0 and f(0, 4, 0, 1) == 0
    assert f(0, 1 << 22, 1000, 1) == 0 and f(0, 1, (1 << 30) + 1, 1) == 0
    for dt in (0, 1):
        for V in (1, 50, 8192, 32769, 151936, 1 << 20, 1 << 30):
            last = 0
            for rows in (1, 2, 7, 64, 255, 256, 1000, 4096, 100000, (1 << 22) - 1):
                assert 0 <= f(dt, rows, V, 1) < 1 << 30


# ------------------------------------------------------------------ the binding
@pytest.fixture()
def s(lib, monkeypatch):  # noqa: F811
    """A sampler of host tensors (device -1) whose library records its calls."""
    calls = []

    def record(*args):
        calls.append(args)
        return 0

    fake = types.SimpleNamespace(
        norm_quantize_rows=record, token_logprobs=record, token_logprobs_grad=record,
        distill_topk=record, token_logprobs_workspace=lambda *a: 48,
        distill_topk_workspace=lambda *a: 0)
    monkeypatch.setattr(tsr, "load_library", lambda: fake)
    monkeypatch.setattr(tsr, "_stream_on", lambda device, stream: 7)
    s = tsr.Sampler.__new__(tsr.Sampler)
    s._h, s.device, s.calls, s._ws_bytes = ctypes.c_void_p(), -1, calls, {}
    return s


def test_binding_norm(s):
    x, w = torch.zeros(3, 10), torch.ones(10)
    codes, scale = s.norm_quantize_rows(x, w)
    assert codes.shape == (3, 10) and codes.stride(0) == 128 and scale.shape == (3,)
    out = s.norm_quantize_rows(x.bfloat16(), w, residual=x.bfloat16())
    assert len(out) == 3 and out[2].dtype is torch.bfloat16 and out[2].shape == (3, 10)
    r = torch.zeros(3, 12)[:, :10]
    assert s.norm_quantize_rows(x, residual=r, out_residual=r)[2] is r
    assert s.calls[-1][6] is None and s.calls[-1][12] == 12
    for bad in (dict(weight=torch.ones(9)), dict(weight=torch.ones(20)[::2]),
                dict(residual=torch.zeros(3, 9)), dict(residual=x.bfloat16()),
                dict(out_residual=x), dict(residual=x, out_residual=x.bfloat16()),
                dict(residual=x, out_residual=torch.zeros(2, 10)), dict(out=torch.zeros(3, 10)),
                dict(out=torch.zeros(3, 9, dtype=torch.int8)), dict(scale=torch.zeros(2))):
        n = len(s.calls)
        with pytest.raises(ValueError):
            s.norm_quantize_rows(x, **bad)
        assert len(s.calls) == n
    for bad in (torch.zeros(10), torch.zeros(3, 0), torch.zeros(10, 3).t(),
                torch.zeros(1, 10).expand(3, 10)):
        with pytest.raises(ValueError):
            s.norm_quantize_rows(bad)
    with pytest.raises(TypeError):
        s.norm_quantize_rows(x.half())
    with pytest.raises(TypeError):
        s.norm_quantize_rows(x, w.half())
    assert s.norm_quantize_rows(torch.zeros(0, 10))[0].shape == (0, 10)


def test_binding_logprobs(s):
    z, t = torch.zeros(3, 10), torch.zeros(3, 2, dtype=torch.int32)
    got = s.token_logprobs(z, t, top_k=4)
    assert got.logprob.shape == (3, 2) and got.top_ids.shape == got.top_logprob.shape == (3, 4)
    assert got.norm.shape == (3, 2) and got.entropy.shape == (3,) and got.status is None
    args = s.calls[-1]
    assert args[8:10] == (2, 4) and args[11] is not None and args[12] == 48 and args[13] == 7
    got = s.token_logprobs(z.bfloat16(), t[:, 0].contiguous(), entropy=False, norm=False)
    assert got.logprob.shape == (3,) and got.logprob.dtype is torch.float32
    assert got[1:] == (None,) * 5
    assert s.token_logprobs(z).logprob is None and s.calls[-1][7] is None
    for args, kw in (((z, t.long()), {}), ((z, t[:2]), {}), ((z, t[:, :1]), {}),
                     ((z, t[:, :, None]), {}), ((z[0], t), {}), ((z[:, ::2], t), {}),
                     ((z, t), dict(status=torch.zeros(3)))):
        n = len(s.calls)
        with pytest.raises(ValueError):
            s.token_logprobs(*args, **kw)
        assert len(s.calls) == n
    with pytest.raises(TypeError):
        s.token_logprobs(z.double(), t)


def test_binding_logprobs_grad(s):
    z, t = torch.zeros(3, 10), torch.zeros(3, 2, dtype=torch.int32)
    norm, g, H = torch.zeros(3, 2), torch.zeros(3, 2), torch.zeros(3)
    out = torch.zeros(3, 16)[:, :10]
    assert s.token_logprobs_grad(z, t, norm, g, H, H, out=out) is out and s.calls[-1][14] == 16
    assert s.token_logprobs_grad(z.bfloat16(), t, norm, g).dtype is torch.bfloat16
    assert s.token_logprobs_grad(z, None, norm, None, H, H).shape == (3, 10)
    for args, kw in (((z, t, norm, None), {}), ((z, None, norm, g), {}), ((z, t, norm, g[:, :1]), {}),
                     ((z, t, g[:, 0], g), {}), ((z, t, norm, g, None, H), {}),
                     ((z, t, norm, g, H, H[:2]), {}), ((z, t, norm, g), dict(out=out.bfloat16())),
                     ((z, t, norm, g), dict(out=out[:2])), ((z, t, norm.double(), g), {})):
        n = len(s.calls)
        with pytest.raises(ValueError):
            s.token_logprobs_grad(*args, **kw)
        assert len(s.calls) == n


def test_binding_distill(s):
    z, ids, lp = torch.zeros(3, 10), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4)
    loss, grad = s.distill_topk(z, ids, lp)
    assert loss.shape == (3,) and grad.shape == (3, 10)
    assert s.distill_topk(z, ids, lp, grad=False)[1] is None and s.calls[-1][13] is None
    out = torch.zeros(3, 16)[:, :10]
    assert s.distill_topk(z, ids, lp, grad=out, tail=True)[1] is out
    assert s.calls[-1][10] == 1 and s.calls[-1][14] == 16
    for args, kw in (((z, ids.long(), lp), {}), ((z, ids[:, :0], lp[:, :0]), {}),
                     ((z, ids[0], lp[0]), {}), ((z, ids, lp[:, :3]), {}), ((z, ids, lp.double()), {}),
                     ((z, ids, lp), dict(row_weight=torch.ones(2))),
                     ((z, ids, lp), dict(status=torch.zeros(3))),
                     ((z, ids, lp), dict(grad=out.bfloat16())), ((z, ids, lp), dict(grad=out[:2]))):
        n = len(s.calls)
        with pytest.raises(ValueError):
            s.distill_topk(*args, **kw)
        assert len(s.calls) == n


def test_binding_keeps_few_sizes(s):
    """A server whose batches never have the same rows twice."""
    z, p = torch.zeros(3000, 4), torch.zeros(3000, 2, 4)
    fake = tsr.load_library()
    fake.verify_probs_ex, fake.verify_probs_workspace = fake.token_logprobs, lambda *a: 0
    s._vp_bytes = {}
    x, u, v = torch.zeros(3000, 1, dtype=torch.int32), torch.zeros(3000, 1), torch.zeros(3000)
    for rows in range(1, 3000):
        s.token_logprobs(z[:rows])
        s.verify_probs(p[:rows], None, x[:rows], u[:rows], v[:rows])
    assert len(s.calls) == 2 * 2999 and all(c[12] == 48 for c in s.calls[::2])
    assert 0 < len(s._ws_bytes) <= 1024 and 0 < len(s._vp_bytes) <= 1024


def test_binding_refuses_tokens_without_rows(s):
    """A single number is no [rows] of tokens, though there is but one row."""
    z, t = torch.zeros(1, 10), torch.tensor(3, dtype=torch.int32)
    for call in (lambda: s.token_logprobs(z, t),
                 lambda: s.token_logprobs_grad(z, t, torch.zeros(1, 2), torch.zeros(()))):
        with pytest.raises(ValueError):
            call()
    assert s.calls == []
