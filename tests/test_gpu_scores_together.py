"""The calls around the logits as they are used: a step from a block's output to tokens
and their scores, a draft's distillation step on a target's top tokens, on other streams,
and in graphs that run at the same time."""
import pytest

from tests.gpu_common import device, gpu_available, torch
from tests.test_gpu_distill import check as check_distill
from tests.test_gpu_logprobs import check as check_logprobs, check_grad
from tests.test_gpu_norm_quantize import check as check_norm

import token_sampling_row_amd as tsr

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=512, max_vocab=1 << 17, max_k=8, seed=3) as h:
        yield h


def model(V, W, seed):
    g = torch.Generator(device()).manual_seed(seed)
    head = 0.05 * torch.randn(V, W, device=device(), generator=g)
    return (torch.exp(0.1 * torch.randn(W, device=device(), generator=g)), head.bfloat16())


def step(s, x, r, norm_w, head, **kw):
    """Residual sum, norm, projection, draw and the draw's scores."""
    codes, scale, h = s.norm_quantize_rows(x, norm_w, 1e-6, r, **kw)
    z = s.int8_logits(codes, scale, *head, **kw)
    token = s.sample_rows(z, {"temperature": 0.8, "top_k": 50}, 3, **kw)
    return h, codes, scale, z, token, s.token_logprobs(z, token, top_k=8, temperature=0.8, **kw)


@pytest.mark.parametrize("rows,V", [(1, 32000), (5, 8191), (64, 50001)])
def test_from_a_blocks_output_to_scored_tokens(s, rows, V):
    W = 1024
    w, full = model(V, W, V)
    head = s.quantize_rows(full)
    g = torch.Generator(device()).manual_seed(1)
    x = torch.randn(rows, W, device=device(), generator=g).bfloat16()
    r = (3 * torch.randn(rows, W, device=device(), generator=g)).bfloat16()
    h, codes, scale, z, token, got = step(s, x, r, w, head)
    check_norm((codes, scale, h), x, w, 1e-6, r)
    check_logprobs(got, z, token.cpu().numpy()[:, None], 8, 0.8, range(min(rows, 4)))
    # the drawn tokens' own log p, which the sampler gives for the unfiltered distribution
    lp = torch.empty(rows, device=device())
    again = s.sample_rows_masked(z, None, {"temperature": 0.8}, 3, logprob=lp)
    mine = s.token_logprobs(z, again, temperature=0.8).logprob
    assert bool(((mine - lp).abs() <= 1e-5 * lp.abs().clamp(min=1.0)).all())


def test_scores_of_verified_drafts(s):
    """The tokens that a verify step leaves, padding behind them, scored against its rows."""
    B, K, V = 6, 4, 5003
    g = torch.Generator(device()).manual_seed(2)
    z = 2 * torch.randn(B, K + 1, V, device=device(), generator=g)
    d = z[:, :K] + torch.randn(B, K, V, device=device(), generator=g)
    x = torch.stack([s.sample_rows(d[:, j].contiguous(), {}, j) for j in range(K)], 1)
    tokens, kept = s.spec_verify(z, d.contiguous(), x.contiguous(), {}, 9)
    flat = z.view(B * (K + 1), V)
    got = s.token_logprobs(flat, tokens.view(-1))
    check_logprobs(got, flat, tokens.view(-1, 1).cpu().numpy(), 0, 1.0)
    up = torch.randn(B * (K + 1), device=device(), generator=g)
    grad = s.token_logprobs_grad(flat, tokens.view(-1), got.norm, up)
    check_grad(grad, flat, tokens.view(-1, 1).cpu().numpy(), got.norm, up)
    assert bool((got.logprob.view(B, K + 1)[tokens == -1] == 0).all())


@pytest.mark.parametrize("tail", [False, True])
def test_a_draft_follows_its_target(s, tail):
    """A target's top tokens into a draft's loss and gradient, as the calls give them."""
    rows, V, T = 7, 9001, 1.5
    g = torch.Generator(device()).manual_seed(3)
    target = 2 * torch.randn(rows, V, device=device(), generator=g)
    draft = (target + torch.randn(rows, V, device=device(), generator=g)).bfloat16()
    top = s.token_logprobs(target, top_k=30, temperature=T)
    w = torch.full((rows,), 1.0 / rows, device=device())
    got = s.distill_topk(draft, top.top_ids, top.top_logprob, T, tail, w)
    check_distill(got, draft, top.top_ids.cpu().numpy(), top.top_logprob.cpu().numpy(), T, tail,
                  w.cpu().numpy())
    # a target with fewer tokens than entries: padded entries, as they come
    target[:, 12:] = float("-inf")
    top = s.token_logprobs(target, top_k=30, temperature=T)
    assert bool((top.top_ids[:, 12:] == -1).all())
    got = s.distill_topk(draft, top.top_ids, top.top_logprob, T, tail, w)
    check_distill(got, draft, top.top_ids.cpu().numpy(), top.top_logprob.cpu().numpy(), T, tail,
                  w.cpu().numpy())


def all_calls(s, a, stream=None):
    kw = dict(stream=stream)
    fwd = s.token_logprobs(a["z"], a["tok"], top_k=40, **kw)
    grad = s.token_logprobs_grad(a["z"], a["tok"], fwd.norm, a["g"], fwd.entropy, a["ge"], **kw)
    top = s.token_logprobs(a["t"], top_k=40, **kw)
    loss, dg = s.distill_topk(a["z"], top.top_ids, top.top_logprob, 1.0, True, **kw)
    codes, scale, h = s.norm_quantize_rows(a["x"], a["w"], 1e-6, a["r"], **kw)
    return [fwd.logprob, fwd.entropy, fwd.norm, fwd.top_ids, fwd.top_logprob, grad, top.top_ids,
            loss, dg, codes, scale, h]


def inputs(rows, V, W, seed, dtype):
    g = torch.Generator(device()).manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, device=device(), generator=g)

    z = 2 * rand(rows, V)
    return dict(z=z.to(dtype), t=(z + rand(rows, V)).to(dtype), g=rand(rows, 2), ge=rand(rows),
                tok=torch.randint(0, V, (rows, 2), device=device(), generator=g).int(),
                x=rand(rows, W).to(dtype), r=rand(rows, W).to(dtype), w=rand(W))


SETS = [(3, 100003, 4099, torch.bfloat16), (40, 60001, 512, torch.float32),
        (300, 9000, 1000, torch.bfloat16)]


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_calls_of_one_handle_on_several_streams(s):
    """Each again and again on a stream of its own, results allocated there: as alone."""
    sets = [inputs(r, V, W, V, dt) for r, V, W, dt in SETS]
    want = [all_calls(s, a) for a in sets]
    torch.cuda.synchronize()
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], [], []]
    for _ in range(6):
        for k, a in enumerate(sets):
            got[k].append(all_calls(s, a, streams[k]))
    torch.cuda.synchronize()
    for k, w in enumerate(want):
        assert all(same(g, w) for g in got[k])


def test_graphs_replayed_at_the_same_time(s):
    """Two graphs captured on one handle, replayed on two streams at once on new inputs, with
    eager work between: each replay equal to the eager result."""
    sets = [inputs(r, V, W, V, dt) for r, V, W, dt in SETS[:2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a in sets:
        all_calls(s, a, side)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for a in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(all_calls(s, a))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(5):
        for i, a in enumerate(sets):
            for name in ("z", "t", "g", "ge", "x", "r"):
                a[name].normal_(generator=torch.Generator(device()).manual_seed(10 * turn + i))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for a, out in zip(sets, outs):
            assert same(out, all_calls(s, a))


def test_results_do_not_vary(s):
    a = inputs(40, 60001, 512, 1, torch.bfloat16)
    want = all_calls(s, a)
    for _ in range(5):
        assert same(all_calls(s, a), want)


def test_a_workspace_of_the_callers():
    """Nothing behind its bytes is written, and what it held before does not matter."""
    lib = tsr.load_library()
    rows, V, k = 5, 120001, 40
    z = torch.randn(rows, V, device=device())
    need = lib.token_logprobs_workspace(0, rows, V, k)
    with tsr.Sampler(0, max_rows=1, max_vocab=10) as h:
        want = h.token_logprobs(z, top_k=k)
        loss = h.distill_topk(z, want.top_ids, want.top_logprob, 1.0, True)
        for fill in (0, 77, 255):
            ws = torch.full((need + 64,), fill, dtype=torch.uint8, device=device())
            top = torch.empty(rows, k, device=device())
            ids = torch.empty(rows, k, dtype=torch.int32, device=device())
            o = tsr._Logprobs(None, None, ids.data_ptr(), top.data_ptr(), None, None)
            rc = lib.token_logprobs(h._h, z.data_ptr(), 0, rows, V, V, 1.0, None, 0, k,
                                    o, ws.data_ptr(), need,
                                    torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert rc == 0 and torch.equal(ids, want.top_ids) and torch.equal(top, want.top_logprob)
            assert bool((ws[need:] == fill).all())
            size = lib.distill_topk_workspace(0, rows, V, 1)
            ws = torch.full((size + 64,), fill, dtype=torch.uint8, device=device())
            l2, g2 = torch.empty(rows, device=device()), torch.empty_like(z)
            rc = lib.distill_topk(h._h, z.data_ptr(), 0, rows, V, V, 1.0, ids.data_ptr(),
                                  top.data_ptr(), k, 1, None, l2.data_ptr(), g2.data_ptr(), V,
                                  None, ws.data_ptr(), size,
                                  torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            assert rc == 0 and torch.equal(l2, loss[0]) and torch.equal(g2, loss[1])
            assert bool((ws[size:] == fill).all())
