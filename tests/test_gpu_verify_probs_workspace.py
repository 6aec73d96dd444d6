"""The workspace of verify_probs: what a handle holds for it, and calls that run at
the same time."""
import pytest

from tests.gpu_common import device, gpu_available, torch

import token_sampling_row_amd as tsr

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_handles_of_short_rows_hold_none():
    """Rows of up to 32 groups of 1024 ids are summed by one workgroup each. 32 such
    handles: what else they hold is under 1 MB each, and an allocation may be
    rounded up to 2 MB, so 64 MB in all; 1024 sums of 8 bytes for each of 512
    sequences would be 134 MB. The first handle is not counted: the library's code
    is loaded with it."""
    device()
    tsr.Sampler(0, max_rows=512, max_vocab=32768, max_k=1).close()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info(0)[0]
    handles = [tsr.Sampler(0, max_rows=512, max_vocab=32768, max_k=1) for _ in range(32)]
    held = free - torch.cuda.mem_get_info(0)[0]
    for h in handles:
        h.close()
    assert held <= 80 << 20, held


@pytest.mark.parametrize("max_vocab", [32769, 100003, (1 << 20) + 1])
@pytest.mark.parametrize("max_rows", [7, 512, 600])
def test_handles_hold_enough_for_their_largest_batches(max_rows, max_vocab):
    """The last sequence of the largest batch, and of the most that share
    workgroups, draws as it does alone."""
    K = 1
    for dtype in (torch.float32, torch.bfloat16):
        with tsr.Sampler(0, max_rows=max_rows, max_vocab=max_vocab, max_k=K) as s:
            for V in {max_vocab, min(max_vocab, 40000)}:
                p = torch.rand(3, K + 1, V, device=device()).to(dtype)
                for rows in {max_rows, min(max_rows, 512)}:
                    at = torch.arange(rows, device=device())
                    x = (at % V).int()[:, None]
                    u = torch.full((rows, K), 0.999, device=device())
                    v = (at.float() + 0.5) / rows
                    many = p[:1].expand(rows, K + 1, V)
                    tokens, kept = s.verify_probs(many, None, x, u, v)
                    for r in {0, rows // 2, rows - 1}:
                        t, a = s.verify_probs(p[:1], None, x[r:r + 1], u[r:r + 1], v[r:r + 1])
                        assert torch.equal(t, tokens[r:r + 1]) and torch.equal(a, kept[r:r + 1])


def batch(rows, K, V, seed):
    g = torch.Generator(device()).manual_seed(seed)
    z = 1.5 * torch.randn(rows, K + 1, V, device=device(), generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :K] + 0.8 * torch.randn(rows, K, V, device=device(), generator=g), -1)
    x = torch.multinomial(q.view(rows * K, V), 1, generator=g).view(rows, K).int()
    return (p, q, x, torch.rand(rows, K, device=device(), generator=g),
            torch.rand(rows, device=device(), generator=g))


def test_calls_of_one_handle_on_several_streams():
    """Batches whose sequences are summed by several workgroups each, on three streams
    of one handle at once, the default stream among them, each again and again: as
    each alone."""
    sets = [batch(rows, 2, V, rows) for rows, V in ((48, 90001), (64, 70001), (33, 100003))]
    with tsr.Sampler(0, max_rows=64, max_vocab=1 << 17, max_k=2) as s:
        want = [s.verify_probs(*a) for a in sets]
        torch.cuda.synchronize()
        streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
        got = [[], [], []]
        for _ in range(10):
            for k, a in enumerate(sets):
                got[k].append(s.verify_probs(*a, stream=streams[k]))
        torch.cuda.synchronize()
    for k, (tokens, kept) in enumerate(want):
        for t, a in got[k]:
            assert torch.equal(t, tokens) and torch.equal(a, kept)


def test_graphs_of_one_handle_replayed_at_the_same_time():
    """Two graphs captured on one handle, replayed on two streams at once, on new
    uniforms each time, with eager work between."""
    sets = [batch(rows, 2, V, rows) for rows, V in ((40, 90001), (56, 70001))]
    with tsr.Sampler(0, max_rows=64, max_vocab=1 << 17, max_k=2) as s:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for a in sets:
            s.verify_probs(*a, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        graphs, outs = [], []
        for a in sets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(s.verify_probs(*a))
            graphs.append(g)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(6):
            for a in sets:
                a[3].uniform_()
                a[4].uniform_()
            torch.cuda.synchronize()
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
            torch.cuda.synchronize()
            for a, out in zip(sets, outs):
                tokens, kept = s.verify_probs(*a)
                assert torch.equal(out[0], tokens) and torch.equal(out[1], kept)


def test_a_workspace_of_the_callers():
    """The same tokens as with the handle's; nothing behind its bytes is written; one
    that is too small or not aligned is refused, and nothing is enqueued."""
    rows, K, V = 20, 2, 50001
    p, q, x, u, v = batch(rows, K, V, 1)
    lib = tsr.load_library()
    need = lib.verify_probs_workspace(0, rows, V)
    assert need == rows * (16 + 49 * 8)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device=device())
    with tsr.Sampler(0, max_rows=rows, max_vocab=V, max_k=K) as s:
        def call(fn, *more):
            t = torch.full((rows, K + 1), -9, dtype=torch.int32, device=device())
            a = torch.full((rows,), -9, dtype=torch.int32, device=device())
            rc = fn(s._h, p.data_ptr(), (K + 1) * V, V, q.data_ptr(), K * V, V, 0, x.data_ptr(),
                    None, u.data_ptr(), v.data_ptr(), rows, K, V, t.data_ptr(), a.data_ptr(), None,
                    *more, torch.cuda.current_stream().cuda_stream)
            torch.cuda.synchronize()
            return rc, t, a

        rc, tokens, kept = call(lib.verify_probs)
        assert rc == 0 and bool((kept >= 0).all())
        for more in ((ws.data_ptr(), need), (None, 0), (None, need)):
            rc, t, a = call(lib.verify_probs_ex, *more)
            assert rc == 0 and torch.equal(t, tokens) and torch.equal(a, kept)
        assert bool((ws[need:] == 77).all()) and not bool((ws[:need] == 77).all())
        for more in ((ws.data_ptr(), need - 1), (ws.data_ptr(), 0), (ws.data_ptr() + 8, need + 8)):
            rc, t, a = call(lib.verify_probs_ex, *more)
            assert rc == 1 and bool((t == -9).all()) and bool((a == -9).all())
