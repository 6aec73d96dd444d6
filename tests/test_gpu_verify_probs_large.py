"""verify_probs on batches that outgrow the caches (48 MiB of target rows on),
whose rows are read past them: against the plain reference on some sequences,
and all of them against the same sequences in small batches, which stay in the
caches (the sums are formed in the same order, so the tokens are the same)."""
import numpy as np
import pytest

from tests.gpu_common import device, gpu_available, torch
from tests.test_gpu_verify_probs import check

import token_sampling_row_amd as tsr

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=1024, max_vocab=1 << 18, max_k=8, seed=3) as h:
        yield h


def large(rows, K, V, dtype, seed):
    """p, q, drafts, uniforms and draft counts (0 to K) of a batch, on the GPU."""
    g = torch.Generator(device()).manual_seed(seed)
    z = 1.5 * torch.randn(rows, K + 1, V, device=device(), generator=g)
    p = torch.softmax(z, -1).to(dtype)
    z = z[:, :K] + 0.8 * torch.randn(rows, K, V, device=device(), generator=g)
    q = torch.softmax(z, -1).to(dtype)
    x = torch.multinomial(q.float().view(rows * K, V), 1, generator=g).view(rows, K).int()
    u = torch.rand(rows, K, device=device(), generator=g)
    v = torch.rand(rows, device=device(), generator=g)
    lens = torch.randint(0, K + 1, (rows,), device=device(), generator=g).int()
    lens[:3] = torch.tensor([0, K, K], dtype=torch.int32)
    return p, q, x, u, v, lens


def compare(s, p, q, x, u, v, lens, step):
    rows = len(x)
    status = torch.full((rows,), -7, dtype=torch.int32, device=device())
    tokens, kept = s.verify_probs(p, q, x, u, v, draft_lens=lens, out_status=status)
    few = [s.verify_probs(p[r:r + step], None if q is None else q[r:r + step], x[r:r + step],
                          u[r:r + step], v[r:r + step],
                          draft_lens=None if lens is None else lens[r:r + step])
           for r in range(0, rows, step)]
    assert torch.equal(tokens, torch.cat([t for t, _ in few]))
    assert torch.equal(kept, torch.cat([a for _, a in few]))
    some = [0, 1, 2, rows // 2, rows - 1]

    def host(t, to):
        return None if t is None else t[some].to(to).cpu().numpy()

    check((tokens[some], kept[some]), host(p, torch.float64), host(q, torch.float64),
          x[some].cpu().numpy(), host(lens, torch.int32), host(u, torch.float32),
          host(v, torch.float32), status[some])
    return kept


TD = {"f32": torch.float32, "bf16": torch.bfloat16}


# by several workgroups a sequence, by one each (few ids; more sequences than the
# workspace), a whole number of spans and not
@pytest.mark.parametrize("dtype,rows,V", [
    ("f32", 128, 100003), ("f32", 50, 262144), ("f32", 600, 24001), ("f32", 520, 40007),
    ("bf16", 256, 100003), ("bf16", 200, 131072), ("bf16", 520, 60001)])
def test_large_batches(s, dtype, rows, V):
    p, q, x, u, v, lens = large(rows, 2, V, TD[dtype], V)
    assert p[:, 0].numel() * p.element_size() >= 48 << 20
    for ln in (None, lens):
        for qq in (q, None):
            compare(s, p, qq, x, u, v, ln, 16)


@pytest.mark.parametrize("dtype,rows,V", [("f32", 128, 100003), ("f32", 600, 24001),
                                          ("bf16", 256, 100003)])
def test_large_batches_with_empty_residuals(s, dtype, rows, V):
    """q = 2 p in every second sequence, refused by u 0.75: nothing is left of the
    target, and the draw is from the target itself."""
    p, q, x, u, v, _ = large(rows, 2, V, TD[dtype], V)
    q[::2] = p[::2, :2] * 2
    u[::2] = 0.75
    kept = compare(s, p, q, x, u, v, None, 16)
    assert bool((kept[::2] == 0).all())


@pytest.mark.parametrize("rows,V", [(128, 100003), (600, 24001)])
def test_bad_values_in_large_batches(s, rows, V):
    """A NaN, an infinity or a negative value in the rows drawn from, at either
    end and in the partial span; the other sequences are as they were."""
    p, q, x, u, v, _ = large(rows, 2, V, torch.float32, V + 1)
    x[:8] = 11
    p[:8, :, 11] = 0.0                                   # the first draft is refused:
    q[:8, :, 11] = 0.5                                   # row 0 is drawn from
    p[0, 0, 0], p[1, 0, V - 1], p[2, 0, V // 2] = float("nan"), float("inf"), -1.0
    q[3, 0, V - 1], q[4, 0, 5] = float("nan"), -0.5
    p[5, 1, 3] = float("nan")                            # not drawn from
    p[6, 0] = 0.0                                        # nothing to draw from
    p[7, 0, 100:200] = -0.0
    status = torch.full((rows,), -7, dtype=torch.int32, device=device())
    tokens, kept = s.verify_probs(p, q, x, u, v, out_status=status)
    assert status[:8].tolist() == [1, 1, 1, 1, 1, 0, 2, 0]
    assert bool((status[8:] == 0).all())
    bad = status != 0
    assert bool((tokens[bad] == -1).all()) and bool((kept[bad] == 0).all())
    some = [5, 7, rows - 1]
    check((tokens[some], kept[some]), p[some].double().cpu().numpy(), q[some].double().cpu().numpy(),
          x[some].cpu().numpy(), None, u[some].cpu().numpy(), v[some].cpu().numpy(), status[some])
