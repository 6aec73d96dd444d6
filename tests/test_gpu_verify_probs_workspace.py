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
