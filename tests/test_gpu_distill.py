"""distill_topk against its reference in 64 bits (oracle/scores.py, which derives the
bounds)."""
import numpy as np
import pytest

from tests.gpu_common import device, gpu_available, torch
from tests.test_gpu_logprobs import NP, TD, VOCABS, dev, logits, new_status, within

import token_sampling_row_amd as tsr
from oracle import scores as sc

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=8, max_vocab=1000, max_k=1, seed=3) as h:
        yield h


def teacher_of(rng, z, k, T, noise=0.8):
    """The top entries of rows near z: (ids, log probabilities)."""
    t = (z.double().cpu().numpy() + rng.normal(0, noise, z.shape)) / T
    ids = np.argsort(-t, 1)[:, :k]
    lse = np.log(np.exp(t - t.max(1, keepdims=True)).sum(1, keepdims=True)) + t.max(1, keepdims=True)
    return ids.astype(np.int32), (np.take_along_axis(t, ids, 1) - lse).astype(np.float32)


def check(got, z, ids, lp, T=1.0, tail=False, weight=None, status=None, rows=None):
    loss, grad = got
    zv = z.float().cpu().numpy()
    for r in range(len(zv)) if rows is None else rows:
        w = sc.distill(zv[r], ids[r], lp[r], T, tail, 1.0 if weight is None else float(weight[r]),
                       NP[z.dtype])
        within(loss[r].item(), w["loss"], w["off_loss"])
        if grad is not None:
            within(grad[r].float().cpu().numpy(), w["grad"], w["off_grad"])
        if status is not None:
            assert status[r].item() == w["status"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("k", [1, 8, 64])
def test_matches(s, dtype, V, tail, k):
    rng = np.random.default_rng([V, k])
    k = min(k, V)
    z = logits(rng, 3, V, dtype)
    weight = rng.normal(0, 1, 3).astype(np.float32)
    for T in (1.0, 1.7):
        ids, lp = teacher_of(rng, z, k, T)
        st = new_status(3)
        got = s.distill_topk(z, dev(ids), dev(lp), T, tail, dev(weight), status=st)
        check(got, z, ids, lp, T, tail, weight, st)
        alone = s.distill_topk(z, dev(ids), dev(lp), T, tail, dev(weight), grad=False)
        check(alone, z, ids, lp, T, tail, weight)
        assert alone[1] is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(40, 32771), (270, 9001), (300, 70001), (1100, 33001),
                                    (600, 151936)])
@pytest.mark.parametrize("tail", [False, True])
def test_many_rows(s, dtype, rows, V, tail):
    """However rows are divided: some against the reference, the losses of all as in small
    batches, to twice the bounds."""
    g = torch.Generator(device()).manual_seed(V)
    z = torch.randn(rows, V, device=device(), generator=g).mul_(2).to(TD[dtype])
    t = z.float() + 0.8 * torch.randn(rows, V, device=device(), generator=g)
    top, ids = t.topk(20, 1)
    lp = top - torch.logsumexp(t, 1, keepdim=True)
    del t
    ids = ids.int()
    w = torch.rand(rows, device=device(), generator=g)
    w[1] = 0.0
    got = s.distill_topk(z, ids, lp, 1.0, tail, w)
    check(got, z, ids.cpu().numpy(), lp.cpu().numpy(), 1.0, tail, w.cpu().numpy(),
          rows=[0, 1, rows // 2, rows - 1])
    for a in range(0, rows, 7):
        b = min(rows, a + 7)
        loss, grad = s.distill_topk(z[a:b], ids[a:b], lp[a:b], 1.0, tail, w[a:b])
        assert bool(((loss - got[0][a:b]).abs() <= 4 * 60 * sc.U * (1 + loss.abs())).all())
        d = (grad.float() - got[1][a:b].float()).abs()
        lim = (2 * sc.HALF_STEP[dtype] + 4 * 60 * sc.U) * grad.float().abs() + 8 * 60 * sc.U
        assert bool((d <= lim).all())


@pytest.mark.parametrize("dtype,rows,V", [("bf16", 11200, 12003), ("f32", 9100, 7499),
                                          ("bf16", 4500, 30001), ("f32", 3400, 20001),
                                          ("bf16", 2800, 50001), ("f32", 2100, 32003),
                                          ("bf16", 1500, 90001), ("f32", 1600, 45003),
                                          ("bf16", 1100, 128253), ("f32", 1100, 65531),
                                          ("bf16", 900, 151935), ("f32", 850, 80003),
                                          ("bf16", 700, 200003)])
def test_gradients_larger_than_the_caches(s, dtype, rows, V):
    """More than 256 MiB, by workgroups of each size: entries' own values over what was put
    past the caches, twice over the same memory."""
    assert rows * V * (4 if dtype == "f32" else 2) > 256 << 20
    g = torch.Generator(device()).manual_seed(V)
    z = torch.empty(rows, V, dtype=TD[dtype], device=device()).normal_(generator=g)
    ids = torch.randint(0, V, (rows, 9), device=device(), generator=g).int()
    ids[:, 2] = ids[:, 6]
    ids[:, 3] = V - 1
    lp = torch.log_softmax(2 * torch.randn(rows, 10, device=device(), generator=g), 1)[:, :9]
    lp = lp.contiguous()
    w = torch.rand(rows, device=device(), generator=g)
    w[1] = 0.0
    some = sorted({0, 1, rows // 3, rows - 1})
    out = torch.full((rows, V), 7.0, dtype=TD[dtype], device=device())
    for tail in (True, False):
        loss, grad = s.distill_topk(z, ids, lp, 0.9, tail, w, grad=out)
        check((loss[some], grad[some]), z[some], ids[some].cpu().numpy(), lp[some].cpu().numpy(),
              0.9, tail, w[some].cpu().numpy())
        # of every row the sum is 0 but for roundings: half a step of each element (counted of
        # the rounded ones: 1 + 2^-7 of it), 4 x 60 U of each as in test_many_rows, 8 x 60 U of
        # each entry and twice that of q_r / p_r for all the others together
        total = grad.sum(1, dtype=torch.float64).abs()
        size = grad.abs().sum(1, dtype=torch.float64)
        lim = (sc.HALF_STEP[dtype] * (1 + 2.0 ** -7) + 240 * sc.U) * size + 11 * 480 * sc.U
        assert bool((total <= lim).all())


@pytest.mark.parametrize("dtype,rows,V", [("f32", 200, 32000), ("bf16", 140, 128256),
                                          ("bf16", 130, 33003), ("f32", 400, 32003),
                                          ("bf16", 1000, 128253), ("bf16", 120, 300005),
                                          ("f32", 8195, 100003), ("bf16", 20000, 1003),
                                          ("bf16", 3000, 33003), ("bf16", 2, 5_000_011)])
def test_every_way_that_rows_are_divided(s, dtype, rows, V):
    """A workgroup of each size to a row, slices joined in each tile or by themselves, more
    rows than the workspace holds at a time, read from the caches or past them: rows on
    either side of the limits against the reference."""
    g = torch.Generator(device()).manual_seed(V)
    z = torch.empty(rows, V, dtype=TD[dtype], device=device()).normal_(generator=g)
    ids = torch.randint(0, V, (rows, 12), device=device(), generator=g).int()
    ids[:, 5] = ids[:, 6]
    ids[:, 7] = V - 1
    ids[:, 8] = -1
    lp = torch.log_softmax(2 * torch.randn(rows, 13, device=device(), generator=g), 1)[:, :12]
    lp = lp.contiguous()
    w = torch.rand(rows, device=device(), generator=g)
    st = new_status(rows)
    if rows > 2:
        w[1] = 0.0
        z[rows - 2, V - 1] = float("nan")
    some = sorted({0, 1, 8191 % rows, 8192 % rows, rows // 2, max(0, rows - 2), rows - 1})
    for tail in (True, False):
        loss, grad = s.distill_topk(z, ids, lp, 1.3, tail, w, status=st)
        check((loss[some], grad[some]), z[some], ids[some].cpu().numpy(), lp[some].cpu().numpy(),
              1.3, tail, w[some].cpu().numpy(), st[some])
        alone, _ = s.distill_topk(z, ids, lp, 1.3, tail, w, grad=False)
        d = (alone - loss).abs()   # the sums may be divided otherwise: twice their bound
        assert bool((d <= 4 * 60 * sc.U * (1 + loss.abs())).logical_or(d.isnan()).all())
        assert int((st != 0).sum()) == (rows > 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 40003])
def test_special_rows(s, dtype, V):
    rng = np.random.default_rng(5)
    k, R = 6, 22
    z = logits(rng, R, V, dtype).float()
    ids, lp = teacher_of(rng, z, k, 1.0)
    w = np.ones(R, dtype=np.float32)
    z[0, V - 1] = float("nan")
    z[1, 3] = float("inf")
    z[2] = float("-inf")
    ids[3, 2] = V
    ids[4, 0] = -2
    lp[5, 1] = np.nan
    lp[6, 5] = np.inf
    lp[7] = -np.inf
    ids[8] = -1
    ids[9, 1:] = -1                            # one entry
    lp[10, :3] = -np.inf
    z[11, ids[11, 2]] = float("-inf")          # the draft excludes what the teacher gives
    z[12, ids[12, 0]] = float("-inf")
    lp[12, 0] = -np.inf                        # nor does the teacher
    ids[13, 1] = ids[13, 0]                    # an id twice
    z[14], ids[14], lp[14], w[14] = float("nan"), V + 9, np.nan, 0.0
    z[15, ids[15, 0]] = 90.0                   # nearly everything on one entry
    keep = z[16, ids[16]].clone()
    z[16] = float("-inf")                      # the draft gives the rest nothing
    z[16, ids[16]] = keep
    lp[17] += 3.0                              # probabilities past 1
    z[18] += 1e4
    lp[19] = np.log(np.float32(1.0 / k))       # nothing is left over
    z[20] = 0.0
    lp[21, 0], lp[21, 1:] = 0.0, -40.0         # certain
    w[15], w[13] = -2.5, 1e-3
    t = z.to(TD[dtype])
    for tail in (False, True):
        st = new_status(R)
        got = s.distill_topk(t, dev(ids), dev(lp), 1.0, tail, dev(w), status=st)
        check(got, t, ids, lp, 1.0, tail, w, st)
        assert st.tolist()[:10] == [1, 1, 2, 3, 3, 1, 1, 2, 2, 0]
        assert got[0][14].item() == 0 and not bool(got[1][14].any())
        assert got[0][11].item() == np.inf
        assert (got[0][16].item() == np.inf) == tail


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_rest_where_entries_hold_nearly_all(s, dtype):
    """p_r down to 1e-9 of the whole: the loss and the gradient of the other ids keep their
    precision (the bounds are relative to each element)."""
    rng = np.random.default_rng(9)
    V = 33001
    z = logits(rng, 6, V, dtype, 1.0).float()
    ids = np.stack([rng.permutation(V)[:5] for _ in range(6)]).astype(np.int32)
    for r in range(6):
        z[r, ids[r]] += 12.0 + 4.0 * r
    lp = np.log(np.full((6, 5), 0.19, dtype=np.float32))
    t = z.to(TD[dtype])
    check(s.distill_topk(t, dev(ids), dev(lp), 1.0, True), t, ids, lp, 1.0, True)


def test_gradient_against_differences(s):
    """Along random directions d in [-1, 1]: the losses at z +- h d. The third derivative of
    every log p along d (that of the rest too) stays below 8 for |d| <= 1, and the
    weights of the logs sum to 1: h^2 / 6 of it, and the losses' own errors over h."""
    V, h = 3001, 2.0 ** -6
    rng = np.random.default_rng(7)
    z = logits(rng, 1, V, "f32")
    for tail in (False, True):
        ids, lp = teacher_of(rng, z, 9, 1.0)

        def value(zz):
            return float(s.distill_topk(zz, dev(ids), dev(lp), 1.0, tail, grad=False)[0][0])

        grad = s.distill_topk(z, dev(ids), dev(lp), 1.0, tail)[1][0].double()
        for _ in range(10):
            d = dev(rng.uniform(-1, 1, (1, V)).astype(np.float32))
            diff = (value(z + h * d) - value(z - h * d)) / (2 * h)
            assert abs(diff - float(grad @ d[0].double())) < h * h / 6 * 16 + 4 * 60 * sc.U * 4 / h


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 5])
@pytest.mark.parametrize("V", [13, 9001, 70003])
def test_strided_rows(s, dtype, off, V):
    rng = np.random.default_rng(off)
    z = logits(rng, 6, V + 37, dtype)[:, off:off + V]
    ids, lp = teacher_of(rng, z, 5, 1.0)
    out = torch.full((6, V + 29), 77.0, dtype=TD[dtype], device=device())
    got = s.distill_topk(z, dev(ids), dev(lp), tail=True, grad=out[:, off:off + V])
    check(got, z, ids, lp, 1.0, True)
    assert bool((out[:, :off] == 77).all()) and bool((out[:, off + V:] == 77).all())


@pytest.mark.parametrize("T", [1e-6, 1e6, 1e30])
@pytest.mark.parametrize("V", [9001, 150003])
def test_temperatures_far_from_one(s, T, V):
    rng = np.random.default_rng(12)
    z = rng.normal(0, 3, (3, V)).astype(np.float32)
    z[1, ::5] = -np.inf
    z[2] *= 1e10
    ids = np.stack([rng.permutation(V)[:4] for _ in range(3)]).astype(np.int32)
    ids[:, 0] = z.argmax(1)
    ids[1, 1:] = [1, 2, 3]
    lp = np.log(np.full((3, 4), 0.2, dtype=np.float32))
    for tail in (False, True):
        t = dev(z)
        check(s.distill_topk(t, dev(ids), dev(lp), T, tail), t, ids, lp, T, tail)


@pytest.mark.parametrize("rows", [3, 130])
def test_gradient_in_columns_of_one_matrix(s, rows):
    """The gradient beside its logits in the rows of one tensor."""
    rng = np.random.default_rng(13)
    V = 40001
    big = torch.zeros(rows, 2 * V, device=device())
    z = big[:, :V]
    z.copy_(logits(rng, rows, V, "f32"))
    ids, lp = teacher_of(rng, z, 5, 1.0)
    before = z.clone()
    got = s.distill_topk(z, dev(ids), dev(lp), 1.0, True, grad=big[:, V:])
    assert torch.equal(z, before)
    check(got, z, ids, lp, 1.0, True, rows=[0, rows - 1])
    with pytest.raises(tsr.TsrError):
        s.distill_topk(z, dev(ids), dev(lp), 1.0, True, grad=big[:, V - 1:-1])


def test_refusals(s):
    z = torch.zeros(2, 100, device=device())
    ids = torch.zeros(2, 65, dtype=torch.int32, device=device())
    lp = torch.zeros(2, 65, device=device())
    with pytest.raises(tsr.TsrError):
        s.distill_topk(z, ids, lp)
    with pytest.raises(tsr.TsrError):
        s.distill_topk(z, ids[:, :4].contiguous(), lp[:, :4].contiguous(), temperature=-1.0)
    with pytest.raises(tsr.TsrError):   # the gradient in the logits' place
        s.distill_topk(z, ids[:, :4].contiguous(), lp[:, :4].contiguous(), grad=z)
    loss, grad = s.distill_topk(z[:0], ids[:0, :4].contiguous(), lp[:0, :4].contiguous())
    assert loss.shape == (0,) and grad.shape == (0, 100)


def test_a_vocabulary_of_millions(s):
    V = 5_000_003
    g = torch.Generator(device()).manual_seed(2)
    z = torch.randn(2, V, device=device(), generator=g)
    ids = np.array([[V - 1, 5, 3_000_000], [0, 70_000, 9]], dtype=np.int32)
    lp = np.log(np.array([[0.5, 0.2, 0.1], [0.3, 0.3, 0.3]], dtype=np.float32))
    for tail in (False, True):
        check(s.distill_topk(z, dev(ids), dev(lp), 1.0, tail), z, ids, lp, 1.0, tail)
