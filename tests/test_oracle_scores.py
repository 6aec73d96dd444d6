"""The references of the calls around the logits (oracle/scores.py): closed forms,
gradients against differences of the reference's own loss, and the identities that the
definitions imply."""
import fractions

import numpy as np
import pytest

from oracle import scores as sc


def test_codes_are_the_exact_quotients():
    """Against rational arithmetic, ties among them (a weight of ones and whole
    values: 127 t / m is a half for every odd t where m is 254)."""
    rng = np.random.default_rng(0)
    x = np.stack([rng.integers(-254, 255, 60).astype(np.float32),
                  rng.normal(0, 1, 60).astype(np.float32)])
    x[0, 0] = 254.0
    for w in (None, rng.normal(1, 0.3, 60).astype(np.float32)):
        codes, scale, h = sc.norm_quantize(x, w)
        for r in range(2):
            t = [fractions.Fraction(float(v)) * fractions.Fraction(1.0 if w is None else float(c))
                 for v, c in zip(h[r], w if w is not None else x[r])]
            m = max(abs(v) for v in t)
            assert [round(127 * v / m) for v in t] == codes[r].tolist()


def test_codes_and_scales_stand_for_the_normed_rows():
    rng = np.random.default_rng(1)
    x, r = rng.normal(0, 2, (2, 5, 300)).astype(np.float32)
    w = rng.normal(1, 0.2, 300).astype(np.float32)
    codes, scale, h = sc.norm_quantize(x, w, 1e-5, r)
    y = h.astype(np.float64) * w / np.sqrt((h.astype(np.float64) ** 2).mean(1) + 1e-5)[:, None]
    assert (np.abs(codes * scale[:, None] - y) <= scale[:, None] * (0.5 + 1e-9)).all()
    assert np.allclose(np.abs(codes).max(1), 127)


def test_rows_without_a_norm():
    x = np.zeros((4, 6), dtype=np.float32)
    x[1, 2], x[2, 3] = np.inf, np.nan
    x[3] = 1.0
    w = np.zeros(6, dtype=np.float32)
    codes, scale, _ = sc.norm_quantize(x)
    assert scale[0] == 0 and np.isnan(scale[1:3]).all() and scale[3] > 0
    assert not codes[:3].any() and (codes[3] == 127).all()
    codes, scale, _ = sc.norm_quantize(x, w)
    assert scale[0] == 0 and scale[3] == 0 and np.isnan(scale[1:3]).all() and not codes.any()


def test_bf16_rounding():
    v = np.array([1.0, 1.00390625, 1.01171875, 3.4e38, np.inf, -2.0], dtype=np.float32)
    assert sc.round_bf16(v)[:3].tolist() == [1.0, 1.0, 1.015625]
    assert np.isinf(sc.round_bf16(v)[3:5]).all() and sc.round_bf16(v)[5] == -2.0


def test_logprobs_closed_forms():
    z = np.zeros(8)
    r = sc.logprobs(z, [3, -1, 8], 3)
    assert r["status"] == 3 and np.isclose(r["logprob"][0], -np.log(8)) and r["logprob"][1] == 0
    assert np.isnan(r["logprob"][2]) and np.isclose(r["entropy"], np.log(8))
    assert r["top_ids"].tolist() == [0, 1, 2] and r["norm"].tolist() == [0.0, 8.0]
    z = np.full(5, -np.inf)
    z[2], z[4] = 1.0, 1.0 + np.log(3.0)
    r = sc.logprobs(z, [2, 0], 4)
    assert np.allclose(np.exp(r["logprob"]), [0.25, 0.0]) and r["top_ids"].tolist() == [4, 2, -1, -1]
    assert np.isclose(r["entropy"], -0.25 * np.log(0.25) - 0.75 * np.log(0.75))
    assert sc.logprobs(np.full(3, -np.inf), [1], 1)["status"] == 2
    assert sc.logprobs(np.array([0.0, np.inf]), [1], 1)["status"] == 1


@pytest.mark.parametrize("T", [1.0, 0.6, 2.5])
def test_logprobs_gradient_against_differences(T):
    rng = np.random.default_rng(2)
    z = rng.normal(0, 2, 40)
    z[5] = -np.inf
    tokens, g, ge = [3, 7, 3, -1], rng.normal(0, 1, 4), 0.3

    def value(z):
        r = sc.logprobs(z, tokens, 0, T)
        return sum(gi * v for gi, v, t in zip(g, r["logprob"], tokens) if t != -1) + \
            ge * r["entropy"]

    r = sc.logprobs(z, tokens, 0, T)
    got, _ = sc.logprobs_grad(z, tokens, r["norm"], g, T, r["entropy"], ge)
    assert got[5] == 0
    for j in range(40):
        if j == 5:
            continue
        step = np.zeros(40)
        step[j] = 1e-5
        assert abs((value(z + step) - value(z - step)) / 2e-5 - got[j]) < 1e-8


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [1.0, 0.6, 2.5])
def test_distill_gradient_against_differences(tail, T):
    rng = np.random.default_rng(3)
    z, t = rng.normal(0, 2, 30), rng.normal(0, 2, 30)
    z[4] = -np.inf
    lp = t - np.log(np.exp(t).sum())
    ids = [9, 2, -1, 17, 2]
    teacher = lp[[9, 2, 0, 17, 2]]
    got = sc.distill(z, ids, teacher, T, tail, 0.7)
    assert got["grad"][4] == 0
    for j in range(30):
        if j == 4:
            continue
        step = np.zeros(30)
        step[j] = 1e-5
        up, down = (sc.distill(z + s, ids, teacher, T, tail, 0.7)["loss"] for s in (step, -step))
        assert abs((up - down) / 2e-5 - got["grad"][j]) < 1e-8


def test_distill_closed_forms():
    """A draft that agrees with its teacher has loss and gradient 0, with every id given or
    with the rest as one; without a tail any constant may be added to the entries."""
    rng = np.random.default_rng(4)
    z = rng.normal(0, 1, 12)
    lp = z - np.log(np.exp(z).sum())
    for tail, ids in ((True, [3, 8, 1]), (True, list(range(12))), (False, list(range(12)))):
        r = sc.distill(z, ids, lp[ids], 1.0, tail)
        assert abs(r["loss"]) < 1e-7 and np.abs(r["grad"]).max() < 1e-7
    a, b = (sc.distill(z, [3, 8], np.array([-1.0, -2.0]) + s) for s in (0.0, 4.0))
    assert np.isclose(a["loss"], b["loss"]) and np.allclose(a["grad"], b["grad"])
    # the whole of the teacher on one id: cross entropy
    r = sc.distill(z, [5], [0.0], 1.0, True)
    assert np.isclose(r["loss"], -lp[5], atol=1e-12)
    assert np.allclose(r["grad"], np.exp(lp) - (np.arange(12) == 5), atol=1e-12)


def test_distill_rows_that_do_not_count():
    z = np.zeros(6)
    assert sc.distill(z, [7], [0.0])["status"] == 3
    assert sc.distill(z, [2], [np.nan])["status"] == 1
    assert sc.distill(z, [-1, 2], [0.0, -np.inf])["status"] == 2
    assert sc.distill(np.full(6, -np.inf), [2], [0.0])["status"] == 2
    assert sc.distill(z * np.nan, [2], [0.0])["status"] == 1
    r = sc.distill(z * np.nan, [9], [np.nan], weight=0.0)
    assert r["status"] == 0 and r["loss"] == 0 and not r["grad"].any()
    z[2] = -np.inf
    assert sc.distill(z, [2, 1], [-1.0, -1.0])["loss"] == np.inf
