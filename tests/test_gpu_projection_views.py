"""int8_logits on views: a single row, by whose stride nothing is read, and hidden
rows that start at words under large weights in whole lines. Scales of one and
float32 logits: sums below 2^24 are held exactly."""
import pytest

from tests.gpu_common import device, gpu_available, torch

import token_sampling_row_amd as tsr

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def s():
    with tsr.Sampler(0, max_rows=2048, max_vocab=1 << 18, max_k=8, seed=3) as h:
        yield h


def matrix(rows, width, stride, off, seed):
    """[rows, width] random codes at byte `off` of rows `stride` bytes apart."""
    g = torch.Generator(device()).manual_seed(seed)
    big = torch.randint(-128, 128, (rows, stride), dtype=torch.int8, device=device(), generator=g)
    return big[:, off:off + width]


def check(s, c, w):
    ones = torch.ones(max(len(c), len(w)), device=device())
    got = s.int8_logits(c, ones[:len(c)], w, ones[:len(w)], dtype=torch.float32)
    want = c.double() @ w.double().t()
    assert float(want.abs().max()) < 2.0 ** 24
    assert torch.equal(got.double(), want)


FAR = 1 << 22   # rows of more than one row may not lie this far apart


@pytest.mark.parametrize("width,off", [(300, 0), (901, 128), (512, 4), (643, 1)])
def test_one_row_of_a_matrix_with_far_rows(s, width, off):
    """The stride of a single row is never used: hidden state, channel or both."""
    one, many = matrix(2, width, FAR + 256, off, 1)[1:2], matrix(70, width, 1024, 0, 2)
    check(s, one, many)
    check(s, many, one)
    check(s, one, matrix(3, width, FAR, off, 3)[2:])


def test_one_row_through_the_path_to_tokens(s):
    """sample_hidden against a single channel whose row is far from the next."""
    w = matrix(2, 256, FAR, 0, 5)[:1]
    hidden = torch.randn(3, 256, device=device())
    got = s.sample_hidden(hidden, w, torch.ones(1, device=device()), {"temperature": 0.0}, 0)
    assert got.tolist() == [0, 0, 0]


@pytest.mark.parametrize("rows", [2, 70])
def test_far_rows_are_refused_where_there_are_several(s, rows):
    far, near = matrix(2, 64, FAR, 0, 6), matrix(rows, 64, 64, 0, 7)
    ones = torch.ones(rows, device=device())
    for c, w in ((far, near), (near, far)):
        with pytest.raises(tsr.TsrError) as e:
            s.int8_logits(c, ones[:len(c)], w, ones[:len(w)])
        assert e.value.code == 4


@pytest.mark.parametrize("width", [640, 901, 4095])
@pytest.mark.parametrize("off", [0, 4, 64])
def test_one_row_of_any_width_at_a_word(s, width, off):
    check(s, matrix(1, width, width + off, off, width), matrix(700, width, 4224, 128, 8))


@pytest.mark.parametrize("rows", [1, 9, 30, 60, 100, 128, 200, 320, 384, 700])
@pytest.mark.parametrize("stride,off", [(1404, 0), (1408, 4), (1536, 64)])
def test_large_weights_under_rows_at_words(s, rows, stride, off):
    """Weights that outgrow the caches in whole lines, hidden rows that start at
    words or halves of lines, with a partial stage behind."""
    check(s, matrix(rows, 1399, stride, off, rows), matrix(40001, 1399, 1408, 0, 9))


def test_a_device_number_as_text():
    """As it comes from an environment variable; every call takes it as a number."""
    with tsr.Sampler("0", max_rows=8, max_vocab=64, max_k=1) as s:
        codes, scale = s.quantize_rows(torch.ones(2, 16, device=device()))
        assert bool((codes == 127).all())
        logits = s.int8_logits(codes, scale, codes, scale, dtype=torch.float32)
        assert s.sample_rows(logits, {"temperature": 0.0}, 0).tolist() == [0, 0]
        p = torch.ones(1, 2, 4, device=device())
        x = torch.zeros(1, 1, dtype=torch.int32, device=device())
        u = torch.zeros(1, 1, device=device())
        assert s.verify_probs(p, None, x, u, u[0])[1].tolist() == [1]
