"""verify_probs' workspace without a GPU: its size by the batch's sizes, and that the
binding gives each call one of its own."""
import ctypes
import types

import pytest

import token_sampling_row_amd as tsr
from tests.test_abi import lib  # noqa: F401


def test_workspace_sizes(lib):  # noqa: F811
    """16 bytes and a double per group of 1024 fp32 or 2048 bf16 ids, 1024 groups at
    most; none up to 32 groups and past 512 sequences."""
    size = lib.verify_probs_workspace
    for dtype, unit in ((0, 1024), (1, 2048)):
        assert size(dtype, 512, 32 * unit) == 0
        assert size(dtype, 1, 32 * unit + 1) == 16 + 33 * 8
        assert size(dtype, 512, 32 * unit + 1) == 512 * (16 + 33 * 8)
        assert size(dtype, 513, 1 << 20) == 0
        assert size(dtype, 512, 1024 * unit) == 512 * (16 + 1024 * 8)
        assert size(dtype, 512, 1024 * unit + 1) == 512 * (16 + 513 * 8)   # two units a group
        assert size(dtype, 512, 1 << 30) <= 512 * (16 + 1024 * 8)
    for bad in ((2, 4, 100000), (0, 0, 100000), (0, -1, 100000), (0, 4, 0)):
        assert size(*bad) == 0


def test_a_null_handle(lib):  # noqa: F811
    assert lib.verify_probs_ex(None, None, 0, 0, None, 0, 0, 0, None, None, None, None, 1, 1, 1,
                               None, None, None, None, 0, None) == 1


@pytest.mark.parametrize("raw", [0, 7])
@pytest.mark.parametrize("rows,vocab,takes", [(3, 40000, True), (3, 32000, False),
                                              (600, 40000, False)])
def test_each_call_brings_its_workspace(lib, monkeypatch, rows, vocab, takes, raw):  # noqa: F811
    """The binding against a library that records what it is given (host tensors).
    On the default stream (0) the handle's workspace is taken."""
    torch = pytest.importorskip("torch")
    calls = []

    def record(*args):
        calls.append(args)
        return 0

    fake = types.SimpleNamespace(verify_probs=record, verify_probs_ex=record,
                                 verify_probs_workspace=lib.verify_probs_workspace)
    monkeypatch.setattr(tsr, "load_library", lambda: fake)
    monkeypatch.setattr(tsr, "_stream_on", lambda device, stream: raw)
    s = tsr.Sampler.__new__(tsr.Sampler)
    s._h, s.device, s._vp_bytes = ctypes.c_void_p(), -1, {}   # -1: the host
    p = torch.zeros(1, 2, vocab).expand(rows, 2, vocab)
    x, u, v = torch.zeros(rows, 1, dtype=torch.int32), torch.zeros(rows, 1), torch.zeros(rows)
    for _ in range(2):
        s.verify_probs(p, None, x, u, v)
    for args in calls:
        assert len(args) == 21
        workspace, size = args[18], args[19]
        assert size == (lib.verify_probs_workspace(0, rows, vocab) if raw else 0)
        assert (workspace is not None and workspace % 16 == 0) == (takes and raw != 0)
        assert args[20] == raw
