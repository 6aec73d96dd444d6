"""The 8-bit projection's and verify_probs' C entry points without a GPU: null
handles are refused, and the binding's mirror of tsr_head has the C layout."""
import ctypes


import token_sampling_row_amd as tsr
from tests.test_abi import lib  # noqa: F401


def test_null_handles(lib):  # noqa: F811
    head = tsr._Head(None, 1, None, None, 1, 1)
    prm = tsr._Params(1.0, 0, 1.0, 0.0, 0)
    assert lib.quantize_rows(None, None, 0, 1, 1, 1, None, 1, None, None) == 1
    assert lib.int8_logits(None, None, 1, None, 1, ctypes.byref(head), None, 0, 1, None) == 1
    assert lib.sample_hidden(None, None, 0, 1, 1, ctypes.byref(head), None, 1, None, None, 0,
                             ctypes.byref(prm), 0, None, None, None) == 1
    assert lib.verify_probs(None, None, 0, 0, None, 0, 0, 0, None, None, None, None, 1, 1, 1,
                            None, None, None, None) == 1


def test_head_layout():
    assert ctypes.sizeof(tsr._Head) == 40
    assert tsr._Head.weight_stride.offset == 8 and tsr._Head.scale.offset == 16
    assert tsr._Head.bias.offset == 24 and tsr._Head.vocab.offset == 32
    assert tsr._Head.width.offset == 36
