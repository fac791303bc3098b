"""Argument checks of the windowed attention and distillation calls that need no device."""
import ctypes

import pytest

from tests._util import ensure_built
from transformer_esm_layer_gb300 import binding

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    return binding.load_library()


def test_null_handles_are_rejected(lib):
    n = ctypes.c_size_t()
    w = binding.EsmAttnWindow(1, 1, 0)
    assert lib.esm_encoder_set_attention_window(None, ctypes.byref(w)) == 1
    assert lib.esm_op_attention_window_workspace_size(None, 4, 1, ctypes.byref(w), 0, ctypes.byref(n)) == 1
    assert lib.esm_op_attention_window(None, None, None, 1, 1, 1, ctypes.byref(w), None, None, None, 0, None) == 1
    assert lib.esm_op_attention_window_backward(None, None, None, None, None, None, 1, 1, 1, ctypes.byref(w), None,
                                                None, 0, None) == 1
    assert lib.esm_op_distill_loss_workspace_size(None, 4, 33, ctypes.byref(n)) == 1
    assert lib.esm_op_distill_loss(None, None, 0, 33, None, None, 1, 1, 33, 1.0, None, None, None, None, None, 0,
                                   None) == 1
    assert lib.esm_op_distill_loss_backward(None, None, 0, 33, None, None, 1, 1, 33, 1.0, None, None, None, 33,
                                            None) == 1
    assert lib.esm_encoder_lm_head_distill_backward(None, None, None, 1, None, None, 1, 1.0, None, None, None, None,
                                                    None, None, 0, None) == 1


class _NoDevice(binding.EsmEncoder):
    """The binding's own checks, without a handle behind them."""

    def __init__(self, precision="bf16"):
        self.precision, self.hidden, self.handle = precision, 256, None
        self.cfg = binding.EsmConfig(1, 256, 4, 512, 33, 1026, 1e-5, 1e4, 1.0, 1, 1, 16)


def test_host_tensors_are_rejected_before_any_call():
    enc = _NoDevice()
    qkv = torch.zeros(8, 768, dtype=torch.bfloat16)
    o = torch.zeros(8, 256, dtype=torch.bfloat16)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    lse = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_attention_window(qkv, cu, 8, (1, 1, 0), o)
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_attention_window_backward(qkv, o, lse, o, cu, 8, (1, 1, 0), qkv)
    z, ids, tl = torch.zeros(8, 33), torch.zeros(8, 2, dtype=torch.int32), torch.zeros(8, 2)
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_distill_loss(z, ids, tl, 1.0, torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_distill_loss_backward(z, ids, tl, 1.0, torch.zeros(8), z)
    with pytest.raises(ValueError, match="CUDA"):
        enc.lm_head_distill_backward(None, o, ids, tl, 1.0)


def test_one_row_may_report_any_stride():
    one = torch.zeros(5, 7)[:1]
    assert binding.EsmEncoder._row_stride(one) == 7
    assert binding.EsmEncoder._row_stride(torch.zeros(1, 7).as_strided((1, 7), (1, 1))) == 7
    assert binding.EsmEncoder._row_stride(torch.zeros(3, 9)[:, :4]) == 9


def test_integers_that_the_library_cannot_take_are_refused():
    """ctypes would keep the low 32 bits: a side of 2^32 became one of 0."""
    for window in ((2 ** 32, 0, 0), (0, 2 ** 31, 0), (1, 1, 2 ** 63), (-2 ** 31 - 1, 0, 0)):
        with pytest.raises(ValueError, match="32"):
            binding._window_struct(window)
    for window in ((1.5, 0, 0), (1, "2", 0), (1, 1, float("nan"))):
        with pytest.raises(ValueError):
            binding._window_struct(window)
    w = binding._window_struct((torch.tensor(7), 2 ** 31 - 1, 4.0))
    assert (w.left, w.right, w.sinks) == (7, 2 ** 31 - 1, 4)
    assert binding._c_int("f", "max_seqlen", 5) == 5
    for n in (2 ** 32 + 64, 64.7):
        with pytest.raises(ValueError, match="max_seqlen"):
            binding._c_int("f", "max_seqlen", n)
