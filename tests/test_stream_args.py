"""Argument checks of the residual stream's operators (dropout, embedding, block norm) that need no device."""
import ctypes

import pytest

from tests._util import ensure_built
from transformer_esm_layer_gb300 import binding
from transformer_esm_layer_gb300.binding import BlockNorm, Dropout

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    return binding.load_library()


def test_null_handles_are_rejected(lib):
    n = ctypes.c_size_t()
    norm, grads = binding.EsmBlockNorm(0, 1.0), binding.EsmBlockNormGrads()
    assert lib.esm_op_dropout(None, None, 0, 8, None, 0, None, 0, 8, 1, 8, None, None) == 1
    assert lib.esm_op_embed(None, None, 1, None, 0, 33, 8, 1.0, None, None, None, 0, 8, None) == 1
    assert lib.esm_op_embed_backward_workspace_size(None, 1, 33, 8, ctypes.byref(n)) == 1
    assert lib.esm_op_embed_backward(None, None, 1, None, 0, 8, 1.0, None, None, None, 33, 8, 0, None, 0, None) == 1
    assert lib.esm_op_block_norm(None, norm, None, 0, None, None, None, None, None, None, 1, 8, None) == 1
    assert lib.esm_op_block_norm_backward_workspace_size(None, 1, 8, ctypes.byref(n)) == 1
    assert lib.esm_op_block_norm_backward(None, norm, None, 0, None, None, None, None, None, None, None, None, grads, 1,
                                          8, None, 0, None) == 1


class _NoDevice(binding.EsmEncoder):
    """The binding's own checks, without a handle behind them."""

    def __init__(self, precision="bf16"):
        self.precision, self.hidden, self.handle = precision, 256, None
        self.cfg = binding.EsmConfig(1, 256, 4, 512, 33, 1026, 1e-5, 1e4, 1.0, 1, 1, 16)


def test_host_tensors_are_rejected_before_any_call():
    enc = _NoDevice()
    x, y = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_dropout(x, x, None)
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_embed(ids, torch.zeros(33, 8), x)
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_embed_backward(ids, x, torch.zeros(33, 8))
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_block_norm(BlockNorm(), x, y, x)
    with pytest.raises(ValueError, match="CUDA"):
        enc.op_block_norm_backward(BlockNorm(), x, y, None, x, None, x, y, {})
    with pytest.raises(ValueError, match="CUDA"):
        Dropout(0.1, torch.zeros(2, dtype=torch.int64))


def test_the_steps_dropout_lies_on_the_steps_device():
    enc = _NoDevice()
    enc._dropout = object.__new__(Dropout)
    enc._dropout._set(device=torch.device("cuda", 1))
    tok, cu = torch.zeros(4, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="rng must be on"):
        enc.forward_train(None, tok, cu, 4, None, None)


def test_block_norm_parameters():
    g = torch.ones(8)
    with pytest.raises(ValueError, match="kind"):
        BlockNorm("batch")
    with pytest.raises(ValueError, match="post_beta needs"):
        BlockNorm(post_beta=g)
    with pytest.raises(ValueError, match="pre_beta needs"):
        BlockNorm(post_gamma=g, pre_beta=g)
    with pytest.raises(ValueError, match="1-D"):
        BlockNorm(pre_gamma=torch.ones(2, 4))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        BlockNorm(pre_gamma=g.double())
    with pytest.raises(ValueError, match="CUDA"):
        BlockNorm(post_gamma=g)
    n = BlockNorm("rms", residual_scale=0.5)
    assert (n.struct.kind, n.struct.residual_scale, n.struct.post_gamma) == (1, 0.5, None)


def test_handles_of_a_call_cannot_be_changed():
    """The structs hold addresses and values: a new value would not reach them."""
    n = BlockNorm("rms")
    with pytest.raises(AttributeError):
        n.residual_scale = 2.0
    with pytest.raises(AttributeError):
        n.pre_gamma = torch.ones(8)


def test_sizes_that_the_library_cannot_take_are_refused():
    enc = _NoDevice()
    for call in (lambda: enc.op_embed_backward_workspace(2 ** 32 + 1, 33, 8),
                 lambda: enc.op_embed_backward_workspace(1, 2.5, 8),
                 lambda: enc.op_block_norm_backward_workspace(2 ** 31, 8)):
        with pytest.raises(ValueError, match="32-bit"):
            call()
