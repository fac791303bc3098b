"""Two handles in two host threads: a call's launches must not depend on what the other thread launches
(one handle is for one thread at a time; two handles are not).

Each case makes one call on narrow rows in one thread and on wide rows in the other, some ten thousand times
on streams and buffers of their own, by the C entry points themselves (between two of them a thread then spends
little time that it does not share), and compares the results with those of the same call alone."""
import ctypes
import threading

import pytest

from tests._util import ensure_built
from transformer_esm_layer_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CALLS = 20000


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _side_by_side(made):
    """made: (function, its arguments, outputs) for each thread."""
    alone = []
    for fn, args, out in made:
        assert fn(*args) == 0
        torch.cuda.synchronize()
        alone.append([t.clone() for t in out])
        for t in out:
            t.fill_(0)
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(made)), [0] * len(made)

    def run(i):
        fn, args, _ = made[i]
        start.wait()
        for _ in range(CALLS):
            failed[i] += fn(*args) != 0

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(made)
    for (_, _, out), want in zip(made, alone):
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("precision", ["bf16", "fp32"])
@pytest.mark.parametrize("narrow,wide", [(64, 1280), (5120, 8192), (2699, 4095), (4099, 8191)])
def test_block_norm_backward(kind, precision, narrow, wide):
    from transformer_esm_layer_gb300.binding import BlockNorm, EsmBlockNormGrads, EsmEncoder
    rows, keep = 3, []

    def make(cols):
        enc = EsmEncoder.from_geometry(synth.Geometry(num_layers=1, hidden=256, heads=4, ffn=512), precision)
        g = torch.Generator(device="cuda").manual_seed(cols)
        f32 = lambda *shape: torch.randn(*shape, device="cuda", generator=g)
        act = lambda *shape: f32(*shape).to(enc.out_dtype)
        gamma = act(cols)
        norm = BlockNorm(kind, post_gamma=gamma, pre_gamma=gamma)
        x, y, x_out, h, stats = f32(rows, cols), act(rows, cols), f32(rows, cols), act(rows, cols), f32(rows, 4)
        enc.op_block_norm(norm, x, y, x_out, h, stats=stats)
        d_x, d_h, dx, dy = f32(rows, cols), act(rows, cols), f32(rows, cols), act(rows, cols)
        d_post, d_pre = f32(cols), f32(cols)
        grads = EsmBlockNormGrads(post_gamma=d_post.data_ptr(), pre_gamma=d_pre.data_ptr())
        ws, stream = enc.op_block_norm_backward_workspace(rows, cols), torch.cuda.Stream()
        keep.append((enc, norm, x_out, y, stats, d_x, d_h, grads, ws, stream))
        p = [t.data_ptr() for t in (x_out, y, stats, d_x, d_h, dx, dy)]
        args = (enc.handle, ctypes.byref(norm.struct), None, 0, None, *p, ctypes.byref(grads), rows, cols, ws.data_ptr(),
                ws.nbytes, stream.cuda_stream)
        return enc.lib.esm_op_block_norm_backward, args, [dx, dy, d_post, d_pre]

    _side_by_side([make(narrow), make(wide)])


def _head(precision, hidden, vocab, seed):
    from transformer_esm_layer_gb300.binding import DeviceLmHead, EsmEncoder
    g = synth.Geometry(num_layers=1, hidden=hidden, heads=hidden // 64, ffn=512, vocab=vocab)
    emb = synth.model_weights(g, seed, precision)["emb"]
    return EsmEncoder.from_geometry(g, precision), DeviceLmHead(synth.lm_head_weights(g, seed, precision, emb), precision)


@pytest.mark.parametrize("precision,narrow,wide", [("bf16", (256, 33), (1280, 33)), ("bf16", (512, 60), (1280, 64)),
                                                   ("fp32", (576, 20), (768, 33))])
def test_lm_head(precision, narrow, wide):
    T, keep = 5, []

    def make(hidden, vocab):
        enc, head = _head(precision, hidden, vocab, hidden)
        h = torch.randn(T, hidden, device="cuda").to(enc.out_dtype)
        logits, ws, stream = torch.zeros(T, vocab, device="cuda"), enc.lm_head_workspace(T), torch.cuda.Stream()
        keep.append((enc, head, h, ws, stream))
        args = (enc.handle, ctypes.byref(head.struct), h.data_ptr(), T, None, logits.data_ptr(), None, None, None,
                ws.data_ptr(), ws.numel(), stream.cuda_stream)
        return enc.lib.esm_encoder_lm_head, args, [logits]

    _side_by_side([make(*narrow), make(*wide)])


@pytest.mark.parametrize("narrow,wide", [(20, 33), (33, 64)])
def test_lm_head_backward(narrow, wide):
    from transformer_esm_layer_gb300.binding import LM_HEAD_NAMES, EsmLmHeadGrads
    T, keep = 5, []

    def make(vocab):
        enc, head = _head("bf16", 256, vocab, vocab)
        h = torch.randn(T, 256, device="cuda").bfloat16()
        targets = torch.arange(T, device="cuda", dtype=torch.int32)
        d_h, ws = torch.zeros(T, 256, device="cuda"), enc.lm_head_backward_workspace(T)
        grads = [torch.zeros(tuple(head.t[k].shape), device="cuda") for k in LM_HEAD_NAMES]
        gs, stream = EsmLmHeadGrads(*[t.data_ptr() for t in grads]), torch.cuda.Stream()
        keep.append((enc, head, h, targets, gs, ws, stream))
        args = (enc.handle, ctypes.byref(head.struct), h.data_ptr(), T, targets.data_ptr(), d_h.data_ptr(), ctypes.byref(gs),
                None, None, None, ws.data_ptr(), ws.numel(), stream.cuda_stream)
        return enc.lib.esm_encoder_lm_head_backward, args, [d_h, *grads]

    _side_by_side([make(narrow), make(wide)])
