"""A training step with dropout, and with a vocabulary whose gradient is summed from sorted tokens, against
torch autograd of an independent float64 formulation with the same masks.

Tolerances (relative L2), as for the step without dropout: 1e-2 for the output and 2e-2 per parameter
gradient; a block's output rows are rounded to bf16 once more (2^-9 of a term of the residual stream),
which these bounds, for some four such roundings per layer, leave room for."""
import numpy as np
import pytest

from oracle import stream as S
from tests._util import ensure_built, rel_l2, to_np
from transformer_esm_layer_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LENGTHS = [37, 130, 5, 64, 1]
SEED, BASE, OFFSET = 99, 1000, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _reference(w, tok, heads, d_out, final_ln, p, lengths=LENGTHS):
    """Output and gradients: hidden states in packed order, a dict of parameter gradients."""
    T, d = len(tok), w["emb"].shape[1]
    L = len(w["layers"])
    t = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float64)).requires_grad_()
    P = {"emb": t(w["emb"]), "lnf_g": t(w["lnf_g"]), "lnf_b": t(w["lnf_b"]),
         "layers": [{k: t(v) for k, v in wl.items()} for wl in w["layers"]]}

    def drop(x, site):
        return x if p == 0 else x * torch.from_numpy(S.dropout_factors(T, d, p, SEED, BASE, OFFSET + site))

    def norm(x, g, b):
        return torch.nn.functional.layer_norm(x, (d,), g, b, 1e-5)

    dh = d // heads
    pos = torch.cat([torch.arange(n) for n in lengths]).double()
    ang = pos[:, None] * 10000.0 ** (-torch.arange(dh // 2).double() * 2 / dh)
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]

    def rope(x):
        a, b = x[..., :dh // 2], x[..., dh // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    x = drop(P["emb"][torch.from_numpy(tok).long()], 0)
    for l, q in enumerate(P["layers"]):
        qkv = norm(x, q["ln1_g"], q["ln1_b"]) @ q["w_qkv"].T + q["b_qkv"]
        qq, kk, vv = (m.view(T, heads, dh) for m in qkv.chunk(3, 1))
        qq, kk = rope(qq), rope(kk)
        out, start = [], 0
        for n in lengths:
            i = slice(start, start + n)
            att = torch.softmax(torch.einsum("qhd,khd->hqk", qq[i], kk[i]) / dh ** 0.5, -1)
            out.append(torch.einsum("hqk,khd->qhd", att, vv[i]).reshape(n, d))
            start += n
        x = x + drop(torch.cat(out) @ q["w_o"].T + q["b_o"], 1 + 2 * l)
        u = torch.nn.functional.gelu(norm(x, q["ln2_g"], q["ln2_b"]) @ q["w_1"].T + q["b_1"])
        x = x + drop(u @ q["w_2"].T + q["b_2"], 2 + 2 * l)
    if final_ln:
        x = norm(x, P["lnf_g"], P["lnf_b"])
    x.backward(torch.from_numpy(d_out.astype(np.float64)))
    return x.detach().numpy(), P


def _setup(vocab=33, final_ln=True, layers=2):
    from transformer_esm_layer_gb300.binding import DeviceGrads, DeviceWeights, EsmEncoder, packed_inputs
    g = synth.Geometry(num_layers=layers, hidden=256, heads=4, ffn=512, vocab=vocab)
    w = synth.model_weights(g, 5, "bf16")
    tok = np.random.default_rng(6).integers(0, vocab, sum(LENGTHS)).astype(np.int32)
    d_out = np.random.default_rng(7).standard_normal((len(tok), g.hidden)).astype(np.float32)
    enc = EsmEncoder.from_geometry(g, "bf16", final_ln)
    t, cu = packed_inputs(tok, LENGTHS)
    state = dict(g=g, w=w, tok=tok, d_out=d_out, enc=enc, dw=DeviceWeights(w, "bf16"), t=t, cu=cu,
                 grads=DeviceGrads(g, layers), d=torch.from_numpy(d_out).cuda(),
                 ws=enc.workspace(len(tok), len(LENGTHS)), tb=enc.train_buffer(len(tok)))
    return state


def _step(s):
    enc = s["enc"]
    for x in s["grads"].tensors():
        x.fill_(float("nan"))
    h = enc.forward_train(s["dw"], s["t"], s["cu"], max(LENGTHS), s["tb"], s["ws"])
    enc.backward(s["dw"], s["d"], s["grads"], s["tb"], s["ws"])
    enc.check()
    return h


def _rng(base=BASE):
    return torch.tensor([SEED, base], dtype=torch.int64, device="cuda")


def _compare(s, h, P, want, final_ln):
    assert rel_l2(to_np(h), want) < 1e-2
    names = [("emb", s["grads"].emb, P["emb"])]
    if final_ln:
        names += [("lnf_g", s["grads"].lnf_g, P["lnf_g"]), ("lnf_b", s["grads"].lnf_b, P["lnf_b"])]
    for l, q in enumerate(P["layers"]):
        names += [(f"{l}.{k}", s["grads"].layers[l][k], v) for k, v in q.items()]
    for name, got, ref in names:
        assert rel_l2(to_np(got), ref.grad.numpy()) < 2e-2, name


@pytest.mark.parametrize("final_ln", [True, False])
@pytest.mark.parametrize("vocab,p", [(33, 0.1), (33, 0.5), (300, 0.1), (300, 0.0), (97, 0.0)])
def test_step_against_autograd(final_ln, vocab, p):
    from transformer_esm_layer_gb300.binding import Dropout
    s = _setup(vocab, final_ln)
    s["enc"].set_dropout(Dropout(p, _rng(), OFFSET))
    h = _step(s)
    want, P = _reference(s["w"], s["tok"], 4, s["d_out"], final_ln, p)
    _compare(s, h, P, want, final_ln)


def test_dropout_leaves_other_calls_and_can_be_taken_back():
    from transformer_esm_layer_gb300.binding import Dropout
    s = _setup()
    enc = s["enc"]
    plain = _step(s)
    grads = [x.clone() for x in s["grads"].tensors()]
    inference = enc.forward(s["dw"], s["t"], s["cu"], max(LENGTHS))
    enc.set_dropout(Dropout(0.3, _rng(), OFFSET))
    assert torch.equal(enc.forward(s["dw"], s["t"], s["cu"], max(LENGTHS)), inference)
    assert not torch.equal(_step(s), plain)
    for none in (None, Dropout(0.0, _rng()), Dropout(1e-6, _rng())):
        enc.set_dropout(Dropout(0.3, _rng(), OFFSET))
        enc.set_dropout(none)
        assert torch.equal(_step(s), plain)
        for a, b in zip(grads, s["grads"].tensors()):
            assert rel_l2(to_np(b), to_np(a)) < 1e-5  # (dq is added in arrival order)


def test_the_mask_goes_by_the_base_on_the_device():
    from transformer_esm_layer_gb300.binding import Dropout
    s = _setup()
    rng = _rng()
    s["enc"].set_dropout(Dropout(0.2, rng, OFFSET))
    first = _step(s)
    assert torch.equal(_step(s), first)
    rng[1] += 5  # 2 * 2 + 1 offsets per step
    second = _step(s)
    assert not torch.equal(second, first)
    rng[1] -= 5
    assert torch.equal(_step(s), first)


def test_captured_step_draws_new_masks():
    from transformer_esm_layer_gb300.binding import Dropout
    s = _setup()
    rng = _rng()
    s["enc"].set_dropout(Dropout(0.2, rng, OFFSET))
    out = torch.empty(len(s["tok"]), 256, dtype=torch.bfloat16, device="cuda")
    run = lambda: (s["enc"].forward_train(s["dw"], s["t"], s["cu"], max(LENGTHS), s["tb"], s["ws"], out=out),
                   s["enc"].backward(s["dw"], s["d"], s["grads"], s["tb"], s["ws"]))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for base in (BASE, BASE + 5, BASE):
        rng[1] = base
        graph.replay()
        torch.cuda.synchronize()
        got, emb = out.clone(), s["grads"].emb.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and rel_l2(to_np(s["grads"].emb), to_np(emb)) < 1e-5


def test_the_backward_uses_its_forwards_dropout():
    """Taking the dropout back between the two changes nothing for the step in hand."""
    from transformer_esm_layer_gb300.binding import Dropout
    s = _setup()
    enc = s["enc"]
    enc.set_dropout(Dropout(0.3, _rng(), OFFSET))
    _step(s)
    want = [x.clone() for x in s["grads"].tensors()]
    enc.forward_train(s["dw"], s["t"], s["cu"], max(LENGTHS), s["tb"], s["ws"])
    enc.set_dropout(None)
    enc.backward(s["dw"], s["d"], s["grads"], s["tb"], s["ws"])
    for a, b in zip(want, s["grads"].tensors()):
        assert rel_l2(to_np(b), to_np(a)) < 1e-5


@pytest.mark.parametrize("vocab", [33, 300])
@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("bad", [-1, 300])
def test_ids_out_of_range_are_reported(vocab, p, bad):
    """With a dropout as without one: -1 is no token of an encoder's step."""
    from transformer_esm_layer_gb300.binding import Dropout
    s = _setup(vocab)
    s["enc"].set_dropout(Dropout(p, _rng(), OFFSET))
    s["t"][3] = bad
    s["enc"].forward_train(s["dw"], s["t"], s["cu"], max(LENGTHS), s["tb"], s["ws"])
    assert s["enc"].check_status() == 4  # ESM_ERR_TOKEN_RANGE
    s["enc"].backward(s["dw"], s["d"], s["grads"], s["tb"], s["ws"])
    assert torch.isfinite(s["grads"].emb).all()


def test_refusals():
    import ctypes

    from transformer_esm_layer_gb300 import binding
    from transformer_esm_layer_gb300.binding import Dropout, EsmEncoder, EsmError
    g = synth.Geometry(num_layers=1, hidden=256, heads=4, ffn=512)
    enc = EsmEncoder.from_geometry(g, "bf16")
    with pytest.raises(ValueError):
        enc.set_dropout(0.1)
    for bad in (binding.EsmDropout(None, 0, 0.1), binding.EsmDropout(_rng().data_ptr(), 0, 1.5)):
        assert enc.lib.esm_encoder_set_dropout(enc.handle, ctypes.byref(bad)) == 1
    for precision in ("fp32", "fp8"):
        with pytest.raises(EsmError, match="UNSUPPORTED"):
            EsmEncoder.from_geometry(g, precision).set_dropout(Dropout(0.1, _rng()))


def _dropped(T, d, p, site, x):
    return S.dropout_factors(T, d, p, SEED, BASE, OFFSET + site) * x.astype(np.float64)


@pytest.mark.parametrize("p", [0.1, 0.5, 1.0])
def test_bias_gradients_are_sums_of_float32_rows(p):
    """Without a final LayerNorm the last block's rows get the dropped d_out itself, so the gradient of its bias
    is their sum: products by a rounded factor (two roundings each) and at most T additions of float32."""
    from transformer_esm_layer_gb300.binding import Dropout
    s = _setup(final_ln=False, layers=1)
    s["enc"].set_dropout(Dropout(p, _rng(), OFFSET))
    _step(s)
    T, d = s["d_out"].shape
    terms = _dropped(T, d, p, 2, s["d_out"])
    bound = (T + 2) * 2.0 ** -24 * np.abs(terms).sum(0)
    assert (np.abs(to_np(s["grads"].layers[0]["b_2"]) - terms.sum(0)) <= bound).all()


# The embedding's gradient goes by size: up to 256 tokens (512 of more than 64 ids) a search through them, above by
# chunks of tokens up to 64 ids, by a sort above; the latter two keep partial sums and lists in the train buffer.
LONGER = {"chunks": [300, 37, 211, 1, 402], "sort": [300, 37, 211, 1, 402, 5]}


@pytest.mark.parametrize("how,vocab,p", [("chunks", 33, 0.1), ("chunks", 64, 0.3), ("sort", 65, 0.1), ("sort", 96, 0.2),
                                         ("sort", 97, 0.0), ("sort", 300, 0.0), ("sort", 300, 0.2)])
@pytest.mark.parametrize("room", [0, 777])  # tokens that the buffers are made for beyond the batch
def test_longer_steps_against_autograd(how, vocab, p, room):
    from transformer_esm_layer_gb300.binding import DeviceGrads, DeviceWeights, Dropout, EsmEncoder, packed_inputs
    lengths = LONGER[how]
    T = sum(lengths)
    g = synth.Geometry(num_layers=1, hidden=256, heads=4, ffn=512, vocab=vocab)
    w = synth.model_weights(g, 15, "bf16")
    rng = np.random.default_rng(16)
    tok = rng.integers(0, vocab, T).astype(np.int32)
    d_out = rng.standard_normal((T, g.hidden)).astype(np.float32)
    enc = EsmEncoder.from_geometry(g, "bf16")
    enc.set_dropout(Dropout(p, _rng(), OFFSET))
    t, cu = packed_inputs(tok, lengths)
    tb = enc.train_buffer(T + room)
    guarded = torch.full((tb.numel() + 2 ** 20,), 0x5A, dtype=torch.uint8, device="cuda")
    s = dict(grads=DeviceGrads(g, 1))
    dw, ws, tb = DeviceWeights(w, "bf16"), enc.workspace(T + room, len(lengths)), guarded[:tb.numel()]
    for x in s["grads"].tensors():
        x.fill_(float("nan"))
    h = enc.forward_train(dw, t, cu, max(lengths), tb, ws)
    enc.backward(dw, torch.from_numpy(d_out).cuda(), s["grads"], tb, ws)
    enc.check()
    assert (guarded[tb.numel():] == 0x5A).all()  # nothing behind the buffer was written
    want, P = _reference(w, tok, 4, d_out, True, p, lengths)
    _compare(s, h, P, want, True)
