"""Windowed attention with sinks (forward, backward, and inside the encoder) against float64.

Tolerances are elementwise and follow from the roundings, each off by at most half a step (2^-8
relative for bf16, 2^-24 for fp32).  Forward: P is rounded to bf16 before P V and o once more, so
|o - o64| <= (2^-8 + 2^-12) sum_j p_j |v_j| + 2^-8 |o64|; the 2^-12 covers the fp32 score sums,
the scaled exponent (|t| 2^-23 with |t| < 2^7) and the hardware exponential (2^-22).  lse: fp32
sums of 64 products of size s, 2^-17 (1 + max |s|).  Backward: P and dS are rounded to bf16, dP - D
is an fp32 difference of two sums of 64 products, and P = exp(s - lse) carries |s - lse| and lse's own
errors, 2^-12 relative: E_dS = (2^-8 + 2^-12) |dS| + 2^-17 P (|dO| |V|^T + |dO| |O|), then
|d - d64| <= sum E |operand| + 2^-8 |d64| with E_P = (2^-8 + 2^-12) P for dV."""
import numpy as np
import pytest

from oracle import backward as B
from oracle import esm_oracle as O
from tests._util import ensure_built, rel_l2, to_np
from transformer_esm_layer_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SMALL = synth.Geometry(num_layers=2, hidden=256, heads=4, ffn=512)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _enc(heads=4, precision="bf16", max_positions=65536):
    from transformer_esm_layer_gb300.binding import EsmEncoder
    return EsmEncoder(1, 64 * heads, heads, 128 * heads, max_positions=max_positions, precision=precision)


def visible(L, window, n_keys=None, device="cpu", rows=None):
    """[rows, L] truth values: query i sees key j."""
    left, right, sinks = window
    i = torch.arange(L, device=device)[:, None] if rows is None else rows[:, None]
    j = torch.arange(L, device=device)[None]
    ok = (j >= i - left) | (j < sinks) if left >= 0 else torch.ones(len(i), L, dtype=torch.bool, device=device)
    if right >= 0:
        ok = ok & (j <= i + right)
    return ok if n_keys is None else ok & (j < n_keys)


def _split(x, heads):
    """[L, n * 64 * heads] -> n tensors [heads, L, 64] in float64."""
    x = x.double()
    return x.view(len(x), x.shape[1] // (64 * heads), heads, 64).permute(1, 2, 0, 3)


def _reference(qkv, lengths, heads, window):
    """o, bound of o, lse, bound of lse in float64."""
    T, d = len(qkv), 64 * heads
    o = torch.zeros(T, d, dtype=torch.float64, device=qkv.device)
    a = torch.zeros_like(o)
    lse = torch.zeros(heads, T, dtype=torch.float64, device=qkv.device)
    el = torch.zeros_like(lse)
    at = 0
    for L in lengths:
        q, k, v = _split(qkv[at:at + L], heads)
        s = q @ k.transpose(1, 2) / 8
        ok = visible(L, window, device=qkv.device)
        el[:, at:at + L] = 2.0 ** -17 * (1 + s.abs().masked_fill(~ok, 0).amax(2)) if L else 0
        s = s.masked_fill(~ok, -float("inf"))
        if L:
            lse[:, at:at + L] = s.logsumexp(2)
            p = (s - s.logsumexp(2, keepdim=True)).exp()
            o[at:at + L] = (p @ v).transpose(0, 1).reshape(L, d)
            a[at:at + L] = (p @ v.abs()).transpose(0, 1).reshape(L, d)
        at += L
    return o, (2.0 ** -8 + 2.0 ** -12) * a + 2.0 ** -8 * o.abs() + 1e-30, lse, el


def _inputs(lengths, heads, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lengths)
    qkv = (1.5 * torch.randn(T, 3 * 64 * heads, device="cuda", generator=g)).to(dtype)
    cu = torch.from_numpy(synth.cu_seqlens_from_lengths(lengths)).cuda()
    return qkv, cu, g


def _guarded(shape, dtype, extra=3):
    """A tensor at the front of a larger buffer, and the rows behind it."""
    buf = torch.full((shape[0] + extra,) + tuple(shape[1:]), 7.0, dtype=dtype, device="cuda")
    return buf[:shape[0]], buf[shape[0]:]


def _forward(enc, qkv, cu, lengths, window, heads, lse=True, **kw):
    T = len(qkv)
    o, behind = _guarded((T, 64 * heads), qkv.dtype)
    o.fill_(float("nan"))
    l = torch.full((heads, T), float("nan"), device="cuda") if lse else None
    enc.op_attention_window(qkv, cu, max(lengths), window, o, lse=l, **kw)
    assert enc.check_status() == 0
    assert torch.all(behind == 7)
    return o, l


RAGGED = [0, 1, 127, 128, 129, 300, 2, 0, 515]
WINDOWS = [(0, 0, 0), (0, 0, 5), (1, 2, 1), (16, 0, 33), (64, 64, 1), (100, 30, 100), (128, 128, 128), (200, 10, 20),
           (127, 1, 16), (-1, 0, 0), (-1, 5, 0), (3, -1, 4), (1, 70000, 17), (70000, 0, 3), (300, 300, 4)]


@pytest.mark.parametrize("window", WINDOWS)
def test_forward_matches_float64(window):
    heads = 4
    qkv, cu, _ = _inputs(RAGGED, heads, 5)
    o, lse = _forward(_enc(heads), qkv, cu, RAGGED, window, heads)
    ro, bo, rl, bl = _reference(qkv, RAGGED, heads, window)
    assert torch.all((o.double() - ro).abs() <= bo)
    assert torch.all((lse.double() - rl).abs() <= bl)


@pytest.mark.parametrize("lengths", [[1], [1] * 300, [1500], [1024, 1, 1024], [129] * 40])
@pytest.mark.parametrize("window", [(32, 32, 1), (5, 0, 2), (256, 256, 40)])
def test_forward_lengths(lengths, window):
    heads = 8
    qkv, cu, _ = _inputs(lengths, heads, 6)
    o, lse = _forward(_enc(heads), qkv, cu, lengths, window, heads)
    ro, bo, rl, bl = _reference(qkv, lengths, heads, window)
    assert torch.all((o.double() - ro).abs() <= bo)
    assert torch.all((lse.double() - rl).abs() <= bl)


def test_unlimited_window_is_full_attention():
    heads = 4
    enc = _enc(heads)
    qkv, cu, _ = _inputs(RAGGED, heads, 7)
    ref = torch.empty(len(qkv), 64 * heads, dtype=torch.bfloat16, device="cuda")
    enc.op_attention(qkv, cu, max(RAGGED), ref)
    for window in [(-1, -1, 0), (65536, 1 << 30, 0), (-1, -1, 9)]:
        o, _ = _forward(enc, qkv, cu, RAGGED, window, heads, lse=False)
        assert torch.equal(o, ref)
    # a window wider than every sequence sees the same keys (through the windowed kernel)
    o, _ = _forward(enc, qkv, cu, RAGGED, (600, 600, 0), heads, lse=False)
    _, bo, _, _ = _reference(qkv, RAGGED, heads, (-1, -1, 0))
    assert torch.all((o.double() - ref.double()).abs() <= 2 * bo)


def test_longest_sequences_at_sampled_rows():
    """Five sequences of 65536 tokens at 40 heads: 2.5e9 elements of q | k | v."""
    heads, L, B, window = 40, 65536, 5, (256, 100, 6)
    qkv, cu, _ = _inputs([L] * B, heads, 8)
    assert qkv.numel() > 2 ** 31
    o, lse = _forward(_enc(heads), qkv, cu, [L] * B, window, heads)
    x = qkv.view(B, L, 3, heads, 64)[-1]
    o, lse = o.view(B, L, heads, 64)[-1], lse.view(heads, B, L)[:, -1]
    for r in (0, 1, 255, 256, 261, 262, 263, 300, 4095, 32767, 40000, 65407, 65408, 65534, 65535):
        ok = visible(L, window, device="cuda", rows=torch.tensor([r], device="cuda"))[0]
        j = ok.nonzero().squeeze(1)
        q, k, v = x[r, 0].double(), x[j, 1].double(), x[j, 2].double()
        s = torch.einsum("hd,jhd->hj", q, k) / 8
        p = s.softmax(1)
        ro = torch.einsum("hj,jhd->hd", p, v)
        bo = (2.0 ** -8 + 2.0 ** -12) * torch.einsum("hj,jhd->hd", p, v.abs()) + 2.0 ** -8 * ro.abs()
        assert torch.all((o[r].double() - ro).abs() <= bo), r
        assert torch.all((lse[:, r].double() - s.logsumexp(1)).abs() <= 2.0 ** -17 * (1 + s.abs().amax(1))), r


@pytest.mark.parametrize("window", [(0, 0, 3), (20, 7, 2), (-1, 0, 0), (3, -1, 5)])
def test_forward_fp32(window):
    """fp32: sums of at most 300 terms of fp32 products, 2^-14 of sum p |v|."""
    heads, lengths = 4, [0, 1, 33, 300, 64]
    qkv, cu, _ = _inputs(lengths, heads, 9, torch.float32)
    o, _ = _forward(_enc(heads, "fp32"), qkv, cu, lengths, window, heads, lse=False)
    ro, bo, _, _ = _reference(qkv, lengths, heads, window)
    assert torch.all((o.double() - ro).abs() <= 2.0 ** -6 * bo)


@pytest.mark.parametrize("lengths", [[1] * 70, [7, 0, 3] * 20, [700], [31, 33, 1, 64, 65, 500], [32] * 9])
@pytest.mark.parametrize("window", [(5, 0, 2), (100, 30, 40), (0, 0, 0), (-1, 0, 0), (3, -1, 128), (2000, 64, 1)])
@pytest.mark.parametrize("heads,dh", [(4, 64), (3, 20), (8, 32), (2, 2)])
def test_forward_fp32_batches(lengths, window, heads, dh):
    """Blocks of several sequences, head sizes below 64; the bound of the test above."""
    from transformer_esm_layer_gb300.binding import EsmEncoder
    d, T = heads * dh, sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(T + heads)
    qkv = 1.5 * torch.randn(T, 3 * d, device="cuda", generator=g)
    cu = torch.from_numpy(synth.cu_seqlens_from_lengths(lengths)).cuda()
    enc = EsmEncoder(1, d, heads, 2 * d, max_positions=4096, precision="fp32")
    o, behind = _guarded((T, d), torch.float32)
    o.fill_(float("nan"))
    enc.op_attention_window(qkv, cu, max(lengths), window, o)
    assert enc.check_status() == 0 and torch.all(behind == 7)
    at = 0
    for L in lengths:
        q, k, v = qkv[at:at + L].double().view(L, 3, heads, dh).permute(1, 2, 0, 3)
        p = (q @ k.transpose(1, 2) / dh ** 0.5).masked_fill(~visible(L, window, device="cuda"), -float("inf")).softmax(2)
        ref, a = ((p @ x).transpose(0, 1).reshape(L, d) for x in (v, v.abs()))
        assert torch.all((o[at:at + L].double() - ref).abs() <= 2.0 ** -14 * (a + ref.abs()) + 1e-30)
        at += L


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_unseen_keys_and_values_have_no_influence_fp32(bad):
    heads, lengths, window = 4, [200, 150, 400], (30, 20, 2)
    qkv, cu, _ = _inputs(lengths, heads, 12, torch.float32)
    enc = _enc(heads, "fp32")
    want, _ = _forward(enc, qkv, cu, lengths, window, heads, lse=False)
    spoiled = qkv.clone()
    spoiled[[205, 450, 749], 64 * heads:] = bad
    o, _ = _forward(enc, spoiled, cu, lengths, window, heads, lse=False)
    sees = torch.zeros(len(qkv), dtype=torch.bool, device="cuda")
    start = 0
    for L in lengths:
        ok = visible(L, window, device="cuda")
        for r in (205, 450, 749):
            if start <= r < start + L:
                sees[start:start + L] |= ok[:, r - start]
        start += L
    ro, bo, _, _ = _reference(qkv, lengths, heads, window)
    assert torch.all((o[~sees].double() - ro[~sees]).abs() <= 2.0 ** -6 * bo[~sees])
    if bad != bad:
        assert torch.isnan(o[sees]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_unseen_keys_and_values_have_no_influence(bad):
    heads, lengths, window = 4, [200, 150, 400], (30, 20, 2)
    enc = _enc(heads)
    qkv, cu, _ = _inputs(lengths, heads, 10)
    spoiled = qkv.clone()
    at = [205, 450, 749]  # positions 5 of the second, 100 and 399 of the third sequence
    d = 64 * heads
    spoiled[at, d:] = bad          # k and v
    o, lse = _forward(enc, spoiled, cu, lengths, window, heads)
    ro, bo, rl, bl = _reference(qkv, lengths, heads, window)
    sees = torch.zeros(len(qkv), dtype=torch.bool, device="cuda")
    start = 0
    for L in lengths:
        ok = visible(L, window, device="cuda")
        for r in at:
            if start <= r < start + L:
                sees[start:start + L] |= ok[:, r - start]
        start += L
    assert torch.all((o[~sees].double() - ro[~sees]).abs() <= bo[~sees])
    assert torch.all((lse[:, ~sees].double() - rl[:, ~sees]).abs() <= bl[:, ~sees])
    assert not torch.isfinite(o[sees]).all(dim=1).any() or bad == float("inf")
    if bad != bad:
        assert torch.isnan(o[sees]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [(-1, -1, 0), (70000, 70000, 3), (-1, 0, 0), (3, -1, 1), (600, 600, 0)])
def test_other_sequences_have_no_influence_under_wide_windows(window, bad):
    """A sequence's last key tile reaches into the next one; nothing of that may show."""
    heads, lengths = 4, [200, 150, 400, 1, 90]
    enc = _enc(heads)
    qkv, cu, _ = _inputs(lengths, heads, 37)
    ro, bo, rl, bl = _reference(qkv, lengths, heads, window)
    d, other = 64 * heads, torch.ones(len(qkv), dtype=torch.bool, device="cuda")
    other[200:350] = False
    other[751:] = False
    spoiled = qkv.clone()
    spoiled[200:350, d:] = bad     # k and v of the second and the last sequence
    spoiled[751:, d:] = bad
    for lse in (False, True):
        o, l = _forward(enc, spoiled, cu, lengths, window, heads, lse=lse)
        assert torch.all((o[other].double() - ro[other]).abs() <= bo[other])
        if lse:
            assert torch.all((l[:, other].double() - rl[:, other]).abs() <= bl[:, other])
        if bad != bad:
            assert torch.isnan(o[~other]).all()


@pytest.mark.parametrize("precision", ["bf16", "fp32"])
def test_rows_whose_visible_scores_are_all_minus_infinity(precision):
    """A softmax over nothing but -inf is NaN; -inf beside finite scores is a weight of 0, also in a
    row that is summed again because of a NaN that it does not see."""
    heads, window = 4, (2, 0, 1)
    dt = torch.float32 if precision == "fp32" else torch.bfloat16
    lengths, d = [150, 40], 64 * heads
    qkv, cu, _ = _inputs(lengths, heads, 38, dt)
    qkv[:, :d] = qkv[:, :d].abs() + 0.1      # q > 0: a key of -inf scores -inf
    enc = _enc(heads, precision)
    gone = torch.zeros(190, dtype=torch.bool, device="cuda")
    x = qkv.clone()
    for k in (0, 60, 61, 62, 100):           # the sink too
        x[k, d:2 * d] = -float("inf")
    gone[[0, 62]] = True                     # rows that see no other key: 0 itself; 0, 60, 61 and 62
    x[120, 2 * d:] = float("nan")            # a value that most rows of its tile do not see
    nan = gone.clone()
    nan[120:123] = True
    lse = None if precision == "fp32" else torch.empty(heads, 190, device="cuda")
    o = torch.zeros(190, d, dtype=dt, device="cuda")
    enc.op_attention_window(x, cu, 150, window, o, lse=lse)
    assert enc.check_status() == 0
    assert torch.isnan(o[nan]).all() and torch.isfinite(o[~nan]).all()
    y = x.clone()
    y[120, 2 * d:] = 0
    ro, bo, rl, bl = [r.nan_to_num(nan=0.0, posinf=0.0, neginf=0.0) for r in _reference(y, lengths, heads, window)]
    ok = ~nan
    # _reference's bound of sum p |v| misses nothing here: the -inf scores have weight 0
    assert torch.all((o[ok].double() - ro[ok]).abs() <= (2.0 ** -6 if precision == "fp32" else 1) * bo[ok])
    if lse is not None:
        assert torch.all(lse[:, gone] == -float("inf"))


def test_scores_far_apart():
    """Rows whose first key tile scores far below (and far above) the later ones."""
    heads, lengths, window = 4, [700], (400, 0, 1)
    qkv, cu, _ = _inputs(lengths, heads, 11)
    d = 64 * heads
    scale = torch.linspace(0.1, 6, 700, device="cuda")[:, None]
    for s in (scale, scale.flip(0)):
        x = qkv.clone()
        x[:, d:2 * d] = (x[:, d:2 * d].float() * s).to(torch.bfloat16)
        o, lse = _forward(_enc(heads), x, cu, lengths, window, heads)
        ro, bo, rl, bl = _reference(x, lengths, heads, window)
        assert torch.all((o.double() - ro).abs() <= bo)
        assert torch.all((lse.double() - rl).abs() <= bl)


# --------------------------------------------------------------------------- backward
def _backward_reference(qkv, o, lse, d_o, lengths, heads, window):
    """dqkv and its elementwise bound in float64, from the given o and lse."""
    T = len(qkv)
    ref = torch.zeros(T, 3, heads, 64, dtype=torch.float64, device=qkv.device)
    bound = torch.zeros_like(ref)
    at = 0
    for L in lengths:
        q, k, v = _split(qkv[at:at + L], heads)
        do, oo = _split(d_o[at:at + L], heads)[0], _split(o[at:at + L], heads)[0]
        ok = visible(L, window, device=qkv.device)
        p = (q @ k.transpose(1, 2) / 8 - lse[:, at:at + L, None].double()).exp().masked_fill(~ok, 0)
        dp = do @ v.transpose(1, 2)
        D = (do * oo).sum(2, keepdim=True)
        ds = p * (dp - D)
        e = (2.0 ** -8 + 2.0 ** -12) * ds.abs() + 2.0 ** -17 * p * (do.abs() @ v.abs().transpose(1, 2)
                                                                    + (do * oo).abs().sum(2, keepdim=True))
        ep = (2.0 ** -8 + 2.0 ** -12) * p
        for n, (x, b) in enumerate([(ds @ k / 8, e @ k.abs() / 8),
                                    (ds.transpose(1, 2) @ q / 8, e.transpose(1, 2) @ q.abs() / 8),
                                    (p.transpose(1, 2) @ do, ep.transpose(1, 2) @ do.abs())]):
            ref[at:at + L, n] = x.transpose(0, 1)
            bound[at:at + L, n] = (b + 2.0 ** -8 * x.abs() + 1e-30).transpose(0, 1)
        at += L
    return ref.view(T, -1), bound.view(T, -1)


def _backward_case(lengths, window, heads, seed):
    enc = _enc(heads)
    qkv, cu, g = _inputs(lengths, heads, seed)
    o, lse = _forward(enc, qkv, cu, lengths, window, heads)
    o = o.contiguous()
    d_o = torch.randn(len(qkv), 64 * heads, device="cuda", generator=g).to(torch.bfloat16)
    dqkv, behind = _guarded(qkv.shape, torch.bfloat16)
    dqkv.fill_(float("nan"))
    enc.op_attention_window_backward(qkv, o, lse, d_o, cu, max(lengths), window, dqkv)
    assert enc.check_status() == 0
    assert torch.all(behind == 7)
    return enc, qkv, cu, o, lse, d_o, dqkv


@pytest.mark.parametrize("window", WINDOWS + [(-1, -1, 0)])
def test_backward_matches_float64(window):
    heads = 4
    _, qkv, _, o, lse, d_o, dqkv = _backward_case(RAGGED, window, heads, 21)
    ref, bound = _backward_reference(qkv, o, lse, d_o, RAGGED, heads, window)
    assert torch.all((dqkv.double() - ref).abs() <= bound)


@pytest.mark.parametrize("lengths,window", [([1], (3, 3, 1)), ([1] * 200, (0, 0, 1)), ([1024, 3, 1200], (64, 64, 1)),
                                            ([1217, 1216, 1218], (64, 64, 4)), ([3300, 70, 1300], (64, 0, 4)),
                                            ([40, 5600], (30, 17, 128)), ([2500, 2500], (1, 1, 1))])
def test_backward_lengths_and_distant_sinks(lengths, window):
    """Sinks are seen from the whole sequence: past some length their gradients are summed from
    parts (from 1153 + left tokens on, in parts of 2048 queries)."""
    heads = 4
    _, qkv, _, o, lse, d_o, dqkv = _backward_case(lengths, window, heads, 22)
    ref, bound = _backward_reference(qkv, o, lse, d_o, lengths, heads, window)
    assert torch.all((dqkv.double() - ref).abs() <= bound)


@pytest.mark.parametrize("window", [(64, 64, 5), (30, 0, 33), (16, 16, 127)])
@pytest.mark.parametrize("lengths", [[1300, 17, 33, 1], [5, 1477, 61], [3, 31, 65, 97]])
def test_backward_of_key_tiles_that_part_a_warp(lengths, window):
    """Warps whose lanes hold sinks (fp32 partial sums), other keys, and rows behind the tile's last."""
    heads = 4
    _, qkv, _, o, lse, d_o, dqkv = _backward_case(lengths, window, heads, 39)
    ref, bound = _backward_reference(qkv, o, lse, d_o, lengths, heads, window)
    assert torch.all((dqkv.double() - ref).abs() <= bound)


def test_backward_against_differences():
    """dL/dx along a random direction, L = sum(o64 * d_o), by central differences in float64:
    the directional derivative of the kernel's gradient within its summed bound."""
    heads, lengths, window = 4, [150, 40], (12, 5, 3)
    _, qkv, _, o, lse, d_o, dqkv = _backward_case(lengths, window, heads, 23)
    ref, bound = _backward_reference(qkv, o, lse, d_o, lengths, heads, window)
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn(qkv.shape, device="cuda", generator=g, dtype=torch.float64)
    h = 1e-5
    f = [(_reference(qkv.double() + s * h * u, lengths, heads, window)[0] * d_o.double()).sum() for s in (1, -1)]
    diff = (f[0] - f[1]) / (2 * h)
    # o is rounded to bf16 before D = rowsum(dO * O): D moves by up to 2^-8 sum |dO o|
    slack = 2.0 ** -8 * (d_o.double() * o.double()).abs().sum() * qkv.double().abs().max()
    assert abs((dqkv.double() * u).sum() - diff) <= (bound * u.abs()).sum() + slack


def test_backward_of_scores_far_apart():
    """Scores of up to about +-100 (lse of that size enters the exponent as a sum of three bf16)."""
    heads, lengths, window = 4, [500, 130], (200, 10, 2)
    enc = _enc(heads)
    qkv, cu, g = _inputs(lengths, heads, 25)
    d = 64 * heads
    scale = torch.linspace(0.1, 8, len(qkv), device="cuda")[:, None]
    for s in (scale, scale.flip(0)):
        x = qkv.clone()
        x[:, d:2 * d] = (x[:, d:2 * d].float() * s).to(torch.bfloat16)
        o, lse = _forward(enc, x, cu, lengths, window, heads)
        o = o.contiguous()
        d_o = torch.randn(len(x), d, device="cuda", generator=g).to(torch.bfloat16)
        dqkv = torch.empty_like(x)
        enc.op_attention_window_backward(x, o, lse, d_o, cu, max(lengths), window, dqkv)
        ref, bound = _backward_reference(x, o, lse, d_o, lengths, heads, window)
        assert torch.all((dqkv.double() - ref).abs() <= bound)
    assert enc.check_status() == 0


@pytest.mark.parametrize("B", [1, 31, 32, 33, 300])
def test_small_batches_with_and_without_a_work_list(B):
    """Batches whose items are found from the offsets (up to 32 sequences and one item per block), and
    their neighbours that go by the work list."""
    heads, window = 4, (9, 3, 2)
    lengths = [(7 * i) % 61 for i in range(B)]
    lengths[-1] = 190
    enc = _enc(heads)
    qkv, cu, _ = _inputs(lengths, heads, 26)
    o, lse = _forward(enc, qkv, cu, lengths, window, heads)
    ro, bo, rl, bl = _reference(qkv, lengths, heads, window)
    assert torch.all((o.double() - ro).abs() <= bo)
    assert torch.all((lse.double() - rl).abs() <= bl)


@pytest.mark.parametrize("B", [257, 1024, 1500])
def test_many_sequences(B):
    """More sequences than a block of the work list's kernels has threads, in both directions."""
    heads, window = 4, (40, 20, 1)
    lengths = [(11 * i) % 37 for i in range(B)]
    lengths[B // 2] = 700
    _, qkv, _, o, lse, d_o, dqkv = _backward_case(lengths, window, heads, 27)
    ro, bo, _, _ = _reference(qkv, lengths, heads, window)
    assert torch.all((o.double() - ro).abs() <= bo)
    ref, bound = _backward_reference(qkv, o, lse, d_o, lengths, heads, window)
    assert torch.all((dqkv.double() - ref).abs() <= bound)


@pytest.mark.parametrize("heads", [4, 12, 20])
def test_outputs_off_32_bytes(heads):
    """o, dqkv 16-byte but not 32-byte aligned."""
    lengths, window = [150, 70], (30, 30, 1)
    enc = _enc(heads)
    qkv, cu, g = _inputs(lengths, heads, 28)
    T, d = len(qkv), 64 * heads
    want, lse = _forward(enc, qkv, cu, lengths, window, heads)
    o = torch.empty(T * d + 8, dtype=torch.bfloat16, device="cuda")[8:].view(T, d)
    enc.op_attention_window(qkv, cu, 150, window, o)
    assert torch.equal(o, want)
    d_o = torch.randn(T, d, device="cuda", generator=g).to(torch.bfloat16)
    a = torch.empty_like(qkv)
    b = torch.empty(T * 3 * d + 8, dtype=torch.bfloat16, device="cuda")[8:].view(T, 3 * d)
    for out in (a, b):
        enc.op_attention_window_backward(qkv, o, lse, d_o, cu, 150, window, out)
    assert torch.equal(a[:, d:], b[:, d:])
    assert enc.check_status() == 0


def test_backward_is_repeatable_but_for_dq():
    heads, lengths, window = 4, [3000, 500], (100, 100, 4)
    enc, qkv, cu, o, lse, d_o, dqkv = _backward_case(lengths, window, heads, 24)
    again = torch.empty_like(dqkv)
    enc.op_attention_window_backward(qkv, o, lse, d_o, cu, max(lengths), window, again)
    assert torch.equal(again[:, 256:], dqkv[:, 256:])


def test_backward_of_the_longest_sequences_at_sampled_rows():
    """Five sequences of 65536 tokens at 40 heads: gradients past 2^31 elements, and sinks that 65536
    queries see (their bound is that of _backward_reference, over one key's queries)."""
    heads, L, B, window = 40, 65536, 5, (256, 100, 6)
    enc = _enc(heads)
    qkv, cu, g = _inputs([L] * B, heads, 29)
    o = torch.empty(len(qkv), 64 * heads, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(heads, len(qkv), device="cuda")
    enc.op_attention_window(qkv, cu, L, window, o, lse=lse)
    d_o = torch.randn(len(qkv), 64 * heads, device="cuda", generator=g, dtype=torch.bfloat16)
    dqkv = torch.empty_like(qkv)
    enc.op_attention_window_backward(qkv, o, lse, d_o, cu, L, window, dqkv)
    assert enc.check_status() == 0
    x, grad = qkv.view(B, L, 3, heads, 64)[-1], dqkv.view(B, L, 3, heads, 64)[-1]
    oo, do, ll = o.view(B, L, heads, 64)[-1], d_o.view(B, L, heads, 64)[-1], lse.view(heads, B, L)[:, -1]

    def pairs(i, j):
        """P, dS and the bound of dS for one query and its keys, or one key and its queries: [n, heads]."""
        q, k, v, dd = x[i, 0].double(), x[j, 1].double(), x[j, 2].double(), do[i].double()
        p = ((q * k).sum(-1) / 8 - ll.t()[i].double()).exp()
        ds = p * ((dd * v).sum(-1) - (dd * oo[i].double()).sum(-1))
        size = (dd.abs() * v.abs()).sum(-1) + (dd * oo[i].double()).abs().sum(-1)
        return p, ds, (2.0 ** -8 + 2.0 ** -12) * ds.abs() + 2.0 ** -17 * p * size, q, k, dd

    def check(got, w, e, other):
        ref = (w[..., None] * other).sum(0)
        assert torch.all((got.double() - ref).abs() <= (e[..., None] * other.abs()).sum(0) + 2.0 ** -8 * ref.abs() + 1e-30)

    for r in (0, 5, 6, 300, 1383, 1384, 3431, 3432, 40000, 65407, 65408, 65535):
        t = torch.tensor([r], device="cuda")
        j = visible(L, window, device="cuda", rows=t)[0].nonzero().squeeze(1)
        p, ds, e, _, k, _ = pairs(t, j)
        check(grad[r, 0], ds / 8, e / 8, k)
        lo = 0 if window[1] >= r else r - window[1]
        hi = L if r < window[2] else min(L, r + window[0] + 1)
        p, ds, e, q, _, dd = pairs(torch.arange(lo, hi, device="cuda"), t)
        check(grad[r, 1], ds / 8, e / 8, q)
        check(grad[r, 2], p, (2.0 ** -8 + 2.0 ** -12) * p, dd)


# --------------------------------------------------------------------------- calls
def test_other_stream_graph_replay_and_two_workspaces():
    heads, lengths, window = 4, [300, 77, 129], (40, 40, 2)
    enc = _enc(heads)
    qkv, cu, g = _inputs(lengths, heads, 31)
    want, lse = _forward(enc, qkv, cu, lengths, window, heads)
    want = want.clone()
    d_o = torch.randn(len(qkv), 256, device="cuda", generator=g).to(torch.bfloat16)
    dref = torch.empty_like(qkv)
    enc.op_attention_window_backward(qkv, want, lse, d_o, cu, 300, window, dref)
    torch.cuda.synchronize()
    ws = [enc.op_attention_window_workspace(len(qkv), 3, window) for _ in range(2)]
    wb = enc.op_attention_window_workspace(len(qkv), 3, window, backward=True)
    outs = [torch.zeros_like(want) for _ in range(2)]
    lses = [torch.zeros_like(lse) for _ in range(2)]
    dq = torch.zeros_like(qkv)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, w, o, l in zip(streams, ws, outs, lses):  # at once, each with its own workspace
        enc.op_attention_window(qkv, cu, 300, window, o, lse=l, workspace=w, stream=st)
    torch.cuda.synchronize()
    for o, l in zip(outs, lses):
        assert torch.equal(o, want) and torch.equal(l, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        enc.op_attention_window(qkv, cu, 300, window, outs[0], lse=lses[0], workspace=ws[0])
        enc.op_attention_window_backward(qkv, outs[0], lses[0], d_o, cu, 300, window, dq, workspace=wb)
    for k in range(3):
        outs[0].zero_()
        dq.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want)
        assert torch.equal(dq[:, 256:], dref[:, 256:])
    # new values and offsets in the captured buffers
    other, _, _ = _inputs(lengths, heads, 32)
    qkv.copy_(other)
    cu.copy_(torch.tensor([0, 5, 206, 506], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ro, bo, _, _ = _reference(qkv, [5, 201, 300], heads, window)
    assert torch.all((outs[0].double() - ro).abs() <= bo)
    assert enc.check_status() == 0


def test_malformed_offsets_are_reported_and_stay_in_bounds():
    heads = 4
    enc = _enc(heads)
    qkv, _, _ = _inputs([400], heads, 33)
    for cu in ([0, 300, 200, 400], [5, 400], [0, 399], [-3, 100, 400], [0, 500, 400], [0, 100, 400]):
        off = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, behind = _guarded((400, 256), torch.bfloat16)
        lse = torch.zeros(heads, 400, device="cuda")
        enc.op_attention_window(qkv, off, 250, (20, 20, 3), o, lse=lse)
        assert enc.check_status() == 3
        assert torch.all(behind == 7)
        dq, behind = _guarded((400, 768), torch.bfloat16)
        enc.op_attention_window_backward(qkv, o.contiguous(), lse, o.contiguous(), off, 250, (20, 20, 3), dq)
        assert enc.check_status() == 3
        assert torch.all(behind == 7)
    ok = torch.tensor([0, 200, 400], dtype=torch.int32, device="cuda")
    enc.op_attention_window(qkv, ok, 250, (20, 20, 3), o)
    assert enc.check_status() == 0


@pytest.mark.parametrize("window", [(20, 20, 3), (-1, 0, 0)])
@pytest.mark.parametrize("cu", [[0, 1024, 0, 1024], [0, 1024, 0, 1024, 0, 1024, 0, 1024]])
def test_overlapping_offsets_in_a_small_batch_stay_in_bounds(cu, window):
    """More tiles than an honest batch of this size can have, found from the offsets."""
    heads, T = 4, 1024
    enc = _enc(heads)
    qkv, _, _ = _inputs([T], heads, 35)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, behind = _guarded((T, 256), torch.bfloat16)
    lse, lse_behind = _guarded((heads, T), torch.float32)
    for _ in range(2):
        enc.op_attention_window(qkv, off, T, window, o, lse=lse)
        assert enc.check_status() == 3
        assert torch.all(behind == 7) and torch.all(lse_behind == 7)
    ok = torch.tensor([0, 400, T], dtype=torch.int32, device="cuda")
    enc.op_attention_window(qkv, ok, T, window, o, lse=lse)
    assert enc.check_status() == 0
    ro, bo, rl, bl = _reference(qkv, [400, 624], heads, window)
    assert torch.all((o.double() - ro).abs() <= bo)
    assert torch.all((lse.double() - rl).abs() <= bl)


@pytest.mark.parametrize("window", [(20, 20, 3), (-1, 0, 0)])
@pytest.mark.parametrize("cu", [[0, 2048] * 4, [0, 2048] * 40])
def test_overlapping_offsets_in_a_work_list_stay_in_bounds(cu, window):
    """More tiles than the list has room for; 40 pairs of offsets are past what the forward finds
    without a list."""
    heads, T = 4, 2048
    enc = _enc(heads)
    qkv, _, g = _inputs([T], heads, 36)
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, behind = _guarded((T, 256), torch.bfloat16)
    lse, lse_behind = _guarded((heads, T), torch.float32)
    enc.op_attention_window(qkv, off, T, window, o, lse=lse)
    assert enc.check_status() == 3
    assert torch.all(behind == 7) and torch.all(lse_behind == 7)
    d_o = torch.randn(T, 256, device="cuda", generator=g).to(torch.bfloat16)
    dq, behind = _guarded((T, 768), torch.bfloat16)
    enc.op_attention_window_backward(qkv, d_o, torch.zeros_like(lse), d_o, off, T, window, dq)
    assert enc.check_status() == 3
    assert torch.all(behind == 7)
    ok = torch.tensor([0, 900, T], dtype=torch.int32, device="cuda")
    enc.op_attention_window(qkv, ok, T, window, o, lse=lse)
    o = o.contiguous()
    enc.op_attention_window_backward(qkv, o, lse, d_o, ok, T, window, dq)
    assert enc.check_status() == 0
    ref, bound = _backward_reference(qkv, o, lse, d_o, [900, 1148], heads, window)
    assert torch.all((dq.double() - ref).abs() <= bound)


def test_refusals():
    from transformer_esm_layer_gb300.binding import EsmError
    heads = 4
    enc = _enc(heads, max_positions=512)
    qkv, cu, _ = _inputs([300], heads, 34)
    o = torch.empty(300, 256, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(heads, 300, device="cuda")
    for window in ((-2, 0, 0), (0, -2, 0), (1, 1, -1), (1, 1, 129)):
        with pytest.raises(EsmError) as e:
            enc.op_attention_window(qkv, cu, 300, window, o)
        assert e.value.status == 1
        with pytest.raises(EsmError):
            enc.set_attention_window(window)
    for n in (0, 513):
        with pytest.raises(EsmError) as e:
            enc.op_attention_window(qkv, cu, n, (1, 1, 0), o)
        assert e.value.status == 1
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(EsmError) as e:
        enc.op_attention_window(qkv, cu, 300, (1, 1, 0), o, workspace=small)
    assert e.value.status == 5
    with pytest.raises(EsmError) as e:  # the forward's workspace is too small for the backward
        enc.op_attention_window_backward(qkv, o, lse, o, cu, 300, (1, 1, 0), torch.empty_like(qkv),
                                         workspace=enc.op_attention_window_workspace(300, 1, (1, 1, 0)))
    assert e.value.status == 5
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 21, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            enc.op_attention_window(qkv, cu, 300, (1, 1, 0), o, workspace=ws)
    for bad in (dict(o=o.float()), dict(o=o[:299]), dict(o=o.t().contiguous().t()), dict(lse=lse.double()),
                dict(lse=lse.t().contiguous()), dict(o=o.cpu())):
        args = dict(o=o, lse=lse)
        args.update(bad)
        with pytest.raises(ValueError):
            enc.op_attention_window(qkv, cu, 300, (1, 1, 0), args["o"], lse=args["lse"])
    buf = torch.zeros(300 * 4 * 256, dtype=torch.bfloat16, device="cuda")   # outputs over inputs
    inside = buf[:300 * 768].view(300, 768)
    with pytest.raises(EsmError) as e:
        enc.op_attention_window(inside, cu, 300, (1, 1, 0), buf[300 * 767:300 * 767 + 300 * 256].view(300, 256))
    assert e.value.status == 1
    with pytest.raises(EsmError) as e:
        enc.op_attention_window_backward(qkv, o, lse, o, cu, 300, (1, 1, 0), qkv)
    assert e.value.status == 1
    with pytest.raises(EsmError) as e:
        enc.op_attention_window_backward(qkv, o, lse, buf[256 * 8:256 * 308].view(300, 256), cu, 300, (1, 1, 0), inside)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        enc.op_attention_window(qkv[:, :-1], cu, 300, (1, 1, 0), o)
    with pytest.raises(ValueError):
        enc.op_attention_window(qkv, cu.long(), 300, (1, 1, 0), o)
    with pytest.raises(ValueError):
        enc.op_attention_window_backward(qkv, o, lse, o, cu, 300, (1, 1, 0), torch.empty(300, 256, device="cuda"))
    f32 = _enc(heads, "fp32", 512)
    with pytest.raises(EsmError) as e:
        f32.op_attention_window(qkv.float(), cu, 300, (1, 1, 0), o.float(), lse=lse)
    assert e.value.status == 2
    with pytest.raises(EsmError) as e:
        f32.op_attention_window_workspace(300, 1, (1, 1, 0), backward=True)
    assert e.value.status == 2
    empty = torch.empty(0, 768, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    enc.op_attention_window(empty, zero, 1, (1, 1, 0), empty[:, :256].contiguous())
    assert enc.check_status() == 0


# --------------------------------------------------------------------------- in the encoder
def _oracle_window(monkeypatch, window):
    """The oracle's attention (and its gradient) under a window."""
    def mask(L, n_keys=None):
        return visible(L, window, n_keys).numpy()

    def attention(q, k, v, n_keys=None):
        s = np.einsum("ihd,jhd->hij", q, k) / 8
        ok = mask(len(q), n_keys)
        s = np.where(ok, s, -np.inf)
        m = s.max(-1, keepdims=True)
        p = np.where(ok, np.exp(s - np.where(np.isfinite(m), m, 0)), 0)
        l = p.sum(-1, keepdims=True)
        return np.einsum("hij,jhd->ihd", p / np.where(l > 0, l, 1), v)

    def attention_backward(q, k, v, do):
        s = np.where(mask(len(q)), np.einsum("ihd,jhd->hij", q, k) / 8, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        dp = np.einsum("ihd,jhd->hij", do, v)
        ds = p * (dp - (p * dp).sum(-1, keepdims=True))
        return (np.einsum("hij,jhd->ihd", ds, k) / 8, np.einsum("hij,ihd->jhd", ds, q) / 8,
                np.einsum("hij,ihd->jhd", p, do))

    monkeypatch.setattr(O, "attention", attention)
    monkeypatch.setattr(B, "attention", attention)
    monkeypatch.setattr(B, "attention_backward", attention_backward)


@pytest.mark.parametrize("precision,window,bound", [("bf16", (20, 20, 1), 1e-2), ("bf16", (50, 0, 4), 1e-2),
                                                    ("fp32", (20, 20, 1), 1e-4), ("fp32", (-1, 0, 0), 1e-4)])
def test_encoder_forward_under_a_window(monkeypatch, precision, window, bound):
    """The bounds are those of the full-attention forward."""
    from transformer_esm_layer_gb300.binding import DeviceWeights, EsmEncoder, packed_inputs
    lengths = [90, 1, 33, 300]
    w = synth.model_weights(SMALL, 3, precision, ln_random=True)
    tok = synth.tokens_for_lengths(np.random.default_rng(3), lengths)
    enc = EsmEncoder.from_geometry(SMALL, precision)
    dw = DeviceWeights(w, precision)
    t, cu = packed_inputs(tok, lengths)
    full = to_np(enc.forward(dw, t, cu, 300, check=True))
    enc.set_attention_window(window)
    got = to_np(enc.forward(dw, t, cu, 300, check=True))
    host = [torch.from_numpy(a).pin_memory() for a in (tok, synth.cu_seqlens_from_lengths(lengths))]
    hout = torch.empty(len(tok), SMALL.hidden, dtype=torch.int16 if precision == "bf16" else torch.float32).pin_memory()
    ws = enc.workspace(len(tok), len(lengths))

    def from_host():
        enc.forward_host(dw, host[0].numpy(), host[1].numpy(), 300, hout.numpy(), ws)
        return to_np(hout.view(torch.bfloat16) if precision == "bf16" else hout)

    for _ in range(3):  # eager, captured, replayed
        assert np.array_equal(from_host(), got)
    enc.set_attention_window(None)
    assert np.array_equal(to_np(enc.forward(dw, t, cu, 300, check=True)), full)
    assert np.array_equal(from_host(), full)     # not the graph of the windowed call
    _oracle_window(monkeypatch, window)
    ref = O.encode_packed(tok, O.cu_seqlens(lengths), w, SMALL.heads)
    ref = np.concatenate([ref[i] for i in range(len(lengths))])
    assert rel_l2(got, ref) < bound
    assert rel_l2(full, ref) > 2 * bound         # the window matters


def test_padded_forward_under_a_window(monkeypatch):
    """Padding queries far behind the last key see nothing; the real rows are the packed ones."""
    from transformer_esm_layer_gb300.binding import DeviceWeights, EsmEncoder
    lengths, S, window = [70, 1, 200, 129], 384, (20, 20, 1)
    w = synth.model_weights(SMALL, 4, "bf16", ln_random=True)
    tok = synth.tokens_for_lengths(np.random.default_rng(4), lengths)
    dw = DeviceWeights(w, "bf16")
    padded = torch.from_numpy(synth.pad_tokens(tok, lengths, S)).cuda()
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for win in (window, (20, 20, 0)):
        enc = EsmEncoder.from_geometry(SMALL, "bf16")
        enc.set_attention_window(win)
        out = to_np(enc.forward_padded(dw, padded, lens, check=True))
        with monkeypatch.context() as m:
            _oracle_window(m, win)
            ref = O.encode_padded(padded.cpu().numpy(), lengths, w, SMALL.heads)
        for b, L in enumerate(lengths):
            assert rel_l2(out[b, :L], ref[b][:L]) < 1e-2
            assert np.all(out[b, L:] == 0)


@pytest.mark.parametrize("layers", [("fp8", "bf16"), ("fp4", "fp8")])
def test_fp8_encoder_under_a_window(monkeypatch, layers):
    """FP8 and FP4 layers take their attention output quantised or with its amax from the kernel.
    With the attention windowed in both, the encoder is as far from the bf16 one as without."""
    from transformer_esm_layer_gb300.binding import DeviceWeights, EsmEncoder
    lengths, S = [300, 1, 129, 64], 320
    g = synth.Geometry(num_layers=2, hidden=256, heads=4, ffn=512)
    w = synth.model_weights(g, 5, "bf16", ln_random=True)
    tok = synth.tokens_for_lengths(np.random.default_rng(5), lengths)
    dw = DeviceWeights(w, "bf16")
    padded = torch.from_numpy(synth.pad_tokens(tok, lengths, S)).cuda()
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    far = {}
    for window in (None, (10, 10, 1)):
        outs = {}
        for precision in ("bf16", "fp8"):
            enc = EsmEncoder.from_geometry(g, precision)
            if precision == "fp8":
                enc.set_layer_precision(layers)
            enc.set_attention_window(window)
            for _ in range(4):  # the delayed scales settle
                out = enc.forward_padded(dw, padded, lens, check=True)
            outs[precision] = to_np(out)
        assert np.isfinite(outs["fp8"]).all()
        far[window] = rel_l2(outs["fp8"], outs["bf16"])
    assert far[(10, 10, 1)] < 1.5 * far[None]


@pytest.mark.parametrize("window", [(20, 20, 1), (40, 0, 3), (-1, 0, 0)])
def test_training_step_under_a_window(monkeypatch, window):
    """forward_train and backward against the oracle's chain; 2e-2 as for full attention."""
    from transformer_esm_layer_gb300.binding import DeviceGrads, DeviceWeights, EsmEncoder, packed_inputs
    lengths = [90, 1, 33, 260]
    rng = np.random.default_rng(6)
    w = synth.model_weights(SMALL, 6, "bf16", ln_random=True)
    tok = synth.tokens_for_lengths(rng, lengths)
    T = len(tok)
    enc = EsmEncoder.from_geometry(SMALL, "bf16")
    enc.set_attention_window(window)
    dw = DeviceWeights(w, "bf16")
    t, cu = packed_inputs(tok, lengths)
    ws, tb = enc.workspace(T, len(lengths)), enc.train_buffer(T)
    out = enc.forward_train(dw, t, cu, max(lengths), tb, ws)
    d_out = rng.standard_normal((T, SMALL.hidden)).astype(np.float32)
    grads = DeviceGrads(SMALL, SMALL.num_layers)
    enc.set_attention_window(None)  # the backward goes by its forward's window
    enc.backward(dw, torch.from_numpy(d_out).cuda(), grads, tb, ws)
    assert enc.check_status() == 0
    _oracle_window(monkeypatch, window)
    c = O.cu_seqlens(lengths)
    ref = O.encode_packed(tok, c, w, SMALL.heads)
    assert rel_l2(to_np(out), np.concatenate([ref[i] for i in range(len(lengths))])) < 1e-2
    gref = B.encode_packed_backward(tok, c, w, SMALL.heads, d_out.astype(np.float64))
    assert rel_l2(to_np(grads.emb), gref["emb"]) < 2e-2
    for l in range(SMALL.num_layers):
        for n in B.PARAM_NAMES:
            assert rel_l2(to_np(grads.layers[l][n]), gref["layers"][l][n]) < 2e-2, (l, n)


def test_training_step_of_a_long_sequence_with_distant_sinks(monkeypatch):
    """Sink gradients in parts, turned back through RoPE (one layer, 1500 tokens)."""
    from transformer_esm_layer_gb300.binding import DeviceGrads, DeviceWeights, EsmEncoder, packed_inputs
    g = synth.Geometry(num_layers=1, hidden=256, heads=4, ffn=256, max_positions=2048)
    lengths, window = [1500, 20], (16, 16, 3)
    rng = np.random.default_rng(8)
    w = synth.model_weights(g, 8, "bf16", ln_random=True)
    tok = synth.tokens_for_lengths(rng, lengths)
    T = len(tok)
    enc = EsmEncoder.from_geometry(g, "bf16")
    short = enc.train_buffer(T)
    enc.set_attention_window(window)
    dw = DeviceWeights(w, "bf16")
    t, cu = packed_inputs(tok, lengths)
    ws, tb = enc.workspace(T, len(lengths)), enc.train_buffer(T)
    assert tb.numel() > short.numel()
    from transformer_esm_layer_gb300.binding import EsmError
    with pytest.raises(EsmError) as e:  # sized without the window
        enc.forward_train(dw, t, cu, max(lengths), short, ws)
    assert e.value.status == 5
    enc.forward_train(dw, t, cu, max(lengths), tb, ws)
    d_out = rng.standard_normal((T, g.hidden)).astype(np.float32)
    grads = DeviceGrads(g, 1)
    enc.backward(dw, torch.from_numpy(d_out).cuda(), grads, tb, ws)
    assert enc.check_status() == 0
    _oracle_window(monkeypatch, window)
    gref = B.encode_packed_backward(tok, O.cu_seqlens(lengths), w, g.heads, d_out.astype(np.float64))
    for n in B.PARAM_NAMES:
        assert rel_l2(to_np(grads.layers[0][n]), gref["layers"][0][n]) < 2e-2, n
