"""Distillation from a teacher's top logits (loss, gradient, and the head's backward from it)
against float64.

Tolerances, in steps of fp32 (2^-23): with M = max |z| / t + max |l| / t + |lse| of a row, a
logarithm or a scaled logit is off by a few steps of M and a probability by (4 + M) 2^-21
relative (scaled exponent, the hardware exponential's 2^-22, the sum), so
|loss - loss64| <= t^2 (1 + M) (8 + M) 2^-21, |lse - lse64| <= (4 + M) 2^-21 and
|g - g64| <= t / n (q + p) (4 + M) 2^-21, plus half a step of the output's type."""
import numpy as np
import pytest

from oracle import esm_oracle as O
from tests._util import ensure_built, rel_l2, to_np
from transformer_esm_layer_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SMALL = synth.Geometry(num_layers=2, hidden=256, heads=4, ffn=512)
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


@pytest.fixture(scope="module")
def enc():
    from transformer_esm_layer_gb300.binding import EsmEncoder
    return EsmEncoder.from_geometry(SMALL, "bf16")


def _case(T, V, K, dtype, seed, pad=0, offset=0):
    """logits in rows of a wider buffer (offset columns in), ids with repeats and unused entries."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = (3 * torch.randn(T, V + pad, device="cuda", generator=g)).to(dtype)
    logits = buf[:, offset:offset + V]
    ids = torch.randint(0, V, (T, K), device="cuda", generator=g, dtype=torch.int32)
    tl = 2 * torch.randn(T, K, device="cuda", generator=g)
    drop = torch.rand(T, K, device="cuda", generator=g) < 0.3
    ids[drop] = -1
    tl[torch.rand(T, K, device="cuda", generator=g) < 0.1] = -INF
    ids[::7] = -1
    return buf, logits, ids, tl


def _reference(logits, ids, tl, t):
    z, use = logits.double() / t, (ids >= 0) & (tl != -INF)
    scored = use.any(1)
    lse = z.logsumexp(1)
    a = torch.where(use, tl.double() / t, -INF)
    p = torch.where(use, (a - torch.where(scored, a.logsumexp(1), 0)[:, None]).exp(), 0)
    logq = z.gather(1, ids.long().clamp(min=0)) - lse[:, None]
    term = torch.where(p > 0, p * (p.clamp(min=1e-300).log() - logq), 0)
    loss = torch.where(scored, t * t * term.sum(1), 0)
    q = (z - lse[:, None]).exp()
    hot = torch.zeros_like(z).scatter_add_(1, ids.long().clamp(min=0), p)
    size = z.abs().masked_fill(~torch.isfinite(z), 0).amax(1) + torch.where(use, a.abs(), 0).amax(1) + lse.abs()
    return scored, loss, torch.where(scored, lse, 0), q, hot, size


def _run(enc, logits, ids, tl, t, **kw):
    T = len(logits)
    loss, lse = torch.full((2, T), float("nan"), device="cuda")
    total = torch.full((1,), float("nan"), device="cuda")
    count = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    enc.op_distill_loss(logits, ids, tl, t, loss, lse, loss_sum=total, count=count, **kw)
    return loss, lse, total, count


CASES = [(1, 1, 1, 0, 0), (5, 2, 3, 0, 0), (300, 33, 8, 0, 0), (77, 33, 33, 31, 5), (64, 64, 256, 0, 0), (9, 65, 40, 3, 1),
         (50, 255, 20, 1, 1), (33, 256, 7, 0, 0), (33, 257, 7, 0, 0), (17, 1000, 100, 24, 8), (40, 4099, 64, 0, 0),
         (3, 32000, 32, 0, 0), (2, 131071, 256, 2, 1), (2000, 40, 1, 0, 0), (1300, 700, 5, 0, 0),
         # more rows than resident blocks: a warp per row, with two and with eight entries per lane
         (1000, 300, 64, 3, 1), (900, 2049, 65, 0, 0), (700, 16000, 256, 7, 3), (650, 5000, 33, 0, 0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,K,pad,offset", CASES)
def test_loss_and_gradient_match_float64(enc, T, V, K, pad, offset, dtype):
    for t in (1.0, 2.0, 0.7):
        buf, logits, ids, tl = _case(T, V, K, dtype, T + V + K, pad, offset)
        before = buf.clone()
        loss, lse, total, count = _run(enc, logits, ids, tl, t)
        scored, rloss, rlse, q, hot, M = _reference(logits, ids, tl, t)
        assert torch.equal(buf, before)
        assert int(count) == int(scored.sum())
        assert torch.all((lse.double() - rlse).abs() <= (4 + M) * 2.0 ** -21)
        e = t * t * (1 + M) * (8 + M) * 2.0 ** -21
        assert torch.all((loss.double() - rloss).abs() <= e)
        # the losses' fp32 sum: at most 2^-24 per addition along a chain of under 100 additions
        assert abs(float(total) - float(rloss.sum())) <= float(e.sum()) + 2.0 ** -17 * float(rloss.abs().sum())
        for over in (count, None, torch.tensor([3], dtype=torch.int32, device="cuda")):
            n = 1 if over is None else int(over)
            dbuf = torch.full_like(buf, 5)
            d = dbuf[:, offset:offset + V]
            enc.op_distill_loss_backward(logits, ids, tl, t, lse, d, loss_count=over)
            rd = torch.where(scored[:, None], t / max(n, 1) * (q - hot), 0)
            bd = t / max(n, 1) * (q + hot) * (4 + M[:, None]) * 2.0 ** -21 + torch.finfo(dtype).eps / 2 * rd.abs()
            assert torch.all((d.double() - rd).abs() <= bd + 1e-38)
            assert torch.all(d[~scored] == 0)
            left = dbuf.clone()
            left[:, offset:offset + V] = 5
            assert torch.all(left == 5)     # between the rows
        # in the logits' place
        enc.op_distill_loss_backward(logits, ids, tl, t, lse, logits, loss_count=None)
        one = torch.empty(T, V, dtype=dtype, device="cuda")
        enc.op_distill_loss_backward(before[:, offset:offset + V], ids, tl, t, lse, one, loss_count=None)
        assert torch.equal(logits, one)
        assert enc.check_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,K", [(260, 64), (300, 20), (2100, 256)])
def test_gradient_in_the_logits_place_reads_the_teachers_ids_first(enc, V, K, dtype):
    """A warp per row: each lane's student logits at the teacher's ids are overwritten by other lanes."""
    T = 900
    _, logits, ids, tl = _case(T, V, K, dtype, 11)
    _, lse, _, _ = _run(enc, logits, ids, tl, 1.5)
    want = torch.empty_like(logits)
    enc.op_distill_loss_backward(logits, ids, tl, 1.5, lse, want)
    for _ in range(20):
        z = logits.clone()
        enc.op_distill_loss_backward(z, ids, tl, 1.5, lse, z)
        assert torch.equal(z, want)
    assert enc.check_status() == 0


@pytest.mark.parametrize("V", [33, 900])
def test_gradient_against_differences(enc, V):
    """Along a random direction, against central differences of the float64 loss."""
    t = 2.0
    _, logits, ids, tl = _case(20, V, 9, torch.float32, 3)
    loss, lse, total, count = _run(enc, logits, ids, tl, t)
    d = torch.empty_like(logits)
    enc.op_distill_loss_backward(logits, ids, tl, t, lse, d, loss_count=count)
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.randn(logits.shape, device="cuda", generator=g, dtype=torch.float64)
    h = 1e-5
    f = [_reference(logits.double() + s * h * u, ids, tl, t)[1].sum() / int(count) for s in (1, -1)]
    _, _, _, q, hot, M = _reference(logits, ids, tl, t)
    bound = (t / int(count) * (q + hot) * (4 + M[:, None]) * 2.0 ** -21 * u.abs()).sum() + 1e-8
    assert abs((d.double() * u).sum() - (f[0] - f[1]) / (2 * h)) <= bound


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [33, 200, 1000])
def test_masked_vocabulary_and_extreme_values(enc, V, dtype):
    """-inf and lowest values in the logits, -inf teacher entries, NaN in rows that are not scored."""
    T, K, t = 12, 4, 1.0
    low = torch.finfo(dtype).min
    logits = torch.randn(T, V, device="cuda").to(dtype)
    logits[:, V // 2:] = -INF
    logits[1, :] = low
    logits[1, 3] = 2.0
    logits[2, :] = low                      # a constant row is uniform
    logits[3, :] = float("nan")             # not scored
    logits[4, :] = -INF
    logits[4, 7] = 1.0                      # one token has all the mass
    ids = torch.arange(K, dtype=torch.int32, device="cuda").repeat(T, 1)
    tl = torch.randn(T, K, device="cuda")
    ids[3] = -1
    ids[4] = torch.tensor([7, -1, 7, 2], dtype=torch.int32)
    tl[4] = torch.tensor([0.5, float("nan"), 0.25, -INF])
    tl[1] = torch.tensor([-INF, -INF, -INF, 4.0])
    ids[5] = torch.tensor([V - 1, 0, 1, 2], dtype=torch.int32)   # the teacher wants a masked token
    loss, lse, total, count = _run(enc, logits, ids, tl, t)
    d = torch.empty_like(logits)
    enc.op_distill_loss_backward(logits, ids, tl, t, lse, d)
    assert enc.check_status() == 0
    assert int(count) == T - 1
    assert loss[3] == 0 and lse[3] == 0 and torch.all(d[3] == 0)
    assert abs(float(lse[1]) - 2.0) < 1e-5 and abs(float(loss[1])) < 1e-5
    # log V is lost beside a lowest value of 3.4e38, so only finiteness is asked of lse there
    assert torch.isfinite(lse[2])
    assert float(lse[4]) == 1.0 and abs(float(loss[4]) - float(torch.tensor([0.5, 0.25]).softmax(0).log()
                                                               @ torch.tensor([0.5, 0.25]).softmax(0))) < 1e-6
    assert torch.all(d[4] == 0) or float(d[4].abs().max()) < 1e-6
    assert float(loss[5]) == INF
    assert torch.isfinite(d[5]).all()
    rest = [0, 6, 7, 8, 9, 10, 11]
    scored, rloss, rlse, q, hot, M = _reference(logits[rest], ids[rest], tl[rest], t)
    assert torch.all((loss[rest].double() - rloss).abs() <= (1 + M) * (8 + M) * 2.0 ** -21)
    assert torch.all(d[:1, V // 2:] == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,K", [(12, 33, 4), (12, 200, 7), (12, 1000, 100), (700, 300, 40)])
@pytest.mark.parametrize("t", [0.5, 1.0, 2.0])
def test_teacher_logits_of_the_lowest_value(enc, T, V, K, dtype, t):
    """The lowest float divided by a temperature below 1 is past the type: a row of nothing else is
    uniform, beside other logits it has no weight.  The bounds of the top, with M over the others."""
    low = torch.finfo(torch.float32).min
    g = torch.Generator(device="cuda").manual_seed(T + V)
    logits = (2 * torch.randn(T, V, device="cuda", generator=g)).to(dtype)
    ids = torch.rand(T, V, device="cuda", generator=g).topk(K, dim=1).indices.to(torch.int32).contiguous()
    tl = torch.randn(T, K, device="cuda", generator=g)
    tl[::2] = low
    tl[1::4, : K // 2] = low
    ids[4, 1:] = -1
    loss, lse, total, count = _run(enc, logits, ids, tl, t)
    d = torch.empty_like(logits)
    enc.op_distill_loss_backward(logits, ids, tl, t, lse, d)
    assert enc.check_status() == 0 and int(count) == T
    shown = torch.where((tl == low).all(1, keepdim=True), 0, tl.clamp(min=-1000))
    scored, rloss, rlse, q, hot, M = _reference(logits, ids, shown, t)
    M = logits.double().abs().amax(1) / t + torch.where(shown > -1000, shown, 0).double().abs().amax(1) / t + rlse.abs()
    assert torch.all((loss.double() - rloss).abs() <= t * t * (1 + M) * (8 + M) * 2.0 ** -21)
    bd = t * (q + hot) * (4 + M[:, None]) * 2.0 ** -21 + torch.finfo(dtype).eps / 2 * (t * (q - hot)).abs()
    assert torch.all((d.double() - t * (q - hot)).abs() <= bd + 1e-38)


@pytest.mark.parametrize("V", [33, 900])
def test_extreme_temperatures(enc, V):
    """t^2 and log2(e) / t stay normal floats within the range; beyond it the call is refused."""
    from transformer_esm_layer_gb300.binding import EsmError
    _, logits, ids, tl = _case(20, V, 9, torch.float32, 12)
    for t in (1.2e-19, 1e-6, 5e18):  # (t^2 log V overflows from 7e18 on)
        loss, lse, total, count = _run(enc, logits, ids, tl, t)
        scored, rloss, rlse, q, hot, M = _reference(logits, ids, tl, t)
        assert torch.all((loss.double() - rloss).abs() <= t * t * (1 + M) * (8 + M) * 2.0 ** -21)
        assert torch.all((lse.double() - rlse).abs() <= (4 + M) * 2.0 ** -21)
        assert torch.isfinite(loss).all() and torch.isfinite(lse).all()
    d = torch.empty_like(logits)
    for t in (1e-19, 1e-30, 1.2e-38, 4e-39, 1.9e19, 1e30, 3e38):
        for call in (lambda: enc.op_distill_loss(logits, ids, tl, t, loss),
                     lambda: enc.op_distill_loss_backward(logits, ids, tl, t, lse, d)):
            with pytest.raises(EsmError) as e:
                call()
            assert e.value.status == 1
    assert enc.check_status() == 0


def test_sizes_that_32_bits_cannot_step_through_are_refused(enc):
    from transformer_esm_layer_gb300.binding import EsmError
    for T, V in ((2 ** 30, 33), (5, 2 ** 30)):
        assert enc.op_distill_loss_workspace(T, V).numel() > 0
    for T, V in ((2 ** 30 + 1, 33), (2 ** 31 - 1, 1), (5, 2 ** 30 + 1), (-1, 33), (5, 0)):
        with pytest.raises(EsmError) as e:
            enc.op_distill_loss_workspace(T, V)
        assert e.value.status == 1
    one = torch.zeros(1, 1, device="cuda")
    ids = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for T in (2 ** 30 + 1, 2 ** 32 + 1):  # (of the second the library would see one row)
        with pytest.raises(ValueError, match="30 rows"):
            enc.op_distill_loss(one.expand(T, 1), ids, one, 1.0, one[0])


def test_no_row_scored_and_no_rows(enc):
    for V in (33, 500):
        logits = torch.full((7, V), float("nan"), device="cuda")
        ids = torch.full((7, 3), -1, dtype=torch.int32, device="cuda")
        tl = torch.full((7, 3), float("nan"), device="cuda")
        loss, lse, total, count = _run(enc, logits, ids, tl, 1.0)
        assert torch.all(loss == 0) and torch.all(lse == 0) and float(total) == 0 and int(count) == 0
        d = torch.full_like(logits, 3)
        enc.op_distill_loss_backward(logits, ids, tl, 1.0, lse, d, loss_count=count)
        assert torch.all(d == 0)
        # rows are scored, but the mean is over nothing
        _, z, ids, tl = _case(7, V, 3, torch.float32, 1)
        loss, lse, _, _ = _run(enc, z, ids, tl, 1.0)
        enc.op_distill_loss_backward(z, ids, tl, 1.0, lse, d, loss_count=count)
        assert torch.all(d == 0)
        none = torch.empty(0, V, device="cuda")
        e = torch.empty(0, device="cuda")
        total.fill_(9)
        count.fill_(9)
        enc.op_distill_loss(none, ids[:0], tl[:0], 1.0, e, e, loss_sum=total, count=count)
        enc.op_distill_loss_backward(none, ids[:0], tl[:0], 1.0, e, none)
        assert float(total) == 0 and int(count) == 0
    assert enc.check_status() == 0


def test_ids_out_of_range_are_unused_and_reported(enc):
    for V in (33, 500):
        _, logits, ids, tl = _case(40, V, 6, torch.float32, 4)
        want = _run(enc, logits, ids, tl, 1.0)
        assert enc.check_status() == 0
        wild = ids.clone()
        wild[wild == -1] = V
        wild[5, 2] = -2 if ids[5, 2] == -1 else wild[5, 2]
        got = _run(enc, logits, wild, tl, 1.0)
        assert enc.check_status() == 4                    # ESM_ERR_TOKEN_RANGE
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        d, e = torch.empty_like(logits), torch.empty_like(logits)
        enc.op_distill_loss_backward(logits, ids, tl, 1.0, want[1], d)
        assert enc.check_status() == 0
        enc.op_distill_loss_backward(logits, wild, tl, 1.0, want[1], e)
        assert enc.check_status() == 4
        assert torch.equal(d, e)


def test_offsets_past_32_bits(enc):
    """66000 rows of 33000 values: 2.2e9 elements; the last rows against float64."""
    T, V, K = 66000, 33000, 4
    logits = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    logits[-50:] = torch.randn(50, V, device="cuda").to(torch.bfloat16)
    ids = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    ids[-50:] = torch.randint(0, V, (50, K), dtype=torch.int32, device="cuda")
    tl = torch.randn(T, K, device="cuda")
    loss, lse, total, count = _run(enc, logits, ids, tl, 1.0)
    assert int(count) == 50
    scored, rloss, rlse, q, hot, M = _reference(logits[-50:], ids[-50:], tl[-50:], 1.0)
    assert torch.all((loss[-50:].double() - rloss).abs() <= (1 + M) * (8 + M) * 2.0 ** -21)
    enc.op_distill_loss_backward(logits, ids, tl, 1.0, lse, logits, loss_count=count)
    rd = (q - hot) / 50
    bd = (q + hot) / 50 * (4 + M[:, None]) * 2.0 ** -21 + 2.0 ** -8 * rd.abs() + 1e-38
    assert torch.all((logits[-50:].double() - rd).abs() <= bd)
    assert torch.count_nonzero(logits[:-50]) == 0
    assert enc.check_status() == 0


def test_streams_graphs_and_repeatability(enc):
    for V in (33, 3000):
        _, logits, ids, tl = _case(3000, V, 8, torch.float32, 6)
        want = _run(enc, logits, ids, tl, 2.0)
        d = torch.empty_like(logits)
        enc.op_distill_loss_backward(logits, ids, tl, 2.0, want[1], d, loss_count=want[3])
        torch.cuda.synchronize()
        got = [torch.zeros_like(x) for x in want]
        dd = torch.zeros_like(d)
        ws = enc.op_distill_loss_workspace(3000, V)
        st = torch.cuda.Stream()
        enc.op_distill_loss(logits, ids, tl, 2.0, got[0], got[1], got[2], got[3], workspace=ws, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            enc.op_distill_loss(logits, ids, tl, 2.0, got[0], got[1], got[2], got[3], workspace=ws)
            enc.op_distill_loss_backward(logits, ids, tl, 2.0, got[1], dd, loss_count=got[3])
        for _ in range(3):
            for x in got:
                x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(dd, d)


def test_a_workspace_of_its_own_on_another_stream(enc):
    """Calls on a side stream that allocate their scratch themselves, beside work of the current
    stream that frees and reuses memory of the same sizes."""
    _, logits, ids, tl = _case(3000, 33, 8, torch.float32, 8)
    want = _run(enc, logits, ids, tl, 1.0)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[torch.zeros_like(x) for x in want] for _ in range(20)]
    torch.cuda.synchronize()
    for g in got:
        enc.op_distill_loss(logits, ids, tl, 1.0, g[0], g[1], loss_sum=g[2], count=g[3], stream=st)
        enc.op_distill_loss_workspace(3000, 33).fill_(255)
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_refusals(enc):
    from transformer_esm_layer_gb300.binding import EsmError
    _, z, ids, tl = _case(8, 40, 4, torch.float32, 7)
    loss, lse, total, count = _run(enc, z, ids, tl, 1.0)
    d = torch.empty_like(z)
    for t in (0.0, -1.0, float("nan"), INF, 1e-40):
        with pytest.raises(EsmError) as e:
            enc.op_distill_loss(z, ids, tl, t, loss)
        assert e.value.status == 1
        with pytest.raises(EsmError) as e:
            enc.op_distill_loss_backward(z, ids, tl, t, lse, d)
        assert e.value.status == 1
    with pytest.raises(EsmError) as e:
        enc.op_distill_loss(z, ids.repeat(1, 65), tl.repeat(1, 65), 1.0, loss)     # K = 260
    assert e.value.status == 1
    with pytest.raises(EsmError) as e:
        enc.op_distill_loss(z, ids[:, :0].contiguous(), tl[:, :0].contiguous(), 1.0, loss)
    assert e.value.status == 1
    with pytest.raises(EsmError) as e:
        enc.op_distill_loss(z, ids, tl, 1.0, loss, loss_sum=total, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    for args in ((z.half(), ids, tl), (z.t(), ids[:1], tl[:1]), (z, ids.long(), tl), (z, ids, tl.double()),
                 (z, ids[:4], tl), (z, ids, tl[:, :2]), (z.cpu(), ids, tl), (z, ids.cpu(), tl),
                 (z[:, ::2], ids, tl)):
        with pytest.raises(ValueError):
            enc.op_distill_loss(*args, 1.0, loss)
    wide = torch.zeros(9, 100, device="cuda")
    for zz, dd in ((wide[:8, :40], wide[:8, 39:79]), (wide[:8, 40:80], wide[:8, 1:41]), (wide[:8, :40], wide[1:, :40]),
                   (wide.view(-1)[:480].view(8, 60)[:, :40], wide[:8, :40])):
        with pytest.raises(EsmError) as e:
            enc.op_distill_loss_backward(zz, ids, tl, 1.0, lse, dd)
        assert e.value.status == 1
    wide[:8, :40] = z                                     # side by side in one buffer
    enc.op_distill_loss_backward(wide[:8, :40], ids, tl, 1.0, lse, wide[:8, 60:])
    enc.op_distill_loss_backward(z, ids, tl, 1.0, lse, d)
    assert torch.equal(wide[:8, 60:], d) and torch.equal(wide[:8, :40], z)
    for dd in (d.bfloat16(), d[:4], d.t().contiguous().t(), d.cpu()):
        with pytest.raises(ValueError):
            enc.op_distill_loss_backward(z, ids, tl, 1.0, lse, dd)
    for ws in (torch.empty(4096, dtype=torch.uint8), torch.empty(8192, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            enc.op_distill_loss(z, ids, tl, 1.0, loss, count=count, workspace=ws)
    with pytest.raises(ValueError):
        enc.op_distill_loss(z, ids, tl, 1.0, loss[:4])
    with pytest.raises(ValueError):
        enc.op_distill_loss(z, ids, tl, 1.0, loss, count=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        enc.op_distill_loss_backward(z, ids, tl, 1.0, lse, d, loss_count=torch.zeros(2, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------------- in the head
def _head_reference(h, head, ids, tl, t, n=None):
    """Gradients of the mean distillation loss through the head, by autograd in float64."""
    x = torch.from_numpy(np.asarray(h, np.float64)).requires_grad_()
    p = {k: torch.from_numpy(np.asarray(head[k], np.float64)).requires_grad_() for k in
         ("dense_w", "dense_b", "ln_g", "ln_b", "emb", "bias")}
    a = x @ p["dense_w"].T + p["dense_b"]
    u = 0.5 * a * (1 + torch.erf(a / 2 ** 0.5))
    z = (u - u.mean(1, keepdim=True)) / (u.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt() * p["ln_g"] + p["ln_b"]
    logits = z @ p["emb"].T + p["bias"]
    use = ids >= 0
    scored = use.any(1)
    w = torch.where(use, tl.double() / t, -INF)[scored].softmax(1)
    logq = (logits[scored] / t).log_softmax(1).gather(1, ids[scored].long().clamp(min=0))
    loss = t * t * (torch.xlogy(w, w) - w * logq).sum()
    (loss / (n or int(scored.sum()))).backward()
    return loss.item(), int(scored.sum()), x.grad.numpy(), {k: v.grad.numpy() for k, v in p.items()}


@pytest.mark.parametrize("T,K,n", [(1, 1, None), (200, 8, None), (333, 33, 1000)])
def test_lm_head_distill_backward(enc, T, K, n):
    """Bounds of the head's backward from the cross-entropy: 2e-2 relative L2."""
    from transformer_esm_layer_gb300.binding import DeviceLmHead
    rng = np.random.default_rng(T)
    w = synth.model_weights(SMALL, 9, "bf16")
    head = synth.lm_head_weights(SMALL, 9, "bf16", w["emb"])
    h = synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(rng.standard_normal((T, SMALL.hidden)).astype(np.float32)))
    ids = torch.from_numpy(np.argsort(rng.random((T, SMALL.vocab)), axis=1)[:, :K].astype(np.int32))
    ids[3::5] = -1
    tl = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32))
    lsum = torch.zeros(1, device="cuda")
    cnt = torch.zeros(1, dtype=torch.int32, device="cuda")
    over = None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")
    dh, g = enc.lm_head_distill_backward(DeviceLmHead(head, "bf16"), torch.from_numpy(h).cuda().bfloat16(),
                                         ids.cuda().contiguous(), tl.cuda(), 2.0, loss_sum=lsum, count=cnt,
                                         loss_count=over)
    assert enc.check_status() == 0
    loss, scored, rh, rg = _head_reference(h, head, ids, tl, 2.0, n)
    assert int(cnt) == scored
    assert abs(float(lsum) - loss) < 2e-2 * abs(loss)
    assert rel_l2(to_np(dh), rh) < 2e-2
    for k in rg:
        assert rel_l2(to_np(g[k]), rg[k]) < 2e-2, k


def test_windowed_student_learns_from_a_full_attention_teacher(monkeypatch):
    """The operators as they are used together: a full-attention teacher's top logits are taken
    from its head; a windowed student runs its training forward, the distillation loss through its
    head and its backward.  Loss and every gradient against the float64 chain."""
    from oracle import backward as B
    from tests.test_gpu_window import _oracle_window
    from transformer_esm_layer_gb300.binding import (DeviceGrads, DeviceLmHead, DeviceWeights, EsmEncoder,
                                                     packed_inputs)
    window, lengths, K, t = (24, 24, 1), [90, 33, 200], 6, 2.0
    T = sum(lengths)
    tok = synth.tokens_for_lengths(np.random.default_rng(12), lengths)
    t_tok, t_cu = packed_inputs(tok, lengths)
    tw = synth.model_weights(SMALL, 13, "bf16", ln_random=True)
    teacher = EsmEncoder.from_geometry(SMALL, "bf16")
    hidden = teacher.forward(DeviceWeights(tw, "bf16"), t_tok, t_cu, max(lengths))
    logits = torch.empty(T, SMALL.vocab, device="cuda")
    teacher.lm_head(DeviceLmHead(synth.lm_head_weights(SMALL, 13, "bf16", tw["emb"]), "bf16"), hidden, logits=logits)
    top = logits.topk(K, dim=1)
    ids, tl = top.indices.to(torch.int32).contiguous(), top.values.contiguous()
    ids[::11] = -1

    g = synth.Geometry(num_layers=1, hidden=256, heads=4, ffn=512)
    w = synth.model_weights(g, 14, "bf16", ln_random=True)
    head = synth.lm_head_weights(g, 14, "bf16", w["emb"])
    student = EsmEncoder.from_geometry(g, "bf16")
    student.set_attention_window(window)
    dw, dh = DeviceWeights(w, "bf16"), DeviceLmHead(head, "bf16")
    ws, tb = student.workspace(T, len(lengths)), student.train_buffer(T)
    out = student.forward_train(dw, t_tok, t_cu, max(lengths), tb, ws)
    lsum = torch.zeros(1, device="cuda")
    cnt = torch.zeros(1, dtype=torch.int32, device="cuda")
    d_hidden, hg = student.lm_head_distill_backward(dh, out, ids, tl, t, loss_sum=lsum, count=cnt)
    grads = DeviceGrads(g, 1)
    student.backward(dw, d_hidden, grads, tb, ws)
    assert student.check_status() == 0

    # the same numbers from the operators called one by one on the head's logits
    z = torch.empty(T, g.vocab, device="cuda")
    student.lm_head(dh, out, logits=z)
    loss, lse = torch.empty(2, T, device="cuda")
    lsum2, cnt2 = torch.zeros_like(lsum), torch.zeros_like(cnt)
    student.op_distill_loss(z, ids, tl, t, loss, lse, loss_sum=lsum2, count=cnt2)
    d = torch.empty_like(z)
    student.op_distill_loss_backward(z, ids, tl, t, lse, d, loss_count=cnt2)
    assert torch.equal(lsum, lsum2) and torch.equal(cnt, cnt2)
    # dbias = column sums of d: fp32 sums of T terms
    assert torch.all((hg["bias"].double() - d.double().sum(0)).abs() <= 2.0 ** -14 * d.double().abs().sum(0))

    _oracle_window(monkeypatch, window)
    cu = O.cu_seqlens(lengths)
    hid = O.encode_packed(tok, cu, w, g.heads)
    hid = np.concatenate([hid[i] for i in range(len(lengths))])
    rloss, n, rh, rg = _head_reference(hid, head, ids.cpu(), tl.cpu(), t)
    assert int(cnt) == n and abs(float(lsum) - rloss) < 2e-2 * rloss
    for k in rg:
        assert rel_l2(to_np(hg[k]), rg[k]) < 2e-2, k
    gref = B.encode_packed_backward(tok, cu, w, g.heads, rh)
    # the student's gradient passes through the head's roundings as well: the bounds add
    for name in B.PARAM_NAMES:
        assert rel_l2(to_np(grads.layers[0][name]), gref["layers"][0][name]) < 4e-2, name
