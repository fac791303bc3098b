"""Dropout, scaled embedding and block norms, forward and backward, against float64.

Tolerances, with u = 2^-24 (half a step of fp32) and half a step of the output's type on top:
  * a product of k fp32 factors and sums is off by at most (number of roundings) u of the same formula
    with every term's magnitude in place of the term;
  * a sum of n terms in any order is off by at most (n - 1) u of the sum of magnitudes; a row's sums run
    over at most 40 values in a lane, 5 exchanges in a warp and 32 warps: D = 80 roundings;
  * the forward's norms are followed step by step (_norm_bound): mean, deviations, variance, 1 / root
    (rsqrtf: 2 steps = 4 u), and the affine map.
"""
import numpy as np
import pytest

from oracle import stream as S
from tests._util import ensure_built, to_np
from transformer_esm_layer_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SMALL = synth.Geometry(num_layers=1, hidden=256, heads=4, ffn=512)
U = 2.0 ** -24
D = 80
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF16, F32 = torch.bfloat16, torch.float32
SEED, BASE = 0x1234_5678_9ABC_DEF0, 2 ** 63 - 2  # base + offset runs past the signed 64 bits


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


@pytest.fixture(scope="module")
def encs():
    from transformer_esm_layer_gb300.binding import EsmEncoder
    return {BF16: EsmEncoder.from_geometry(SMALL, "bf16"), F32: EsmEncoder.from_geometry(SMALL, "fp32")}


@pytest.fixture(scope="module")
def enc(encs):
    return encs[BF16]


def _rng(seed=SEED, base=BASE):
    return torch.tensor([seed, base], dtype=torch.int64, device="cuda")


def _drop(p, offset=5, rng=None):
    from transformer_esm_layer_gb300.binding import Dropout
    return Dropout(p, _rng() if rng is None else rng, offset) if p is not None else None


def _factors(rows, cols, p, offset=5, seed=SEED, base=BASE):
    n = rows if np.ndim(rows) == 0 else len(rows)
    return np.ones((n, cols)) if p is None else S.dropout_factors(rows, cols, p, seed, base, offset)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32):
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def _within(got, want, bound, dtype=F32):
    """Element by element: |got - want| <= bound + half a step of the type."""
    got, want = to_np(got), np.asarray(want, dtype=np.float64)
    # (below the normal numbers a step is fixed)
    limit = bound + HALF[dtype] * (np.abs(want) + bound) + 2.0 ** -126
    bad = ~(np.abs(got - want) <= limit)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3],
                           np.broadcast_to(limit, bad.shape)[bad][:3])


# ------------------------------------------------------------------ dropout
SHAPES = [(1, 1), (1, 8), (3, 7), (5, 33), (173, 1280), (64, 256), (37, 1283), (2, 5121), (1000, 24)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("tx,ty", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(enc, rows, cols, tx, ty, residual):
    g = _gen(rows * cols)
    x, res = _randn(g, rows, cols, dtype=tx), _randn(g, rows, cols, dtype=ty) if residual else None
    y = torch.full((rows, cols), float("nan"), device="cuda", dtype=ty)
    f = _factors(rows, cols, 0.3)
    enc.op_dropout(x, y, _drop(0.3), residual=res)
    kept = to_np(x) * f
    r = to_np(res) if residual else 0.0
    _within(y, kept + r, 3 * U * (np.abs(kept) + np.abs(r)), ty)
    if not residual:
        assert (to_np(y)[f == 0] == 0).all()


@pytest.mark.parametrize("p", [None, 0.0, 1e-6, 2.0 ** -17, 1 / 65536, 0.5, 1 - 1 / 65536, 1 - 1e-6, 1.0])
def test_dropout_rates(enc, p):
    x = _randn(_gen(1), 50, 129)
    y = torch.empty_like(x)
    enc.op_dropout(x, y, _drop(p))
    f = _factors(50, 129, p)
    _within(y, to_np(x) * f, 2 * U * np.abs(to_np(x) * f))
    if p is None or p < 2.0 ** -17:  # rounds to none: the very values
        assert torch.equal(x, y)


def test_dropped_values_may_be_anything(enc):
    for bad in (float("nan"), float("inf"), -float("inf")):
        for cols in (64, 33):
            x = torch.full((40, cols), bad, device="cuda")
            y, f = torch.empty_like(x), _factors(40, cols, 0.5)
            enc.op_dropout(x, y, _drop(0.5))
            assert (to_np(y)[f == 0] == 0).all()
            np.testing.assert_array_equal(to_np(y)[f != 0], bad)


@pytest.mark.parametrize("pad,offset", [(5, 0), (8, 0), (8, 8), (3, 1)])
def test_dropout_rows_of_wider_buffers(enc, pad, offset):
    """The mask goes by row and column whatever the strides; what lies between rows stays."""
    g, rows, cols = _gen(3), 77, 264
    xb, yb = _randn(g, rows, cols + pad, dtype=BF16), _randn(g, rows, cols + pad, dtype=BF16)
    before = yb.clone()
    x, y = xb[:, offset:offset + cols], yb[:, offset:offset + cols]
    enc.op_dropout(x, y, _drop(0.25))
    f = _factors(rows, cols, 0.25)
    _within(y, to_np(x) * f, 2 * U * np.abs(to_np(x) * f), BF16)
    out = torch.ones(cols + pad, dtype=torch.bool)
    out[offset:offset + cols] = False
    assert torch.equal(yb[:, out], before[:, out])


def test_dropout_in_place_and_interleaved(enc):
    g = _gen(4)
    x = _randn(g, 130, 320)
    want = torch.empty_like(x)
    enc.op_dropout(x, want, _drop(0.4))
    y = x.clone()
    enc.op_dropout(y, y, _drop(0.4))
    assert torch.equal(y, want)
    res = _randn(g, 130, 320)
    both = torch.empty_like(x)
    enc.op_dropout(x, both, _drop(0.4), residual=res)
    into = res.clone()
    enc.op_dropout(x, into, _drop(0.4), residual=into)
    assert torch.equal(into, both)
    two = torch.empty(130, 2, 320, device="cuda")  # rows of x and y in turn
    two[:, 0] = x
    enc.op_dropout(two[:, 0], two[:, 1], _drop(0.4))
    assert torch.equal(two[:, 1], want) and torch.equal(two[:, 0], x)


def test_dropout_is_its_own_gradient(enc):
    """<w, D(x)> = <D(w), x>, and D's differences are D of the differences."""
    g = _gen(5)
    x, w = _randn(g, 64, 100), _randn(g, 64, 100)
    dx, dw = torch.empty_like(x), torch.empty_like(x)
    enc.op_dropout(x, dx, _drop(0.3))
    enc.op_dropout(w, dw, _drop(0.3))
    a, b = (to_np(w) * to_np(dx)).sum(), (to_np(dw) * to_np(x)).sum()
    assert abs(a - b) <= 4 * U * np.abs(to_np(w) * to_np(dx)).sum()


def test_dropout_past_32_bits(enc):
    """More than 2^32 elements: rows at both ends and around every multiple of 2^32."""
    rows, cols = 600_000, 7200
    x = torch.ones(rows, cols, device="cuda", dtype=BF16)
    enc.op_dropout(x, x, _drop(0.5))
    at = [0, 1, 2 ** 31 // cols, 2 ** 31 // cols + 1, 2 ** 32 // cols, 2 ** 32 // cols + 1, rows - 1]
    np.testing.assert_array_equal(to_np(x[at]), S.dropout_factors(at, cols, 0.5, SEED, BASE, 5))


def test_dropout_masks_differ_and_repeat(enc):
    x = torch.ones(300, 640, device="cuda")
    y = [torch.empty_like(x) for _ in range(5)]
    enc.op_dropout(x, y[0], _drop(0.5))
    enc.op_dropout(x, y[1], _drop(0.5))
    enc.op_dropout(x, y[2], _drop(0.5, offset=6))
    enc.op_dropout(x, y[3], _drop(0.5, rng=_rng(SEED + 1)))
    enc.op_dropout(x, y[4], _drop(0.5, offset=4, rng=_rng(base=BASE + 1)))  # the same sum
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[4])
    for other in (y[2], y[3]):
        share = (y[0] != other).double().mean().item()
        assert abs(share - 0.5) < 5 * 0.5 / x.numel() ** 0.5


# ------------------------------------------------------------------ embedding
EMBED = [(1, 1, 1), (3, 2, 7), (64, 33, 256), (173, 33, 1280), (500, 1, 40), (1000, 300, 33), (77, 5000, 264),
         (2500, 64, 130), (40, 33, 5128)]


def _tokens(g, T, V):
    ids = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    ids[::11] = -1
    if T > 3:
        ids[3] = V - 1
    return ids


@pytest.mark.parametrize("T,V,cols", EMBED)
@pytest.mark.parametrize("tt,to", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("rows,p", [(False, None), (True, 0.2)])
def test_embed(enc, T, V, cols, tt, to, rows, p):
    g = _gen(T + V)
    ids, table = _tokens(g, T, V), _randn(g, V, cols, dtype=tt)
    rs = _randn(g, T) if rows else None
    out = torch.full((T, cols), float("nan"), device="cuda", dtype=to)
    enc.op_embed(ids, table, out, scale=1.7, row_scale=rs, dropout=_drop(p))
    want = S.embed(ids.cpu().numpy(), to_np(table), np.float32(1.7), to_np(rs) if rows else None, _factors(T, cols, p))
    _within(out, want, 5 * U * np.abs(want), to)
    enc.check()


@pytest.mark.parametrize("T,V,cols", EMBED)
@pytest.mark.parametrize("td", [F32, BF16])
@pytest.mark.parametrize("rows,p,accumulate", [(False, None, False), (True, 0.2, True), (False, 0.2, False)])
def test_embed_backward(enc, T, V, cols, td, rows, p, accumulate):
    g = _gen(T + V + 1)
    ids, d = _tokens(g, T, V), _randn(g, T, cols, dtype=td)
    rs = _randn(g, T) if rows else None
    table = _randn(g, V, cols) if accumulate else torch.full((V, cols), float("nan"), device="cuda")
    before = to_np(table) if accumulate else 0.0
    enc.op_embed_backward(ids, d, table, scale=1.7, row_scale=rs, dropout=_drop(p), accumulate=accumulate)
    want, mag = S.embed_backward(ids.cpu().numpy(), to_np(d), V, np.float32(1.7), to_np(rs) if rows else None,
                                 _factors(T, cols, p))
    most = int(torch.bincount(ids[ids >= 0], minlength=V).max()) if (ids >= 0).any() else 0
    _within(table, want + before, (most + 6) * U * (mag + np.abs(before)))
    enc.check()


def _zipf(g, T, V):
    u = torch.rand(T, device="cuda", generator=g, dtype=torch.float64)
    return ((u * np.log(V + 1)).exp() - 1).long().clamp(0, V - 1).to(torch.int32)


@pytest.mark.parametrize("T,V,cols", [(16384, 33, 256), (16384, 50021, 64), (70001, 5, 40), (3000, 131072, 24),
                                      (40000, 700, 33), (1025, 257, 8), (2049, 65536, 16), (9000, 65537, 8)])
def test_embed_backward_of_large_batches(enc, T, V, cols):
    g = _gen(T)
    ids, d = _zipf(g, T, V), _randn(g, T, cols)
    table = torch.full((V, cols), float("nan"), device="cuda")
    enc.op_embed_backward(ids, d, table)
    want, mag = S.embed_backward(ids.cpu().numpy(), to_np(d), V, 1.0, None, np.ones((1, 1)))
    counts = np.bincount(ids.cpu().numpy(), minlength=V)[:, None]
    _within(table, want, (counts + 6) * U * mag)
    again = torch.empty_like(table)
    enc.op_embed_backward(ids, d, again)
    assert torch.equal(table, again)  # the order goes by the ids and the sizes


@pytest.mark.parametrize("T,V,cols", [(1, 8192, 8), (512, 1639, 1280), (511, 1638, 1280), (257, 33, 2056), (512, 3, 12),
                                      (256, 33, 264), (512, 65, 264), (513, 65, 264)])
@pytest.mark.parametrize("ids", ["any", "one", "none"])
def test_embed_backward_of_few_tokens(enc, T, V, cols, ids):
    """On both sides of the search's limits; a token count of zero clears the table or leaves it."""
    g = _gen(T + V)
    t = {"any": torch.randint(-1, V, (T,), device="cuda", generator=g), "one": torch.full((T,), V - 1),
         "none": torch.full((T,), -1)}[ids].to(torch.int32).cuda()
    d, kept = _randn(g, T, cols), _randn(g, V, cols)
    want, mag = S.embed_backward(t.cpu().numpy(), to_np(d), V, 1.0, None, _factors(T, cols, 0.2))
    for n in (T, 0):
        for accumulate in (False, True):
            table = kept.clone() if accumulate else torch.full((V, cols), float("nan"), device="cuda")
            enc.op_embed_backward(t[:n], d[:n], table, dropout=_drop(0.2), accumulate=accumulate)
            before = to_np(kept) if accumulate else 0.0
            _within(table, (want if n else 0.0) + before, (n + 6) * U * ((mag if n else 0.0) + np.abs(before)))


@pytest.mark.parametrize("T,V,cols", [(513, 1, 8), (769, 64, 1283), (2000, 63, 12), (1025, 2, 520), (4097, 33, 1280),
                                      (16384, 33, 1280), (9000, 64, 1283), (40000, 9, 520)])
@pytest.mark.parametrize("ids", ["any", "one", "none", "runs", "first"])
@pytest.mark.parametrize("td", [F32, BF16])
def test_embed_backward_of_few_ids(enc, T, V, cols, ids, td):
    """Sums of chunks: ids that fill a chunk, that a chunk lacks, that change on and off its warps' borders."""
    g = _gen(T + V)
    t = {"any": torch.randint(-1, V, (T,), device="cuda", generator=g), "one": torch.full((T,), V - 1),
         "none": torch.full((T,), -1), "runs": torch.arange(T) // 32 % V,
         "first": torch.cat([torch.zeros(250, dtype=torch.long), torch.arange(T - 250) // 250 % V])}[ids].to(torch.int32).cuda()
    d, rs, kept = _randn(g, T, cols, dtype=td), _randn(g, T), _randn(g, V, cols)
    want, mag = S.embed_backward(t.cpu().numpy(), to_np(d), V, 1.0, to_np(rs), _factors(T, cols, 0.2))
    most = int(torch.bincount(t[t >= 0], minlength=V).max()) if ids != "none" else 0
    for accumulate in (False, True):
        table = kept.clone() if accumulate else torch.full((V, cols), float("nan"), device="cuda")
        enc.op_embed_backward(t, d, table, row_scale=rs, dropout=_drop(0.2), accumulate=accumulate)
        before = to_np(kept) if accumulate else 0.0
        _within(table, want + before, (most + 6) * U * (mag + np.abs(before)))
    if ids == "none":
        assert torch.equal(table, kept)


@pytest.mark.parametrize("ids", ["one", "rising", "none", "last"])
def test_embed_backward_of_uneven_ids(enc, ids):
    T, V, cols = 5000, 5000, 72
    t = {"one": torch.full((T,), 7), "rising": torch.arange(T), "none": torch.full((T,), -1),
         "last": torch.cat([torch.full((T - 1,), V - 1), torch.tensor([0])])}[ids].to(torch.int32).cuda()
    d = _randn(_gen(9), T, cols)
    table = torch.full((V, cols), float("nan"), device="cuda")
    enc.op_embed_backward(t, d, table)
    want, mag = S.embed_backward(t.cpu().numpy(), to_np(d), V, 1.0, None, np.ones((1, 1)))
    _within(table, want, (T + 6) * U * mag)
    kept = _randn(_gen(10), V, cols)
    table = kept.clone()
    enc.op_embed_backward(t, d, table, accumulate=True)
    _within(table, want + to_np(kept), (T + 6) * U * (mag + np.abs(to_np(kept))))
    if ids == "none":
        assert torch.equal(table, kept)


def test_embed_ids_outside_the_table(enc):
    from transformer_esm_layer_gb300.binding import EsmError
    g = _gen(11)
    bad = [33, 2 ** 31 - 1, -2, -2 ** 31]
    ids = torch.tensor([4, *bad, 5, -1], dtype=torch.int32, device="cuda")
    table, d = _randn(g, 33, 64), _randn(g, 7, 64)
    out, grad = torch.empty(7, 64, device="cuda"), torch.empty(33, 64, device="cuda")
    for call in (lambda: enc.op_embed(ids, table, out), lambda: enc.op_embed_backward(ids, d, grad)):
        call()
        with pytest.raises(EsmError, match="TOKEN_RANGE"):
            enc.check()
    assert (to_np(out)[[1, 2, 3, 4, 6]] == 0).all() and torch.equal(out[0], table[4]) and torch.equal(out[5], table[5])
    want = torch.zeros(33, 64, device="cuda")
    want[4], want[5] = d[0], d[5]
    assert torch.equal(grad, want)
    big_ids = torch.randint(0, 33, (5000,), device="cuda", generator=g, dtype=torch.int32)
    big_ids[4321] = 77
    big = torch.empty(33, 64, device="cuda")
    enc.op_embed_backward(big_ids, _randn(g, 5000, 64), big)
    with pytest.raises(EsmError, match="TOKEN_RANGE"):
        enc.check()


def test_embed_values_of_absent_tokens_are_not_read(enc):
    """NaN in rows without an id, in dropped places and in the table's unused rows."""
    ids = torch.tensor([1, -1, 1], dtype=torch.int32, device="cuda")
    d = torch.ones(3, 40, device="cuda")
    d[1] = float("nan")
    grad = torch.empty(3, 40, device="cuda")
    enc.op_embed_backward(ids, d, grad)
    np.testing.assert_array_equal(to_np(grad), [[0.0] * 40, [2.0] * 40, [0.0] * 40])
    f = _factors(3, 40, 0.5)
    d = torch.where(torch.from_numpy(f == 0).cuda(), float("nan"), 1.0)
    enc.op_embed_backward(ids, d, grad, dropout=_drop(0.5))
    np.testing.assert_array_equal(to_np(grad)[1], (f[0] + f[2]))
    table = torch.full((3, 40), float("nan"), device="cuda")
    table[1] = 3.0
    out = torch.empty(3, 40, device="cuda")
    enc.op_embed(ids, table, out)
    np.testing.assert_array_equal(to_np(out), [[3.0] * 40, [0.0] * 40, [3.0] * 40])


def test_embed_strided_rows(enc):
    g = _gen(12)
    ids, table = _tokens(g, 90, 33), _randn(g, 33, 136, dtype=BF16)
    for pad, off in ((8, 0), (3, 2)):
        buf = _randn(g, 90, 136 + pad)
        before, out = buf.clone(), buf[:, off:off + 136]
        enc.op_embed(ids, table, out, scale=2.0)
        want = S.embed(ids.cpu().numpy(), to_np(table), 2.0, None, np.ones((1, 1)))
        np.testing.assert_array_equal(to_np(out), want)
        assert torch.equal(buf[:, off + 136:], before[:, off + 136:]) and torch.equal(buf[:, :off], before[:, :off])
        grad = torch.empty(33, 136, device="cuda")
        enc.op_embed_backward(ids, out, grad)
        want, mag = S.embed_backward(ids.cpu().numpy(), to_np(out), 33, 1.0, None, np.ones((1, 1)))
        _within(grad, want, 90 * U * mag)


def test_embed_backward_of_no_tokens_in_wide_rows(enc):
    """Shapes that no token count takes to the search still have a workspace for none."""
    for V, cols in ((3, 800_000), (9000, 264)):
        ids, d = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, cols, device="cuda")
        table = torch.full((V, cols), float("nan"), device="cuda")
        enc.op_embed_backward(ids, d, table)
        assert (table == 0).all()
        enc.op_embed_backward(ids, d, table.fill_(2.0), accumulate=True)
        assert (table == 2).all()


def test_embed_of_nothing(enc):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table, out = _randn(_gen(1), 9, 16), torch.empty(0, 16, device="cuda")
    enc.op_embed(none, table, out)
    grad = torch.full((9, 16), float("nan"), device="cuda")
    enc.op_embed_backward(none, out, grad)
    assert (grad == 0).all()
    enc.op_embed_backward(none, out, table, accumulate=True)
    assert torch.equal(table, _randn(_gen(1), 9, 16))


def test_embed_tables_past_32_bits(enc):
    """Rows that start beyond 2^31 elements, in the table and in its gradient."""
    V, cols = 1_700_000, 1280
    ids = torch.tensor([0, V - 1, 2 ** 31 // cols, 2 ** 31 // cols + 1, V - 1], dtype=torch.int32, device="cuda")
    table = torch.zeros(V, cols, dtype=BF16, device="cuda")
    rows = _randn(_gen(13), 5, cols, dtype=BF16)
    table[ids.long()] = rows
    out = torch.empty(5, cols, device="cuda")
    enc.op_embed(ids, table, out)
    assert torch.equal(out, table[ids.long()].float())
    del table
    grad = torch.full((V, cols), float("nan"), device="cuda")
    enc.op_embed_backward(ids, rows, grad)
    assert torch.equal(grad[V - 1], rows[1].float() + rows[4].float())
    assert torch.equal(grad[ids[2:4].long()], rows[2:4].float())
    grad[ids.long()] = 0
    assert (grad == 0).all()


# ------------------------------------------------------------------ block norm
EPS = 1e-5
NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (5, 33), (173, 1280), (64, 256), (37, 1283), (9, 2560), (4, 4096), (3, 4104),
               (3, 5120), (2, 8192), (2, 8191), (1500, 64), (700, 260), (701, 1280), (305, 8), (311, 2056), (7, 2304),
               (333, 4088), (309, 904)]
# kind, post, pre, betas, gate, residual scale, dropout
NORMS = [("layer", True, True, True, "vector", 1.0, 0.1), ("layer", True, True, False, "rows", 0.7, None),
         ("rms", True, True, False, "vector", 1.0, 0.3), ("rms", True, True, True, "none", -0.5, None),
         ("layer", False, True, True, "none", 1.0, 0.1), ("layer", True, False, True, "vector", 1.0, 0.2),
         ("rms", False, False, False, "rows", 1.0, 0.5), ("layer", False, True, True, "rows", 0.0, None)]


def _norm_case(dtype, rows, cols, config, seed, offset=0.0):
    from transformer_esm_layer_gb300.binding import BlockNorm
    kind, post, pre, betas, gate, alpha, p = config
    g = _gen(seed)
    t = dict(post_gamma=1 + 0.2 * _randn(g, cols) if post else None, post_beta=_randn(g, cols) if post and betas else None,
             pre_gamma=1 + 0.2 * _randn(g, cols) if pre else None, pre_beta=_randn(g, cols) if pre and betas else None)
    t = {k: None if v is None else v.to(dtype) for k, v in t.items()}
    gt = {"none": None, "vector": _randn(g, cols, dtype=dtype), "rows": _randn(g, rows, cols, dtype=dtype)}[gate]
    x, y = 2 * _randn(g, rows, cols) + offset, (_randn(g, rows, cols) + offset).to(dtype)
    norm = BlockNorm(kind, residual_scale=alpha, **t)
    ref = {k: None if v is None else to_np(v) for k, v in t.items()}
    ref.update(rms=kind == "rms", residual_scale=np.float64(np.float32(alpha)), gate=None if gt is None else to_np(gt))
    return norm, gt, x, y, p, ref


def _norm_bound(z, err, ref, which):
    """Bound of a norm's output of z known to within err, and of its two statistics."""
    n = z.shape[1]
    mean, rstd = S.moments(z, ref["rms"], EPS)
    e_mean = 0.0 if ref["rms"] else D * U * np.abs(z).mean(1, keepdims=True) + np.mean(err, 1, keepdims=True)
    dz = np.abs(z - mean)
    e_dz = err + e_mean + U * dz
    q = (dz ** 2).mean(1, keepdims=True)
    # (the second term of (dz + e)^2 counts where a row is all but constant)
    e_q = (2 * dz * e_dz + e_dz ** 2).mean(1, keepdims=True) + D * U * q
    e_r = 0.5 * e_q / (q + EPS) / (1 - np.minimum(0.5, e_q / (q + EPS))) ** 1.5 + 6 * U
    hat = dz * rstd
    e_hat = rstd * e_dz * (1 + e_r) + hat * (e_r + 2 * U)
    gamma = np.abs(ref[which + "_gamma"])
    beta = 0.0 if ref[which + "_beta"] is None else np.abs(ref[which + "_beta"])
    return gamma * e_hat + 2 * U * (gamma * hat + beta), np.broadcast_to(e_mean, rstd.shape), rstd * e_r


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("config", NORMS)
def test_block_norm(encs, rows, cols, dtype, config):
    norm, gate, x, y, p, ref = _norm_case(dtype, rows, cols, config, rows + cols)
    f = _factors(rows, cols, p)
    x_out = torch.full((rows, cols), float("nan"), device="cuda")
    h = torch.full((rows, cols), float("nan"), device="cuda", dtype=dtype) if config[2] else None
    stats = torch.full((rows, 4), float("nan"), device="cuda")
    encs[dtype].op_block_norm(norm, x, y, x_out, h, gate=gate, dropout=_drop(p), stats=stats)
    _check_forward(x, y, x_out, h, stats, ref, f, dtype)


def _check_forward(x, y, x_out, h, stats, ref, f, dtype):
    want_x, want_h, want_s = S.block_norm(to_np(x), to_np(y), ref, f, EPS)
    e_s = np.zeros_like(want_s)
    if ref["post_gamma"] is not None:
        e_n, e_s[:, 0:1], e_s[:, 1:2] = _norm_bound(to_np(y), np.zeros(y.shape), ref, "post")
        n = S._affine((to_np(y) - want_s[:, 0:1]) * want_s[:, 1:2], ref["post_gamma"], ref["post_beta"])
    else:
        e_n, n = 0.0, to_np(y)
    gate = 1.0 if ref["gate"] is None else np.abs(ref["gate"])
    a = np.abs(ref["residual_scale"] * to_np(x))
    e_x = gate * f * (e_n + 4 * U * np.abs(n)) + 2 * U * a
    _within(x_out, want_x, e_x)
    if h is not None:
        e_h, e_s[:, 2:3], e_s[:, 3:4] = _norm_bound(want_x, e_x + U * np.abs(want_x), ref, "pre")
        _within(h, want_h, e_h, dtype)
    if stats is not None:
        _within(stats, want_s, e_s)


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(0, 64), (2000, 1280)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("config", NORMS)
def test_block_norm_backward(encs, rows, cols, dtype, config):
    norm, gate, x, y, p, ref = _norm_case(dtype, rows, cols, config, 3 * rows + cols)
    g = _gen(rows)
    d_x = None if config[0] == "rms" and config[2] and config[5] < 0 else _randn(g, rows, cols)
    d_h = _randn(g, rows, cols, dtype=dtype) if config[2] else None
    _check_backward(encs[dtype], norm, gate, x, y, p, ref, d_x, d_h, dtype)


@pytest.mark.parametrize("rows,cols", [(500, 4104), (700, 5120), (470, 8192), (471, 6400), (460, 4096), (309, 3592)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("config", NORMS)
def test_block_norm_backward_of_wide_rows(encs, rows, cols, dtype, config):
    """Several rows to a block, and more of them than are on their way at once."""
    test_block_norm_backward(encs, rows, cols, dtype, config)


def _check_backward(enc, norm, gate, x, y, p, ref, d_x, d_h, dtype, **kw):
    rows, cols = y.shape
    f = _factors(rows, cols, p)
    x_out, stats = torch.empty_like(x), torch.empty(rows, 4, device="cuda")
    h = torch.empty_like(y) if ref["pre_gamma"] is not None else None
    enc.op_block_norm(norm, x, y, x_out, h, gate=gate, dropout=_drop(p), stats=stats)
    nan = lambda *s, dt=F32: torch.full(s, float("nan"), device="cuda", dtype=dt)
    dx, dy = nan(rows, cols), nan(rows, cols, dt=dtype)
    grads = {k: nan(cols) for k in ("post_gamma", "post_beta", "pre_gamma", "pre_beta") if ref[k] is not None}
    if gate is not None:
        grads["gate"] = nan(cols) if gate.dim() == 1 else nan(rows, cols, dt=dtype)
    enc.op_block_norm_backward(norm, x_out, y, stats, d_x, d_h, dx, dy, grads, gate=gate, dropout=_drop(p), **kw)
    st, xo, yd = to_np(stats), to_np(x_out), to_np(y)
    dxo, dh = (None if d_x is None else to_np(d_x)), (None if d_h is None else to_np(d_h))
    want = S.block_norm_backward(xo, yd, st, dxo, dh, ref, f)
    # the same formulas with magnitudes, in the order in which the kernel joins a row's sums
    my, ry, mx, rx = (st[:, i:i + 1] for i in range(4))
    n = 1.0 / max(cols, 1)
    e = np.zeros_like(yd) if dxo is None else np.abs(dxo)
    A = B = 0.0
    xh = np.zeros_like(yd)
    if dh is not None:
        xh = np.abs((xo - mx) * rx)
        gg = np.abs(dh * ref["pre_gamma"])
        e = e + rx * gg
        A, B = 0 if ref["rms"] else rx * gg.sum(1, keepdims=True) * n, rx * (gg * xh).sum(1, keepdims=True) * n
    G = e + A + xh * B
    k = f * (1.0 if ref["gate"] is None else np.abs(ref["gate"]))
    post = ref["post_gamma"] is not None
    yh = np.abs((yd - my) * ry) if post else np.abs(yd)
    steps = 2 * D + 20  # two sums of a row, one in the other, and the products around them
    _within(dx, want[0], steps * U * np.abs(ref["residual_scale"]) * G)
    if post:
        c = k * np.abs(ref["post_gamma"])
        m0 = 0 if ref["rms"] else ((c * e).sum(1, keepdims=True) + A * c.sum(1, keepdims=True)
                                   + B * (c * xh).sum(1, keepdims=True)) * n
        m1 = ((c * e * yh).sum(1, keepdims=True) + A * (c * yh).sum(1, keepdims=True)
              + B * (c * xh * yh).sum(1, keepdims=True)) * n
        dy_mag = ry * (c * G + m0 + yh * m1)
    else:
        dy_mag = k * G
    _within(dy, want[1], steps * U * dy_mag, dtype)
    mags = {}
    if dh is not None:
        mags["pre_gamma"], mags["pre_beta"] = np.abs(dh) * xh, np.abs(dh)
    if post:
        mags["post_gamma"], mags["post_beta"] = k * G * yh, k * G
    if gate is not None:
        mags["gate"] = f * G * (yh * np.abs(ref["post_gamma"]) + np.abs(0 if ref["post_beta"] is None else ref["post_beta"])
                                if post else yh)
    for name, got in grads.items():
        if name == "gate" and gate.dim() == 2:
            _within(got, want[2][name], steps * U * mags[name], dtype)
        else:
            _within(got, want[2][name], (steps + rows) * U * mags[name].sum(0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_block_norm_rows_far_from_zero(encs, dtype):
    """A mean a thousand deviations away costs digits of the input, not of the sums."""
    for cols in (1280, 2560, 77):
        norm, gate, x, y, p, ref = _norm_case(dtype, 30, cols, NORMS[0], cols, offset=1000.0)
        x_out, h, stats = torch.empty_like(x), torch.empty_like(y), torch.empty(30, 4, device="cuda")
        encs[dtype].op_block_norm(norm, x, y, x_out, h, gate=gate, dropout=_drop(p), stats=stats)
        _check_forward(x, y, x_out, h, stats, ref, _factors(30, cols, p), dtype)


@pytest.mark.parametrize("cols", [64, 1283, 5120])
def test_block_norm_constant_rows(enc, cols):
    """No variance: the normalised row is 0, its scale 1 / sqrt(eps)."""
    from transformer_esm_layer_gb300.binding import BlockNorm
    one = torch.ones(cols, device="cuda", dtype=BF16)
    norm = BlockNorm("layer", post_gamma=one, pre_gamma=one)
    x, y = torch.full((3, cols), 4.0, device="cuda"), torch.full((3, cols), 2.0, device="cuda", dtype=BF16)
    x_out, h, stats = torch.empty_like(x), torch.empty_like(y), torch.empty(3, 4, device="cuda")
    enc.op_block_norm(norm, x, y, x_out, h, stats=stats)
    assert (x_out == 4).all() and (h == 0).all() and (stats[:, 0] == 2).all() and (stats[:, 2] == 4).all()
    np.testing.assert_allclose(to_np(stats)[:, [1, 3]], EPS ** -0.5, rtol=1e-6)


def test_block_norm_in_place(encs):
    for cols in (1280, 33, 2600):
        norm, gate, x, y, p, ref = _norm_case(BF16, 200, cols, NORMS[0], cols)
        enc, d = encs[BF16], _drop(p)
        x_out, h, stats = torch.empty_like(x), torch.empty_like(y), torch.empty(200, 4, device="cuda")
        enc.op_block_norm(norm, x, y, x_out, h, gate=gate, dropout=d, stats=stats)
        x2, y2, s2 = x.clone(), y.clone(), torch.empty_like(stats)
        enc.op_block_norm(norm, x2, y2, x2, y2, gate=gate, dropout=d, stats=s2)
        assert torch.equal(x2, x_out) and torch.equal(y2, h) and torch.equal(s2, stats)
        g = _gen(cols)
        d_x, d_h = _randn(g, 200, cols), _randn(g, 200, cols, dtype=BF16)
        new = lambda: {k: torch.empty(cols, device="cuda") for k in
                       ("post_gamma", "post_beta", "pre_gamma", "pre_beta", "gate")}
        dx, dy, a = torch.empty_like(x), torch.empty_like(y), new()
        enc.op_block_norm_backward(norm, x_out, y, stats, d_x, d_h, dx, dy, a, gate=gate, dropout=d)
        for place in ("d_h", "y"):
            dx2, dh2, y3, b = d_x.clone(), d_h.clone(), y.clone(), new()
            dy2 = dh2 if place == "d_h" else y3
            enc.op_block_norm_backward(norm, x_out, y3, stats, dx2, dh2, dx2, dy2, b, gate=gate, dropout=d)
            assert torch.equal(dx2, dx) and torch.equal(dy2, dy) and all(torch.equal(a[k], b[k]) for k in a)


def test_block_norm_misaligned(encs):
    """Rows that start off 16 bytes though their length is a multiple of 8."""
    enc, cols = encs[BF16], 264
    norm, gate, x, y, p, ref = _norm_case(BF16, 50, cols, NORMS[0], 1)
    shift = lambda t, n: torch.cat([torch.zeros(n, device="cuda", dtype=t.dtype), t.flatten()])[n:].view_as(t)
    xs, ys = shift(x, 1), shift(y, 3)
    assert ys.data_ptr() % 16
    x_out, h, stats = shift(torch.empty_like(x), 3), shift(torch.empty_like(y), 1), torch.empty(50, 4, device="cuda")
    enc.op_block_norm(norm, xs, ys, x_out, h, gate=shift(gate, 5), dropout=_drop(p), stats=stats)
    _check_forward(x, y, x_out, h, stats, ref, _factors(50, cols, p), BF16)


# aligned rows, rows off 16 bytes, wide rows of both kinds; several groups of warps to a block and one
@pytest.mark.parametrize("rows,cols", [(1000, 64), (400, 1280), (37, 1283), (9, 4096), (5, 5120), (3, 8191)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("config", NORMS)
def test_block_norm_backward_reads_no_absent_norms_stats(encs, rows, cols, dtype, config):
    """The columns of stats of a norm that there is not may hold anything."""
    enc = encs[dtype]
    norm, gate, x, y, p, ref = _norm_case(dtype, rows, cols, config, 4)
    post, pre = config[1], config[2]
    d_x, d_h = _randn(_gen(1), rows, cols), _randn(_gen(2), rows, cols, dtype=dtype) if pre else None
    x_out, stats = torch.empty_like(x), torch.empty(rows, 4, device="cuda")
    enc.op_block_norm(norm, x, y, x_out, torch.empty_like(y) if pre else None, gate=gate, dropout=_drop(p), stats=stats)
    results = []
    for hold in (0.0, float("nan")):
        st = stats.clone()
        if not post:
            st[:, :2] = hold
        if not pre:
            st[:, 2:] = hold
        dx, dy = torch.empty_like(x), torch.empty_like(y)
        grads = {k: torch.empty(cols, device="cuda") for k in ("post_gamma", "post_beta", "pre_gamma", "pre_beta")
                 if ref[k] is not None}
        enc.op_block_norm_backward(norm, x_out if pre else None, y, st, d_x, d_h, dx, dy, grads, gate=gate, dropout=_drop(p))
        results.append([dx, dy] + list(grads.values()))
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("rows,cols", [(1000, 64), (400, 1280), (37, 1283), (9, 4096), (5, 5120), (3, 8191)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("config", [c for c in NORMS if c[6]])
@pytest.mark.parametrize("hold", [float("nan"), float("inf")])
def test_block_norm_backward_of_dropped_places(encs, rows, cols, dtype, config, hold):
    """What d_x_out holds at a dropped place goes to dx there and nowhere else; without a norm after the block,
    what y holds there goes nowhere."""
    enc = encs[dtype]
    norm, gate, x, y, p, ref = _norm_case(dtype, rows, cols, config, 5)
    post, pre = config[1], config[2]
    dropped = torch.from_numpy(_factors(rows, cols, p) == 0).cuda()
    d_x, d_h = _randn(_gen(1), rows, cols), _randn(_gen(2), rows, cols, dtype=dtype) if pre else None
    x_out, stats = torch.empty_like(x), torch.empty(rows, 4, device="cuda")
    h = torch.empty_like(y) if pre else None
    enc.op_block_norm(norm, x, y, x_out, h, gate=gate, dropout=_drop(p), stats=stats)
    results = []
    for there in (False, True):
        d_xt, yt = d_x.clone(), y.clone()
        if there:
            d_xt[dropped] = hold
            if not post:
                yt[dropped] = hold
                again = torch.empty_like(x)
                enc.op_block_norm(norm, x, yt, again, h, gate=gate, dropout=_drop(p))
                assert torch.equal(again, x_out)
        dx, dy = torch.empty_like(x), torch.empty_like(y)
        grads = {k: torch.empty(cols, device="cuda") for k in ("post_gamma", "post_beta", "pre_gamma", "pre_beta")
                 if ref[k] is not None}
        if gate is not None:
            grads["gate"] = torch.empty(cols, device="cuda") if gate.dim() == 1 else torch.empty_like(gate)
        enc.op_block_norm_backward(norm, x_out, yt, stats, d_xt, d_h, dx, dy, grads, gate=gate, dropout=_drop(p))
        results.append([dx.masked_fill(dropped, 0.0), dy] + list(grads.values()))
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("shift", [4, 8])
def test_float32_rows_off_32_bytes(encs, shift):
    """Float32 rows that start `shift` values into their buffer: the same results, wherever they lie."""
    enc, rows, cols, V = encs[F32], 600, 264, 70
    move = lambda t: torch.cat([torch.zeros(shift, device="cuda"), t.flatten()])[shift:].view_as(t)
    g = _gen(3)
    x, table, ids = _randn(g, rows, cols), _randn(g, V, cols), _tokens(g, rows, V)
    for case in range(2):
        at = move if case else (lambda t: t.clone())
        y, out, dt = at(torch.empty_like(x)), at(torch.empty_like(x)), at(torch.empty_like(table))
        enc.op_dropout(at(x), y, _drop(0.3), residual=at(2 * x))
        enc.op_embed(ids, at(table), out, dropout=_drop(0.3))
        enc.op_embed_backward(ids, at(x), dt, dropout=_drop(0.3))
        few = at(torch.empty(33, cols, device="cuda"))
        enc.op_embed_backward(ids % 33, at(x), few, dropout=_drop(0.3))
        now = [y, out, dt, few]
        if case:
            assert all(torch.equal(a, b) for a, b in zip(now[:2], first[:2]))
            for a, b in zip(now[2:], first[2:]):
                torch.testing.assert_close(a, b, rtol=0, atol=64 * U * 64)  # up to 64 terms of some size 8 in another order
        first = now
    norm, gate, x, y, p, ref = _norm_case(F32, 50, cols, NORMS[0], 1)
    x_out, h, stats = move(torch.empty_like(x)), move(torch.empty_like(y)), torch.empty(50, 4, device="cuda")
    enc.op_block_norm(norm, move(x), move(y), x_out, h, gate=gate, dropout=_drop(p), stats=stats)
    _check_forward(x, y, x_out, h, stats, ref, _factors(50, cols, p), F32)
    _check_backward(enc, norm, gate, move(x), move(y), p, ref, move(x), move(y), F32)


def test_some_gradients_alone(encs):
    """Any of the parameters' gradients may be left out."""
    enc, cols = encs[BF16], 640
    norm, gate, x, y, p, ref = _norm_case(BF16, 90, cols, NORMS[0], 2)
    x_out, h, stats = torch.empty_like(x), torch.empty_like(y), torch.empty(90, 4, device="cuda")
    enc.op_block_norm(norm, x, y, x_out, h, gate=gate, dropout=_drop(p), stats=stats)
    d_x, d_h = _randn(_gen(1), 90, cols), _randn(_gen(2), 90, cols, dtype=BF16)
    names = ("post_gamma", "post_beta", "pre_gamma", "pre_beta", "gate")
    full = {k: torch.empty(cols, device="cuda") for k in names}
    dx, dy = torch.empty_like(x), torch.empty_like(y)
    enc.op_block_norm_backward(norm, x_out, y, stats, d_x, d_h, dx, dy, full, gate=gate, dropout=_drop(p))
    for some in ((), ("gate",), ("pre_beta", "post_gamma")):
        part, dx2, dy2 = {k: torch.empty(cols, device="cuda") for k in some}, torch.empty_like(x), torch.empty_like(y)
        enc.op_block_norm_backward(norm, x_out, y, stats, d_x, d_h, dx2, dy2, part, gate=gate, dropout=_drop(p))
        assert torch.equal(dx, dx2) and torch.equal(dy, dy2) and all(torch.equal(part[k], full[k]) for k in some)


# ------------------------------------------------------------------ the set together, streams, graphs
def _step(enc, s, stream=None):
    """Embedding, two blocks (stand-ins: y = their input times a weight) with their norms, and all the way back."""
    kw = dict(stream=stream)
    enc.op_embed(s["ids"], s["table"], s["x0"], scale=2.0, row_scale=s["row_scale"], dropout=s["d0"], **kw)
    enc.op_block_norm(s["n1"], s["x0"], s["y1"], s["x1"], s["h1"], gate=s["gate"], dropout=s["d1"], stats=s["s1"], **kw)
    enc.op_dropout(s["h1"], s["y2"], s["d2"], **kw)  # the second block: dropout alone
    enc.op_block_norm(s["n2"], s["x1"], s["y2"], s["x2"], s["h2"], dropout=s["d3"], stats=s["s2"], **kw)
    enc.op_block_norm_backward(s["n2"], s["x2"], s["y2"], s["s2"], None, s["d_h2"], s["dx1"], s["dy2"], s["g2"],
                               dropout=s["d3"], workspace=s["wn"], **kw)
    enc.op_dropout(s["dy2"], s["dh1"], s["d2"], **kw)
    enc.op_block_norm_backward(s["n1"], s["x1"], s["y1"], s["s1"], s["dx1"], s["dh1"], s["dx0"], s["dy1"], s["g1"],
                               gate=s["gate"], dropout=s["d1"], workspace=s["wn"], **kw)
    enc.op_embed_backward(s["ids"], s["dx0"], s["d_table"], scale=2.0, row_scale=s["row_scale"], dropout=s["d0"],
                          workspace=s["we"], **kw)


OUTPUTS = ("x0", "x1", "h1", "s1", "y2", "x2", "h2", "s2", "dx1", "dy2", "dh1", "dx0", "dy1", "d_table")


def _state(enc, T=1500, V=33, cols=256):
    from transformer_esm_layer_gb300.binding import BlockNorm
    g = _gen(21)
    rng = _rng()
    new = lambda *s, dt=F32: torch.full(s, float("nan"), device="cuda", dtype=dt)
    v = lambda: (1 + 0.2 * _randn(g, cols)).to(BF16)
    s = dict(ids=_tokens(g, T, V), table=_randn(g, V, cols, dtype=BF16), row_scale=torch.rand(T, device="cuda", generator=g),
             y1=_randn(g, T, cols, dtype=BF16), gate=v(), rng=rng, d_h2=_randn(g, T, cols, dtype=BF16),
             n1=BlockNorm("layer", post_gamma=v(), post_beta=v(), pre_gamma=v(), pre_beta=v()),
             n2=BlockNorm("rms", pre_gamma=v(), residual_scale=0.9))
    for i, p in enumerate((0.1, 0.2, 0.3, 0.4)):
        s[f"d{i}"] = _drop(p, offset=i, rng=rng)
    for k in ("x0", "x1", "x2", "dx0", "dx1"):
        s[k] = new(T, cols)
    for k in ("h1", "y2", "h2", "dy2", "dh1", "dy1"):
        s[k] = new(T, cols, dt=BF16)
    s["s1"], s["s2"], s["d_table"] = new(T, 4), new(T, 4), new(V, cols)
    s["g1"] = {k: new(cols) for k in ("post_gamma", "post_beta", "pre_gamma", "pre_beta", "gate")}
    s["g2"] = {"pre_gamma": new(cols)}
    s["wn"], s["we"] = enc.op_block_norm_backward_workspace(T, cols), enc.op_embed_backward_workspace(T, V, cols)
    return s


def _results(s):
    return {**{k: s[k].clone() for k in OUTPUTS}, **{f"{n}.{k}": t.clone() for n in ("g1", "g2") for k, t in s[n].items()}}


def _same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


def test_a_training_step_of_the_set(enc):
    """The whole chain against the float64 one, which rounds only where the operators' types do: every
    tensor's relative error stays within a few of its type's steps."""
    s = _state(enc)
    _step(enc, s)
    T, cols = s["x0"].shape
    n = lambda t: None if t is None else to_np(t)
    f = [_factors(T, cols, p, offset=i) for i, p in enumerate((0.1, 0.2, 0.3, 0.4))]
    ids = s["ids"].cpu().numpy()
    par = lambda b, rms, alpha, gate: dict(rms=rms, residual_scale=alpha, gate=gate, post_gamma=n(b.post_gamma),
                                           post_beta=n(b.post_beta), pre_gamma=n(b.pre_gamma), pre_beta=n(b.pre_beta))
    p1, p2 = par(s["n1"], False, 1.0, n(s["gate"])), par(s["n2"], True, np.float64(np.float32(0.9)), None)
    x0 = S.embed(ids, n(s["table"]), 2.0, n(s["row_scale"]), f[0])
    x1, h1, s1 = S.block_norm(x0, n(s["y1"]), p1, f[1], EPS)
    y2 = S.dropout(h1, f[2])
    x2, h2, s2 = S.block_norm(x1, y2, p2, f[3], EPS)
    dx1, dy2, g2 = S.block_norm_backward(x2, y2, s2, None, n(s["d_h2"]), p2, f[3])
    dh1 = S.dropout(dy2, f[2])
    dx0, dy1, g1 = S.block_norm_backward(x1, n(s["y1"]), s1, dx1, dh1, p1, f[1])
    dt, _ = S.embed_backward(ids, dx0, 33, 2.0, n(s["row_scale"]), f[0])
    # bf16 roundings on the way: h1, y2 forward, dy2, dh1 backward, each at most 2^-8 of an element, entering
    # at most once per branch; a tensor that depends on k of them is held to (k + 1) 2^-8
    want = dict(x0=(x0, 0), x1=(x1, 0), h1=(h1, 1), y2=(y2, 2), x2=(x2, 2), h2=(h2, 3), dx1=(dx1, 3), dy2=(dy2, 4),
                dh1=(dh1, 5), dx0=(dx0, 5), dy1=(dy1, 6), d_table=(dt, 5))
    for k, (w, steps) in want.items():
        rel = np.linalg.norm(to_np(s[k]) - w) / np.linalg.norm(w)
        assert rel <= (steps + 1) * 2.0 ** -8 if steps else rel <= D * U, (k, rel)
    for grads, w in ((s["g1"], g1), (s["g2"], g2)):
        for k, t in grads.items():
            rel = np.linalg.norm(to_np(t) - w[k]) / np.linalg.norm(w[k])
            assert rel <= 7 * 2.0 ** -8, (k, rel)


def test_streams_and_graphs(enc):
    """Another stream, and a captured step whose replays draw new masks when the base moves on."""
    s = _state(enc)
    _step(enc, s)
    torch.cuda.synchronize()
    want = _results(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _step(enc, s, stream=side)
    side.synchronize()
    assert _same(_results(s), want)  # bitwise: nothing depends on scheduling
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(enc, s)
    graph.replay()
    torch.cuda.synchronize()
    assert _same(_results(s), want)
    s["rng"][1] += 4
    graph.replay()
    torch.cuda.synchronize()
    moved = _results(s)
    assert not torch.equal(moved["x0"], want["x0"])
    _step(enc, s)
    torch.cuda.synchronize()
    assert _same(_results(s), moved)
    s["rng"][1] -= 4
    graph.replay()
    torch.cuda.synchronize()
    assert _same(_results(s), want)


def test_calls_without_a_workspace(enc):
    """The binding's own workspace, on the call's stream."""
    s = _state(enc)
    _step(enc, s)
    torch.cuda.synchronize()
    want = _results(s)
    s["wn"] = s["we"] = None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        _step(enc, s, stream=side)
    side.synchronize()
    assert _same(_results(s), want)


# ------------------------------------------------------------------ refusals (host checks: nothing runs)
def test_refusals(enc):
    from transformer_esm_layer_gb300.binding import BlockNorm, Dropout, EsmError
    x = torch.zeros(4, 64, device="cuda")
    xb = x.to(BF16)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    table = torch.zeros(33, 64, device="cuda")
    v = torch.ones(64, device="cuda", dtype=BF16)
    norm = BlockNorm("layer", pre_gamma=v, post_gamma=v)
    stats = torch.zeros(4, 4, device="cuda")
    big = torch.zeros(8, 64, device="cuda")
    bad = (ValueError, EsmError)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError):
            Dropout(p, _rng())
    with pytest.raises(ValueError):
        Dropout(0.1, _rng().float())
    with pytest.raises(ValueError):
        Dropout(0.1, _rng(), 2 ** 63)
    calls = [
        lambda: enc.op_dropout(x.double(), x, None),
        lambda: enc.op_dropout(x, x[:, :32], None),
        lambda: enc.op_dropout(x.t(), x.t(), None),
        lambda: enc.op_dropout(x[0], x[0], None),
        lambda: enc.op_dropout(x[:1].expand(4, 64), torch.empty_like(x), None),
        lambda: enc.op_dropout(x, torch.empty_like(x), None, residual=xb),
        lambda: enc.op_dropout(x, torch.empty_like(x), 0.1),
        lambda: enc.op_dropout(big[:4], big[1:5], None),
        lambda: enc.op_dropout(x, big[:4], None, residual=big[2:6]),
        lambda: enc.op_embed(ids.long(), table, x),
        lambda: enc.op_embed(ids, table[:, :32], x[:, :32]),
        lambda: enc.op_embed(ids, table, x[:3]),
        lambda: enc.op_embed(ids, table, table[:4]),
        lambda: enc.op_embed(ids, table, x, row_scale=torch.zeros(3, device="cuda")),
        lambda: enc.op_embed_backward(ids, x, table.to(BF16)),
        lambda: enc.op_embed_backward(ids, table[:4], table),
        lambda: enc.op_embed_backward(ids, x, table, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: enc.op_embed_backward(ids, x, table, workspace=torch.empty(4096, dtype=torch.uint8)),
        lambda: enc.op_block_norm(norm, xb, xb, x, xb),
        lambda: enc.op_block_norm(norm, x, xb, torch.empty_like(x)),
        lambda: enc.op_block_norm(BlockNorm(), x, xb, torch.empty_like(x), torch.empty_like(xb)),
        lambda: enc.op_block_norm(norm, x[:, :32].contiguous(), xb[:, :32].contiguous(), x[:, :32].contiguous(),
                                  xb[:, :32].contiguous()),
        lambda: enc.op_block_norm(norm, x, xb, torch.empty_like(x), torch.empty_like(xb), gate=v[:32]),
        lambda: enc.op_block_norm(norm, x, xb, torch.empty_like(x), torch.empty_like(xb), gate=v.float()),
        lambda: enc.op_block_norm(norm, x, xb, torch.empty_like(x), torch.empty_like(xb), stats=stats[:, :3]),
        lambda: enc.op_block_norm(norm, big[:4], xb, big[1:5], torch.empty_like(xb)),
        lambda: enc.op_block_norm_backward(norm, x, xb, stats, x, None, x, xb, {}),
        lambda: enc.op_block_norm_backward(norm, x, xb, None, x, xb, x, xb, {}),
        lambda: enc.op_block_norm_backward(norm, x, xb, stats, x, xb, x, xb, {"gate": torch.empty(64, device="cuda")}),
        lambda: enc.op_block_norm_backward(norm, x, xb, stats, x, xb, x, xb, {"other": torch.empty(64, device="cuda")}),
        lambda: enc.op_block_norm_backward(norm, x, xb, stats, x, xb, x, xb, {}),  # dx over x_out
        lambda: enc.op_block_norm_backward(norm, x, xb, stats, None, xb, torch.empty_like(x), torch.empty_like(xb), {},
                                           workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
        lambda: enc.op_block_norm_backward_workspace(4, 8193),
        lambda: enc.op_embed_backward_workspace(4, 0, 8),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(bad):
            call()
            pytest.fail(f"call {i} was taken")
    g = torch.empty(64, device="cuda")
    with pytest.raises(bad):  # one buffer for two gradients
        enc.op_block_norm_backward(norm, x, xb, stats, None, xb.clone(), torch.empty_like(x), torch.empty_like(xb),
                                   {"post_gamma": g, "pre_gamma": g})
    wide = torch.zeros(2, 8193, device="cuda")
    with pytest.raises(EsmError, match="UNSUPPORTED"):
        enc.op_block_norm(BlockNorm(), wide, wide.to(BF16), torch.empty_like(wide))
    enc.check()


@pytest.mark.parametrize("T,V", [(8, 33), (600, 33), (600, 100)])  # a search, chunks, a sort
def test_embed_backward_workspace_lies_apart(enc, T, V):
    from transformer_esm_layer_gb300.binding import EsmError
    cols = 16
    need = enc.op_embed_backward_workspace(T, V, cols).numel()
    buf = torch.zeros(need + 2 ** 18, dtype=torch.uint8, device="cuda")
    ws, table = buf[:need], torch.zeros(V, cols, device="cuda")
    new = dict(ids=torch.zeros(T, dtype=torch.int32, device="cuda"), d_out=torch.ones(T, cols, device="cuda"),
               row_scale=torch.ones(T, device="cuda"), rng=_rng())
    for name, t in new.items():
        for at, taken in ((0, False), (need - 16, False), (need, True)):
            inside = buf[at:at + t.nbytes].view(t.dtype).view(t.shape)
            inside.copy_(t)
            s = {**new, name: inside}

            def call():
                enc.op_embed_backward(s["ids"], s["d_out"], table, row_scale=s["row_scale"], dropout=_drop(0.1, rng=s["rng"]),
                                      workspace=ws)
            if taken:
                call()
                assert torch.isfinite(table).all()
                continue
            with pytest.raises(EsmError, match="INVALID_ARG"):
                call()
                pytest.fail(f"{name} at {at} was taken")
    enc.check()


def test_no_dropout_needs_no_generator(enc, encs):
    """A p that rounds to none is no dropout, whatever rng is, in every call that takes one."""
    from transformer_esm_layer_gb300 import binding
    lib, h = enc.lib, enc.handle
    x = _randn(_gen(30), 5, 64)
    y = torch.empty_like(x)
    for p in (0.0, 2.0 ** -18):
        for rng in (None, 4, _rng().data_ptr()):  # (4: not even aligned)
            none = binding.EsmDropout(rng, 3, p)
            y.fill_(float("nan"))
            assert lib.esm_op_dropout(h, x.data_ptr(), 0, 64, None, 0, y.data_ptr(), 0, 64, 5, 64, none, None) == 0
            assert torch.equal(x, y)
            for e in encs.values():
                assert lib.esm_encoder_set_dropout(e.handle, none) == 0
    for bad in (binding.EsmDropout(None, 0, 0.1), binding.EsmDropout(4, 0, 0.1), binding.EsmDropout(None, 0, -0.1),
                binding.EsmDropout(None, 0, float("nan")), binding.EsmDropout(None, 0, 1.5)):
        assert lib.esm_op_dropout(h, x.data_ptr(), 0, 64, None, 0, y.data_ptr(), 0, 64, 5, 64, bad, None) == 1
        assert lib.esm_encoder_set_dropout(h, bad) == 1
