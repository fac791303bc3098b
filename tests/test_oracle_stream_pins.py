"""The oracle of the residual stream's operators against published answers, finite differences and
torch autograd (CPU)."""
import numpy as np
import pytest

from oracle import stream as S

torch = pytest.importorskip("torch")


def test_philox_published_answers():
    """Known answers of Philox4x32-10 published with the generator."""
    pi = ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0])
    for (c, k), want in (
            (([0] * 4, [0] * 2), [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            (([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2), [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            (pi, [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert [int(x) for x in S.philox4x32(c, k)] == want


def _bits(r, c, cols, seed, o):
    """Word by word, with Python's integers."""
    b = r * (-(-cols // 8)) + c // 8
    x = [b & 0xFFFFFFFF, b >> 32, o & 0xFFFFFFFF, o >> 32]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for i in range(10):
        p0, p1 = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(p1 >> 32) ^ x[1] ^ ((k[0] + i * 0x9E3779B9) & 0xFFFFFFFF), p1 & 0xFFFFFFFF,
             (p0 >> 32) ^ x[3] ^ ((k[1] + i * 0xBB67AE85) & 0xFFFFFFFF), p0 & 0xFFFFFFFF]
    return (x[(c % 8) // 2] >> (16 * (c % 2))) & 0xFFFF


@pytest.mark.parametrize("cols", [1, 7, 8, 33])
def test_dropout_factors_element_by_element(cols):
    seed, base, offset, p = 2 ** 63 + 12345, 2 ** 64 - 3, 5, 0.4
    n = round(p * 65536)
    rows = [0, 1, 2, 2 ** 31 + 7, 2 ** 40]
    got = S.dropout_factors(rows, cols, p, seed, base, offset)
    for i, r in enumerate(rows):
        for c in range(cols):
            kept = _bits(r, c, cols, seed, (base + offset) % 2 ** 64) >= n
            assert got[i, c] == (65536 / (65536 - n) if kept else 0.0)


def test_dropout_rates():
    for p in (0.0, 1e-6, 0.1, 0.5, 0.999, 1.0):
        f = S.dropout_factors(200, 1000, p, 3, 4, 5)
        n = int(np.floor(p * 65536 + 0.5))
        share, q = (f == 0).mean(), n / 65536
        assert abs(share - q) <= 5 * np.sqrt(q * (1 - q) / f.size)
        if 0 < n < 65536:
            assert f.max() == 65536 / (65536 - n)
    assert (S.dropout_factors(9, 9, 1e-6, 3, 4, 5) == 1).all()
    x = np.full((200, 1000), np.nan)
    f = S.dropout_factors(200, 1000, 0.5, 3, 4, 5)
    assert (np.isnan(S.dropout(x, f)) == (f != 0)).all()


def _params(rng, cols, rms, post, pre, gate, rows):
    v = lambda *s: rng.standard_normal(s)
    return dict(rms=rms, residual_scale=0.7, post_gamma=1 + v(cols) if post else None,
                post_beta=v(cols) if post else None, pre_gamma=1 + v(cols) if pre else None,
                pre_beta=v(cols) if pre else None,
                gate={"none": None, "vector": v(cols), "rows": v(rows, cols)}[gate])


CONFIGS = [(rms, post, pre, gate) for rms in (False, True) for post in (False, True) for pre in (False, True)
           for gate in ("none", "vector", "rows")]


@pytest.mark.parametrize("rms,post,pre,gate", CONFIGS)
def test_block_norm_backward_is_the_gradient(rms, post, pre, gate):
    rng = np.random.default_rng(5)
    rows, cols, eps = 5, 11, 1e-3
    x, y = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    p = _params(rng, cols, rms, post, pre, gate, rows)
    f = S.dropout_factors(rows, cols, 0.3, 1, 2, 3)
    wx, wh = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))

    def loss(x, y, p):
        x_out, h, _ = S.block_norm(x, y, p, f, eps)
        return (wx * x_out).sum() + (0 if h is None else (wh * h).sum())

    x_out, h, stats = S.block_norm(x, y, p, f, eps)
    dx, dy, grads = S.block_norm_backward(x_out, y, stats, wx, wh if pre else None, p, f)

    def slope(make, shape, i):
        e = np.zeros(shape)
        e.flat[i] = 1e-6
        return (loss(*make(e)) - loss(*make(-e))) / 2e-6

    for i in range(0, rows * cols, 7):
        assert slope(lambda e: (x + e, y, p), x.shape, i) == pytest.approx(dx.flat[i], rel=1e-6, abs=1e-7)
        assert slope(lambda e: (x, y + e, p), y.shape, i) == pytest.approx(dy.flat[i], rel=1e-6, abs=1e-7)
    for name in ("post_gamma", "post_beta", "pre_gamma", "pre_beta", "gate"):
        if p[name] is None:
            assert name not in grads
            continue
        for i in range(0, p[name].size, 4):
            got = slope(lambda e: (x, y, {**p, name: p[name] + e}), p[name].shape, i)
            assert got == pytest.approx(grads[name].flat[i], rel=1e-6, abs=1e-7)


@pytest.mark.parametrize("rms", [False, True])
def test_block_norm_forward_against_torch(rms):
    rng = np.random.default_rng(6)
    x, y = rng.standard_normal((4, 12)), rng.standard_normal((4, 12))
    p = _params(rng, 12, rms, True, True, "vector", 4)
    t = {k: torch.from_numpy(v) for k, v in p.items() if isinstance(v, np.ndarray)}

    def norm(z, which):
        if rms:
            return torch.nn.functional.rms_norm(z, (12,), t[which + "_gamma"], 1e-5) + t[which + "_beta"]
        return torch.nn.functional.layer_norm(z, (12,), t[which + "_gamma"], t[which + "_beta"], 1e-5)

    x_out, h, _ = S.block_norm(x, y, p, np.ones((4, 12)), 1e-5)
    want = 0.7 * torch.from_numpy(x) + t["gate"] * norm(torch.from_numpy(y), "post")
    np.testing.assert_allclose(x_out, want.numpy(), rtol=1e-12)
    np.testing.assert_allclose(h, norm(want, "pre").numpy(), rtol=1e-11, atol=1e-12)


def test_embedding_against_torch_autograd():
    rng = np.random.default_rng(7)
    ids = np.array([3, -1, 0, 3, 6, 3, -1, 9])  # 9 is outside the table
    row_scale = rng.random(8)
    f = S.dropout_factors(8, 5, 0.4, 1, 2, 3)
    table = torch.from_numpy(rng.standard_normal((7, 5))).requires_grad_()
    ok = (ids >= 0) & (ids < 7)
    out = table[np.where(ok, ids, 0)] * torch.from_numpy(2.5 * row_scale * ok)[:, None] * torch.from_numpy(f)
    got = S.embed(ids, table.detach().numpy(), 2.5, row_scale, f)
    np.testing.assert_allclose(got, out.detach().numpy(), rtol=1e-14)
    d = rng.standard_normal((8, 5))
    out.backward(torch.from_numpy(d))
    grad, mag = S.embed_backward(ids, d, 7, 2.5, row_scale, f)
    np.testing.assert_allclose(grad, table.grad.numpy(), rtol=1e-13, atol=1e-15)
    assert (mag >= np.abs(grad) - 1e-15).all()
