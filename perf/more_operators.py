"""What a training step does to the residual stream outside its products and its attention: the
cases that are measured, their inputs, and their plain forms.

A case's "op" is one of

  embed                out  from token ids and a table: rows of the table times a scale, dropped out
  embed_backward       d_table  from token ids and d_out, summed token by token
  dropout              y  from x (and a residual); its gradient is the same call
  block_norm           x_out, h, stats: the norm after a block, its dropout, gate and residual, and
                       the norm before the next block
  block_norm_backward  dx, dy and the parameters' gradients

Dropout: element (r, c) of [rows, cols] has 16 random bits u.  They come from Philox4x32-10 with the
counter (b, o), both 64 bits, b = r * ceil(cols / 8) + c // 8 and o = rng[1] + offset, and the key
rng[0]; element j = c % 8 takes the lower (j even) or upper half of word j // 2.  With n = p * 65536
rounded, an element is kept if u >= n and then multiplied by 65536 / (65536 - n); others are zero.

Block norm, for a row: u = dropout(post(y)), x_out = residual_scale * x + gate * u, h = pre(x_out), with
post and pre a LayerNorm or an RMS norm (gamma, beta), or, for post, nothing.  stats holds each row's
mean and 1 / deviation of post, then of pre (0 where there is none; an RMS norm's mean is 0).
"""
import functools
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZES = {"fp32": 4, "bf16": 2}


def listed():
    return [
        # one protein at a time, as a service embeds it: latency
        dict(name="embed_one_protein", op="embed", tokens=180, vocab=33, cols=1280, table="bf16", type="fp32",
             per_token=False, p=0.0, skip=0.0),
        # a training batch of a language model's vocabulary, masked tokens' rows scaled away, dropout behind it
        dict(name="embed_vocab", op="embed", tokens=16384, vocab=50021, cols=1280, table="fp32", type="fp32",
             per_token=True, p=0.1, skip=0.0),
        # fine-tuning on a handful of short sequences
        dict(name="embed_bwd_small", op="embed_backward", tokens=173, vocab=33, cols=1280, type="fp32",
             per_token=False, p=0.0, skip=0.0),
        # the packed 650M batch: few ids, each with hundreds of tokens
        dict(name="embed_bwd_packed_650m", op="embed_backward", tokens=16384, vocab=33, cols=1280, type="fp32",
             per_token=True, p=0.1, skip=0.0),
        # a language model's vocabulary: most ids never met, some met a thousand times
        dict(name="embed_bwd_vocab", op="embed_backward", tokens=16384, vocab=50021, cols=1280, type="bf16",
             per_token=False, p=0.0, skip=0.02),
        # one small batch of proteins behind a projection
        dict(name="dropout_small", op="dropout", rows=180, cols=1280, x="bf16", type="bf16", residual=False, pad=0,
             p=0.1),
        # the feed-forward activations of the packed 650M batch
        dict(name="dropout_ffn", op="dropout", rows=16384, cols=5120, x="bf16", type="bf16", residual=False, pad=0,
             p=0.1),
        # odd rows out of a wider buffer, added to the residual stream
        dict(name="dropout_odd", op="dropout", rows=8191, cols=1283, x="bf16", type="fp32", residual=True, pad=5, p=0.25),
        # one protein at a time through a model with norms on both sides of a block
        dict(name="norm_one_protein", op="block_norm", type="bf16", rows=180, cols=1280, rms=False, post=True, pre=True,
             gate="vector", scale=1.0, p=0.0, stats=False),
        # the training forward of the packed 650M batch
        dict(name="norm_packed_650m", op="block_norm", type="bf16", rows=16384, cols=1280, rms=False, post=True, pre=True,
             gate="vector", scale=1.0, p=0.1, stats=True),
        # its backward
        dict(name="norm_bwd_packed_650m", op="block_norm_backward", type="bf16", rows=16384, cols=1280, rms=False,
             post=True, pre=True, gate="vector", scale=1.0, p=0.1),
        # the 3B width, RMS norms, a gate of its own for every token
        dict(name="norm_bwd_3b_rms", op="block_norm_backward", type="bf16", rows=16384, cols=2560, rms=True, post=True,
             pre=True, gate="rows", scale=0.8, p=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    """Mostly the widths models have, some odd ones."""
    usual = [w for w in (128, 320, 480, 640, 1280, 2560, 4096, 5120) if w <= hi]
    return rng.choice([rng.choice(usual), rng.choice(usual), 8 * _log(rng, 8, hi // 8), _log(rng, 33, hi)])


def draw(rng):
    op = rng.choice(["embed", "embed_backward", "dropout", "block_norm", "block_norm_backward"])
    p = rng.choice([0.0, 0.1, 0.1, 0.3])
    types = ["fp32", "bf16"]
    if op.startswith("embed"):
        vocab = rng.choice([33, 33, _log(rng, 2, 256), _log(rng, 257, 65536)])
        cols = _width(rng, min(5120, 2 ** 26 // vocab))
        tokens = _log(rng, 1, min(65536, 2 ** 24 // cols))
        case = dict(op=op, tokens=tokens, vocab=vocab, cols=cols, type=rng.choice(types), per_token=rng.random() < 0.5,
                    p=p, skip=rng.choice([0.0, 0.0, 0.1]))
        if op == "embed":
            case["table"] = rng.choice(types)
        return case
    if op == "dropout":
        cols = _width(rng, 8192)
        return dict(op=op, rows=_log(rng, 1, 2 ** 25 // cols), cols=cols, x=rng.choice(types), type=rng.choice(types),
                    residual=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 5]), p=p or 0.5)
    cols = _width(rng, 4096)
    case = dict(op=op, type=rng.choice(["fp32", "bf16", "bf16", "bf16"]), rows=_log(rng, 1, 2 ** 24 // cols), cols=cols,
                rms=rng.random() < 0.4, post=rng.random() < 0.7, pre=rng.random() < 0.8,
                gate=rng.choice(["none", "vector", "vector", "rows"]), scale=rng.choice([1.0, 1.0, 0.7]), p=p)
    if op == "block_norm":
        case["stats"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _chances(case):
    """How often each id stands in the tokens: residues evenly, a language's ids by rank."""
    V = case["vocab"]
    if V <= 64:
        return np.full(V, 1.0 / V)
    rank = np.arange(1, V + 1)
    return np.log((rank + 1) / rank) / math.log(V + 1)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    dt = DTYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s["rng"] = torch.tensor([int(seed) * 0x9E3779B97F4A7C15 % 2 ** 63, int(seed) % 1000003], device="cuda")
    if case["op"].startswith("embed"):
        T, V, d = case["tokens"], case["vocab"], case["cols"]
        u = uniform(T).double()
        ids = (u * V if V <= 64 else (u * math.log(V + 1)).exp() - 1).long().clamp(0, V - 1)
        s["ids"] = torch.where(uniform(T) < case["skip"], -1, ids).to(torch.int32)
        masked = uniform(T) < 0.12
        s["row_scale"] = torch.where(masked, 0.0, 0.88 / (0.85 + 0.1 * uniform(T))) if case["per_token"] else None
        s["scale"] = math.sqrt(d) if V > 64 else 1.0
        if case["op"] == "embed":
            s["table"] = (normal(V, d) / math.sqrt(d)).to(DTYPES[case["table"]])
            s["table_type"] = case["table"]
        else:
            s["d_out"] = normal(T, d).to(dt)
        return s
    R, C = case["rows"], case["cols"]
    if case["op"] == "dropout":
        s["x"] = normal(R, C + case["pad"]).to(DTYPES[case["x"]])[:, :C]
        s["res"] = normal(R, C).to(dt) if case["residual"] else None
        return s
    s["x_in"] = 2.0 * normal(R, C) + 0.5 * normal(C)
    s["y"] = (0.5 * normal(R, C) + 0.2 * normal(C)).to(dt)
    for name, there in (("post", case["post"]), ("pre", case["pre"])):
        s[name + "_gamma"] = (1.0 + 0.2 * normal(C)).to(dt) if there else None
        s[name + "_beta"] = (0.1 * normal(C)).to(dt) if there and not case["rms"] else None
    s["g"] = {"none": lambda: None, "vector": lambda: (0.3 + 0.1 * normal(C)).to(dt),
              "rows": lambda: uniform(R, C).to(dt)}[case["gate"]]()
    if case["op"] == "block_norm_backward":
        s["x_out"], _, s["st"] = _plain_norm(s)
        s["d_x_out"] = normal(R, C)
        s["d_h"] = normal(R, C).to(dt) if case["pre"] else None
        del s["x_in"]
    return s


# ---------------------------------------------------------------- plain forms
OFFSET = 7
LOW = 0xFFFFFFFF


def _kept(s, rows, cols):
    """The factor of every element: 0 if it is dropped."""
    n = int(s["p"] * 65536 + 0.5)
    if n == 0:
        return 1.0
    b = torch.arange(rows * (-(-cols // 8)), device="cuda")
    o = s["rng"][1] + OFFSET
    c0, c1 = b & LOW, (b >> 32) & LOW
    c2, c3 = (o & LOW).expand_as(b), ((o >> 32) & LOW).expand_as(b)
    k0, k1 = s["rng"][0] & LOW, (s["rng"][0] >> 32) & LOW
    for _ in range(10):
        a, d = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64: the upper words come by shift and mask
        c0, c1, c2, c3 = ((d >> 32) & LOW) ^ c1 ^ k0, d & LOW, ((a >> 32) & LOW) ^ c3 ^ k1, a & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    u = torch.stack([h for w in (c0, c1, c2, c3) for h in (w & 0xFFFF, w >> 16)], 1)
    return torch.where(u.view(rows, -1)[:, :cols] >= n, 65536 / (65536 - n), 0.0)


def _token_scale(s):
    f = torch.full((s["tokens"],), s["scale"], device="cuda")
    if s["row_scale"] is not None:
        f = f * s["row_scale"]
    return torch.where(s["ids"] >= 0, f, 0)[:, None]


def _plain_embed(s):
    rows = s["table"].float()[s["ids"].long().clamp(min=0)]
    return (rows * _token_scale(s) * _kept(s, s["tokens"], s["cols"])).to(DTYPES[s["type"]])


def _plain_embed_backward(s):
    rows = s["d_out"].float() * _kept(s, s["tokens"], s["cols"]) * _token_scale(s)
    out = torch.zeros(s["vocab"], s["cols"], device="cuda")
    return out.index_add_(0, s["ids"].long().clamp(min=0), rows)


def _plain_dropout(s):
    y = s["x"].float() * _kept(s, s["rows"], s["cols"])
    if s["res"] is not None:
        y = s["res"].float() + y
    return y.to(DTYPES[s["type"]])


def _moments(s, z):
    mean = torch.zeros(len(z), 1, device="cuda") if s["rms"] else z.mean(1, keepdim=True)
    rstd = ((z - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
    return mean, rstd


def _affine(s, which, z):
    z = z * s[which + "_gamma"].float()
    return z if s[which + "_beta"] is None else z + s[which + "_beta"].float()


def _plain_norm(s):
    u = s["y"].float()
    none = torch.zeros(len(u), 1, device="cuda")
    stats = [none] * 4
    if s["post"]:
        stats[0], stats[1] = _moments(s, u)
        u = _affine(s, "post", (u - stats[0]) * stats[1])
    u = u * _kept(s, s["rows"], s["cols"])
    if s["g"] is not None:
        u = u * s["g"].float()
    x = s["scale"] * s["x_in"] + u
    h = None
    if s["pre"]:
        stats[2], stats[3] = _moments(s, x)
        h = _affine(s, "pre", (x - stats[2]) * stats[3]).to(s["y"].dtype)
    return x, h, torch.cat(stats, 1)


def _back(s, g, zhat, rstd):
    """Gradient through a norm whose normalised row is zhat, of g = d_out * gamma."""
    g0 = 0 if s["rms"] else g.mean(1, keepdim=True)
    return rstd * (g - g0 - zhat * (g * zhat).mean(1, keepdim=True))


def _plain_norm_backward(s):
    post_mean, post_rstd, pre_mean, pre_rstd = s["st"].split(1, 1)
    grads = {}
    G = s["d_x_out"]
    if s["pre"]:
        xhat, dh = (s["x_out"] - pre_mean) * pre_rstd, s["d_h"].float()
        grads["pre_gamma"] = (dh * xhat).sum(0)
        if s["pre_beta"] is not None:
            grads["pre_beta"] = dh.sum(0)
        G = G + _back(s, dh * s["pre_gamma"].float(), xhat, pre_rstd)
    keep = _kept(s, s["rows"], s["cols"])
    y = s["y"].float()
    yhat = (y - post_mean) * post_rstd if s["post"] else y
    dn = G * keep
    if s["g"] is not None:
        dgate = dn * (_affine(s, "post", yhat) if s["post"] else y)
        grads["gate"] = dgate.sum(0) if s["gate"] == "vector" else dgate.to(s["y"].dtype)
        dn = dn * s["g"].float()
    dy = dn
    if s["post"]:
        grads["post_gamma"] = (dn * yhat).sum(0)
        if s["post_beta"] is not None:
            grads["post_beta"] = dn.sum(0)
        dy = _back(s, dn * s["post_gamma"].float(), yhat, post_rstd)
    return {"dx": s["scale"] * G, "dy": dy.to(s["y"].dtype), **grads}


# ---------------------------------------------------------------- one pass
@functools.lru_cache(maxsize=None)
def _encoder(precision):
    from transformer_esm_layer_gb300.binding import EsmEncoder
    return EsmEncoder(1, 256, 4, 1024, precision=precision, ln_eps=EPS)


def _drop(s):
    from transformer_esm_layer_gb300.binding import Dropout
    if "drop" not in s:
        s["drop"] = Dropout(s["p"], s["rng"], OFFSET) if s["p"] else None
    return s["drop"]


def _norm(s):
    from transformer_esm_layer_gb300.binding import BlockNorm
    if "norm" not in s:
        s["norm"] = BlockNorm("rms" if s["rms"] else "layer", post_gamma=s["post_gamma"], post_beta=s["post_beta"],
                              pre_gamma=s["pre_gamma"], pre_beta=s["pre_beta"], residual_scale=s["scale"])
    return s["norm"]


def _own(s):
    op = s["op"]
    dt = DTYPES[s["type"]]
    if op == "embed":
        out = torch.empty(s["tokens"], s["cols"], dtype=dt, device="cuda")
        _encoder("bf16").op_embed(s["ids"], s["table"], out, scale=s["scale"], row_scale=s["row_scale"], dropout=_drop(s))
        return {"out": out}
    if op == "embed_backward":
        enc = _encoder("bf16")
        if "workspace" not in s:
            s["workspace"] = enc.op_embed_backward_workspace(s["tokens"], s["vocab"], s["cols"])
        d_table = torch.empty(s["vocab"], s["cols"], device="cuda")
        enc.op_embed_backward(s["ids"], s["d_out"], d_table, scale=s["scale"], row_scale=s["row_scale"], dropout=_drop(s),
                              workspace=s["workspace"])
        return {"d_table": d_table}
    R, C = s["rows"], s["cols"]
    if op == "dropout":
        y = torch.empty(R, C, dtype=dt, device="cuda")
        _encoder("bf16").op_dropout(s["x"], y, _drop(s), residual=s["res"])
        return {"y": y}
    enc = _encoder(s["type"])
    if op == "block_norm":
        x_out = torch.empty(R, C, device="cuda")
        h = torch.empty(R, C, dtype=dt, device="cuda") if s["pre"] else None
        stats = torch.empty(R, 4, device="cuda") if s["stats"] else None
        enc.op_block_norm(_norm(s), s["x_in"], s["y"], x_out, h, gate=s["g"], dropout=_drop(s), stats=stats)
        return {"x_out": x_out, "h": h, "stats": stats}
    if "workspace" not in s:
        s["workspace"] = enc.op_block_norm_backward_workspace(R, C)
    dx = torch.empty(R, C, device="cuda")
    dy = torch.empty(R, C, dtype=dt, device="cuda")
    grads = {k: torch.empty(C, device="cuda") for k in ("pre_gamma", "pre_beta", "post_gamma", "post_beta")
             if s[k] is not None}
    if s["g"] is not None:
        grads["gate"] = torch.empty(C, device="cuda") if s["gate"] == "vector" else torch.empty_like(s["g"])
    enc.op_block_norm_backward(_norm(s), s["x_out"], s["y"], s["st"], s["d_x_out"], s["d_h"], dx, dy, grads, gate=s["g"],
                               dropout=_drop(s), workspace=s["workspace"])
    return {"dx": dx, "dy": dy, **grads}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "embed":
        return {"out": _plain_embed(s)}
    if s["op"] == "embed_backward":
        return {"d_table": _plain_embed_backward(s)}
    if s["op"] == "dropout":
        return {"y": _plain_dropout(s)}
    if s["op"] == "block_norm":
        x_out, h, stats = _plain_norm(s)
        return {"x_out": x_out, "h": h, "stats": stats if s["stats"] else None}
    return _plain_norm_backward(s)


# ---------------------------------------------------------------- the least work
PHILOX = 60  # products, exclusive ors and key steps of one call, which serves eight elements


def work(case):
    es = SIZES[case["type"]]
    random = PHILOX / 8 if case["p"] else 0
    if case["op"].startswith("embed"):
        T, V, d = case["tokens"], case["vocab"], case["cols"]
        fixed = 4 * T + (4 * T if case["per_token"] else 0) + es * T * d
        met = float((1.0 - (1.0 - _chances(case)) ** (T * (1.0 - case["skip"]))).sum())
        if case["op"] == "embed":
            return {"bytes": int(fixed + met * d * SIZES[case["table"]]), "flops": int((2 + random) * T * d)}
        return {"bytes": fixed + 4 * V * d, "flops": int((2 + random) * T * d)}
    n = case["rows"] * case["cols"]
    if case["op"] == "dropout":
        return {"bytes": n * (SIZES[case["x"]] + es * (2 if case["residual"] else 1)), "flops": int((2 + random) * n)}
    gate = es if case["gate"] == "rows" else 0
    if case["op"] == "block_norm":
        per = 8 + es + (es if case["pre"] else 0) + gate
        return {"bytes": n * per + (16 * case["rows"] if case["stats"] else 0), "flops": int((18 + random) * n)}
    per = 8 + 2 * es + (4 + es if case["pre"] else 0) + 2 * gate
    return {"bytes": n * per + 16 * case["rows"], "flops": int((32 + random) * n)}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_factors(s, rows, cols):
    """Dropout factors in float64, with the products of the generator taken in 16-bit halves."""
    n = int(round(s["p"] * 65536))
    per_row = (cols + 7) // 8
    if n == 0:
        return torch.ones(rows, cols, dtype=torch.float64, device="cuda")
    seed, base = (int(v) % 2 ** 64 for v in s["rng"].tolist())
    o = (base + OFFSET) % 2 ** 64
    key = [seed % 2 ** 32, seed >> 32]

    def times(x, m):  # 32 x 32 bits -> (upper, lower) words
        x1, x0, m1, m0 = x >> 16, x & 0xFFFF, m >> 16, m & 0xFFFF
        low = x0 * m0
        mid = x1 * m0 + (low >> 16)
        mid2 = x0 * m1 + (mid & 0xFFFF)
        return x1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | (low & 0xFFFF)

    out = torch.empty(rows, per_row * 8, dtype=torch.float64, device="cuda")
    step = max(1, 2 ** 20 // per_row)
    for a in range(0, rows, step):
        r = torch.arange(a, min(rows, a + step), device="cuda")[:, None]
        b = r * per_row + torch.arange(per_row, device="cuda")[None]
        w = [b % 2 ** 32, b // 2 ** 32, torch.full_like(b, o % 2 ** 32), torch.full_like(b, o >> 32)]
        for i in range(10):
            k = [(key[0] + i * 0x9E3779B9) % 2 ** 32, (key[1] + i * 0xBB67AE85) % 2 ** 32]
            h0, l0 = times(w[0], 0xD2511F53)
            h1, l1 = times(w[2], 0xCD9E8D57)
            w = [h1 ^ w[1] ^ k[0], l1, h0 ^ w[3] ^ k[1], l0]
        u = torch.empty(*b.shape, 8, dtype=torch.int64, device="cuda")
        for j in range(8):
            u[..., j] = (w[j // 2] >> (16 * (j % 2))) % 65536
        out[a:a + step] = (u >= n).double().reshape(len(r), -1) * (65536.0 / (65536 - n))
    return out[:, :cols]


def _exact_embed(s, backward):
    T, V, d = s["tokens"], s["vocab"], s["cols"]
    f = _exact_factors(s, T, d)
    ids = s["ids"].long()
    w = s["scale"] * (ids >= 0).double()
    if s["row_scale"] is not None:
        w = w * s["row_scale"].double()
    if not backward:
        return {"out": w[:, None] * f * s["table"].double().index_select(0, ids.clamp(min=0))}
    order = torch.argsort(ids.clamp(min=0), stable=True)
    total = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    rows = (f * w[:, None] * s["d_out"].double()).index_select(0, order)
    if V <= 64:
        counts = torch.bincount(ids.clamp(min=0), minlength=V).tolist()
        start = 0
        for v, c in enumerate(counts):
            total[v] = rows[start:start + c].sum(0)
            start += c
    else:
        total.index_add_(0, ids.clamp(min=0).index_select(0, order), rows)
    return {"d_table": total}


def _exact_norm(s, x_in):
    f = _exact_factors(s, s["rows"], s["cols"])

    def normalise(z, which):
        centre = z.new_zeros(len(z), 1) if s["rms"] else z.sum(1, keepdim=True) / s["cols"]
        dev = (((z - centre) ** 2).sum(1, keepdim=True) / s["cols"] + EPS) ** -0.5
        out = (z - centre) * dev * s[which + "_gamma"].double()[None]
        if s[which + "_beta"] is not None:
            out = out + s[which + "_beta"].double()[None]
        return out, centre, dev

    stats = torch.zeros(s["rows"], 4, dtype=torch.float64, device="cuda")
    n = s["y"].double()
    if s["post"]:
        n, stats[:, 0:1], stats[:, 1:2] = normalise(n, "post")
    x = s["scale"] * x_in.double() + n * f * (1.0 if s["g"] is None else s["g"].double())
    h = None
    if s["pre"]:
        h, stats[:, 2:3], stats[:, 3:4] = normalise(x, "pre")
    return {"x_out": x, "h": h, "stats": stats if s["stats"] else None}


def _exact_norm_backward(s):
    """From the statistics in hand; the sums over rows piece by piece."""
    R, C = s["rows"], s["cols"]
    f = _exact_factors(s, R, C)
    out = {"dx": torch.empty(R, C, dtype=torch.float64, device="cuda"),
           "dy": torch.empty(R, C, dtype=torch.float64, device="cuda")}
    for k in ("pre_gamma", "pre_beta", "post_gamma", "post_beta"):
        if s[k] is not None:
            out[k] = torch.zeros(C, dtype=torch.float64, device="cuda")
    if s["g"] is not None:
        out["gate"] = torch.zeros((R, C) if s["gate"] == "rows" else (C,), dtype=torch.float64, device="cuda")
    step = max(1, 2 ** 22 // C)
    for a in range(0, R, step):
        rows = slice(a, a + step)
        m_y, r_y, m_x, r_x = (s["st"][rows, k].double()[:, None] for k in range(4))
        total = s["d_x_out"][rows].double()
        if s["pre"]:
            e = s["d_h"][rows].double()
            xn = (s["x_out"][rows].double() - m_x) * r_x
            out["pre_gamma"] += torch.einsum("rc,rc->c", e, xn)
            if "pre_beta" in out:
                out["pre_beta"] += e.sum(0)
            e = e * s["pre_gamma"].double()
            e = e - xn * torch.einsum("rc,rc->r", e, xn)[:, None] / C - (0 if s["rms"] else e.sum(1)[:, None] / C)
            total = total + e * r_x
        out["dx"][rows] = s["scale"] * total
        y = s["y"][rows].double()
        yn = (y - m_y) * r_y if s["post"] else y
        n = yn
        if s["post"]:
            n = n * s["post_gamma"].double() + (0 if s["post_beta"] is None else s["post_beta"].double())
        total = total * f[rows]
        if s["gate"] == "rows":
            out["gate"][rows] = total * n
            total = total * s["g"][rows].double()
        elif s["gate"] == "vector":
            out["gate"] += (total * n).sum(0)
            total = total * s["g"].double()
        if s["post"]:
            out["post_gamma"] += (total * yn).sum(0)
            if "post_beta" in out:
                out["post_beta"] += total.sum(0)
            total = total * s["post_gamma"].double()
            total = total - yn * ((total * yn).sum(1) / C)[:, None] - (0 if s["rms"] else (total.sum(1) / C)[:, None])
            total = total * r_y
        out["dy"][rows] = total
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("embed"):
        return _exact_embed(s, case["op"] == "embed_backward")
    if case["op"] == "dropout":
        y = s["x"].double() * _exact_factors(s, s["rows"], s["cols"])
        return {"y": y if s["res"] is None else y + s["res"].double()}
    if case["op"] == "block_norm":
        return _exact_norm(s, s["x_in"])
    return _exact_norm_backward(s)
