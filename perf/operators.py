"""Windowed attention with first-token sinks and distillation from a teacher's top logits,
each with its gradient: the cases that are measured, their inputs, and their plain forms.

A case's "op" is one of

  attention_window           o, lse  from packed q | k | v
  attention_window_backward  dqkv    from qkv, o, lse and d_o
  distill_loss               token_loss, lse, loss_sum, count  from logits and a teacher's top K
  distill_loss_backward      d_logits

Windowed attention: query i of a sequence of length L sees key j of the same sequence if
j <= i + right and (j >= i - left or j < sinks); a side of -1 is unlimited.  Head size 64,
scores scaled by 1/8.  Distillation: q = softmax(logits / t), p = softmax over the row's usable
teacher entries (id >= 0) of teacher_logits / t, loss = t^2 sum_k p_k (log p_k - log q_{id_k});
a row without a usable entry is not scored: its loss, its lse and its gradient are zero.
"""
import functools
import math

import torch

own = False

HEAD = 64
SCALE = 0.125
BLOCK = 128
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}

# The 47 lengths (16384 tokens) of the repository's packed 650M workload.
PACKED_650M = ("336,219,234,69,883,596,247,477,355,215,539,249,246,187,394,283,416,208,324,176,497,336,366,384,"
               "164,480,1024,112,106,122,497,324,573,463,340,356,271,505,152,233,347,884,190,157,214,537,97")


def listed():
    return [
        # one protein at a time, as a service answers it: latency
        dict(name="attn_one_protein", op="attention_window", type="bf16", heads=20, lengths="180", left=32, right=32,
             sinks=1, lse=False),
        # the packed batch of the 650M model, <cls> kept visible
        dict(name="attn_packed_650m", op="attention_window", type="bf16", heads=20, lengths=PACKED_650M, left=128,
             right=128, sinks=1, lse=False),
        # a training forward over one long sequence, far beyond what full attention affords
        dict(name="attn_long", op="attention_window", type="bf16", heads=20, lengths="65536", left=256, right=256,
             sinks=4, lse=True),
        # left context only (next-token training) at the 3B width, ragged lengths
        dict(name="attn_causal", op="attention_window", type="bf16", heads=40,
             lengths="2048,1,1777,640,2001,129,1283,2048,900,1461", left=-1, right=0, sinks=0, lse=True),
        # fine-tuning on a handful of short sequences
        dict(name="attn_bwd_small", op="attention_window_backward", type="bf16", heads=4, lengths="37,130,5,1",
             left=16, right=16, sinks=1),
        # the training step of the packed 650M batch
        dict(name="attn_bwd_packed_650m", op="attention_window_backward", type="bf16", heads=20, lengths=PACKED_650M,
             left=128, right=128, sinks=1),
        # one long sequence with a few short ones, one-sided window
        dict(name="attn_bwd_long", op="attention_window_backward", type="bf16", heads=20, lengths="32768,511,70,1025",
             left=512, right=0, sinks=4),
        # every token of the packed 650M batch against eight stored teacher logits of the 33
        dict(name="distill_esm", op="distill_loss", type="fp32", tokens=16384, vocab=33, k=8, temperature=2.0, pad=0),
        # a language model's vocabulary, bf16 logits
        dict(name="distill_vocab", op="distill_loss", type="bf16", tokens=8192, vocab=32000, k=32, temperature=1.0,
             pad=0),
        # one small batch of proteins
        dict(name="distill_bwd_small", op="distill_loss_backward", type="bf16", tokens=173, vocab=33, k=4,
             temperature=1.0, pad=0),
        dict(name="distill_bwd_esm", op="distill_loss_backward", type="fp32", tokens=16384, vocab=33, k=8,
             temperature=2.0, pad=0),
        # an odd vocabulary (rows that start off 16 bytes), many teacher logits
        dict(name="distill_bwd_vocab", op="distill_loss_backward", type="fp32", tokens=2048, vocab=50021, k=64,
             temperature=1.5, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention_window", "attention_window_backward", "distill_loss", "distill_loss_backward"])
    if op.startswith("distill"):
        vocab = rng.choice([33, _log(rng, 2, 64), _log(rng, 65, 4096), _log(rng, 4097, 131072)])
        tokens = _log(rng, 1, min(65536, 2 ** 26 // max(vocab, 64)))
        return dict(op=op, type=rng.choice(["fp32", "bf16"]), tokens=tokens, vocab=vocab,
                    k=min(vocab, rng.choice([1, 4, 8, 20, 32, 64, 100])), temperature=rng.choice([0.5, 1.0, 2.0, 4.0]),
                    pad=rng.choice([0, 0, 3, 31]))
    kind = "fp32" if op == "attention_window" and rng.random() < 0.15 else "bf16"
    heads = rng.choice([4, 8]) if kind == "fp32" else rng.choice([4, 8, 20, 40])
    tokens = _log(rng, 1, 1024 if kind == "fp32" else 8192 if heads == 40 else 16384)
    lengths, left_over = [], tokens
    while left_over > 0:
        n = min(left_over, _log(rng, 1, 4096) if rng.random() < 0.8 else left_over, 4096 if heads == 40 else 16384)
        lengths.append(n)
        left_over -= n
        if len(lengths) == 63:
            break
    longest = max(lengths)
    left, right = rng.choice([(0, 0), (7, 0), (1, 2), (64, 64), (100, 300), (128, 128), (511, 0), (1024, 1024),
                              (_log(rng, 1, 1500), _log(rng, 1, 1500)), (_log(rng, 1, 3000), 0)])
    if longest <= 2048 and rng.random() < 0.3:
        left = -1
        right = rng.choice([-1, 0, 64])
    case = dict(op=op, type=kind, heads=heads, lengths=",".join(str(n) for n in lengths), left=left, right=right,
                sinks=rng.choice([0, 1, 4, 5, 16, 33, 100]))
    if op == "attention_window":
        case["lse"] = kind == "bf16" and rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs
def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def _random(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def prepare(case, seed):
    g = _random(seed)
    s = dict(case)
    dt = DTYPES[case["type"]]
    if case["op"].startswith("attention"):
        lengths = _lengths(case)
        T, d = sum(lengths), HEAD * case["heads"]
        s["max_seqlen"] = max(lengths)
        s["cu"] = torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0).to(device="cuda", dtype=torch.int32)
        s["qkv"] = (1.25 * torch.randn(T, 3 * d, device="cuda", generator=g)).to(dt)
        if case["op"] == "attention_window_backward":
            s["o"], s["lse"] = _plain_attention(s)
            s["d_o"] = torch.randn(T, d, device="cuda", generator=g).to(dt)
        return s
    T, V, K = case["tokens"], case["vocab"], case["k"]
    rows = (2.0 * torch.randn(T, V + case["pad"], device="cuda", generator=g)).to(dt)
    s["logits"] = rows[:, :V]  # rows of a wider buffer where pad > 0
    teacher = s["logits"] + torch.randn(T, V, device="cuda", generator=g).to(dt)
    top = teacher.float().topk(K, dim=1)
    s["teacher_logits"] = top.values.contiguous()
    ids = top.indices.to(torch.int32)
    # some rows hold fewer entries than K, some tokens (padding, special tokens) are not scored
    have = torch.where(torch.rand(T, 1, device="cuda", generator=g) < 0.2,
                       torch.randint(0, K + 1, (T, 1), device="cuda", generator=g), K)
    s["teacher_ids"] = torch.where(torch.arange(K, device="cuda")[None] < have, ids, -1).contiguous()
    if case["op"] == "distill_loss_backward":
        _, s["lse"], _, s["count"] = _plain_distill(s)
    return s


# ---------------------------------------------------------------- plain forms
def _blocks(s):
    """Rows in blocks of BLOCK queries; per block the key rows that any of them can see, per
    query the sink rows outside its window; and what each query sees of them."""
    T, n = s["qkv"].shape[0], s["max_seqlen"] - 1
    left = n if s["left"] < 0 else min(s["left"], n)
    right = n if s["right"] < 0 else min(s["right"], n)
    cu = s["cu"].long()
    nb = -(-T // BLOCK)
    at = torch.arange(nb * BLOCK, device=cu.device).view(nb, BLOCK)
    keys = at[:, :1] - left + torch.arange(BLOCK + left + right, device=cu.device)[None]
    inside = (keys >= 0) & (keys < T)
    rows, keys = at.clamp(max=T - 1), keys.clamp(0, T - 1)
    seq = torch.searchsorted(cu[1:], rows, right=True)
    kseq = torch.searchsorted(cu[1:], keys, right=True)
    r, k = rows[:, :, None], keys[:, None, :]
    seen = inside[:, None, :] & (kseq[:, None, :] == seq[:, :, None]) & (k >= r - left) & (k <= r + right)
    sinks = cu[seq][:, :, None] + torch.arange(s["sinks"], device=cu.device)
    sink_seen = (sinks < cu[seq + 1][:, :, None]) & (sinks < r - left)
    return rows, keys, seen, sinks.clamp(max=T - 1), sink_seen


def _heads(x, heads):
    return x.float().view(x.shape[0], heads, HEAD)


def _plain_attention(s):
    T, H = s["qkv"].shape[0], s["heads"]
    rows, keys, seen, sinks, sink_seen = _blocks(s)
    q, k, v = (_heads(x, H) for x in s["qkv"].chunk(3, dim=1))
    qb = q[rows]
    a = torch.einsum("bqhd,bkhd->bhqk", qb, k[keys]).mul_(SCALE).masked_fill_(~seen[:, None], -math.inf)
    b = torch.einsum("bqhd,bqshd->bhqs", qb, k[sinks]).mul_(SCALE)
    b = b.masked_fill_(~sink_seen[:, None], -math.inf)
    m = a.amax(-1, keepdim=True)
    if s["sinks"]:
        m = torch.maximum(m, b.amax(-1, keepdim=True))
    a, b = a.sub_(m).exp_(), b.sub_(m).exp_()
    l = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    o = torch.einsum("bhqk,bkhd->bhqd", a, v[keys]) + torch.einsum("bhqs,bqshd->bhqd", b, v[sinks])
    o = (o / l).permute(0, 2, 1, 3).reshape(-1, H * HEAD)[:T].to(s["qkv"].dtype)
    lse = (m + l.log()).squeeze(-1).permute(1, 0, 2).reshape(H, -1)[:, :T].contiguous()
    return o, lse


def _plain_attention_backward(s):
    T, H = s["qkv"].shape[0], s["heads"]
    rows, keys, seen, sinks, sink_seen = _blocks(s)
    q, k, v = (_heads(x, H) for x in s["qkv"].chunk(3, dim=1))
    g = _heads(s["d_o"], H)
    live = (torch.arange(rows.numel(), device=rows.device) < T).view(rows.shape)[:, None, :, None]
    D = (g * _heads(s["o"], H)).sum(-1)[rows].permute(0, 2, 1)[..., None]
    lse = s["lse"].t()[rows].permute(0, 2, 1)[..., None]
    qb, gb, kb, vb, ks, vs = q[rows], g[rows], k[keys], v[keys], k[sinks], v[sinks]
    p = torch.einsum("bqhd,bkhd->bhqk", qb, kb).mul_(SCALE).sub_(lse).exp_().masked_fill_(~(seen[:, None] & live), 0)
    ps = torch.einsum("bqhd,bqshd->bhqs", qb, ks).mul_(SCALE).sub_(lse).exp_()
    ps = ps.masked_fill_(~(sink_seen[:, None] & live), 0)
    ds = torch.einsum("bqhd,bkhd->bhqk", gb, vb).sub_(D).mul_(p)
    dss = torch.einsum("bqhd,bqshd->bhqs", gb, vs).sub_(D).mul_(ps)
    dq = torch.einsum("bhqk,bkhd->bqhd", ds, kb) + torch.einsum("bhqs,bqshd->bqhd", dss, ks)
    dq = dq.reshape(-1, H, HEAD)[:T] * SCALE
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    at, sat = keys.reshape(-1), sinks.reshape(-1)
    dk.index_add_(0, at, torch.einsum("bhqk,bqhd->bkhd", ds, qb).reshape(-1, H, HEAD))
    dv.index_add_(0, at, torch.einsum("bhqk,bqhd->bkhd", p, gb).reshape(-1, H, HEAD))
    if s["sinks"]:
        dk.index_add_(0, sat, torch.einsum("bhqs,bqhd->bqshd", dss, qb).reshape(-1, H, HEAD))
        dv.index_add_(0, sat, torch.einsum("bhqs,bqhd->bqshd", ps, gb).reshape(-1, H, HEAD))
    return torch.cat([x.reshape(T, -1) for x in (dq, dk * SCALE, dv)], 1).to(s["qkv"].dtype)


def _teacher(s):
    """Teacher probabilities and their logarithms over the usable entries (0 elsewhere)."""
    use = s["teacher_ids"] >= 0
    a = (s["teacher_logits"] / s["temperature"]).masked_fill(~use, -math.inf)
    m = a.amax(1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0)
    e = (a - m).exp()
    l = e.sum(1, keepdim=True)
    p = torch.where(use, e / l, 0)
    logp = torch.where(use, a - m - l.log(), 0)
    return use, p, logp


def _plain_distill(s):
    use, p, logp = _teacher(s)
    z = s["logits"].float() / s["temperature"]
    m = z.amax(1, keepdim=True)
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    logq = z.gather(1, s["teacher_ids"].long().clamp(min=0)) - lse
    term = torch.where(p > 0, p * (logp - logq), 0)
    scored = use.any(1)
    loss = torch.where(scored, s["temperature"] ** 2 * term.sum(1), 0)
    lse = torch.where(scored, lse.squeeze(1), 0)
    return loss, lse, loss.double().sum().float().view(1), scored.sum().to(torch.int32).view(1)


def _plain_distill_backward(s):
    use, p, _ = _teacher(s)
    g = (s["logits"].float() / s["temperature"] - s["lse"][:, None]).exp_()
    g.scatter_add_(1, s["teacher_ids"].long().clamp(min=0), -p)
    g *= torch.where(use.any(1, keepdim=True), s["temperature"], 0) / s["count"].clamp(min=1)
    return g.to(s["logits"].dtype)


# ---------------------------------------------------------------- one pass
@functools.lru_cache(maxsize=None)
def _encoder(heads, precision):
    from transformer_esm_layer_gb300.binding import EsmEncoder
    return EsmEncoder(1, HEAD * heads, heads, 4 * HEAD * heads, max_positions=65536, precision=precision)


def _own(s):
    op = s["op"]
    if op.startswith("attention"):
        enc = _encoder(s["heads"], s["type"])
        T, B = s["qkv"].shape[0], s["cu"].numel() - 1
        window = (s["left"], s["right"], s["sinks"])
        backward = op == "attention_window_backward"
        if "workspace" not in s:
            s["workspace"] = enc.op_attention_window_workspace(T, B, window, backward=backward)
        if backward:
            dqkv = torch.empty_like(s["qkv"])
            enc.op_attention_window_backward(s["qkv"], s["o"], s["lse"], s["d_o"], s["cu"], s["max_seqlen"], window,
                                             dqkv, workspace=s["workspace"])
            return {"dqkv": dqkv}
        o = torch.empty(T, HEAD * s["heads"], dtype=s["qkv"].dtype, device="cuda")
        lse = torch.empty(s["heads"], T, device="cuda") if s["lse"] else None
        enc.op_attention_window(s["qkv"], s["cu"], s["max_seqlen"], window, o, lse=lse, workspace=s["workspace"])
        return {"o": o, "lse": lse}
    enc = _encoder(4, "bf16")
    if op == "distill_loss_backward":
        d_logits = torch.empty(s["logits"].shape, dtype=s["logits"].dtype, device="cuda")
        enc.op_distill_loss_backward(s["logits"], s["teacher_ids"], s["teacher_logits"], s["temperature"], s["lse"],
                                     d_logits, loss_count=s["count"])
        return {"d_logits": d_logits}
    T = s["logits"].shape[0]
    if "workspace" not in s:
        s["workspace"] = enc.op_distill_loss_workspace(T, s["vocab"])
    token_loss, lse = torch.empty(2, T, device="cuda")
    loss_sum = torch.empty(1, device="cuda")
    count = torch.empty(1, dtype=torch.int32, device="cuda")
    enc.op_distill_loss(s["logits"], s["teacher_ids"], s["teacher_logits"], s["temperature"], token_loss, lse,
                        loss_sum=loss_sum, count=count, workspace=s["workspace"])
    return {"token_loss": token_loss, "lse": lse, "loss_sum": loss_sum, "count": count}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "attention_window":
        o, lse = _plain_attention(s)
        return {"o": o, "lse": lse if s["lse"] else None}
    if s["op"] == "attention_window_backward":
        return {"dqkv": _plain_attention_backward(s)}
    if s["op"] == "distill_loss":
        return dict(zip(("token_loss", "lse", "loss_sum", "count"), _plain_distill(s)))
    return {"d_logits": _plain_distill_backward(s)}


# ---------------------------------------------------------------- the least work
def _visible(L, left, right, sinks):
    """Visible (query, key) pairs of one sequence."""
    total = 0
    for i in range(L):
        hi = L - 1 if right < 0 else min(L - 1, i + right)
        lo = 0 if left < 0 else max(0, i - left)
        total += hi - lo + 1 + min(sinks, lo)
    return total


def work(case):
    es = 2 if case["type"] == "bf16" else 4
    if case["op"].startswith("attention"):
        lengths, H = _lengths(case), case["heads"]
        T, d = sum(lengths), HEAD * H
        pairs = sum(_visible(n, case["left"], case["right"], case["sinks"]) for n in lengths)
        if case["op"] == "attention_window":
            return {"bytes": es * 4 * T * d + (4 * H * T if case["lse"] else 0), "flops": 4 * HEAD * H * pairs}
        return {"bytes": es * 8 * T * d + 4 * H * T, "flops": 10 * HEAD * H * pairs}
    T, V, K = case["tokens"], case["vocab"], case["k"]
    if case["op"] == "distill_loss":
        return {"bytes": es * T * V + 8 * T * K + 8 * T + 8, "flops": 3 * T * V}
    return {"bytes": 2 * es * T * V + 8 * T * K + 4 * T + 4, "flops": 3 * T * V}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_attention(s, backward):
    H, dev = s["heads"], s["qkv"].device
    x = s["qkv"].double().view(-1, 3, H, HEAD).permute(1, 2, 0, 3)  # [3, H, T, 64]
    out = torch.zeros(x.shape if backward else x.shape[1:], dtype=torch.float64, device=dev)
    lses = torch.zeros(H, x.shape[2], dtype=torch.float64, device=dev)
    start = 0
    for L in _lengths(s):
        q, k, v = x[:, :, start:start + L]
        for a in range(0, L, 512):
            i = torch.arange(a, min(L, a + 512), device=dev)
            lo = 0 if s["left"] < 0 else max(0, a - s["left"])
            hi = L if s["right"] < 0 else min(L, a + len(i) + s["right"])
            j = torch.cat([torch.arange(min(s["sinks"], lo), device=dev), torch.arange(lo, hi, device=dev)])
            ok = j[None] < s["sinks"]
            ok = torch.ones_like(ok) if s["left"] < 0 else ok | (j[None] >= i[:, None] - s["left"])
            if s["right"] >= 0:
                ok = ok & (j[None] <= i[:, None] + s["right"])
            qi, kj, vj = q[:, i], k[:, j], v[:, j]
            z = (qi @ kj.transpose(1, 2) / 8.0).masked_fill(~ok, -math.inf)
            lse = s["lse"][:, start + i].double()[..., None] if backward else z.logsumexp(2, keepdim=True)
            p = (z - lse).exp()
            if not backward:
                out[:, start + i] = p @ vj
                lses[:, start + i] = lse.squeeze(2)
                continue
            do = s["d_o"][start + i].double().view(-1, H, HEAD).transpose(0, 1)
            o = s["o"][start + i].double().view(-1, H, HEAD).transpose(0, 1)
            ds = p * (do @ vj.transpose(1, 2) - (do * o).sum(2, keepdim=True))
            out[0][:, start + i] = ds @ kj / 8.0
            out[1].index_add_(1, start + j, ds.transpose(1, 2) @ qi / 8.0)
            out[2].index_add_(1, start + j, p.transpose(1, 2) @ do)
        start += L
    if backward:
        return {"dqkv": out.permute(2, 0, 1, 3).reshape(x.shape[2], -1)}
    return {"o": out.transpose(0, 1).reshape(x.shape[2], -1), "lse": lses if s["lse"] else None}


def _exact_distill(s, backward):
    t, V = s["temperature"], s["vocab"]
    loss, lses, grad = [], [], []
    scored = (s["teacher_ids"] >= 0).any(1)
    n = max(1, int(scored.sum()))
    step = max(1, 2 ** 25 // V)
    for a in range(0, len(scored), step):
        rows = slice(a, a + step)
        ids, ok = s["teacher_ids"][rows].long(), scored[rows]
        y = s["logits"][rows].double() / t
        lse = s["lse"][rows].double() if backward else y.logsumexp(1)
        w = torch.where(ids >= 0, s["teacher_logits"][rows].double() / t, -math.inf).softmax(1)
        w = torch.where(ok[:, None] & (ids >= 0), w, 0)
        at = ids.clamp(min=0)
        if backward:
            d = (y - lse[:, None]).exp().scatter_add_(1, at, -w) * (t / n)
            grad.append(torch.where(ok[:, None], d, 0))
        else:
            kl = torch.xlogy(w, w) - w * (y.gather(1, at) - lse[:, None])
            loss.append(torch.where(ok, t * t * kl.sum(1), 0))
            lses.append(torch.where(ok, lse, 0))
    if backward:
        return {"d_logits": torch.cat(grad)}
    loss = torch.cat(loss)
    return {"token_loss": loss, "lse": torch.cat(lses), "loss_sum": loss.sum().view(1), "count": None}


def exact(case, seed):
    s = prepare(case, seed)
    backward = case["op"].endswith("_backward")
    return _exact_attention(s, backward) if case["op"].startswith("attention") else _exact_distill(s, backward)
