"""Cases of the packed-prompt operators: rotary positions, attention over packed sequences, log
probabilities of given tokens from logits, and the same from hidden states and the head matrix.

`run` computes a case in plain torch operations (own = False) or through the library's entry
points (own = True) on the same prepared state; `exact` computes it in 64 bits from the
definitions.
"""
import math

import torch

own = False


def listed():
    return [
        # one new token at a far position, query and key heads of the 8B-shaped decoder, positions
        # scaled by bands: latency
        dict(name="rope_one_token", op="rope", rows=1, heads=40, head_dim=128, pad=1024, rot=128, pairs="half",
             dtype="bf16", theta=1.0e6, scaling="bands", factor=4.0, orig=4096.0, low=1.0, high=32.0,
             magnitude=1.125, far=131072),
        # 16 prompts of 512: query and key heads inside the fused projection of the 1.7B-shaped decoder
        dict(name="rope_prompts", op="rope", rows=8192, heads=24, head_dim=128, pad=1024, rot=128, pairs="half",
             dtype="bf16", theta=1.0e6, scaling="none", factor=1.0, orig=0.0, low=0.0, high=0.0,
             magnitude=1.0, far=512),
        # half of each head rotated, neighbouring features paired, fp32, positions interpolated
        dict(name="rope_partial_f32", op="rope", rows=5003, heads=12, head_dim=64, pad=0, rot=32, pairs="interleaved",
             dtype="f32", theta=1.0e4, scaling="linear", factor=8.0, orig=0.0, low=0.0, high=0.0,
             magnitude=1.0, far=16384),
        # three short questions: latency
        dict(name="attention_tiny", op="attention", lens="7,1,19", extra=0, heads=16, kv_heads=8, head_dim=128),
        # classification prompts of mixed lengths in a buffer with room for more
        dict(name="attention_prompts", op="attention", lens=_lens_text(61, 1, 512, 5) + ",0,1,512", extra=77,
             heads=16, kv_heads=8, head_dim=128),
        # one head per key/value head, head dim 64, up to the longest position of those decoders
        dict(name="attention_hd64", op="attention", lens="2048,129,1777,64,1023,2000,300,5", extra=0,
             heads=12, kv_heads=12, head_dim=64),
        # two long documents, four query heads to a key/value head
        dict(name="attention_long", op="attention", lens="8191,4097", extra=0, heads=32, kv_heads=8, head_dim=128),
        # one sampled token with its five alternatives: latency
        dict(name="logprobs_one_row", op="logprobs", rows=1, vocab=50272, pad=0, dtype="bf16", top=5, masked=0.0),
        # all positions of a batch of completions over the large vocabulary
        dict(name="logprobs_batch", op="logprobs", rows=2048, vocab=151936, pad=0, dtype="bf16", top=8, masked=0.0),
        # fp32 logits of an odd vocabulary in padded rows, part of the tokens ruled out
        dict(name="logprobs_masked_f32", op="logprobs", rows=509, vocab=49999, pad=17, dtype="f32", top=20, masked=0.6),
        # a few answers scored against the head of the 125M-shaped decoder: the head is read once
        dict(name="head_few_rows", op="head", rows=5, vocab=50272, width=768),
        # a batch of completions scored against the head of the 1.7B-shaped decoder
        dict(name="head_batch", op="head", rows=4096, vocab=151936, width=2048),
    ]


def _lens_text(count, least, most, start):
    """`count` lengths between least and most, spread over their logarithm by a fixed rule."""
    span = math.log(most / least)
    return ",".join(str(int(least * math.exp(span * ((start + 37 * i) % 101) / 100.0))) for i in range(count))


def _spread(rng, least, most):
    return max(least, min(most, int(round(math.exp(rng.uniform(math.log(least), math.log(most)))))))


def draw(rng):
    op = rng.choice(["rope", "attention", "logprobs", "head"])
    if op == "rope":
        head_dim = rng.choice([64, 80, 96, 128, 256])
        rows = _spread(rng, 1, 30000)
        heads = rng.randint(1, max(1, min(64, (8192 * 24 * 128) // (rows * head_dim))))
        scaling = rng.choice(["none", "linear", "bands"])
        return dict(op="rope", rows=rows, heads=heads, head_dim=head_dim, pad=rng.choice([0, 3, 8, 1024]),
                    rot=rng.choice([head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)]),
                    pairs=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "f32"]),
                    theta=rng.choice([1.0e4, 5.0e5, 1.0e6]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    orig=4096.0 if scaling == "bands" else 0.0, low=1.0 if scaling == "bands" else 0.0,
                    high=rng.choice([4.0, 32.0]) if scaling == "bands" else 0.0,
                    magnitude=rng.choice([1.0, 1.25]), far=_spread(rng, 64, 1000000))
    if op == "attention":
        heads, kv_heads = rng.choice([(12, 12), (16, 8), (32, 8), (56, 56), (10, 2), (8, 1)])
        head_dim = rng.choice([64, 128])
        count = _spread(rng, 1, 64)
        # padded scores of the plain form and the products stay below the largest listed case's
        most = min(8192, int(math.sqrt(2.0 * 32 * 8191 ** 2 / (count * heads))))
        top = _spread(rng, 16, most)
        lens = [top] + [rng.choice([_spread(rng, 1, top), rng.randint(0, top)]) for _ in range(count - 1)]
        rng.shuffle(lens)
        return dict(op="attention", lens=",".join(map(str, lens)), extra=rng.choice([0, 3, 130]), heads=heads,
                    kv_heads=kv_heads, head_dim=head_dim)
    if op == "logprobs":
        vocab = _spread(rng, 1000, 152000)
        dtype = rng.choice(["bf16", "f32"])
        rows = _spread(rng, 1, min(16384, (2048 * 151936) // (vocab * (2 if dtype == "f32" else 1))))
        return dict(op="logprobs", rows=rows, vocab=vocab, pad=rng.choice([0, 0, 1, 64]), dtype=dtype,
                    top=rng.choice([0, 1, 5, 20, 32]), masked=rng.choice([0.0, 0.3, 0.999]))
    width = 8 * _spread(rng, 16, 512)
    vocab = _spread(rng, 1000, 152000)
    rows = _spread(rng, 1, max(1, min(8192, (4096 * 151936 * 2048) // (vocab * width))))
    return dict(op="head", rows=rows, vocab=vocab, width=width)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _rand(gen, *shape, scale=1.0, dtype=torch.float32):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16 if dtype == torch.bfloat16 else torch.float32)
    return x if scale == 1.0 else x.mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=dict(case))
    if case["op"] == "rope":
        # query and key heads inside rows that hold `pad` further features behind them
        dtype, width = _TYPES[case["dtype"]], case["heads"] * case["head_dim"]
        s["x"] = _rand(gen, case["rows"], width + case["pad"], dtype=dtype)
        s["out"] = torch.zeros(case["rows"], width, dtype=dtype, device="cuda")
        s["positions"] = torch.randint(0, case["far"], (case["rows"],), generator=gen, device="cuda", dtype=torch.int32)
    elif case["op"] == "attention":
        lens, e = _lens(case), case["head_dim"]
        total = sum(lens) + case["extra"]
        h, hk = case["heads"], case["kv_heads"]
        s["qkv"] = _rand(gen, total, (h + 2 * hk) * e, dtype=torch.bfloat16)
        s["out"] = torch.zeros(total, h * e, dtype=torch.bfloat16, device="cuda")
        s["cu_seqlens"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["longest"] = max(lens)
    elif case["op"] == "logprobs":
        # logits of a language model: a few tokens stand out, the given one is often among them
        dtype, rows, vocab = _TYPES[case["dtype"]], case["rows"], case["vocab"]
        x = _rand(gen, rows, vocab + case["pad"], scale=2.0, dtype=dtype)
        peak = torch.randint(0, vocab, (rows, 6), generator=gen, device="cuda")
        x.scatter_(1, peak, (8.0 + 4.0 * torch.randn(rows, 6, generator=gen, device="cuda")).to(dtype))
        other = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        targets = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.7, peak[:, 0], other)
        if case["masked"]:
            # part of the tokens is ruled out in every row; the given one stays
            drop = torch.rand(vocab + case["pad"], generator=gen, device="cuda") < case["masked"]
            kept = x.gather(1, targets[:, None])
            x.masked_fill_(drop[None, :], -math.inf)
            x.scatter_(1, targets[:, None], kept)
        if rows > 8:
            targets[::8] = -1  # a prompt's own tokens are not scored
        s["logits"], s["targets"] = x, targets.to(torch.int32)
        s["logprob"] = torch.zeros(rows, dtype=torch.float32, device="cuda")
        s["entropy"] = torch.zeros(rows, dtype=torch.float32, device="cuda")
        s["top_ids"] = torch.zeros(rows, case["top"], dtype=torch.int32, device="cuda")
        s["top_logprobs"] = torch.zeros(rows, case["top"], dtype=torch.float32, device="cuda")
    else:
        rows, vocab, width = case["rows"], case["vocab"], case["width"]
        s["hidden"] = _rand(gen, rows, width, dtype=torch.bfloat16)
        s["head"] = _rand(gen, vocab, width, scale=0.05, dtype=torch.bfloat16)
        s["targets"] = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        if rows > 8:
            s["targets"][::8] = -1
        s["logprob"] = torch.zeros(rows, dtype=torch.float32, device="cuda")
        s["entropy"] = torch.zeros(rows, dtype=torch.float32, device="cuda")
    if own:
        # what a program of the library keeps: its context, the workspace, the rotation's settings
        import zero_order_forward_b200 as zo
        s["ctx"] = _context(zo)
        if case["op"] == "head":
            need = zo.zo_head_logprobs_workspace(case["rows"], case["vocab"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        if case["op"] == "rope":
            s["rope"] = dict(theta=case["theta"], rot_dim=case["rot"], interleaved=case["pairs"] == "interleaved",
                             scaling=case["scaling"], factor=case["factor"], orig_len=case["orig"],
                             band_low=case["low"], band_high=case["high"], magnitude=case["magnitude"])
    return s


_contexts = []


def _context(zo):
    """The one context of the program (these operators read none of its parameters)."""
    if not _contexts:
        _contexts.append(zo.zo_create(torch.zeros(64, dtype=torch.bfloat16, device="cuda")))
    return _contexts[0]


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


def _own(s):
    import zero_order_forward_b200 as zo
    c, ctx = s["case"], s["ctx"]
    if c["op"] == "rope":
        x, out = s["x"], s["out"]
        zo.zo_rope(ctx, x, out, s["positions"], s["rope"], c["rows"], x.shape[1], out.shape[1], c["heads"], c["head_dim"])
        return out
    if c["op"] == "attention":
        h, hk, e = c["heads"], c["kv_heads"], c["head_dim"]
        qkv, out = s["qkv"], s["out"]
        ld = qkv.shape[1]
        zo.zo_attention_packed(ctx, qkv, qkv[:, h * e:], qkv[:, (h + hk) * e:], out, s["cu_seqlens"],
                               s["cu_seqlens"].numel() - 1, qkv.shape[0], ld, ld, ld, h * e, h, hk, e, 1.0 / math.sqrt(e))
        return out
    if c["op"] == "logprobs":
        x = s["logits"]
        zo.zo_logprobs(ctx, x, c["rows"], c["vocab"], x.shape[1], s["targets"], s["logprob"], s["entropy"],
                       c["top"], s["top_ids"], s["top_logprobs"])
        return _with_top(s, s["logprob"], s["entropy"], s["top_ids"], s["top_logprobs"])
    zo.zo_head_logprobs(ctx, s["hidden"], s["head"], c["rows"], c["vocab"], c["width"], c["width"], c["width"],
                        s["targets"], s["logprob"], s["entropy"], s["workspace"])
    return dict(logprob=s["logprob"], entropy=s["entropy"])


def _with_top(s, logprob, entropy, ids, values):
    out = dict(logprob=logprob, entropy=entropy)
    if s["case"]["top"]:
        out.update(top_ids=ids, top_logprobs=values)
    return out


# ---------------------------------------------------------------- plain forms


def _frequencies(c):
    """Radians per position of each pair, in 64 bits."""
    half = torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64)
    f = c["theta"] ** (-half / c["rot"])
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "bands":
        turns = c["orig"] * f / (2.0 * math.pi)
        keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / c["factor"]
    return f


def _plain_rope(s):
    c = s["case"]
    rows, heads, e, rot = c["rows"], c["heads"], c["head_dim"], c["rot"]
    x = s["x"][:, : heads * e].reshape(rows, heads, e)
    angle = s["positions"].double()[:, None] * _frequencies(c)[None, :]
    cos = (angle.cos() * c["magnitude"]).float()[:, None, :]
    sin = (angle.sin() * c["magnitude"]).float()[:, None, :]
    y = x.float()
    if c["pairs"] == "interleaved":
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned.to(x.dtype), x[..., rot:]], dim=-1).reshape(rows, heads * e)


def _plain_attention(s):
    c = s["case"]
    h, hk, e, top = c["heads"], c["kv_heads"], c["head_dim"], s["longest"]
    start, end = s["cu_seqlens"][:-1].long(), s["cu_seqlens"][1:].long()
    at = torch.arange(top, device="cuda")
    inside = at[None, :] < (end - start)[:, None]
    index = (start[:, None] + at[None, :]).where(inside, torch.zeros_like(at)[None, :])
    rows = s["qkv"].float()[index]                      # [sequences][longest][features]
    n = rows.shape[0]
    q = rows[..., : h * e].reshape(n, top, hk, h // hk, e).permute(0, 2, 3, 1, 4)
    k = rows[..., h * e: (h + hk) * e].reshape(n, top, hk, 1, e).permute(0, 2, 3, 4, 1)
    v = rows[..., (h + hk) * e:].reshape(n, top, hk, 1, e).permute(0, 2, 3, 1, 4)
    p = torch.matmul(q, k).mul_(1.0 / math.sqrt(e))
    p.masked_fill_(at[None, :] > at[:, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v).div_(total).permute(0, 3, 1, 2, 4).reshape(n, top, h * e)
    s["out"][index[inside]] = o[inside].to(s["out"].dtype)
    return s["out"]


def _from_logits(x, targets):
    """(logprob, entropy, log of the sum) of fp32 rows; a negative target scores 0."""
    top = x.amax(-1, keepdim=True)
    shifted = x - top
    p = shifted.exp()
    total = p.sum(-1, keepdim=True)
    weighted = (p * shifted.clamp(min=-1.0e30)).sum(-1, keepdim=True)
    log_total = total.log()
    lse = top + log_total
    given = shifted.gather(1, targets.long().clamp(min=0)[:, None]) - log_total
    logprob = torch.where(targets < 0, torch.zeros_like(given[:, 0]), given[:, 0])
    return logprob, (log_total - weighted / total)[:, 0], lse


def _plain_logprobs(s):
    c = s["case"]
    x = s["logits"][:, : c["vocab"]]
    f = x.float()
    logprob, entropy, lse = _from_logits(f, s["targets"])
    if not c["top"]:
        return _with_top(s, logprob, entropy, None, None)
    # order by value, then by lowest index: one whole number for both
    bits = (f + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = order * 2 ** 31 + (2 ** 31 - 1 - torch.arange(c["vocab"], device="cuda"))
    ids = (2 ** 31 - 1) - (key.topk(c["top"], dim=1).values % 2 ** 31)
    return _with_top(s, logprob, entropy, ids.to(torch.int32), f.gather(1, ids) - lse)


def _plain_head(s):
    x = torch.matmul(s["hidden"].float(), s["head"].float().t())
    logprob, entropy, _ = _from_logits(x, s["targets"])
    return dict(logprob=logprob, entropy=entropy)


_PLAIN = dict(rope=_plain_rope, attention=_plain_attention, logprobs=_plain_logprobs, head=_plain_head)


# ---------------------------------------------------------------- from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _exact_rope(c, s)
    if c["op"] == "attention":
        return _exact_attention(c, s)
    if c["op"] == "logprobs":
        rows = s["logits"][:, : c["vocab"]]
        return _exact_scores(s, c["rows"], 64, lambda a, b: rows[a:b].double(), c["top"])
    head = s["head"].double()
    return _exact_scores(s, c["rows"], 256, lambda a, b: s["hidden"][a:b].double() @ head.T, 0)


def _exact_rope(c, s):
    rows, heads, e, rot = c["rows"], c["heads"], c["head_dim"], c["rot"]
    x = s["x"][:, : heads * e].reshape(rows, heads, e).double()
    rate = []
    for i in range(rot // 2):
        f = math.pow(c["theta"], -2.0 * i / rot)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "bands":
            share = (c["orig"] * f / (2.0 * math.pi) - c["low"]) / (c["high"] - c["low"])
            share = min(1.0, max(0.0, share))
            f = share * f + (1.0 - share) * (f / c["factor"])
        rate.append(f)
    angle = torch.outer(s["positions"].double(), torch.tensor(rate, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(angle, c["magnitude"]), angle)[:, None, :]
    first = slice(0, rot, 2) if c["pairs"] == "interleaved" else slice(0, rot // 2)
    second = slice(1, rot, 2) if c["pairs"] == "interleaved" else slice(rot // 2, rot)
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y.reshape(rows, heads * e)


def _exact_attention(c, s):
    h, hk, e = c["heads"], c["kv_heads"], c["head_dim"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for n in _lens(c):
        for g in range(h if n else 0):
            kv = g // (h // hk)
            part = s["qkv"][at: at + n].double()
            q = part[:, g * e: (g + 1) * e]
            k = part[:, (h + kv) * e: (h + kv + 1) * e]
            v = part[:, (h + hk + kv) * e: (h + hk + kv + 1) * e]
            score = q @ k.T / math.sqrt(e)
            score += torch.full_like(score, -math.inf).triu(1)
            out[at: at + n, g * e: (g + 1) * e] = torch.softmax(score, -1) @ v
        at += n
    return out


def _exact_scores(s, count, step, logits, top):
    logprob, entropy, ids, values = [], [], [], []
    for a in range(0, count, step):
        logp = torch.log_softmax(logits(a, min(a + step, count)), -1)
        t = s["targets"][a: a + step].long()
        logprob.append(torch.where(t >= 0, logp[torch.arange(len(t), device="cuda"), t.clamp(min=0)], 0.0))
        entropy.append(-torch.special.xlogy(logp.exp(), logp.exp()).sum(-1))
        if top:
            best, index = logp.sort(dim=-1, descending=True, stable=True)
            ids.append(index[:, :top].to(torch.int32))
            values.append(best[:, :top])
    out = dict(logprob=torch.cat(logprob), entropy=torch.cat(entropy))
    if top:
        out.update(top_ids=torch.cat(ids), top_logprobs=torch.cat(values))
    return out


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=2 * c["rows"] * c["heads"] * c["head_dim"] * size + 4 * c["rows"],
                    flops=3 * c["rows"] * c["heads"] * c["rot"])
    if c["op"] == "attention":
        tokens = sum(_lens(c))
        return dict(bytes=2 * tokens * c["head_dim"] * 2 * (c["heads"] + c["kv_heads"]),
                    flops=4 * c["head_dim"] * c["heads"] * sum(n * (n + 1) // 2 for n in _lens(c)))
    if c["op"] == "logprobs":
        size = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=c["rows"] * (c["vocab"] * size + 12 + 8 * c["top"]), flops=5 * c["rows"] * c["vocab"])
    return dict(bytes=2 * c["width"] * (c["vocab"] + c["rows"]) + 12 * c["rows"],
                flops=2 * c["rows"] * c["vocab"] * c["width"])
