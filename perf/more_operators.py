"""Measured cases of the operators between a language model's matrix products: the embedding of tokens, layer norm and
dropout with their gradients, and the log probabilities of given tokens with their gradient.

``run`` computes a case in plain torch operations, or, with ``own``, through the library's entry points.  Tokens fall as
words do, the n-th most frequent about 1/n times as often as the first; a share of them is padding (-1)."""

import functools
import math

import torch

own = False

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
SEED, OFFSET = 0x9E3779B97F4A7C15 >> 1, 12


# ---------------------------------------------------------------- cases

def listed():
    return [
        # BERT-large's table in fp32 as the optimizer holds it, embedded for a forward pass in bf16
        dict(name="embed_many", op="embed", tokens=65536, vocab=30522, dim=1024, table="f32", dtype="bf16", scale=32.0,
             padding=0.0, long=True),
        # the gradient of one micro-batch of ragged sequences, into a gradient field that every row of is written
        dict(name="embed_back_ragged", op="embed_back", tokens=4093, vocab=30522, dim=1024, dtype="bf16", table="f32",
             scale=1.0, padding=0.12, long=False, accumulate=False),
        # GPT-2-medium's table, which the output projection shares: added to the gradient that is there
        dict(name="embed_back_many", op="embed_back", tokens=65536, vocab=50257, dim=1024, dtype="bf16", table="f32",
             scale=1.0, padding=0.0, long=True, accumulate=True),
        # a token or a few at a time, where a call is all latency
        dict(name="norm_few", op="norm", rows=3, dim=1024, dtype="f32", params="f32", bias=True, pad=0),
        # a layer of BERT-large or GPT-2-medium over 64 sequences of 1,024
        dict(name="norm_many", op="norm", rows=65536, dim=1024, dtype="bf16", params="f32", bias=True, pad=0),
        # rows of no round size, as views of wider ones
        dict(name="norm_back_odd", op="norm_back", rows=1531, dim=769, dtype="f32", params="f32", bias=True, pad=3),
        # the gradient of the large layer, with the weight's and the bias's over 65,536 rows
        dict(name="norm_back_many", op="norm_back", rows=65536, dim=1024, dtype="bf16", params="f32", bias=True, pad=0),
        # a small odd branch in fp32; without a residual the same call is the gradient's
        dict(name="drop_odd", op="drop", rows=197, dim=1023, dtype="f32", p=0.1, residual=False),
        # the residual branch of the large layer
        dict(name="drop_many", op="drop", rows=65536, dim=1024, dtype="bf16", p=0.1, residual=True),
        # generation: a few sequences' next tokens over GPT-2's vocabulary, with the alternatives
        dict(name="logp_few", op="logp", rows=4, vocab=50257, dtype="bf16", top=8, entropy=True, masked=0.0, scale=1.0,
             pad=0),
        # the loss of 8 sequences of 1,024 over GPT-2's vocabulary, a tenth of them padding
        dict(name="logp_many", op="logp", rows=8192, vocab=50257, dtype="bf16", top=0, entropy=True, masked=0.1, scale=1.0,
             pad=47),
        # and its gradient
        dict(name="logp_back_many", op="logp_back", rows=8192, vocab=50257, dtype="bf16", entropy=True, masked=0.1,
             scale=1.0, pad=47),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["embed", "embed_back", "norm", "norm_back", "drop", "drop", "logp", "logp_back"])
    dtype = rng.choice(["f32", "bf16"])
    if op.startswith("embed"):
        dim = log(8, 4096)
        case = dict(op=op, tokens=min(log(1, 65536), 67_000_000 // dim), vocab=min(log(64, 200_000), 51_000_000 // dim),
                    dim=dim, table=rng.choice(["f32", "bf16"]), dtype=dtype, scale=rng.choice([1.0, math.sqrt(dim)]),
                    padding=rng.choice([0.0, rng.uniform(0.01, 0.5)]), long=rng.choice([True, False]))
        if op == "embed_back":
            case["accumulate"] = case["table"] == "f32" and rng.choice([True, False])
        return case
    if op.startswith("norm"):
        dim = log(8, 16384)
        return dict(op=op, rows=min(log(1, 65536), 67_000_000 // dim), dim=dim, dtype=dtype,
                    params=rng.choice(["f32", "bf16"]), bias=rng.choice([True, False]), pad=rng.choice([0, 0, rng.randint(1, 64)]))
    if op == "drop":
        dim = log(8, 16384)
        return dict(op=op, rows=min(log(1, 65536), 67_000_000 // dim), dim=dim, dtype=dtype, p=rng.uniform(0.01, 0.6),
                    residual=rng.choice([True, False]))
    vocab = log(2, 200_000)
    case = dict(op=op, rows=min(log(1, 8192), (400_000_000 if dtype == "bf16" else 200_000_000) // vocab), vocab=vocab,
                dtype=dtype, entropy=rng.choice([True, False]), masked=rng.choice([0.0, rng.uniform(0.01, 0.5)]),
                scale=rng.choice([1.0, 1 / rng.uniform(0.5, 1.5)]), pad=rng.choice([0, 0, rng.randint(1, 64)]))
    if op == "logp":
        case["top"] = rng.choice([0, rng.randint(1, min(20, vocab))])
    return case


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    make = dict(embed=_prepare_embed, norm=_prepare_norm, drop=_prepare_drop, logp=_prepare_logp)
    make[case["op"].split("_")[0]](s, case, gen)
    return s


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _tokens(gen, n, vocab, padding, long):
    """Words by their frequency's rank, which is spread over the vocabulary."""
    rank = torch.exp(torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * math.log(vocab)).long() - 1
    tokens = (rank.clamp(0, vocab - 1) * 7919 + 101) % vocab
    tokens = torch.where(torch.rand(n, generator=gen, device="cuda") < padding, -1, tokens)
    return tokens if long else tokens.int()


def _rows(gen, rows, dim, pad, dtype):
    """Rows with an offset each and columns that some of are much larger than others, as a residual stream has them."""
    x = _normal(gen, rows, dim + pad) * torch.exp(_normal(gen, dim + pad) * 0.5) + _normal(gen, rows, 1) * 0.5
    return x.to(KINDS[dtype])[:, :dim]


def _prepare_embed(s, c, gen):
    s["tokens"] = _tokens(gen, c["tokens"], c["vocab"], c["padding"], c["long"])
    if c["op"] == "embed":
        s["table"] = (_normal(gen, c["vocab"], c["dim"]) * 0.02).to(KINDS[c["table"]])
        s["out"] = torch.empty(c["tokens"], c["dim"], dtype=KINDS[c["dtype"]], device="cuda")
    else:
        s["grad"] = (_normal(gen, c["tokens"], c["dim"]) * 1e-3).to(KINDS[c["dtype"]])
        s["out"] = (_normal(gen, c["vocab"], c["dim"]) * 1e-3).to(KINDS[c["table"]])


def _prepare_norm(s, c, gen):
    s["x"] = _rows(gen, c["rows"], c["dim"], c["pad"], c["dtype"])
    s["weight"] = (1 + _normal(gen, c["dim"]) * 0.1).to(KINDS[c["params"]])
    s["bias"] = (_normal(gen, c["dim"]) * 0.1).to(KINDS[c["params"]]) if c["bias"] else None
    s["out"] = torch.empty(c["rows"], c["dim"], dtype=KINDS[c["dtype"]], device="cuda")
    if c["op"] == "norm_back":
        s["grad"] = (_normal(gen, c["rows"], c["dim"]) * 1e-3).to(KINDS[c["dtype"]])
        s["stats"] = _norm_plain(s)[1]
        s["grad_weight"] = torch.empty_like(s["weight"])
        s["grad_bias"] = torch.empty_like(s["weight"]) if c["bias"] else None


def _prepare_drop(s, c, gen):
    s["x"] = _rows(gen, c["rows"], c["dim"], 0, c["dtype"])
    s["residual"] = _rows(gen, c["rows"], c["dim"], 0, c["dtype"]) if c["residual"] else None
    s["out"] = torch.empty_like(s["x"])
    s["seed"] = SEED + int(torch.randint(1 << 40, (1,), generator=gen, device="cuda"))


def _prepare_logp(s, c, gen):
    n, v = c["rows"], c["vocab"]
    # a vocabulary that some words of are likelier everywhere, and what this place says
    x = _normal(gen, n, v + c["pad"])
    s["logits"] = x.mul_(2.0).add_(_normal(gen, v + c["pad"])).to(KINDS[c["dtype"]])[:, :v]
    del x
    s["targets"] = _tokens(gen, n, v, c["masked"], True)
    if c["op"] == "logp_back":
        s["grad_logp"] = _normal(gen, n) / n
        s["grad_entropy"] = _normal(gen, n) * 0.01 / n if c["entropy"] else None
        plain = _logp_plain(dict(s, case=dict(c, top=0)))
        s["stats"], s["entropy"] = plain["stats"], plain.get("entropy")
        s["out"] = torch.empty(n, v, dtype=KINDS[c["dtype"]], device="cuda")


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    return dict(embed=_embed_plain, embed_back=_embed_back_plain, norm=_norm_plain, norm_back=_norm_back_plain,
                drop=_drop_plain, logp=_logp_plain, logp_back=_logp_back_plain)[op](s)


def _run_own(s, op):
    import reduction_reducer_gb300 as lib
    c = s["case"]
    if op == "embed":
        return lib.embed(s["table"], s["tokens"], scale=c["scale"], out=s["out"])
    if op == "embed_back":
        return lib.embed_backward(s["grad"], s["tokens"], s["out"], scale=c["scale"], accumulate=c["accumulate"])
    if op == "norm":
        return lib.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out=s["out"])
    if op == "norm_back":
        return lib.layer_norm_backward(s["grad"], s["x"], s["stats"], s["weight"], grad_weight=s["grad_weight"],
                                       grad_bias=s["grad_bias"], out=s["out"])
    if op == "drop":
        return lib.drop(s["x"], c["p"], s["seed"], offset=OFFSET, residual=s["residual"], out=s["out"])
    if op == "logp":
        got = lib.logprobs(s["logits"], s["targets"], top=c["top"], scale=c["scale"], entropy=c["entropy"])
        return {n: x for n, x in got._asdict().items() if x is not None}
    return lib.logprobs_backward(s["grad_logp"], s["logits"], s["targets"], s["stats"], scale=c["scale"],
                                 entropy=s["entropy"], grad_entropy=s["grad_entropy"], out=s["out"])


# ---------------------------------------------------------------- plain forms

def _embed_plain(s):
    c, t = s["case"], s["tokens"].long()
    y = s["table"][t.clamp(min=0)].float() * c["scale"]
    return torch.where((t >= 0).unsqueeze(1), y, 0.0).to(KINDS[c["dtype"]])


def _embed_back_plain(s):
    c, t = s["case"], s["tokens"].long()
    g = torch.where((t >= 0).unsqueeze(1), s["grad"].float() * c["scale"], 0.0)
    if c["accumulate"]:
        return s["out"].index_add_(0, t.clamp(min=0), g)
    d = torch.zeros(c["vocab"], c["dim"], device="cuda").index_add_(0, t.clamp(min=0), g)
    return s["out"].copy_(d)


def _norm_plain(s):
    """y, and each row's mean and 1 / sqrt(variance + eps)."""
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + EPS).sqrt()
    y = (x - mean) * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype), torch.cat([mean, rstd], 1)


def _norm_back_plain(s):
    x, dy, w = s["x"].float(), s["grad"].float(), s["weight"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xh, g = (x - mean) * rstd, dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dw = (dy * xh).sum(0).to(s["weight"].dtype)
    return dx.to(s["x"].dtype), dw, None if s["bias"] is None else dy.sum(0).to(s["weight"].dtype)


def _philox_round(counter, key):
    """One round of Philox4x32 on words held in 64 bits; products past 63 bits wrap, and keep their bits."""
    c0, c1, c2, c3 = counter
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    low = 0xFFFFFFFF
    return ((b >> 32) & low) ^ c1 ^ key[0], b & low, ((a >> 32) & low) ^ c3 ^ key[1], a & low


def _random_plain(n, seed, offset):
    """32 random bits for each of n elements: eight of them take their upper halves from the four words of one block
    of Philox4x32-10, and their lower halves from those of another."""
    group = torch.arange(-(-n // 8), device="cuda")
    keys = [((seed + i * 0x9E3779B9) & 0xFFFFFFFF, ((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF) for i in range(10)]
    zero = torch.zeros_like(group)
    upper, lower = (torch.stack(functools.reduce(_philox_round, keys, (
        group & 0xFFFFFFFF, group >> 32, zero + (offset & 0xFFFFFFFF), zero + (offset >> 32 | which << 31))), 1)
        for which in (0, 1))
    bits = torch.stack([(upper & 0xFFFF) << 16 | (lower & 0xFFFF), (upper >> 16) << 16 | lower >> 16], 2)
    return bits.view(-1)[:n]


def _drop_plain(s):
    c, x = s["case"], s["x"]
    keep = _random_plain(x.numel(), s["seed"], OFFSET).view(x.shape) >= round(c["p"] * 2 ** 32)
    y = torch.where(keep, x.float() * (1 / (1 - c["p"])), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype)


def _logp_plain(s):
    """A row without a target (-1) is left out: zeros, and alternatives of -1."""
    c, t = s["case"], s["targets"]
    live = t >= 0
    z = s["logits"].float() * c["scale"]
    top = z.amax(1, keepdim=True)
    z = z - top
    e = torch.exp(z)
    total = e.sum(1)
    out = dict(logp=torch.where(live, z.gather(1, t.clamp(min=0).unsqueeze(1)).squeeze(1) - total.log(), 0.0),
               stats=torch.where(live.unsqueeze(1), torch.cat([top, total.log().unsqueeze(1)], 1), 0.0))
    if c["entropy"]:
        out["entropy"] = torch.where(live, total.log() - e.mul_(z).sum(1) / total, 0.0)
    del e
    if c["top"]:
        order = s["logits"].sort(dim=1, descending=True, stable=True).indices[:, :c["top"]]
        out["top_index"] = torch.where(live.unsqueeze(1), order, -1).int()
        out["top_logp"] = torch.where(live.unsqueeze(1), z.gather(1, order) - total.log().unsqueeze(1), 0.0)
    return out


def _logp_back_plain(s):
    c, t = s["case"], s["targets"]
    live = (t >= 0).unsqueeze(1)
    logp = s["logits"].float() * c["scale"] - s["stats"][:, :1] - s["stats"][:, 1:]
    p = torch.exp(logp)
    g = s["grad_logp"].unsqueeze(1)
    if c["entropy"]:
        d = p * -(s["grad_entropy"].unsqueeze(1) * (logp + s["entropy"].unsqueeze(1)) + g)
    else:
        d = p * -g
    d = d.scatter_add_(1, t.clamp(min=0).unsqueeze(1), g).mul_(c["scale"])
    return torch.where(live, d, 0.0).to(s["logits"].dtype)


# ---------------------------------------------------------------- work

def work(case):
    size = {"f32": 4, "bf16": 2}
    op, act = case["op"], size[case["dtype"]]
    if op.startswith("embed"):
        n, v, d, table = case["tokens"], case["vocab"], case["dim"], size[case["table"]]
        met = _distinct(n * (1 - case["padding"]), v)
        tokens = n * (8 if case["long"] else 4)
        if op == "embed":
            return {"bytes": int(tokens + met * d * table + n * d * act), "flops": n * d}
        read = n * (1 - case["padding"]) * d * act
        return {"bytes": int(tokens + read + (met * 2 if case["accumulate"] else v) * d * table), "flops": n * d}
    if op.startswith("logp"):
        n, v, live = case["rows"], case["vocab"], case["rows"] * (1 - case["masked"])
        if op == "logp":
            return {"bytes": int(live * v * act + n * (20 + 4 * case["entropy"] + 8 * case["top"])), "flops": int(live * v * 6)}
        return {"bytes": int((live + n) * v * act + n * (20 + 8 * case["entropy"])), "flops": int(live * v * 6)}
    n, d = case["rows"], case["dim"]
    if op == "drop":
        return {"bytes": n * d * act * (3 if case["residual"] else 2), "flops": n * d * 2}
    params = size[case["params"]] * d * (2 if case["bias"] else 1)
    if op == "norm":
        return {"bytes": 2 * n * d * act + 8 * n + params, "flops": n * d * 8}
    return {"bytes": 3 * n * d * act + 8 * n + params + size[case["params"]] * d, "flops": n * d * 14}


def _distinct(n, vocab):
    """About how many words of the vocabulary n tokens of ``_tokens`` meet: the r-th falls with probability
    log((r + 1) / r) / log(vocab)."""
    steps = 400
    edges = [vocab ** (i / steps) for i in range(steps + 1)]
    return sum((b - a) * -math.expm1(-n / ((a + b) / 2 * math.log(vocab))) for a, b in zip(edges, edges[1:]))


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return dict(embed=_exact_embed, embed_back=_exact_embed_back, norm=_exact_norm, norm_back=_exact_norm_back,
                drop=_exact_drop, logp=_exact_logp, logp_back=_exact_logp_back)[case["op"]](s)


def _exact_embed(s):
    y = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    there = s["tokens"] >= 0
    y[there] = s["table"].double()[s["tokens"][there].long()] * s["case"]["scale"]
    return y


def _exact_embed_back(s):
    """Sums of the sorted tokens' rows, as differences of one running sum for each column block."""
    c = s["case"]
    d = s["out"].double() if c["accumulate"] else torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    tokens, order = s["tokens"].long().sort(stable=True)
    words, count = tokens.unique_consecutive(return_counts=True)
    end = count.cumsum(0)
    for a in range(0, c["dim"], 256):
        run_ = s["grad"][:, a:a + 256].double()[order].cumsum(0)[end - 1]
        part = torch.cat([run_[:1], run_[1:] - run_[:-1]]) * c["scale"]
        d[words[words >= 0], a:a + 256] += part[words >= 0]
    return d


def _exact_norm(s):
    x = s["x"].double()
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = torch.rsqrt(var + EPS)
    y = torch.addcmul(torch.zeros((), dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double(),
                      (x - mean[:, None]) * rstd[:, None], s["weight"].double())
    return y, torch.stack([mean, rstd], 1)


def _exact_norm_back(s):
    """By differentiating the definition."""
    x, w = s["x"].double().requires_grad_(True), s["weight"].double().requires_grad_(True)
    b = torch.zeros_like(w).requires_grad_(True)
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    y = (x - mean) / (var + EPS).sqrt() * w + b
    dx, dw, db = torch.autograd.grad(y, (x, w, b), s["grad"].double())
    return dx, dw, None if s["bias"] is None else db


def _exact_words(lo, hi, seed, offset, which):
    """Philox4x32-10 with its products taken in parts of 16 bits."""
    def product(x, m):
        p = [(x & 0xFFFF) * (m & 0xFFFF), (x >> 16) * (m & 0xFFFF), (x & 0xFFFF) * (m >> 16), (x >> 16) * (m >> 16)]
        mid = (p[0] >> 16) + (p[1] & 0xFFFF) + (p[2] & 0xFFFF)
        return p[3] + (p[1] >> 16) + (p[2] >> 16) + (mid >> 16), (mid & 0xFFFF) << 16 | p[0] & 0xFFFF
    x = [lo, hi, torch.full_like(lo, offset % 2 ** 32), torch.full_like(lo, offset // 2 ** 32 + which * 2 ** 31)]
    k = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = product(x[0], 0xD2511F53)
        h1, l1 = product(x[2], 0xCD9E8D57)
        x = [torch.bitwise_xor(torch.bitwise_xor(h1, x[1]), torch.full_like(lo, k[0])), l1,
             torch.bitwise_xor(torch.bitwise_xor(h0, x[3]), torch.full_like(lo, k[1])), l0]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return x


def _exact_drop(s):
    c, x = s["case"], s["x"].double().reshape(-1)
    element = torch.arange(x.numel(), device="cuda")
    group, place = element // 8, element % 8
    u = 0
    for which in (0, 1):
        words = torch.stack(_exact_words(group[::8] % 2 ** 32, group[::8] // 2 ** 32, s["seed"], OFFSET, which))
        word = words[place // 2, group]
        u = u * 65536 + torch.where(place % 2 == 1, word // 65536, word % 65536)
    y = torch.where(u < round(c["p"] * 2 ** 32), 0.0, x / (1 - c["p"]))
    return (y if s["residual"] is None else y + s["residual"].double().reshape(-1)).view(s["x"].shape)


def _exact_logp(s):
    """Row block by row block."""
    c = s["case"]
    parts = []
    for a in range(0, c["rows"], 1024):
        t = s["targets"][a:a + 1024]
        live = (t >= 0).double()
        logp = torch.log_softmax(s["logits"][a:a + 1024].double() * c["scale"], 1)
        part = [logp[torch.arange(len(t), device="cuda"), t.clamp(min=0)] * live]
        top = s["logits"][a:a + 1024].amax(1).double() * c["scale"]
        log_sum = torch.logsumexp(s["logits"][a:a + 1024].double() * c["scale"] - top.unsqueeze(1), 1)
        part.append(torch.stack([top, log_sum], 1) * live.unsqueeze(1))
        if c["entropy"]:
            part.append(torch.special.entr(logp.exp()).sum(1) * live)
        if c["top"]:
            part.append(logp.topk(c["top"], 1).values * live.unsqueeze(1))
        parts.append(part)
    names = ["logp", "stats"] + ["entropy"] * c["entropy"] + ["top_logp"] * (c["top"] > 0)
    out = {n: torch.cat([p[i] for p in parts]) for i, n in enumerate(names)}
    return dict(out, top_index=None) if c["top"] else out


def _exact_logp_back(s):
    """By differentiating the definition, row block by row block."""
    c = s["case"]
    out = []
    for a in range(0, c["rows"], 1024):
        x = s["logits"][a:a + 1024].double().requires_grad_(True)
        t = s["targets"][a:a + 1024]
        logp = torch.log_softmax(x * c["scale"], 1)
        total = logp.gather(1, t.clamp(min=0).unsqueeze(1)).squeeze(1) * s["grad_logp"][a:a + 1024]
        if c["entropy"]:
            total = total - (logp.exp() * logp).sum(1) * s["grad_entropy"][a:a + 1024]
        out.append(torch.autograd.grad((total * (t >= 0)).sum(), x)[0])
    return torch.cat(out)
