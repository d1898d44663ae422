"""Measured cases of the operators around the gradient path: the AdamW step over many tensors (moments in 32 or in 8
bits), the global gradient norm it clips by, and the routing of tokens to experts with its gradient.

``run`` computes a case in plain torch operations, or, with ``own``, through the library's entry points.  Parameters,
moments and their scales live in flat buffers in which every tensor starts on a block of 256 elements; the gradients
lie in a bucket arena, in reverse registration order and without padding, as a reduction leaves them."""

import itertools
import math
import random

import torch

own = False

BLOCK = 256                      # elements that share one scale of an 8-bit moment
BETA1, BETA2, EPS, LR = 0.9, 0.999, 1e-8, 1e-3
DECAY, MAX_NORM, STEP = 0.01, 1.0, 100
TOP_M, TOP_V = 448.0, 57344.0    # largest finite e4m3 and e5m2 values


# ---------------------------------------------------------------- cases

def listed():
    return [
        # Linear(10, 10), the worked example: 110 elements, where a step is all latency
        dict(name="adamw32_linear", op="adamw", bits=32, model="linear", weights="f32", unused=0.0),
        # ResNet-50: 161 tensors, most of them vectors of 64 to 2048 elements
        dict(name="adamw32_resnet50", op="adamw", bits=32, model="resnet50", weights="f32", unused=0.0),
        # BERT-large, the largest step: 335 M elements of 32-bit everything
        dict(name="adamw32_bert_large", op="adamw", bits=32, model="bert_large", weights="f32", unused=0.0),
        # GPT-2-medium in mixed precision: bf16 weights beside an fp32 master copy
        dict(name="adamw32_gpt2_medium", op="adamw", bits=32, model="gpt2_medium", weights="bf16", unused=0.0),
        # 97 ragged tensors of which a third got no gradient in this step (experts that no token reached)
        dict(name="adamw8_ragged", op="adamw", bits=8, model="random", tensors=97, elements=3_000_017, spread=11,
             weights="f32", unused=0.33),
        # GPT-2-medium in mixed precision with moments in 8 bits, the largest of its kind
        dict(name="adamw8_gpt2_medium", op="adamw", bits=8, model="gpt2_medium", weights="bf16", unused=0.0),
        # the norm to clip by, of ResNet-50's and of BERT-large's gradients
        dict(name="norm_resnet50", op="norm", model="resnet50", unused=0.0),
        dict(name="norm_bert_large", op="norm", model="bert_large", unused=0.0),
        # the last, nearly empty micro-batch of a small softmax router
        dict(name="route_few", op="route", tokens=3, experts=64, k=4, score="softmax", renorm=True, bias=False,
             groups=1, top_groups=1, scale=1.0, dtype="bf16", masked=0.0),
        # a large batch over many experts: sigmoid scores, balanced by a bias, limited to groups; 2 % padding tokens
        dict(name="route_many", op="route", tokens=65536, experts=256, k=8, score="sigmoid", renorm=True, bias=True,
             groups=8, top_groups=4, scale=2.5, dtype="f32", masked=0.02),
        # the gradient of a softmax router whose weights are not renormalised: every expert's logit gets one
        dict(name="route_back_softmax", op="route_back", tokens=4097, experts=60, k=4, score="softmax", renorm=False,
             bias=False, groups=1, top_groups=1, scale=1.0, dtype="f32", masked=0.0),
        # the gradient of the large batch, in bf16
        dict(name="route_back_many", op="route_back", tokens=65536, experts=256, k=8, score="sigmoid", renorm=True,
             bias=True, groups=8, top_groups=4, scale=2.5, dtype="bf16", masked=0.02),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["adamw", "adamw", "norm", "route", "route_back"])
    if op in ("adamw", "norm"):
        elements = log(100, 300_000_000)
        case = dict(op=op, model="random", tensors=min(log(1, 400), elements), elements=elements,
                    spread=rng.randrange(1 << 20), unused=rng.choice([0.0, 0.0, rng.uniform(0.05, 0.6)]))
        if op == "adamw":
            case.update(bits=rng.choice([32, 8]), weights=rng.choice(["f32", "bf16"]))
        return case
    # a bias and groups come with sigmoid scores; softmax scores choose by themselves
    score = rng.choice(["softmax", "sigmoid"])
    groups = rng.choice([1, 2, 4, 8]) if score == "sigmoid" else 1
    experts = groups * log(max(1, 8 // groups), 512 // groups)
    top_groups = rng.randint(1, groups)
    k = rng.randint(1, min(12, top_groups * (experts // groups)))
    return dict(op=op, tokens=min(log(1, 65536), 16_000_000 // experts), experts=experts, k=k, score=score,
                renorm=k > 1 and rng.choice([True, False]), bias=score == "sigmoid" and rng.choice([True, False]),
                groups=groups, top_groups=top_groups, scale=rng.choice([1.0, 2.5]),
                dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, rng.uniform(0.01, 0.5)]))


# ---------------------------------------------------------------- parameter shapes

def _sizes(case):
    """Element counts in registration order."""
    model = case["model"]
    if model == "linear":
        return [100, 10]
    if model == "bert_large":
        h, f = 1024, 4096
        layer = [h * h, h] * 4 + [h, h] + [f * h, f, h * f, h, h, h]
        return [30522 * h, 512 * h, 2 * h, h, h] + layer * 24 + [h * h, h]
    if model == "gpt2_medium":
        d = 1024
        layer = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d, 4 * d * d, d]
        return [50257 * d, 1024 * d] + layer * 24 + [d, d]
    if model == "resnet50":
        def block(cin, c, first):
            return ([cin * c, c, c, 9 * c * c, c, c, 4 * c * c, 4 * c, 4 * c]
                    + ([4 * cin * c, 4 * c, 4 * c] if first else []))
        stages = [(64, 64, 3), (256, 128, 4), (512, 256, 6), (1024, 512, 3)]
        body = [n for cin, c, count in stages for b in range(count) for n in block(cin if b == 0 else 4 * c, c, b == 0)]
        return [9408, 64, 64] + body + [2_048_000, 1000]
    rng = random.Random(case["spread"])
    share = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(case["tensors"])]
    left = case["elements"] - case["tensors"]
    sizes = [1 + int(left * x / sum(share)) for x in share]
    sizes[0] += case["elements"] - sum(sizes)
    return sizes


def _unused(case, count):
    """Which tensors got no gradient; never all of them."""
    rng = random.Random(case.get("spread", 0) + 1)
    return [v > 0 and rng.random() < case["unused"] for v in range(count)]


def _starts(counts):
    return [0, *itertools.accumulate(counts)]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_route(case, gen) if case["op"].startswith("route") else _prepare_step(case, gen)


def _prepare_step(case, gen):
    sizes = _sizes(case)
    used = [not u for u in _unused(case, len(sizes))]
    rows = [-(-n // BLOCK) for n in sizes]
    row0 = _starts(rows)
    total = row0[-1] * BLOCK
    back = _starts(sizes[::-1])[:-1][::-1]                     # arena offsets: the last tensor comes first
    arena = torch.randn(sum(sizes), generator=gen, device="cuda") * 1e-3
    s = dict(case=case, sizes=sizes, row0=row0, arena=arena, t=STEP, used=None,
             grads=[arena[o:o + n] for o, n in zip(back, sizes)])
    if not all(used):
        s["used"] = torch.tensor(used, device="cuda").to(torch.uint8)
        rows_t = torch.tensor(rows, device="cuda")
        s["used_arena"] = torch.repeat_interleave(s["used"].flip(0).bool(), torch.tensor(sizes[::-1], device="cuda"))
        s["used_rows"] = torch.repeat_interleave(s["used"].bool(), rows_t).unsqueeze(1)
    s["mine"] = [v for v, u in enumerate(used) if u]           # the tensors of this step, as the host knows them
    if case["op"] == "norm":
        s["out"] = torch.zeros(1, device="cuda")
        if own:
            from reduction_reducer_gb300 import AdamW
            s["opt"] = AdamW(sizes)
            s["opt"].bind_grads(s["grads"])
        return s

    def views(flat):
        return [flat[r * BLOCK:r * BLOCK + n] for r, n in zip(row0, sizes)]

    # weights, and moments as after many steps on gradients of this scale; the blocks' ends past a tensor hold zeros
    inside = torch.zeros(total, device="cuda")
    torch._foreach_add_(views(inside), 1.0)
    weight = torch.randn(total, generator=gen, device="cuda") * 0.02 * inside
    m = torch.randn(total, generator=gen, device="cuda") * 3e-4 * inside
    v = torch.exp(torch.randn(total, generator=gen, device="cuda")) * 1e-6 * inside
    del inside
    decay = [DECAY if n >= 4096 else 0.0 for n in sizes]       # none for biases and norms
    s["decay_rows"] = torch.repeat_interleave(torch.tensor(decay, device="cuda"),
                                              torch.tensor(rows, device="cuda")).unsqueeze(1)
    s["norm"] = torch.linalg.vector_norm(arena).reshape(1).clamp(min=1e-3)
    s["weight"] = weight
    s["param"] = weight.to(torch.bfloat16) if case["weights"] == "bf16" else None
    if case["bits"] == 8:
        for name, x, top, kind in (("m", m, TOP_M, torch.float8_e4m3fn), ("v", v, TOP_V, torch.float8_e5m2)):
            scale = x.view(-1, BLOCK).abs().amax(1, keepdim=True) / top
            s[name] = (x.view(-1, BLOCK) / scale.clamp(min=1e-30)).clamp(-top, top).to(kind).view(-1)
            s[name + "_scale"] = scale.view(-1).contiguous()
    else:
        s["m"], s["v"] = m, v
    if own:
        from reduction_reducer_gb300 import AdamW
        bf16, eight = case["weights"] == "bf16", case["bits"] == 8

        def scales(flat):
            return [flat[row0[i]:row0[i + 1]] for i in range(len(sizes))]

        s["opt"] = AdamW(sizes, param_dtype=case["weights"], state_bits=case["bits"])
        s["opt"].bind(views(s["param"] if bf16 else weight), s["grads"], views(s["m"]), views(s["v"]),
                      weight_decay=decay, master=views(weight) if bf16 else None,
                      exp_avg_scale=scales(s["m_scale"]) if eight else None,
                      exp_avg_sq_scale=scales(s["v_scale"]) if eight else None)
    return s


def _prepare_route(case, gen):
    T, E, k = case["tokens"], case["experts"], case["k"]
    # a token's affinities, and experts that are liked more than others
    logits = torch.randn(T, E, generator=gen, device="cuda") * 1.5 + torch.randn(E, generator=gen, device="cuda") * 0.5
    s = dict(case=case, logits=logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits, bias=None, mask=None,
             counts=torch.zeros(E, dtype=torch.int32, device="cuda"))
    if case["bias"]:
        s["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.05
    if case["masked"] > 0:
        s["mask"] = torch.rand(T, generator=gen, device="cuda") >= case["masked"]
    s["indices"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    s["weights"] = torch.empty(T, k, device="cuda")
    if case["op"] == "route_back":
        s["indices"], s["weights"], _ = _route_plain(s)
        s["grad"] = torch.randn(T, k, generator=gen, device="cuda")
        s["out"] = torch.empty_like(s["logits"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op == "adamw":
        s["t"] += 1
        (_step_own if own else _step_plain)(s)
        return {name: s[name] for name in ("weight", "param", "m", "v", "m_scale", "v_scale") if s.get(name) is not None}
    if op == "norm":
        return s["opt"].grad_norm(s["out"], used=s["used"]) if own else _norm_plain(s)
    if op == "route":
        return _route_own(s) if own else _route_plain(s)
    return _route_back_own(s) if own else _route_back_plain(s)


def _step_own(s):
    s["opt"].step(s["t"], lr=LR, betas=(BETA1, BETA2), eps=EPS, norm=s["norm"], max_norm=MAX_NORM, used=s["used"],
                  seed=s["t"])


def _route_own(s):
    from reduction_reducer_gb300 import route
    c = s["case"]
    indices, weights = route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                             top_groups=c["top_groups"], renorm=c["renorm"], scale=c["scale"], mask=s["mask"],
                             counts=s["counts"], out=(s["indices"], s["weights"]))
    return indices, weights, s["counts"]


def _route_back_own(s):
    from reduction_reducer_gb300 import route_backward
    c = s["case"]
    return route_backward(s["grad"], s["logits"], s["indices"], s["weights"], score=c["score"], renorm=c["renorm"],
                          scale=c["scale"], out=s["out"])


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    """sqrt of the sum of squares over the tensors that have a gradient."""
    if s["used"] is None:
        return s["arena"].square().sum().sqrt().reshape(1)
    return torch.where(s["used_arena"], s["arena"], 0.0).square().sum().sqrt().reshape(1)


def _step_plain(s):
    case, t = s["case"], s["t"]
    g = torch.zeros_like(s["weight"])                          # the gradients in the weights' layout
    torch._foreach_copy_([g[r * BLOCK:r * BLOCK + n] for r, n in zip(s["row0"], s["sizes"])], s["grads"])
    g = g.view(-1, BLOCK) * (MAX_NORM / (s["norm"] + 1e-6)).clamp(max=1.0)
    w = s["weight"].view(-1, BLOCK)
    if case["bits"] == 8:
        m = s["m"].view(-1, BLOCK).float() * s["m_scale"].unsqueeze(1)
        v = s["v"].view(-1, BLOCK).float() * s["v_scale"].unsqueeze(1)
    else:
        m, v = s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK)
    m1 = m * BETA1 + g * (1 - BETA1)
    v1 = v * BETA2 + (g * g) * (1 - BETA2)
    denom = v1.sqrt() * (1 / math.sqrt(1 - BETA2 ** t)) + EPS
    w1 = w * (1 - LR * s["decay_rows"]) - (LR / (1 - BETA1 ** t)) * m1 / denom
    keep = s.get("used_rows")
    if case["bits"] == 8:
        m_code, m_scale, v_code, v_scale = _store_plain(m1, v1, t)
        new = dict(m_scale=m_scale, v_scale=v_scale)
        bits = dict(m=m_code, v=v_code)
    else:
        new, bits = dict(m=m1, v=v1), {}
    new["weight"] = w1
    if s["param"] is not None:
        new["param"] = w1.to(torch.bfloat16)
    _write(s, new, keep)
    _write({n: s[n].view(torch.uint8) for n in bits}, bits, keep)


def _write(s, new, keep):
    """Into the state, but for the tensors that got no gradient."""
    old = [s[n].view(x.shape) for n, x in new.items()]
    fresh = list(new.values()) if keep is None else [torch.where(keep, x, o) for x, o in zip(new.values(), old)]
    [o.copy_(x) for o, x in zip(old, fresh)]


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_plain(rows, seed):
    """32 random bits for each element: a counter of the seed, the block and the place in it, mixed twice."""
    lo, hi = seed & 0xFFFFFFFF, seed >> 32
    block = torch.arange(rows, device="cuda").unsqueeze(1)
    key = _mix((_mix((block & 0xFFFFFFFF) ^ lo) + hi) & 0xFFFFFFFF)
    place = torch.arange(BLOCK, device="cuda").unsqueeze(0)
    return _mix((key + place * 0x9E3779B9) & 0xFFFFFFFF)


def _grid_plain(y, u, least, mantissa):
    """Codes of non-negative y on a floating grid with `mantissa` bits, rounded up with the probability of the rest.
    `least` is the exponent below which the spacing stays the same."""
    e = ((y.view(torch.int32) >> 23) - 127).clamp(min=least)
    n = torch.floor(y * ((127 + mantissa - e) << 23).view(torch.float32) + u).to(torch.int32)
    return n + ((e - least) << mantissa)


def _store_plain(m, v, seed):
    h = _random_plain(m.shape[0], seed)
    m_scale = m.abs().amax(1, keepdim=True) / TOP_M
    v_scale = v.amax(1, keepdim=True) / TOP_V
    tiny = 2.0 ** -126                                         # blocks of no more than that are zeros
    m_scale, v_scale = m_scale * (m_scale >= tiny), v_scale * (v_scale >= tiny)
    m_y = m.abs() * torch.where(m_scale > 0, 1 / m_scale, 0.0)
    v_y = v * torch.where(v_scale > 0, 1 / v_scale, 0.0)
    m_code = _grid_plain(m_y, (h >> 16).float() * 2.0 ** -16, -6, 3).clamp(max=126) | ((m < 0).int() << 7)
    v_code = _grid_plain(v_y, (h & 0xFFFF).float() * 2.0 ** -16, -14, 2).clamp(max=123)
    v_code = torch.where((v_y > 0) & (v_code == 0), 1, v_code)  # a second moment that is not zero stays so
    return m_code.to(torch.uint8), m_scale, v_code.to(torch.uint8), v_scale


def _scores_plain(s):
    x = s["logits"].float()
    if s["case"]["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        return x, e / e.sum(1, keepdim=True)
    return x, 1 / (1 + torch.exp(-x))


def _route_plain(s):
    c = s["case"]
    T, E, k, G = c["tokens"], c["experts"], c["k"], c["groups"]
    x, score = _scores_plain(s)
    # without a bias and groups the scores' order is the logits'
    choice = x if s["bias"] is None and G == 1 else score if s["bias"] is None else score + s["bias"]
    if G > 1:
        best = choice.view(T, G, E // G).topk(min(2, E // G)).values.sum(2)
        first = best.argsort(dim=1, descending=True, stable=True)[:, :c["top_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, first, True)
        choice = torch.where(open_.repeat_interleave(E // G, dim=1), choice, -math.inf)
    order = choice.argsort(dim=1, descending=True, stable=True)[:, :k]
    live = torch.ones(T, 1, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].unsqueeze(1)
    live = live.expand(T, k)
    w = torch.where(live, score.gather(1, order), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    s["counts"].scatter_add_(0, order.reshape(-1), live.reshape(-1).int())
    return torch.where(live, order, -1).int(), w * c["scale"], s["counts"]


def _route_back_plain(s):
    c = s["case"]
    x, score = _scores_plain(s)
    live = s["indices"] >= 0
    at = s["indices"].clamp(min=0).long()
    g = torch.where(live, s["grad"], 0.0)
    gw = g * s["weights"]
    if c["renorm"]:                                            # w_j (g_j - sum_l g_l w_l / scale)
        part = s["weights"] * (g - gw.sum(1, keepdim=True) / c["scale"])
    else:
        part = gw
    if c["score"] == "sigmoid":
        part = part * (1 - score.gather(1, at))
    d = torch.zeros_like(x).scatter_add_(1, at, torch.where(live, part, 0.0))
    if c["score"] == "softmax":
        d = d - score * torch.where(live, part, 0.0).sum(1, keepdim=True)
    return d.to(s["logits"].dtype)


# ---------------------------------------------------------------- work

def work(case):
    if case["op"].startswith("route"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        logits = T * E * (2 if case["dtype"] == "bf16" else 4)
        mask = T if case["masked"] > 0 else 0
        if case["op"] == "route":
            return {"bytes": logits + mask + 8 * T * k + 4 * E * (2 if case["bias"] else 1), "flops": T * E * 4}
        whole = case["score"] == "softmax" and not case["renorm"]
        some = 0 if whole or case["score"] == "softmax" else T * k * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": logits * (2 if whole else 1) + some + 12 * T * k, "flops": T * (E * 3 if whole else k * 6)}
    sizes = _sizes(case)
    n = sum(x for x, u in zip(sizes, _unused(case, len(sizes))) if not u)
    if case["op"] == "norm":
        return {"bytes": 4 * n + 4, "flops": 2 * n}
    each = 12 + (4 if case["bits"] == 8 else 16) + (2 if case["weights"] == "bf16" else 0)
    return {"bytes": each * n + (16 * -(-n // BLOCK) if case["bits"] == 8 else 0), "flops": 16 * n}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    keep, globals()["own"] = own, False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = keep
    return {"adamw": _exact_step, "norm": _exact_norm, "route": _exact_route, "route_back": _exact_back}[case["op"]](s)


def _exact_norm(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for v in s["mine"]:
        total += torch.dot(s["grads"][v].double(), s["grads"][v].double())
    return total.sqrt().reshape(1)


def _exact_step(s):
    """Tensor by tensor, in double; the 8-bit rounding from the formats' spacings."""
    case, t = s["case"], s["t"] + 1
    eight = case["bits"] == 8
    clip = min(1.0, MAX_NORM / (float(s["norm"]) + 1e-6))
    out = {n: s[n].double() for n in ("weight", "param", "m", "v", "m_scale", "v_scale") if s.get(n) is not None}
    for v in s["mine"]:
        n, r0, r1 = s["sizes"][v], s["row0"][v], s["row0"][v + 1]
        a = r0 * BLOCK
        g = s["grads"][v].double() * clip
        w, m1, v1 = out["weight"][a:a + n], out["m"][a:a + n], out["v"][a:a + n]
        block = torch.arange(n, device="cuda") // BLOCK
        if eight:
            old_m, old_v = m1 * out["m_scale"][r0:r1][block], v1 * out["v_scale"][r0:r1][block]
        else:
            old_m, old_v = m1, v1
        new_m = BETA1 * old_m + (1 - BETA1) * g
        new_v = BETA2 * old_v + (1 - BETA2) * g ** 2
        m_hat, v_hat = new_m / (1 - BETA1 ** t), new_v / (1 - BETA2 ** t)
        new_w = w - LR * (m_hat / (v_hat.sqrt() + EPS) + float(s["decay_rows"][r0]) * w)
        w.copy_(new_w)
        if s["param"] is not None:
            out["param"][a:a + n] = new_w
        if not eight:
            m1.copy_(new_m)
            v1.copy_(new_v)
            continue
        bits = _exact_bits(t, r0 + block, torch.arange(n, device="cuda") % BLOCK)
        for name, code, x, top, mantissa, least, u in (("m", m1, new_m, TOP_M, 3, -6, bits >> 16),
                                                       ("v", v1, new_v, TOP_V, 2, -14, bits & 0xFFFF)):
            peak = torch.zeros(r1 - r0, dtype=torch.float64, device="cuda").scatter_reduce_(0, block, x.abs(), "amax")
            out[name + "_scale"][r0:r1] = peak / top
            y = torch.where(peak[block] > 0, x.abs() * top / peak[block], 0.0)
            exponent = torch.frexp(y).exponent - 1
            q = torch.exp2(exponent.clamp(min=least).double() - mantissa)
            z = torch.floor(y / q + u.double() / 65536) * q
            if name == "v":
                z = torch.where((y > 0) & (z == 0), 2.0 ** (least - mantissa), z)
            code.copy_(torch.copysign(z.clamp(max=top), x))
    return out


def _exact_bits(seed, block, place):
    def scramble(x):
        for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
            x = torch.bitwise_xor(x, torch.bitwise_right_shift(x, shift)) * factor % 2 ** 32
        return torch.bitwise_xor(x, torch.bitwise_right_shift(x, 16))
    key = scramble((scramble(torch.bitwise_xor(block % 2 ** 32, seed % 2 ** 32)) + seed // 2 ** 32) % 2 ** 32)
    return scramble((key + place * 0x9E3779B9) % 2 ** 32)


def _exact_scores(s):
    x = s["logits"].double()
    return x, (x - torch.logsumexp(x, 1, keepdim=True)).exp() if s["case"]["score"] == "softmax" else torch.sigmoid(x)


def _exact_route(s):
    """The best expert k times over; only the weights have a 64-bit value."""
    c = s["case"]
    T, E, G = c["tokens"], c["experts"], c["groups"]
    x, score = _exact_scores(s)
    choice = score.clone() if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        group = choice.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        barred = group.argsort(dim=1, descending=True)[:, c["top_groups"]:]
        choice = choice.view(T, G, E // G).clone()
        choice[torch.arange(T, device="cuda").unsqueeze(1), barred] = -math.inf
        choice = choice.view(T, E)
    picked = []
    for _ in range(c["k"]):
        at = choice.argmax(1, keepdim=True)
        picked.append(score.gather(1, at))
        choice.scatter_(1, at, -math.inf)
    w = torch.cat(picked, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    if s["mask"] is not None:
        w[~s["mask"]] = 0.0
    return None, w, None


def _exact_back(s):
    """By differentiating the weights' definition at the given choice."""
    c = s["case"]
    x = s["logits"].double().requires_grad_(True)
    score = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    live = s["indices"] >= 0
    w = score.gather(1, s["indices"].clamp(min=0).long())
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    (w * c["scale"] * s["grad"].double() * live).sum().backward()
    return x.grad
