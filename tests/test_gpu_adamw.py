"""The AdamW step and the gradient norm on the GPU against the 64-bit oracle.

Bounds (u = 2^-24, fp32 rounding): the clip factor is two roundings from the
exact one, the clipped gradient three; m' is a sum of two products, v' of two
non-negative ones:  |m' err| <= 6u (|b1 m| + |b1c g'|),  |v' err| <= 10u v'.
The update's relative error adds the square root (half of v's, and 1), two
products, a sum, a product and a quotient: 12u times b = (|b1 m| + |b1c g'|) /
denominator, and the weight two roundings and that of 1 - lr wd: 4u |w|.
"""

import numpy as np
import pytest
import torch

from oracle import adamw as A
from reduction_reducer_gb300 import AdamW, Reducer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-7)
SIZES = {"one": [1], "block_edges": [255, 256, 257, 1, 511, 513], "empties": [7, 0, 513, 0, 1000, 64, 0],
         "linear": [100, 10], "many_small": [1 + (37 * i) % 70 for i in range(300)], "large": [70_001, 3, 4096]}
GUARD = 12345.0


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


class Case:
    """Tensors of one optimizer in guarded flat buffers, all at element offset `shift` from 16-byte alignment."""

    def __init__(self, sizes, dtype="f32", bits=32, shift=0, seed=0, arena=False):
        self.sizes, self.bits, self.bf16 = sizes, bits, dtype == "bf16"
        rng = np.random.default_rng(seed)
        draw = lambda f: [f(n).astype(np.float32) for n in sizes]          # noqa: E731
        self.w = draw(lambda n: rng.normal(size=n) * 0.05)
        self.g = draw(lambda n: rng.normal(size=n) * 0.01 * np.exp(rng.normal(size=n)))
        self.m = draw(lambda n: rng.normal(size=n) * 0.004)
        self.v = draw(lambda n: np.exp(rng.normal(size=n) * 1.5) * 1e-5)
        self.wd = [0.1 if v % 3 else 0.0 for v in range(len(sizes))]
        self.flats = {}
        put = self.put
        self.grads = put("grads", self.g, torch.float32, 1 if arena else 64, shift)
        self.weights = put("w", self.w, torch.float32, 64, shift)
        self.params = self.weights
        if self.bf16:
            self.params = put("p", [np.full(n, 9.0, np.float32) for n in sizes], torch.bfloat16, 64, shift)
        state = {}
        if bits == 8:
            self.code, self.scale = {}, {}
            for name, x, kind, fmt in (("m", self.m, torch.float8_e4m3fn, A.E4M3), ("v", self.v, torch.float8_e5m2, A.E5M2)):
                made = [A.encode(t, np.full(t.size, 32768), **fmt) for t in x]
                scales = [s.astype(np.float32) for _, s, _ in made]
                values = [z for z, _, _ in made]
                self.scale[name] = put(name + "_scale", scales, torch.float32, 1, shift)
                self.code[name] = put(name, [z.astype(np.float32) for z in values], kind, 64, shift)
                # what the state stands for from here on
                setattr(self, name, [z * np.repeat(s.astype(np.float64), A.BLOCK)[:z.size] for z, s in zip(values, scales)])
            state = dict(exp_avg_scale=self.scale["m"], exp_avg_sq_scale=self.scale["v"])
            m, v = self.code["m"], self.code["v"]
        else:
            m, v = self.m_t, self.v_t = put("m", self.m, torch.float32, 64, shift), put("v", self.v, torch.float32, 64, shift)
        self.opt = AdamW(sizes, dtype, bits)
        self.opt.bind(self.params, self.grads, m, v, weight_decay=self.wd, master=self.weights if self.bf16 else None, **state)

    def put(self, name, arrays, dtype, align, shift):
        starts, at = [], shift
        for a in arrays:
            starts.append(at)
            at += -(-a.size // align) * align + (8 if align > 1 else 0)
        size = torch.empty(0, dtype=dtype).element_size()
        flat = (torch.full((at + 64,), GUARD).to(dtype) if size > 1
                else torch.full((at + 64,), 0x55, dtype=torch.uint8).view(dtype))
        inside = torch.zeros(at + 64, dtype=torch.bool)
        for a, o in zip(arrays, starts):
            if a.size == 0:
                continue
            flat.view(torch.uint8).view(-1, size)[o:o + a.size] = torch.from_numpy(a).to(dtype).view(torch.uint8).view(-1, size)
            inside[o:o + a.size] = True
        dev = flat.view(torch.uint8).cuda().view(dtype)
        self.flats[name] = (dev, flat, inside)
        return [dev[o:o + a.size] for a, o in zip(arrays, starts)]

    def check_guards(self):
        for name, (dev, was, inside) in self.flats.items():
            size = was.element_size()
            now = dev.view(torch.uint8).cpu().view(-1, size)
            assert torch.equal(now[~inside], was.view(torch.uint8).view(-1, size)[~inside]), name

    def snapshot(self):
        return {n: dev.view(torch.uint8).cpu() for n, (dev, _, _) in self.flats.items()}

    def check(self, t, clip, used=None, seed=0):
        """The tensors after one step t from the case's initial values."""
        torch.cuda.synchronize()
        self.check_guards()
        block0 = 0
        for v, n in enumerate(self.sizes):
            blocks = -(-n // A.BLOCK)
            first, block0 = block0, block0 + blocks
            if n == 0:
                continue
            w = self.weights[v].cpu().numpy().astype(np.float64)
            if used is not None and not used[v]:
                assert np.array_equal(w, self.w[v].astype(np.float64))
                continue
            b1, b2 = HYPER["beta1"], HYPER["beta2"]
            want_w, want_m, want_v = A.adamw(self.w[v], self.g[v], self.m[v], self.v[v], t, wd=self.wd[v], clip=clip,
                                             **HYPER)
            size = np.abs(b1 * np.asarray(self.m[v], np.float64)) + np.abs((1 - b1) * clip * self.g[v].astype(np.float64))
            denom = np.sqrt(want_v / (1 - b2 ** t)) + HYPER["eps"]
            b = HYPER["lr"] / (1 - b1 ** t) * size / denom
            # hyperparameters reach the kernel in fp32 too: 1 - beta and the corrections, 4u more
            assert np.all(np.abs(w - want_w) <= 4 * U * np.abs(self.w[v]) + 24 * U * b), v
            if self.bf16:
                assert torch.equal(self.params[v], self.weights[v].to(torch.bfloat16))
            if self.bits == 32:
                assert np.all(np.abs(self.m_t[v].cpu().numpy() - want_m) <= 8 * U * size), v
                assert np.all(np.abs(self.v_t[v].cpu().numpy() - want_v) <= 12 * U * want_v), v
                continue
            place = np.arange(n)
            bits = A.random_bits(seed, first + place // A.BLOCK, place % A.BLOCK)
            for name, x, err, fmt, r16 in (("m", want_m, 8 * U * size, A.E4M3, bits >> np.uint64(16)),
                                           ("v", want_v, 12 * U * want_v, A.E5M2, bits & np.uint64(0xFFFF))):
                z, scale, at = A.encode(x, r16, **fmt)
                got_scale = self.scale[name][v].cpu().numpy()
                got = self.code[name][v].float().cpu().numpy().astype(np.float64)
                most = np.zeros(blocks)
                np.maximum.at(most, place // A.BLOCK, err)
                assert np.all(np.abs(got_scale - scale) <= most / fmt["top"] + 2 * U * scale), (name, v)
                per = np.repeat(scale, A.BLOCK)[:n]
                y = np.divide(np.abs(x), per, out=np.zeros(n), where=per > 0)
                q = A.spacing(y, fmt["mantissa"], fmt["least"])
                if name == "v":
                    z = np.where((y > 0) & (z == 0), q, z)
                # the same number, but where the rounded-up place is nearer to a whole one than fp32 tells
                off = np.divide(err + np.repeat(most, A.BLOCK)[:n] * y / fmt["top"], per, out=np.zeros(n), where=per > 0) / q
                near = np.abs(at - np.round(at)) <= off + 6 * U * (at + 1)
                assert np.all((got == z) | (near & (np.abs(got - z) <= 1.01 * q))), (name, v)
                assert near.mean() < 0.01 or n < 1000


def run(case, t, clip_at=0.0, used=None, seed=0, stream=None):
    norm = None
    clip = 1.0
    if clip_at:
        norm = torch.empty(1, device="cuda")
        case.opt.grad_norm(norm, used=used)
        live = [g for v, g in enumerate(case.g) if used is None or bool(used[v])]
        exact = A.grad_norm(live)
        assert abs(float(norm) - exact) <= 64 * U * exact
        clip = A.clip_factor(exact, clip_at)
        # the clip's own error is the norm's: give the oracle the kernel's norm
        clip = A.clip_factor(float(norm), clip_at)
    case.opt.step(t, lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"], norm=norm,
                  max_norm=clip_at, used=used, seed=seed, stream=stream)
    return clip


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", SIZES)
def test_step(sizes, dtype, bits):
    case = Case(SIZES[sizes], dtype, bits)
    seed = (5 << 32) + 17
    clip = run(case, 3, seed=seed)
    case.check(3, clip, seed=seed)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_step_at_odd_addresses(shift, dtype, bits):
    case = Case([513, 1, 70, 2000, 255], dtype, bits, shift=shift, arena=True)
    clip = run(case, 1, clip_at=0.05, seed=9)
    assert clip < 1
    case.check(1, clip, seed=9)


@pytest.mark.parametrize("bits", [32, 8])
def test_step_with_gradients_in_an_arena_alone_misaligned(bits):
    case = Case([101, 900, 33, 5000], "f32", bits, arena=True)       # weights and moments aligned, gradients not
    clip = run(case, 1000, clip_at=0.05)
    case.check(1000, clip)


@pytest.mark.parametrize("bits", [32, 8])
def test_unused_tensors_stay(bits):
    case = Case([300, 5, 0, 1024, 700], "bf16", bits)
    before = case.snapshot()
    used = torch.tensor([1, 0, 1, 0, 1], dtype=torch.uint8, device="cuda")
    clip = run(case, 2, clip_at=0.1, used=used, seed=4)
    case.check(2, clip, used=used.cpu().tolist(), seed=4)
    for v in (1, 3):
        for views, was in ((case.params, case.flats["p"]), (case.weights, case.flats["w"])):
            lo = views[v].data_ptr() - was[0].data_ptr()
            now = was[0].view(torch.uint8).cpu()[lo:lo + views[v].nbytes]
            name = "p" if was is case.flats["p"] else "w"
            assert torch.equal(now, before[name][lo:lo + views[v].nbytes])
    none = torch.zeros(5, dtype=torch.bool, device="cuda")
    before = case.snapshot()
    norm = case.opt.grad_norm(torch.full((1,), 7.0, device="cuda"), used=none)
    case.opt.step(3, used=none)
    torch.cuda.synchronize()
    assert float(norm) == 0.0
    assert all(torch.equal(a, b) for a, b in zip(before.values(), case.snapshot().values()))


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_norm_skips_when_asked(bits):
    case = Case([300, 40], "f32", bits)
    case.grads[1][7] = float("nan")
    norm = case.opt.grad_norm(torch.zeros(1, device="cuda"))
    assert bool(torch.isnan(norm))
    before = case.snapshot()
    case.opt.step(1, norm=norm, max_norm=1.0, skip_nonfinite=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before.values(), case.snapshot().values()))
    case.opt.step(1, norm=norm, max_norm=1.0)                      # asked not to: it shows
    torch.cuda.synchronize()
    assert bool(torch.isnan(case.weights[0]).all())
    case.grads[1][7] = float("-inf")
    assert float(case.opt.grad_norm(norm)) == float("inf")


def test_nonfinite_gradient_stays_in_its_block():
    """Without clipping, a NaN or infinite gradient spoils its own block's 8-bit moments and no other's."""
    case = Case([2000], "f32", 8)
    case.grads[0][300] = float("inf")
    case.grads[0][800] = float("nan")
    case.opt.step(1)
    torch.cuda.synchronize()
    for name in ("m", "v"):
        bad = torch.isnan(case.scale[name][0]).cpu().tolist()
        assert bad == [i in (1, 3) for i in range(8)]
        assert bool(torch.isfinite(case.code[name][0].float()).all())
    w = case.weights[0].cpu()
    assert torch.isfinite(w).sum() == 1998 and not torch.isfinite(w[[300, 800]]).any()


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_zero_state(bits):
    n = [700]
    opt = AdamW(n, "f32", bits)
    w = torch.ones(700, device="cuda")
    g = torch.zeros(700, device="cuda")
    state = opt.zero_state()
    opt.bind([w], [g], weight_decay=0.5, **state)
    opt.step(1, lr=0.25)
    torch.cuda.synchronize()
    assert torch.equal(w, torch.full_like(w, 0.875))               # decay alone
    assert all(float(x.float().abs().sum()) == 0 for views in state.values() for x in views)
    g[3] = 2.0
    opt.step(2, lr=0.25)
    torch.cuda.synchronize()
    assert float(state["exp_avg"][0].float()[3]) != 0 and float(state["exp_avg"][0].float().abs().sum()) == float(state["exp_avg"][0].float()[3])


def test_tiny_second_moments_are_never_stored_as_zero():
    n = 256
    opt = AdamW([n], "f32", 8)
    w, g = torch.zeros(n, device="cuda"), torch.full((n,), 1e-12, device="cuda")
    g[0] = 1.0
    state = opt.zero_state()
    opt.bind([w], [g], **state)
    for t in range(1, 20):
        opt.step(t, seed=t)
    torch.cuda.synchronize()
    assert bool((state["exp_avg_sq"][0].float() > 0).all())
    assert bool(torch.isfinite(w).all()) and float(w.abs().max()) <= 19 * 1e-3 * 1.05


def test_eight_bit_second_moment_follows_the_32_bit_one():
    """Over 3000 steps at beta2 = 0.999 a step moves v by about a thousandth, an e5m2 number's neighbours lie a quarter
    apart: only unbiased rounding follows.  The mean over 65,536 elements (noise of the rounding 30 % an element,
    0.12 % in the mean) lies within 2 % of the 32-bit run's, from a start four times too high."""
    n, sigma = 65536, 1e-2
    gen = torch.Generator("cuda").manual_seed(1)
    runs = {}
    for bits in (32, 8):
        opt = AdamW([n], "f32", bits)
        w, g = torch.zeros(n, device="cuda"), torch.empty(n, device="cuda")
        state = opt.zero_state()
        if bits == 32:
            state["exp_avg_sq"][0].fill_(4 * sigma ** 2)
        else:
            state["exp_avg_sq"][0].copy_(torch.ones(n, device="cuda").to(torch.float8_e5m2))
            state["exp_avg_sq_scale"][0].fill_(4 * sigma ** 2)
        opt.bind([w], [g], **state)
        gen.manual_seed(2)
        for t in range(1, 3001):
            g.normal_(generator=gen).mul_(sigma)
            opt.step(t, seed=t)
        x = state["exp_avg_sq"][0].float()
        if bits == 8:
            x = x * state["exp_avg_sq_scale"][0].repeat_interleave(256)
        runs[bits] = float(x.mean())
    assert abs(runs[32] / sigma ** 2 - (1 + 3 * 0.999 ** 3000)) < 0.02
    assert abs(runs[8] / runs[32] - 1) < 0.02


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("shift", [0, 1])
def test_norm(sizes, shift):
    case = Case(SIZES[sizes], shift=shift, arena=True)
    norm = torch.empty(1, device="cuda")
    a = case.opt.grad_norm(norm).clone()
    b = case.opt.grad_norm(norm).clone()
    exact = A.grad_norm(case.g)
    # a lane's squares are summed in fp32, all else in twice its digits: errors of either sign, of which 16u of the square
    # (8u of its root) are far out
    assert abs(float(a) - exact) <= 8 * U * exact
    assert torch.equal(a, b)
    alone = AdamW(case.sizes)
    alone.bind_grads(case.grads)
    assert torch.equal(alone.grad_norm(norm), a)


def test_norm_of_nothing():
    for sizes in ([], [0, 0]):
        opt = AdamW(sizes)
        opt.bind_grads([torch.empty(0, device="cuda") for _ in sizes])
        assert float(opt.grad_norm(torch.full((1,), 3.0, device="cuda"))) == 0.0
        opt.bind(*[[torch.empty(0, device="cuda") for _ in sizes] for _ in range(4)])
        opt.step(1)


def test_norm_grid_changes_between_calls():
    """The norm's count of finished CTAs serves every grid: bindings of other sizes, calls in a row."""
    for sizes in ([10], [3_000_000], [100], [700_000, 5]):
        g = [torch.full((n,), 0.5, device="cuda") for n in sizes]
        opt = AdamW(sizes)
        opt.bind_grads(g)
        for _ in range(3):
            assert float(opt.grad_norm(torch.zeros(1, device="cuda"))) == pytest.approx(0.5 * sum(sizes) ** 0.5, rel=1e-6)


def test_other_stream_and_graph():
    case = Case([1000, 33], "f32", 32)
    twin = Case([1000, 33], "f32", 32)
    norm, other = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    case.opt.grad_norm(norm, stream=side)
    hyper = dict(lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"])
    case.opt.step(1, norm=norm, max_norm=0.1, stream=side, **hyper)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twin.opt.grad_norm(other)
        twin.opt.step(1, norm=other, max_norm=0.1, **hyper)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, other) and float(norm) > 0
    for a, b in zip(case.weights + case.m_t + case.v_t, twin.weights + twin.m_t + twin.v_t):
        assert torch.equal(a, b)
    case.check(1, A.clip_factor(float(norm), 0.1))


def test_a_step_on_another_stream_straight_after_bind():
    """bind has put its table in place when it returns, for streams that wait for no other too."""
    sizes = [1 + v % 5 for v in range(900)]
    g = [torch.full((n,), 2.0, device="cuda") for n in sizes]
    w = [torch.zeros(n, device="cuda") for n in sizes]
    opt = AdamW(sizes, "f32", 32)
    state = opt.zero_state()
    side = torch.cuda.Stream()
    norm = torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        opt.bind(w, g, **state)
        opt.grad_norm(norm, stream=side)
        side.synchronize()
        assert float(norm) == pytest.approx(2.0 * sum(sizes) ** 0.5, rel=1e-6)
        norm.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    """One tensor of 2^31 + 301 elements: zeros but for its ends."""
    n = 2 ** 31 + 301
    opt = AdamW([n], "f32", bits)
    w, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g[:3] = 2.0
    g[-3:] = 3.0
    state = opt.zero_state()
    opt.bind([w], [g], **state)
    norm = opt.grad_norm(torch.zeros(1, device="cuda"))
    assert float(norm) == pytest.approx((3 * 4 + 3 * 9) ** 0.5, rel=1e-6)
    opt.step(1, lr=0.5)
    torch.cuda.synchronize()
    m = state["exp_avg"][0]
    assert torch.allclose(w[:4], torch.tensor([-0.5, -0.5, -0.5, 0.0], device="cuda"))
    assert torch.allclose(w[-4:], torch.tensor([0.0, -0.5, -0.5, -0.5], device="cuda"))
    assert int((w != 0).sum()) == 6 and int((m.view(torch.uint8) != 0).any().item()) == 1
    assert int((m.float() != 0).sum()) == 6 if bits == 32 else float(state["exp_avg_scale"][0][-1]) > 0


def test_after_a_reduction():
    """Gradients reduced into the arena, their norm and the step on the bucket views: the formula on the replicas' mean."""
    numel = [300, 7, 1025, 64]
    red = Reducer(numel, "f32", 1200)
    gen = torch.Generator("cuda").manual_seed(0)
    replicas = [[torch.randn(n, generator=gen, device="cuda") for n in numel] for _ in range(4)]
    arena = torch.empty(red.arena_numel(), device="cuda")
    red.bind(replicas, arena, None)
    _, offs = red.get_bucket_info()
    views = [arena[offs[b] + o:offs[b] + o + n] for b, _, o, n in red.get_locators()]
    weights = [torch.randn(n, generator=gen, device="cuda") for n in numel]
    start = [w.cpu().numpy().astype(np.float64) for w in weights]
    opt = AdamW(numel)
    opt.bind(weights, views, weight_decay=0.01, **opt.zero_state())
    red.reduce_all()
    norm = opt.grad_norm(torch.empty(1, device="cuda"))
    opt.step(1, norm=norm, max_norm=1.0)
    torch.cuda.synchronize()
    mean = [np.mean([r[v].cpu().numpy().astype(np.float64) for r in replicas], axis=0) for v in range(4)]
    exact = A.grad_norm(mean)
    assert float(norm) == pytest.approx(exact, rel=1e-6)
    for v, n in enumerate(numel):
        want, _, _ = A.adamw(start[v], mean[v], np.zeros(n), np.zeros(n), 1, 1e-3, 0.9, 0.999, 1e-8, 0.01,
                             A.clip_factor(exact, 1.0))
        # a first step moves by lr whatever the gradient is, but where it is near eps: none is
        np.testing.assert_allclose(weights[v].cpu().numpy(), want, rtol=0, atol=4 * U * 5 + 40 * U * 1e-3)


def test_gradient_step_against_differences():
    """The step is a function of the gradient: its slope in g, by differences of the oracle's, agrees with the kernel's
    own response to a changed gradient."""
    n = 64
    rng = np.random.default_rng(0)
    g0, dg = rng.normal(size=n).astype(np.float32), np.float32(2.0 ** -4)
    moved = []
    for g in (g0 - dg, g0 + dg):
        opt = AdamW([n])
        w, gt = torch.zeros(n, device="cuda"), torch.from_numpy(g).cuda()
        m, v = torch.full((n,), 0.5, device="cuda"), torch.full((n,), 2.0, device="cuda")
        opt.bind([w], [gt], [m], [v])
        opt.step(10, lr=1.0)
        moved.append(w.cpu().numpy().astype(np.float64))
    want = [A.adamw(np.zeros(n), g, np.full(n, 0.5), np.full(n, 2.0), 10, 1.0, 0.9, 0.999, 1e-8, 0.0)[0]
            for g in (g0 - dg, g0 + dg)]
    # each side is within 24u of a value of about 0.1 / sqrt(200)
    np.testing.assert_allclose(moved[1] - moved[0], want[1] - want[0], rtol=0, atol=48 * U * 0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_twenty_thousand_tensors(bits):
    """Tensors of 1 to 60 elements, one block each: every fp32 moment and weight of the first step from zero state, where
    m' = (1 - b1) g, v' = (1 - b2) g^2 and the update is lr g / (|g| + eps sqrt-corrected) to 12u."""
    sizes = [1 + (i * 7919) % 60 for i in range(20_000)]
    flat = torch.randn(sum(sizes), generator=torch.Generator("cuda").manual_seed(0), device="cuda")
    weight = torch.zeros(sum(sizes), device="cuda")
    opt = AdamW(sizes, state_bits=bits)
    state = opt.zero_state()
    opt.bind(list(weight.split(sizes)), list(flat.split(sizes)), **state)
    norm = opt.grad_norm(torch.empty(1, device="cuda"))
    opt.step(1, lr=0.5, eps=1e-30)
    torch.cuda.synchronize()
    exact = float(flat.double().square().sum().sqrt())
    assert abs(float(norm) - exact) <= 8 * U * exact
    assert torch.allclose(weight, -0.5 * torch.sign(flat), rtol=24 * U, atol=0)
    if bits == 32:
        m = torch.cat(state["exp_avg"])
        assert torch.allclose(m, flat * np.float32(1 - 0.9), rtol=2 * U, atol=0)
    else:
        peak = torch.stack([x.abs().amax() for x in flat.split(sizes)[:200]])
        got = torch.stack([x[0] for x in state["exp_avg_scale"][:200]])
        assert torch.allclose(got, peak * np.float32(1 - 0.9) / 448, rtol=4 * U, atol=0)
