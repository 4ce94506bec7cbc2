"""GPU parity of lrm_adamw and lrm_grad_norm against 64-bit forms.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding to nearest):
  * m = b1 m + (1 - b1) g factor: the constants, the factor's product and the sum are rounded: 4 u of the terms'
    magnitudes.  v the same with g squared: 6 u of v itself (its terms have one sign).
  * w: decay and sum 3 u |w|; the update u_t = rate m / (sqrt(v) / sqrt(c2) + eps) has m's error over the denominator
    and 24 u of itself (fast quotient 4 u, fast root 2 u, half of v's 6 u, c1, c2, their roots and quotients, rate).
    One rounding to the type of w more: half a step, 2^-9 |w| for bf16, doubled to 2^-8.
  * 8-bit states: the value before rounding errs by 2^-20 relative at most, so the code is one of the two neighbours of
    the 64-bit value (that much further apart), and it is the one that the 16 random bits choose but where they fall
    within that error: at most 2^-15 of the elements, 2^-10 allowed.
"""
import numpy as np
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def mix(h):
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def random_bits(at, seed, step, ident):
    key = mix(mix((seed + 0x9E3779B9 * (ident + 1)) & 0xFFFFFFFF) ^ step)
    return mix(((at & 0xFFFFFFFF) * 0x9E3779B1 + (at >> 32) * 0xC2B2AE3D + key) & 0xFFFFFFFF)


def values(q, scale):
    """What 8-bit states stand for, in 64 bits."""
    return q.double() * scale.double().repeat_interleave(256)[: q.numel()].view(q.shape)


class Case:
    """Tensors with a state of some steps ago, and what a step makes of them in 64 bits."""

    def __init__(self, sizes, w_dt, g_dt, bits, copy=False, seed=1, std=1e-3):
        g = gen(seed)

        def make(n, scale, dt):
            return (torch.randn(n, generator=g, device="cuda") * scale).to(dt)

        self.bits, self.sizes = bits, sizes
        self.w = [make(n, 0.02, w_dt) for n in sizes]
        self.g = [make(n, std, g_dt) for n in sizes]
        self.copy = [make(n, 1.0, BF16) for n in sizes] if copy else None
        m, r = [make(n, 0.3 * std, F32) for n in sizes], [make(n, std, F32).abs() + 0.1 * std for n in sizes]
        if bits == 32:
            self.state = {"m": m, "v": [a.square() for a in r]}
        else:
            self.state = {"m": [], "v": [], "m_scale": [], "v_scale": []}
            for key, each in (("m", m), ("v", r)):
                for a in each:
                    n = a.numel()
                    p = torch.nn.functional.pad(a, (0, -n % 256)).view(-1, 256)
                    top = p.abs().amax(1, keepdim=True).clamp_min(1e-30)
                    self.state[key].append((p * (448 / top)).to(FP8).view(-1)[:n].contiguous())
                    self.state[key + "_scale"].append((top / 448).view(-1))

    def moments(self, i):
        if self.bits == 32:
            return self.state["m"][i].double(), self.state["v"][i].double()
        return (values(self.state["m"][i], self.state["m_scale"][i]),
                values(self.state["v"][i], self.state["v_scale"][i]).square())

    def optimiser(self, lrm, **kw):
        return lrm.AdamW(self.w, self.g, copies=self.copy, state_bits=self.bits, state=self.state, **kw)

    def expect(self, lr, b1, b2, eps, wd, step, factor=1.0, lr_scale=1.0, only=None):
        """(w, m, v and bounds on their errors before the last rounding) of each tensor."""
        out = []
        for i in range(len(self.sizes)) if only is None else [only]:
            g = self.g[i].double() * factor
            m0, v0 = self.moments(i)
            m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
            em, ev = 4 * U * ((b1 * m0).abs() + ((1 - b1) * g).abs()), 6 * U * v
            den = v.sqrt() / (1 - b2 ** step) ** 0.5 + eps
            rate = lr * lr_scale / (1 - b1 ** step)
            up = rate * m / den
            w = self.w[i].double() * (1 - lr * lr_scale * wd) - up
            ew = 3 * U * (self.w[i].double().abs() + w.abs()) + rate * em / den + 24 * U * up.abs()
            out.append((w, ew, m, em, v, ev))
        return out

    def check(self, want, step=1, seed=0):
        for i, (w, ew, m, em, v, ev) in enumerate(want):
            ulp = 2.0 ** -8 if self.w[i].dtype == BF16 else 2 * U
            assert bool(((self.w[i].double() - w).abs() <= ew + ulp * w.abs()).all()), i
            if self.copy is not None:
                assert torch.equal(self.copy[i], self.w[i].bfloat16())
            if self.bits == 32:
                assert bool(((self.state["m"][i].double() - m).abs() <= em + U * m.abs()).all())
                assert bool(((self.state["v"][i].double() - v).abs() <= ev).all())
            elif self.sizes[i]:
                bits = random_bits(torch.arange(self.sizes[i], device="cuda"), seed, step, i)
                self.check_state(i, "m", m, bits & 0xFFFF, 0.0)
                self.check_state(i, "v", v.sqrt(), bits >> 16, 2.0 ** -9)

    def check_state(self, i, key, a, rnd, least):
        n = a.numel()
        top = torch.nn.functional.pad(a.abs(), (0, -n % 256)).view(-1, 256).amax(1).clamp_min(2.0 ** -120)
        scale = self.state[key + "_scale"][i].double()
        assert bool(((scale - top / 448).abs() <= 2.0 ** -20 * top / 448).all())
        y = a.abs() / top.repeat_interleave(256)[:n] * 448
        step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)  # e4m3's spacing at y
        low = torch.floor(y / step) * step
        chosen = torch.where((y - low) / step + rnd.double() / 65536 >= 1, low + step, low).clamp_max(448)
        chosen = torch.where((a != 0) & (chosen < least), torch.full_like(chosen, least), chosen)
        got = self.state[key][i].double()
        assert bool((torch.signbit(got) == torch.signbit(a))[got != 0].all())
        got = got.abs()
        near = (got - y).abs() <= step + 2.0 ** -18 * y + (least if least else 0)
        assert bool(near.all())
        assert int((got != chosen).sum()) <= 2 + n / 1024
        if least:
            assert bool((got[a > 0] > 0).all())


HYPER = dict(lr=3e-4, betas=(0.9, 0.95), eps=1e-8)
TYPES = [(BF16, F32, 8, False), (BF16, BF16, 8, False), (F32, F32, 8, False), (F32, BF16, 8, True),
         (BF16, F32, 32, False), (BF16, BF16, 32, False), (F32, F32, 32, True), (F32, BF16, 32, False)]


@pytest.mark.parametrize("types", TYPES, ids=str)
def test_step(types):
    import pruned_expert_backward_gb300 as lrm
    sizes = [1, 3, 4, 127, 128, 130, 255, 256, 257, 511, 8191, 8192, 8193, 100003]
    c = Case(sizes, *types)
    want = c.expect(3e-4, 0.9, 0.95, 1e-8, 0.1, 7)
    opt = c.optimiser(lrm, **HYPER, weight_decay=0.1, seed=99)
    assert opt.step(step=7) is None
    c.check(want, 7, 99)
    assert int(opt.dev_status.item()) == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_many_tensors_with_clipping_and_their_own_rates(bits):
    """More tensors than one launch takes, empty ones among them."""
    import pruned_expert_backward_gb300 as lrm
    sizes = [(i * 37) % 1000 if i % 50 else 0 for i in range(300)] + [20000]
    c = Case(sizes, BF16, F32, bits, std=0.1)
    norm = torch.cat([g.double() for g in c.g]).norm().item()
    assert norm > 2
    decay, scale = [0.1 * (i % 3) for i in range(301)], [1.0 + i % 2 for i in range(301)]
    factor = 0.5 / (norm + 1e-6)
    want = []
    for i in range(301):
        wanted = sizes[i] > 0 and i % 10 == 0
        want.append(c.expect(3e-4, 0.9, 0.95, 1e-8, decay[i], 3, factor, scale[i], only=i)[0] if wanted else None)
    opt = c.optimiser(lrm, **HYPER, weight_decay=decay, lr_scale=scale, max_norm=0.5, seed=5)
    got = opt.step(step=3)
    assert abs(got.item() / norm - 1) < 1e-6
    for i in range(0, 301, 10):
        if want[i] is not None:
            part = Case.__new__(Case)
            part.bits, part.sizes = c.bits, [sizes[i]]
            part.w, part.copy = [c.w[i]], None
            part.state = {k: [v[i]] for k, v in c.state.items()}
            w, ew, m, em, v, ev = want[i]
            # the factor has errors of its own: the norm's and its quotient's, 1e-6
            slack = 2e-6 * c.g[i].double().abs() * factor
            den = v.sqrt() / (1 - 0.95 ** 3) ** 0.5 + 1e-8
            ew = ew + 3e-4 * scale[i] / (1 - 0.9 ** 3) * (0.1 * slack / den + 2e-6 * m.abs() / den)
            if bits == 32:
                part.check([(w, ew, m, em + 0.1 * slack, v, ev + 4e-6 * v)])
            else:
                assert bool(((c.w[i].double() - w).abs() <= ew + 2.0 ** -8 * w.abs()).all())
                bits_i = random_bits(torch.arange(sizes[i], device="cuda"), 5, 3, i)
                part.check_state(0, "m", m, bits_i & 0xFFFF, 0.0)
                part.check_state(0, "v", v.sqrt(), bits_i >> 16, 2.0 ** -9)


def test_norm_of_long_and_odd_gradients():
    import pruned_expert_backward_gb300 as lrm
    for dt in (BF16, F32):
        for sizes in ([1], [3, 5], [8192 * 700 + 11, 7], [1 << 24]):
            g = [torch.randn(n, generator=gen(n), device="cuda").to(dt) for n in sizes]
            opt = lrm.AdamW([torch.zeros(n, device="cuda") for n in sizes], g, max_norm=1.0)
            want = sum(float(a.double().square().sum()) for a in g) ** 0.5
            # 32 squares a partial sum in fp32: 33 roundings at most, then 64 bits and one rounding
            assert abs(opt.step().item() / want - 1) <= 17 * U + U
    opt = lrm.AdamW([torch.zeros(0, device="cuda")], [torch.zeros(0, device="cuda")], max_norm=1.0)
    assert opt.step().item() == 0.0


def test_same_bits_again():
    import pruned_expert_backward_gb300 as lrm
    out = []
    for _ in range(2):
        c = Case([1 << 20, 777], BF16, F32, 8)
        opt = c.optimiser(lrm, **HYPER, max_norm=0.1, seed=3)
        opt.step()
        opt.step()
        codes = [a.view(torch.uint8) for k in ("m", "v") for a in c.state[k]]
        out.append([*c.w, *codes, *c.state["m_scale"], opt.norm])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_states_repeat_in_a_host_programs_fp32():
    """Two steps' 8-bit states, bit for bit from fp32 operations that are each rounded by themselves."""
    import pruned_expert_backward_gb300 as lrm
    f, n = np.float32, 256 * 500 + 77
    c = Case([n], F32, F32, 8, seed=8)
    opt = c.optimiser(lrm, **HYPER, max_norm=0.01, seed=21)

    def host(a):
        return a.float().cpu().numpy()

    def state(a, rnd, least):
        top = np.maximum(np.abs(np.pad(a, (0, -n % 256))).reshape(-1, 256).max(1), f(2.0 ** -120))
        y = np.abs(a) * np.repeat(f(448) * (f(1) / top), 256)[:n]
        shift = np.where(y < f(2.0 ** -6), f(2.0 ** -6), f(0))
        up = ((y + shift).view(np.uint32) + (rnd.astype(np.uint32) << np.uint32(4))) & np.uint32(0xFFF00000)
        y = up.view(f) - shift
        y = np.where((a != 0) & (y < least), f(least), y)
        return np.copysign(y, a), top * (f(1) / f(448))

    for step in (1, 2):
        m, r = (host(c.state[k][0]) * np.repeat(host(c.state[k + "_scale"][0]), 256)[:n] for k in ("m", "v"))
        v = r * r
        norm = f(opt.step().item())
        g = host(c.g[0]) * (f(1) / (norm + f(1e-6)) * f(0.01))
        m = m * f(0.9) + g * f(1 - 0.9)
        v = v * f(0.95) + g * g * f(1 - 0.95)
        bits = random_bits(torch.arange(n), 21, step, 0).numpy()
        for key, a, rnd, least in (("m", m, bits & 0xFFFF, 0.0), ("v", np.sqrt(v), bits >> 16, 2.0 ** -9)):
            q, scale = state(a, rnd, least)
            assert np.array_equal(host(c.state[key][0]), q) and np.array_equal(host(c.state[key + "_scale"][0]), scale)


def test_random_rounding_keeps_the_mean():
    """A sqrt(v) that shrinks by 0.05 % a step does so in 8 bits too; to nearest it would stand still (half a step is 3
    to 6 %).  100000 equal values after 400 steps of no gradient: the mean's deviation, a walk of 400 steps of at most
    1/8 relative each over 100000 values, is below 400^0.5 / 8 / 100000^0.5 < 0.8 %; five of them are allowed."""
    import pruned_expert_backward_gb300 as lrm
    n = 100096
    r = torch.full((n,), 0.3, device="cuda")
    r[::256] = 1.0  # the largest of each block, whose scale follows it exactly
    state = {"m": [torch.zeros(n, device="cuda").to(FP8)], "v": [(r * 448).to(FP8)],
             "m_scale": [torch.zeros(n // 256, device="cuda")],
             "v_scale": [torch.full((n // 256,), 1 / 448, device="cuda")]}
    start = values(state["v"][0], state["v_scale"][0])
    g = torch.zeros(n, device="cuda")
    big = torch.zeros(n, dtype=torch.bool, device="cuda")
    big[::256] = True
    g[big] = 1.0  # the largest stay at 1, so that the others shrink against their scale
    opt = lrm.AdamW([torch.zeros(n, device="cuda")], [g], lr=0.0, betas=(0.9, 0.999), state_bits=8, state=state,
                    seed=11)
    for _ in range(400):
        opt.step()
    now = values(state["v"][0], state["v_scale"][0])
    ratio = (now[~big].mean() / start[~big].mean()).item()
    assert abs(ratio / 0.999 ** 200 - 1) < 0.04
    assert bool(((now[big] - 1).abs() < 1e-3).all())


def test_elements_without_gradient_do_not_explode():
    """A value far below its block's largest keeps a sqrt(v) above 0, so its m over it stays small."""
    import pruned_expert_backward_gb300 as lrm
    n = 512
    w, g = torch.zeros(n, device="cuda"), torch.full((n,), 1e-6, device="cuda")
    g[0] = g[300] = 1e4
    opt = lrm.AdamW([w], [g], lr=1e-3, betas=(0.9, 0.95), weight_decay=0.0, state_bits=8, seed=1)
    opt.step()
    g.zero_()
    for _ in range(20):
        opt.step()
    assert w.abs().max().item() < 0.1 and bool(torch.isfinite(w).all())
    assert bool((opt.state["v"][0].float() > 0).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_gradients_that_are_not_finite(bits):
    import pruned_expert_backward_gb300 as lrm
    for bad in (float("nan"), float("inf"), float("-inf")):
        c = Case([1000, 300], BF16, F32, bits)
        before = [a.clone() for a in (*c.w, *c.state["m"], *c.state["v"])]
        c.g[0][513] = bad
        opt = c.optimiser(lrm, **HYPER, max_norm=1.0)
        assert not np.isfinite(opt.step().item()) and int(opt.dev_status.item()) == 7
        after = [*c.w, *c.state["m"], *c.state["v"]]
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, after))
        # without the common norm it spoils itself (32 bits), or its 256 elements from the next step on (8 bits)
        opt = c.optimiser(lrm, **HYPER)
        opt.step()
        opt.step()
        broken = ~torch.isfinite(c.w[0])
        assert bool(broken[513]) and not bool(broken[:512].any()) and not bool(broken[768:].any())
        assert bits == 8 or int(broken.sum()) == 1
        assert bool(torch.isfinite(c.w[1]).all())


def test_extreme_states_and_first_steps():
    """Zeroed states, tiny and huge gradients, betas of zero, no decay: as the formula says."""
    import pruned_expert_backward_gb300 as lrm
    for scale in (1e-12, 1e-6, 1.0, 1e9, 1e15):
        for betas in ((0.9, 0.999), (0.0, 0.0), (0.0, 0.9)):
            for bits in (8, 32):
                w, g = torch.zeros(700, device="cuda"), torch.randn(700, generator=gen(4), device="cuda") * scale
                opt = lrm.AdamW([w], [g], lr=1e-2, betas=betas, eps=0.0, weight_decay=0.0, state_bits=bits)
                opt.step()
                # the first step moves every weight by the rate against its gradient's sign
                assert bool(((w + 1e-2 * g.sign()).abs() <= 1e-2 * 64 * U).all()), (scale, betas, bits)


def test_captured_steps():
    import pruned_expert_backward_gb300 as lrm
    for bits in (8, 32):
        a, b = Case([5000, 33], BF16, F32, bits), Case([5000, 33], BF16, F32, bits)
        eager = a.optimiser(lrm, **HYPER, max_norm=0.5, seed=7)
        graphed = b.optimiser(lrm, **HYPER, max_norm=0.5, seed=7, capturable=True)
        graph = torch.cuda.CUDAGraph()
        graphed.step_dev.fill_(-1)
        with torch.cuda.graph(graph):
            graphed.step()
        graphed.step_dev.zero_()
        for k in range(3):
            for c in (a, b):
                for g in c.g:
                    g.mul_(1.5)
            if k == 2:
                graphed.lr_dev.fill_(1e-4)
            graph.replay()
            eager.step(lr=1e-4 if k == 2 else None)
        torch.cuda.synchronize()
        assert int(graphed.step_dev.item()) == 3
        for x, y in zip((*a.w, *a.state["m"], *a.state["v"]), (*b.w, *b.state["m"], *b.state["v"])):
            if x.dtype == FP8:
                assert int((x.view(torch.uint8) != y.view(torch.uint8)).sum()) <= 2 + x.numel() / 256
            else:
                assert torch.allclose(x.float(), y.float(), rtol=2.0 ** -7, atol=1e-9)


def test_another_stream_and_new_gradients():
    import pruned_expert_backward_gb300 as lrm
    c = Case([3000], F32, F32, 32)
    want = c.expect(3e-4, 0.9, 0.95, 1e-8, 0.01, 1)
    opt = c.optimiser(lrm, **HYPER)
    fresh = [g.clone() for g in c.g]
    opt.set_grads([torch.full_like(g, float("nan")) for g in c.g])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step(grads=fresh)
    side.synchronize()
    c.check(want)


def test_params_of_two_types():
    import pruned_expert_backward_gb300 as lrm
    a, b = Case([500, 70], BF16, F32, 32), Case([300], F32, F32, 32, copy=True)
    wa, wb = a.expect(3e-4, 0.9, 0.95, 1e-8, 0.01, 1), b.expect(3e-4, 0.9, 0.95, 1e-8, 0.01, 1)
    state = {k: [a.state[k][0], b.state[k][0], a.state[k][1]] for k in ("m", "v")}
    opt = lrm.AdamW([a.w[0], b.w[0], a.w[1]], [a.g[0], b.g[0], a.g[1]], copies=[None, b.copy[0], None], state=state,
                    max_norm=1e3, **HYPER)
    norm = opt.step().item()
    assert abs(norm / torch.cat([t.double() for t in (*a.g, *b.g)]).norm().item() - 1) < 1e-6
    a.check(wa)
    b.check(wb)


def test_more_than_32_bits_of_elements():
    """A tensor whose element numbers pass 32 bits: its last elements, and their random bits."""
    import pruned_expert_backward_gb300 as lrm
    n = 2 ** 32 + 777
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    w, g = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    at = 2 ** 32 - 512
    w[at:] = torch.randn(n - at, generator=gen(1), device="cuda").bfloat16()
    g[at:] = torch.randn(n - at, generator=gen(2), device="cuda").bfloat16()
    w0, g0 = w[at:].double(), g[at:].double()
    opt = lrm.AdamW([w], [g], lr=1e-2, betas=(0.9, 0.95), weight_decay=0.0, state_bits=8, seed=21, max_norm=1e9)
    norm = opt.step().item()
    assert abs(norm / g0.norm().item() - 1) < 1e-6
    m, v = 0.1 * g0, 0.05 * g0 * g0
    want = w0 - 1e-2 * g0.sign()
    assert bool(((w[at:].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all())
    part = Case.__new__(Case)
    part.bits, part.sizes = 8, [n - at]
    part.state = {"m": [opt.state["m"][0][at:]], "v": [opt.state["v"][0][at:]],
                  "m_scale": [opt.state["m_scale"][0][at // 256:]], "v_scale": [opt.state["v_scale"][0][at // 256:]]}
    bits = random_bits(torch.arange(at, n, device="cuda"), 21, 1, 0)
    part.check_state(0, "m", m, bits & 0xFFFF, 0.0)
    part.check_state(0, "v", v.sqrt(), bits >> 16, 2.0 ** -9)
    assert int(torch.count_nonzero(w[:at].view(torch.int16)).item()) == 0


def test_refusals():
    import pruned_expert_backward_gb300 as lrm
    w, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    for call in (lambda: lrm.AdamW([], []), lambda: lrm.AdamW([w], [g], state_bits=16), lambda: lrm.AdamW([w], [g, g]),
                 lambda: lrm.AdamW([w], [g[:32]]), lambda: lrm.AdamW([w.cpu()], [g]),
                 lambda: lrm.AdamW([w], [g], max_norm=0),
                 lambda: lrm.AdamW([w], [g], weight_decay=[0.1, 0.2]), lambda: lrm.AdamW([w[::2]], [g[:32]]),
                 lambda: lrm.AdamW([w], [g], state={"m": [w[:3]], "v": [g]}), lambda: lrm.AdamW([w], [g]).step(step=0),
                 lambda: lrm.AdamW([w], [g], copies=[w[:5].bfloat16()]),
                 lambda: lrm.AdamW([w, w], [g, g]), lambda: lrm.AdamW([w, w[32:]], [g, g[32:]]),
                 lambda: lrm.AdamW([w], [g], state={"m": [w], "v": [g]}),
                 lambda: lrm.AdamW([w], [g], capturable=True).step(step=3)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lrm.AdamW([w.half()], [g]), lambda: lrm.AdamW([w], [g.double()]),
                 lambda: lrm.AdamW([w, w.clone()], [g, g.bfloat16()]),
                 lambda: lrm.AdamW([w.bfloat16()], [g], copies=[w.bfloat16()]),
                 lambda: lrm.AdamW([w], [g], state={"m": [w.bfloat16()], "v": [w]})):
        with pytest.raises(TypeError):
            call()
    for kw in (dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=float("nan"))):
        with pytest.raises(lrm.LrmError):
            lrm.AdamW([w], [g], **kw).step()
    with pytest.raises(lrm.LrmError):
        lrm.AdamW([w[1:33]], [g[1:33]]).step()  # off the 16 bytes
    opt = lrm.AdamW([w, w.bfloat16()], [g, g.clone()])
    with pytest.raises(lrm.LrmError):
        opt.step(grads=[g, torch.zeros(65, device="cuda")[1:]])
    with pytest.raises(ValueError):
        opt.step(step=0)
    assert opt.steps == 0 and opt.step() is None and opt.steps == 1
    assert torch.count_nonzero(w) == 0
