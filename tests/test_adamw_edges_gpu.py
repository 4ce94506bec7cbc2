"""Edges of lrm_adamw and AdamW: blocks of 8-bit states that are zero or near the floor of their scale, steps counted on
the device, tensors that moved and states that are loaded."""
import pytest
import torch

from helpers import ensure_built
from test_adamw_gpu import BF16, F32, FP8, Case, gen, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


FLOOR = 2.0 ** -119  # of the largest magnitude of 256 elements' states: 448 / FLOOR is an fp32 value


def all_finite(opt):
    return all(bool(torch.isfinite(t.float()).all()) for key in opt.state for t in opt.state[key])


@pytest.mark.parametrize("g_dt", [BF16, F32], ids=["bf16", "f32"])
def test_zero_blocks_stay_zero(g_dt):
    """An expert without a token: zero states and zero gradients for some steps, then gradients for a part of it."""
    import pruned_expert_backward_gb300 as lrm
    n = (1 << 20) + 77
    w = (torch.randn(n, generator=gen(3), device="cuda") * 0.1).bfloat16()
    start, g = w.clone(), torch.zeros(n, dtype=g_dt, device="cuda")
    opt = lrm.AdamW([w], [g], lr=1e-2, betas=(0.9, 0.95), weight_decay=0.0, state_bits=8, max_norm=1.0)
    for _ in range(3):
        opt.step()
        assert all_finite(opt)
        for key in ("m", "v"):
            assert int(torch.count_nonzero(opt.state[key][0].float())) == 0
            scale = opt.state[key + "_scale"][0].double()
            assert bool(((scale - FLOOR / 448).abs() <= 2.0 ** -149).all())  # (a subnormal's spacing)
    assert torch.equal(w, start) and opt.norm.item() == 0.0
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    live[:5000] = live[-1] = True
    g[live] = 1e-3
    for _ in range(3):
        opt.step()
        assert all_finite(opt) and bool(torch.isfinite(w).all())
    assert torch.equal(w[~live], start[~live])
    assert bool((w[live].float() < start[live].float()).all())
    for key in ("m", "v"):
        held = opt.state[key][0].float()
        assert int(torch.count_nonzero(held[~live])) == 0 and bool((held[live] > 0).all())
    assert int(opt.dev_status.item()) == 0


def test_states_near_the_floor_of_their_scale():
    """Halved first moments whose largest is 2^-110 to 2^-140, and none: held within a step of e4m3 (2^-3 of the value,
    2^-9 of the scale for the smallest), with the scale within its own spacing (2^-149, on 448 steps)."""
    import pruned_expert_backward_gb300 as lrm
    powers = [-110, -116, -117, -118, -118.25, -118.5, -118.75, -119, -119.5, -120, -125, -130, -140, None]
    n = 256 * len(powers)
    q = torch.rand(n, generator=gen(5), device="cuda") * 446 + 1
    q[::256] = 448
    q[1::256] = -448
    q[2::256] = 2.0 ** -9
    q[3::256] = 0
    m = q.to(FP8)
    for i, p in enumerate(powers):
        if p is None:
            m[256 * i:256 * (i + 1)] = torch.zeros(256, device="cuda").to(FP8)
    scale = torch.tensor([0.0 if p is None else 2.0 ** p / 448 for p in powers], device="cuda")
    state = {"m": [m], "m_scale": [scale], "v": [torch.zeros(n, device="cuda").to(FP8)],
             "v_scale": [torch.zeros(len(powers), device="cuda")]}
    want = values(m, scale) / 2
    w, g = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    opt = lrm.AdamW([w], [g], lr=1e-2, betas=(0.5, 0.9), weight_decay=0.0, state_bits=8, state=state, seed=3)
    opt.step()
    assert all_finite(opt)
    top = want.abs().view(-1, 256).amax(1).clamp_min(FLOOR)
    new = opt.state["m_scale"][0].double()
    assert bool(((new - top / 448).abs() <= 2.0 ** -20 * top / 448 + 2.0 ** -148).all())
    held, spacing = values(opt.state["m"][0], opt.state["m_scale"][0]), new.repeat_interleave(256)
    assert bool(((held - want).abs() <= 2.0 ** -3 * want.abs() + 2.0 ** -9 * spacing + 448 * 2.0 ** -148).all())
    assert bool((held[want == 0] == 0).all())
    assert torch.equal(w, torch.ones_like(w))  # m / eps is below 2^-80
    for _ in range(3):
        opt.step()
        assert all_finite(opt) and bool(torch.isfinite(w).all())


def test_zero_elements_past_32_bits():
    """Every state of a tensor whose element numbers pass 32 bits, without gradient but for its end."""
    import pruned_expert_backward_gb300 as lrm
    n = 2 ** 32 + 777
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    w, g = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    g[-300:] = 0.5
    opt = lrm.AdamW([w], [g], lr=1e-2, betas=(0.9, 0.95), weight_decay=0.0, state_bits=8, seed=21)
    for _ in range(2):
        opt.step()
        for key in ("m", "v"):
            codes = opt.state[key][0].view(torch.uint8)
            for part in codes[:-300].split(1 << 30):
                assert int(torch.count_nonzero(part & 0x7F)) == 0
            assert bool(torch.isfinite(codes[-300:].view(FP8).float()).all())
            assert bool(torch.isfinite(opt.state[key + "_scale"][0]).all())
    assert int(torch.count_nonzero(w[:-300].view(torch.int16))) == 0 and bool((w[-300:] < 0).all())


def test_a_device_step_below_1_counts_as_1():
    """Bias corrections and random bits alike."""
    import pruned_expert_backward_gb300 as lrm
    out = []
    for first in (0, -1, -1000):
        c = Case([5000], F32, F32, 8)
        opt = c.optimiser(lrm, lr=3e-4, seed=7, capturable=True)
        opt.step_dev.fill_(first)
        opt.step()
        assert int(opt.step_dev.item()) == first + 1
        out.append([c.w[0], *(c.state[k][0].view(torch.uint8) for k in c.state)])
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


def moved(t):
    """The tensor's values elsewhere, as a module that is moved leaves it; where they were."""
    old = t.data_ptr()
    t.data = t.data.clone()
    assert t.data_ptr() != old
    return old


def test_memory_that_the_tables_address_stays():
    """A param, copy, gradient or state whose tensor got other memory: nobody else gets the old, and where a copy, or a
    param without one, moved, a step is refused before it changes anything."""
    import pruned_expert_backward_gb300 as lrm
    for which, copy in (("w", False), ("copy", True), ("w", True), ("g", False), ("m", True), ("v", False)):
        c = Case([70001, 300], F32, F32, 32, copy=copy)
        other = Case([70001, 300], F32, F32, 32, copy=copy)
        opt, twin = c.optimiser(lrm, lr=1e-3), other.optimiser(lrm, lr=1e-3)
        t = c.state[which][0] if which in c.state else getattr(c, which)[0]
        old = moved(t)
        taken = [torch.full_like(t, 9.0) for _ in range(64)]
        assert all(a.data_ptr() != old for a in taken)
        if which == "copy" or (which == "w" and not copy):
            with pytest.raises(ValueError):
                opt.step()
            assert opt.steps == 0
            assert all(torch.equal(a, b) for k in c.state for a, b in zip(c.state[k], other.state[k]))
        else:  # the step goes on where the tables point
            opt.step()
            twin.step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(c.copy if copy else c.w, other.copy if copy else other.w))
        assert all(bool((a == 9.0).all()) for a in taken)


@pytest.mark.parametrize("bits", [8, 32])
def test_state_is_read_only_and_loaded(bits):
    import io

    import pruned_expert_backward_gb300 as lrm
    sizes, kw = [5000, 300, 1], dict(lr=1e-3, seed=4, max_norm=1.0)
    a, b = Case(sizes, BF16, F32, bits, seed=1), Case(sizes, BF16, F32, bits, seed=2)
    first = a.optimiser(lrm, **kw)
    first.step()
    saved = io.BytesIO()
    torch.save(first.state, saved)
    saved.seek(0)
    state = torch.load(saved, map_location="cpu")
    second = b.optimiser(lrm, **kw)
    for name in ("params", "copies", "grads", "state", "state_bits"):
        with pytest.raises(AttributeError):
            setattr(second, name, getattr(second, name))
    for call in (lambda: second.state.update(state), lambda: second.state.pop("m"),
                 lambda: second.state.__setitem__("m", state["m"]), lambda: second.state["m"].__setitem__(0, None),
                 lambda: second.params.__setitem__(0, None),
                 lambda: second.load_state(dict(state, m=[t.double() for t in state["m"]]))):
        with pytest.raises((TypeError, AttributeError)):
            call()
    for bad in (state["m"][:2], state["m"][::-1]):
        with pytest.raises(ValueError):
            second.load_state(dict(state, m=bad))
    b.state["m"][0] = None  # (the caller's own list)
    second.load_state(state)
    for own, t, g, u in zip(second.params, first.params, second.grads, first.grads):
        own.copy_(t)
        g.copy_(u)
    second.steps = first.steps
    first.step()
    second.step()
    for t, u in zip((*first.params, *(t for k in first.state for t in first.state[k])),
                    (*second.params, *(t for k in second.state for t in second.state[k]))):
        assert torch.equal(t.view(torch.uint8) if t.dtype == FP8 else t, u.view(torch.uint8) if u.dtype == FP8 else u)
    with pytest.raises(ValueError):
        lrm.AdamW(b.w, b.g, state_bits=bits, state={k: second.state[k][:2] for k in second.state})


@pytest.mark.parametrize("captured", [False, True])
def test_steps_on_the_device_that_are_skipped_or_refused_do_not_count(captured):
    """A first step whose norm is not finite, then two as if it had not been; a refused one changes no count."""
    import pruned_expert_backward_gb300 as lrm
    for bad in (float("inf"), float("nan")):
        a, b = Case([5000, 33], F32, F32, 8), Case([5000, 33], F32, F32, 8)
        kw = dict(lr=1e-3, max_norm=0.5, seed=7, capturable=True)
        opt, plain = a.optimiser(lrm, **kw), b.optimiser(lrm, **kw)
        for name, value in (("lr", -1.0), ("betas", (0.9, 1.0)), ("eps", float("nan"))):
            good = getattr(opt, name)
            setattr(opt, name, value)
            with pytest.raises(lrm.LrmError):
                opt.step()
            setattr(opt, name, good)
        assert int(opt.step_dev.item()) == 0 and opt.norm.item() == 0.0
        run = opt.step
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                opt.step()
            run = graph.replay
        kept = a.g[0][7].clone()
        a.g[0][7] = bad
        run()
        assert int(opt.step_dev.item()) == 0 and int(opt.dev_status.item()) == 7
        a.g[0][7] = kept
        for count in (1, 2):
            run()
            plain.step()
            assert int(opt.step_dev.item()) == int(plain.step_dev.item()) == count
        for t, u in zip((*a.w, *sum(a.state.values(), [])), (*b.w, *sum(b.state.values(), []))):
            assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))
    opt = Case([100], F32, F32, 32).optimiser(lrm, lr=1e-3, capturable=True)  # without a norm every step counts
    opt.step()
    opt.step()
    assert int(opt.step_dev.item()) == 2


def test_the_smallest_eps():
    """2^-126, with zero and tiny gradients: 0 where there is none, the formula's quotient elsewhere."""
    import pruned_expert_backward_gb300 as lrm
    for bits in (8, 32):
        w, g = torch.zeros(600, device="cuda"), torch.zeros(600, device="cuda")
        g[300:] = 1e-3
        opt = lrm.AdamW([w], [g], lr=1e-2, eps=2.0 ** -126, weight_decay=0.0, state_bits=bits)
        opt.step()
        assert int(torch.count_nonzero(w[:300])) == 0
        assert bool(((w[300:] + 1e-2).abs() <= 1e-2 * 2.0 ** -18).all())
        for bad in (1e-40, 1.17e-38):
            with pytest.raises(lrm.LrmError):
                lrm.AdamW([w], [g], eps=bad).step()


@pytest.mark.parametrize("bits", [8, 32])
def test_tensors_of_several_launches(bits):
    """More tensors than two launches hold (384 each), of two types: every state, random bit and weight, and the norm
    over all launches' sums."""
    import pruned_expert_backward_gb300 as lrm
    a = Case([1 + (i * 37) % 700 if i % 50 else 0 for i in range(800)] + [20000], BF16, F32, bits, seed=1)
    b = Case([1 + (i * 53) % 300 for i in range(400)], F32, F32, bits, seed=2)
    wa, wb = (c.expect(3e-4, 0.9, 0.95, 1e-8, 0.1, 3) for c in (a, b))
    state = {k: a.state[k] + b.state[k] for k in a.state}
    opt = lrm.AdamW(a.w + b.w, a.g + b.g, lr=3e-4, betas=(0.9, 0.95), weight_decay=0.1, state_bits=bits, state=state,
                    max_norm=1e6, seed=5)
    norm = opt.step(step=3).item()
    want = torch.cat([g.double() for g in a.g + b.g]).norm().item()
    assert abs(norm / want - 1) < 1e-6
    whole = Case.__new__(Case)
    whole.bits, whole.copy, whole.state = bits, None, state
    whole.w, whole.sizes = a.w + b.w, a.sizes + b.sizes
    whole.check(wa + wb, 3, 5)
    assert int(opt.dev_status.item()) == 0
