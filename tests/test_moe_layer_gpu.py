"""GPU parity of the MoE layer's forward operators and their gradients against 64-bit plain forms.

Tolerances, from the arithmetic:
  * u is the output type's rounding: 2^-9 for bf16 (8 significant bits, to nearest), 2^-24 for fp32; one
    rounding of a value v errs by at most u |v|, so u is doubled to 2^-8 / 2^-23 for the comparison.
  * a sum of n products in fp32, in any order, each step rounded or truncated, errs by at most
    (n + 1) 2^-23 sum |a b|.  Through an activation that error is multiplied by its slope (at most 1.13
    for GELU and 1.1 for SiLU; through SwiGLU's gate, also by |up|).
  * fp32 expf / erff and the divide add a few units in 2^-23 of the activation's value (8 allowed).
"""
import numpy as np
import pytest
import torch

from helpers import ensure_built

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ULP = {BF16: 2.0 ** -8, F32: 2.0 ** -23}
EPS = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


@pytest.fixture
def status():
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    yield st
    torch.cuda.synchronize()
    assert int(st.item()) == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dt=BF16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def check(got, want, slack, dt=None):
    """|got - want| <= ulp |want| + slack, elementwise; NaN and infinities in the same places."""
    dt = got.dtype if dt is None else dt
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    slack = slack if torch.is_tensor(slack) else torch.full_like(want, float(slack))
    over = ((got - want).abs() - (ULP[dt] * want.abs() + slack))[fine]
    assert over.numel() == 0 or over.max().item() <= 0, f"over by {over.max().item():.3e}"


# ------------------------------------------------------------------------------------- sort -----
def routing(g, T, k, E, skew=1.0, masked=0.0):
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits -= skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=F32))
    top, idx = torch.topk(logits, k, dim=1)
    idx = idx.to(torch.int32)
    if masked:
        drop = torch.rand(T, k, generator=g, device="cuda") < masked
        drop |= torch.rand(T, 1, generator=g, device="cuda") < masked
        idx = torch.where(drop, torch.full_like(idx, -1), idx)
    return idx.contiguous(), torch.softmax(top, 1).contiguous()


def plain_sort(idx, E):
    flat = idx.cpu().numpy().reshape(-1)
    rows, pairs, seg = np.full(flat.size, -1, np.int64), np.full(flat.size, -1, np.int64), [0]
    at = 0
    for e in range(E):
        for u in np.flatnonzero(flat == e):
            rows[u], pairs[at] = at, u
            at += 1
        seg.append(at)
    return np.array(seg), pairs, rows


SORTS = [  # T, k, E, H, dtype, skew, masked
    (1, 8, 128, 2048, BF16, 1.0, 0.0), (1, 1, 1, 8, F32, 0.0, 0.0), (3, 16, 16, 24, BF16, 0.0, 0.0),
    (33, 2, 7, 520, F32, 1.5, 0.3), (255, 8, 256, 256, BF16, 1.0, 0.0), (256, 8, 256, 64, BF16, 1.0, 0.2),
    (257, 8, 256, 64, BF16, 1.0, 0.2), (100, 4, 257, 72, F32, 0.0, 0.1), (64, 16, 1024, 40, BF16, 1.0, 0.0),
    (5003, 6, 60, 136, F32, 1.0, 0.2), (4097, 2, 2, 8, BF16, 1.5, 0.0), (3000, 1, 1, 264, BF16, 0.0, 0.0),
    (20000, 8, 128, 16, BF16, 1.0, 0.05),
]


@pytest.mark.parametrize("case", SORTS, ids=str)
def test_sort(case, status):
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, dt, skew, masked = case
    g = gen(T + E)
    idx, _ = routing(g, T, k, E, skew, masked)
    x = randn(g, T, H, dt=dt)
    seg, pair, row, x_s = lrm.lrm_sort_tokens(idx, x, E, dev_status=status)
    wseg, wpair, wrow = plain_sort(idx, E)
    assert np.array_equal(seg.cpu().numpy(), wseg)
    assert np.array_equal(pair.cpu().numpy(), wpair)
    assert np.array_equal(row.cpu().numpy(), wrow)
    n = int(wseg[-1])
    assert torch.equal(x_s[:n], x[torch.from_numpy(wpair[:n] // k).cuda()])
    assert torch.count_nonzero(x_s[n:]) == 0
    # the index arrays alone, without rows
    seg2, pair2, row2, none = lrm.lrm_sort_tokens(idx, None, E, dev_status=status)
    assert none is None and torch.equal(seg2, seg) and torch.equal(pair2, pair) and torch.equal(row2, row)
    # the gradient: <sort(x), d> = <x, scatter(d)> for every d
    d = randn(g, T * k, H, dt=dt)
    d[n:] = 0
    dx = lrm.lrm_scatter_dx(row, d, T, k, dev_status=status)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    want.index_add_(0, torch.from_numpy(wpair[:n] // k).cuda(), d[:n].double())
    total = torch.zeros_like(want).index_add_(0, torch.from_numpy(wpair[:n] // k).cuda(), d[:n].double().abs())
    check(dx, want, k * EPS * total)


def test_sort_empty_masked_and_bad_ids():
    import pruned_expert_backward_gb300 as lrm
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for E in (4, 300):  # both forms
        idx = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
        seg, pair, row, x_s = lrm.lrm_sort_tokens(idx, torch.zeros(0, 16, device="cuda"), E, dev_status=st)
        assert torch.count_nonzero(seg) == 0 and pair.numel() == row.numel() == x_s.numel() == 0
    for T in (5, 3000):
        idx = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
        x = torch.ones(T, 16, device="cuda")
        seg, pair, row, x_s = lrm.lrm_sort_tokens(idx, x, 4, dev_status=st)
        assert torch.count_nonzero(seg) == 0 and torch.count_nonzero(x_s) == 0
        assert bool((pair == -1).all()) and bool((row == -1).all())
        assert int(st.item()) == 0
        # ids outside [0, E) other than -1 count as not routed and are reported
        idx[:] = 1
        idx[0, 0], idx[T - 1, 1], idx[2, 0] = 4, -7, 2 ** 31 - 1
        seg, pair, row, x_s = lrm.lrm_sort_tokens(idx, x, 4, dev_status=st)
        assert int(st.item()) == 9
        st.zero_()
        assert seg.tolist() == [0, 0, 2 * T - 3, 2 * T - 3, 2 * T - 3]
        assert row[0].item() == row[2 * T - 1].item() == row[4].item() == -1


# ---------------------------------------------------------------------------------- combine -----
COMBINES = [  # T, k, E, H, dtype, masked, residual
    (1, 8, 128, 2048, BF16, 0.0, True), (1, 1, 1, 8, F32, 0.0, False), (2047, 3, 9, 72, F32, 0.3, True),
    (2048, 3, 9, 72, BF16, 0.3, False), (2051, 16, 32, 264, BF16, 0.1, True), (4100, 11, 64, 520, F32, 0.2, False),
    (65, 8, 16, 4096, BF16, 0.0, False), (7, 9, 12, 4104, F32, 0.5, True),
]


def combine_inputs(case, seed):
    T, k, E, H, dt, masked, residual = case
    import pruned_expert_backward_gb300 as lrm
    g = gen(seed)
    idx, alpha = routing(g, T, k, E, 1.0, masked)
    _, _, row, _ = lrm.lrm_sort_tokens(idx, None, E)
    return g, row, alpha, randn(g, T * k, H, dt=dt), randn(g, T, H, dt=dt) if residual else None


def plain_combine(row, alpha, y_s, residual):
    T, k = alpha.shape
    r = row.long()
    rows = y_s.double()[r.clamp(min=0)].view(T, k, -1)
    live = (r >= 0).view(T, k, 1)
    terms = torch.where(live, alpha.double()[:, :, None] * rows, torch.zeros((), dtype=torch.float64, device="cuda"))
    base = residual.double() if residual is not None else torch.zeros_like(terms[:, 0])
    return base + terms.sum(1), terms.abs().sum(1) + base.abs()


@pytest.mark.parametrize("case", COMBINES, ids=str)
def test_combine_and_its_gradient(case, status):
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, dt, _, _ = case
    g, row, alpha, y_s, residual = combine_inputs(case, T)
    y_s[(row < 0).sum().neg().item() or T * k:] = float("nan")  # rows of no pair are never read
    y = lrm.lrm_combine(row, alpha, y_s, residual=residual, dev_status=status)
    want, total = plain_combine(row, alpha, y_s, residual)
    check(y, want, (k + 2) * EPS * total)
    if residual is not None:  # in place of the residual
        into = residual.clone()
        assert torch.equal(lrm.lrm_combine(row, alpha, y_s, residual=into, y=into, dev_status=status), y)
    dy = randn(g, T, H, dt=dt)
    dy_s = torch.full((T * k, H), 7.0, dtype=dt, device="cuda")
    _, dalpha = lrm.lrm_combine_backward(row, alpha, dy, y_s, dy_s=dy_s, dev_status=status)
    r = row.long().view(T, k)
    live = r >= 0
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    named[r[live]] = True
    assert bool((dy_s[~named] == 7.0).all())
    want_s = (alpha.double()[:, :, None] * dy.double()[:, None])[live]
    check(dy_s[r[live]], want_s, EPS * want_s.abs())
    prod = dy.double()[:, None] * y_s.double()[r.clamp(min=0)]
    prod = torch.where(live[:, :, None], prod, torch.zeros((), dtype=torch.float64, device="cuda"))
    check(dalpha, prod.sum(2), (H + 1) * EPS * prod.abs().sum(2))
    assert torch.count_nonzero(dalpha[~live]) == 0
    only = torch.full((T * k, H), 7.0, dtype=dt, device="cuda")
    assert lrm.lrm_combine_backward(row, alpha, dy, None, dy_s=only, dev_status=status)[1] is None
    assert torch.equal(only, dy_s)


def test_combine_gradient_against_differences(status):
    import pruned_expert_backward_gb300 as lrm
    T, k, H = 40, 4, 64
    g, row, alpha, y_s, _ = combine_inputs((T, k, 8, H, F32, 0.2, False), 5)
    dy = randn(g, T, H, dt=F32)
    dy_s, dalpha = lrm.lrm_combine_backward(row, alpha, dy, y_s, dy_s=torch.zeros_like(y_s), dev_status=status)

    def loss(a, s):
        return (lrm.lrm_combine(row, a, s, dev_status=status).double() * dy.double()).sum().item()

    # the operator is linear in each argument: central differences err only by fp32 rounding of y,
    # k 2^-23 |y| per value against a change of |grad| h
    for grad, moved in ((dalpha, lambda d: (alpha + d, y_s)), (dy_s, lambda d: (alpha, y_s + d))):
        step = grad / grad.norm()
        diff = (loss(*moved(step)) - loss(*moved(-step))) / 2
        assert abs(diff - grad.double().norm().item()) <= 1e-4 * grad.norm().item()


def test_combine_reports_a_row_out_of_range():
    import pruned_expert_backward_gb300 as lrm
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    row = torch.tensor([0, 5, -2, 1], dtype=torch.int32, device="cuda")
    y = lrm.lrm_combine(row, torch.ones(2, 2, device="cuda"), torch.ones(2, 16, device="cuda"), dev_status=st)
    assert int(st.item()) == 9 and bool((y == 1).all())
    st.zero_()
    dy_s, dalpha = lrm.lrm_combine_backward(row, torch.ones(2, 2, device="cuda"), torch.ones(2, 16, device="cuda"),
                                            torch.ones(2, 16, device="cuda"), dev_status=st)
    assert int(st.item()) == 9 and dalpha.tolist() == [[16.0, 0.0], [0.0, 16.0]]


# ----------------------------------------------------------------------------------- linear -----
def segments(kind, R, E, g):
    """Segment ends of R rows: 'even', 'ragged' (random, some empty), 'one' (all in one expert), 'short' (some rows
    belong to no expert)."""
    if kind == "even":
        cut = [R * e // E for e in range(E + 1)]
    elif kind == "one":
        cut = [0] * (E // 2 + 1) + [R] * (E - E // 2)
    else:
        top = R if kind == "ragged" else R - R // 3
        mid = sorted(torch.randint(0, top + 1, (E - 1,), generator=g, device="cuda").tolist())
        cut = [0] + mid + [top]
    return torch.tensor(cut, dtype=torch.int32, device="cuda")


def rows_of(seg, R):
    if seg is None:
        return [(0, 0, R)]
    s = seg.tolist()
    return [(e, s[e], s[e + 1]) for e in range(len(s) - 1)]


def act64(z, act):
    if act == "swiglu":
        n = z.shape[1] // 2
        return z[:, :n] * torch.special.expit(z[:, :n]) * z[:, n:]
    return {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.special.expit(v),
            "gelu": lambda v: v * torch.special.ndtr(v)}[act](z)


def act_slack(z, ez, act):
    """Error of act(z) when z errs by ez, with the activation's own fp32 arithmetic."""
    if act == "swiglu":
        n = z.shape[1] // 2
        g, u, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
        s = (g * torch.special.expit(g)).abs()
        return 1.1 * eg * (u.abs() + eu) + s * eu + 10 * EPS * s * u.abs()
    return 1.13 * ez + 10 * EPS * z.abs()


ACTS = ("none", "relu", "gelu", "silu", "swiglu")
LINEARS = [  # dtype, R, N, K, act, bias, residual, save_z, out_f32
    (BF16, 1, 8, 8, "none", False, False, False, False), (F32, 1, 8, 8, "swiglu", True, True, True, False),
    (BF16, 1, 1408, 4096, "swiglu", True, False, False, False), (BF16, 2, 72, 4104, "gelu", True, True, True, False),
    (BF16, 5, 776, 64, "relu", False, True, False, False), (BF16, 8, 4096, 1408, "none", True, True, False, False),
    (BF16, 9, 128, 2048, "none", True, False, False, True), (BF16, 16, 520, 72, "silu", True, True, True, False),
    (BF16, 17, 264, 1032, "swiglu", False, True, True, False), (BF16, 33, 256, 256, "gelu", True, False, True, False),
    (BF16, 63, 520, 512, "silu", True, True, False, False), (BF16, 64, 264, 128, "swiglu", True, True, True, False),
    (BF16, 65, 40, 136, "relu", True, True, True, False), (BF16, 127, 128, 192, "none", False, False, False, True),
    (BF16, 128, 256, 64, "swiglu", True, True, True, False), (BF16, 129, 136, 72, "gelu", True, True, True, False),
    (BF16, 255, 512, 1000, "silu", False, True, False, False),
    (BF16, 257, 776, 1032, "swiglu", True, True, True, False),
    (BF16, 513, 64, 320, "none", True, False, True, True), (BF16, 1537, 776, 1032, "gelu", True, True, True, False),
    (BF16, 3001, 1416, 520, "swiglu", True, False, True, False),
    (BF16, 4000, 128, 2048, "none", True, False, False, True),
    (BF16, 70, 8, 8, "gelu", True, True, True, False), (BF16, 33, 16, 24, "swiglu", True, True, True, False),
    (BF16, 300, 8, 2048, "relu", True, False, False, True), (F32, 70, 8, 8, "silu", True, True, True, False),
    # many rows and K an odd multiple of 8: weights copied to aligned rows
    (BF16, 4096, 136, 72, "silu", True, True, True, False), (BF16, 5000, 264, 328, "swiglu", True, True, True, False),
    # products with few tiles and a long reduction: summed in parts
    (BF16, 64, 1408, 4096, "swiglu", True, True, True, False), (BF16, 100, 264, 6000, "gelu", True, True, True, False),
    (BF16, 300, 128, 4096, "none", True, False, True, True),
    (F32, 327, 128, 1016, "relu", True, False, True, False), (F32, 53, 72, 3000, "swiglu", True, True, True, False),
    (F32, 600, 264, 2048, "gelu", True, True, False, False), (F32, 33, 8, 4096, "silu", True, True, True, False),
    (F32, 3, 40, 72, "gelu", True, True, True, False), (F32, 70, 136, 264, "swiglu", True, True, True, False),
    (F32, 257, 264, 1032, "silu", True, True, True, False), (F32, 700, 520, 136, "none", False, False, False, False),
    (F32, 1300, 72, 2056, "relu", True, True, False, False), (F32, 40, 520, 2048, "swiglu", False, True, False, False),
]


def linear_inputs(g, dt, R, NP, N, K, bias, residual, E=None):
    lead = (E,) if E else ()
    return (randn(g, R, K, dt=dt), randn(g, *lead, NP, K, dt=dt, std=K ** -0.5),
            randn(g, *lead, NP, dt=dt, std=0.3) if bias else None, randn(g, R, N, dt=dt) if residual else None)


def check_linear(x, w, b, residual, act, seg, y, z):
    R, K = x.shape
    NP = w.shape[-2]
    for e, a, c in rows_of(seg, R):
        if a == c:
            continue
        we, xe = w.view(-1, NP, K)[e].double(), x[a:c].double()
        z64, ez = xe @ we.t(), (K + 1) * EPS * (xe.abs() @ we.abs().t())
        if b is not None:
            z64 = z64 + b.view(-1, NP)[e].double()
            ez = ez + EPS * z64.abs()
        if z is not None:
            check(z[a:c], z64, ez)
        want, slack = act64(z64, act), act_slack(z64, ez, act)
        if residual is not None:
            want = want + residual[a:c].double()
            slack = slack + EPS * (want.abs() + residual[a:c].double().abs())
        check(y[a:c], want, slack)
        rms = want.pow(2).mean().sqrt()
        assert ((y[a:c].double() - want).pow(2).mean().sqrt() <= (2.0 ** -8 if y.dtype == BF16 else 1e-5) * rms + 1e-12)


@pytest.mark.parametrize("simt", [False, True], ids=["default", "simt"])
@pytest.mark.parametrize("case", LINEARS, ids=str)
def test_linear(case, simt, status):
    import pruned_expert_backward_gb300 as lrm
    dt, R, N, K, act, bias, residual, save_z, out_f32 = case
    NP = 2 * N if act == "swiglu" else N
    residual = residual and not out_f32
    x, w, b, res = linear_inputs(gen(R + N), dt, R, NP, N, K, bias, residual)
    y, z = lrm.lrm_linear(x, w, bias=b, residual=res, act=act, save_z=save_z, out_dtype=F32 if out_f32 else None,
                          flags=1 if simt else 0, dev_status=status)
    assert (z is not None) == save_z and y.dtype == (F32 if out_f32 else dt)
    check_linear(x, w, b, res, act, None, y, z)


GROUPED = [  # dtype, R, E, segments, N, K, act, bias, residual, save_z
    (BF16, 1, 4, "one", 64, 72, "swiglu", True, True, True),
    (BF16, 8, 128, "ragged", 768, 256, "swiglu", False, False, False),
    (BF16, 100, 5, "short", 136, 264, "gelu", True, True, True),
    (BF16, 512, 128, "ragged", 264, 520, "swiglu", True, False, True),
    (BF16, 512, 16, "one", 72, 136, "none", True, True, False),
    (BF16, 1000, 3, "even", 520, 72, "silu", True, True, True),
    (BF16, 2000, 7, "short", 264, 328, "swiglu", True, True, True),
    (BF16, 5000, 40, "ragged", 392, 200, "relu", True, False, False),
    (BF16, 3000, 1, "even", 136, 64, "swiglu", False, True, True),
    (BF16, 6000, 1024, "ragged", 72, 64, "none", True, False, False),
    (F32, 60, 6, "ragged", 40, 72, "swiglu", True, True, True),
    (F32, 900, 9, "short", 136, 264, "gelu", True, True, True),
    (F32, 2500, 4, "ragged", 72, 1032, "silu", False, True, False),
    (BF16, 9000, 2, "ragged", 136, 72, "gelu", True, True, True),
    (F32, 200, 5, "short", 72, 2048, "swiglu", True, True, True),
    (F32, 700, 3, "one", 136, 1480, "gelu", True, False, True),
]


@pytest.mark.parametrize("simt", [False, True], ids=["default", "simt"])
@pytest.mark.parametrize("case", GROUPED, ids=str)
def test_grouped_linear(case, simt, status):
    import pruned_expert_backward_gb300 as lrm
    dt, R, E, kind, N, K, act, bias, residual, save_z = case
    NP = 2 * N if act == "swiglu" else N
    g = gen(R + E)
    seg = segments(kind, R, E, g)
    x, w, b, res = linear_inputs(g, dt, R, NP, N, K, bias, residual, E)
    n = int(seg[-1])
    x[n:] = float("nan")  # rows of no expert are never used
    y = torch.full((R, N), 7.0, dtype=dt, device="cuda")
    z = torch.full((R, NP), 7.0, dtype=dt, device="cuda") if save_z else None
    lrm.lrm_linear(x, w, bias=b, residual=res, act=act, seg_offsets=seg, y=y, z=z, flags=1 if simt else 0,
                   dev_status=status)
    check_linear(x, w, b, res, act, seg, y, z)
    assert bool((y[n:] == 7.0).all()) and (z is None or bool((z[n:] == 7.0).all()))


def test_linear_infinities_and_nan_stay_in_their_rows(status):
    """A row with an infinity or a NaN spoils its own outputs only, in every kernel."""
    import pruned_expert_backward_gb300 as lrm
    for R in (3, 300):
        for dt in (BF16, F32):
            x, w, b, res = linear_inputs(gen(R), dt, R, 72, 72, 136, True, True)
            x[0, 3], x[R - 1, 7] = float("inf"), float("nan")
            y, _ = lrm.lrm_linear(x, w, bias=b, residual=res, act="none", dev_status=status)
            assert not bool(torch.isfinite(y[0]).any()) and bool(torch.isnan(y[R - 1]).all())
            check_linear(x[1:R - 1].contiguous(), w, b, res[1:R - 1].contiguous(), "none", None, y[1:R - 1], None)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R", [3, 200])
def test_linear_of_the_lowest_values_and_nan(R, dt, status):
    """The type's lowest value times one weight is itself; ReLU keeps a NaN; -0 and the lowest give 0."""
    import pruned_expert_backward_gb300 as lrm
    low = torch.finfo(dt).min
    x = torch.zeros(R, 16, dtype=dt, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = low, float("nan"), -low
    w = torch.eye(16, dtype=dt, device="cuda")
    y, _ = lrm.lrm_linear(x, w, dev_status=status)
    # (fp32 values are held to 24 bits as three bf16 parts)
    assert abs(y[0, 0].item() / low - 1) <= 2.0 ** -23 and abs(y[2, 0].item() / low + 1) <= 2.0 ** -23
    assert bool((y[0, 1:] == 0).all()) and bool((y[2, 1:] == 0).all())
    r, _ = lrm.lrm_linear(x, w, act="relu", dev_status=status)
    assert r[0, 0].item() == 0 and bool(torch.isnan(r[1, 0])) and r[2, 0].item() == y[2, 0].item()
    assert torch.count_nonzero(r[3:]) == 0


@pytest.mark.parametrize("act", ACTS)
def test_linear_large_pre_activations(act, status):
    """Saturated activations: |z| up to 500 gives 0, z or the product, never NaN."""
    import pruned_expert_backward_gb300 as lrm
    for R in (4, 200):
        NP = 32 if act == "swiglu" else 16
        x = torch.zeros(R, 16, device="cuda")
        x[:, 0] = torch.linspace(-500, 500, R, device="cuda")
        w = torch.zeros(NP, 16, device="cuda")
        w[:, 0] = 1
        for dt in (BF16, F32):
            y, _ = lrm.lrm_linear(x.to(dt), w.to(dt), act=act, dev_status=status)
            assert bool(torch.isfinite(y).all())
            check_linear(x.to(dt), w.to(dt), None, None, act, None, y, None)


# -------------------------------------------------------------------------------- gradients -----
ACT_GRADS = [  # dtype, R, N, E, segments
    (BF16, 1, 8, None, None), (F32, 1, 8, None, None), (BF16, 127, 72, None, None), (BF16, 128, 264, None, None),
    (BF16, 129, 768, None, None), (F32, 1000, 136, None, None), (BF16, 5000, 520, None, None),
    (BF16, 1000, 264, 7, "ragged"), (BF16, 700, 768, 128, "ragged"), (F32, 300, 40, 16, "one"),
    (BF16, 2000, 136, 5, "short"), (BF16, 4096, 72, 32, "even"), (F32, 900, 24, 300, "ragged"),
    (BF16, 20000, 72, 64, "ragged"), (F32, 17001, 24, 100, "one"), (F32, 2049, 16, 2, "short"),
]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("case", ACT_GRADS, ids=str)
def test_act_backward(case, act, status):
    import pruned_expert_backward_gb300 as lrm
    dt, R, N, E, kind = case
    NP = 2 * N if act == "swiglu" else N
    g = gen(R + N)
    seg = segments(kind, R, E, g) if E else None
    dy, z = randn(g, R, N, dt=dt), randn(g, R, NP, dt=dt, std=2.0)
    z.view(-1)[:: 37] = 0  # ReLU's corner
    n = R if seg is None else int(seg[-1])
    dy[n:] = float("nan")
    dz = torch.full((R, NP), 7.0, dtype=dt, device="cuda")
    _, db = lrm.lrm_act_backward(dy, None if act == "none" else z, act=act, seg_offsets=seg, dz=dz, dev_status=status)
    z64, d64 = z[:n].double().requires_grad_(), dy[:n].double()
    if act == "relu":
        want = d64 * (z64 > 0)
    else:
        want = torch.autograd.grad(act64(z64, act), z64, d64)[0]
    zz = z64.detach()
    mag = d64.abs() * (1 + zz.abs()) if act != "swiglu" else torch.cat(
        [d64.abs() * (1 + zz[:, :N].abs()) * zz[:, N:].abs(), d64.abs() * zz[:, :N].abs()], 1)
    slack = 16 * EPS * mag
    check(dz[:n], want, slack)
    assert bool((dz[n:] == 7.0).all())
    for e, a, b in rows_of(seg, R):
        got = db if seg is None else db[e]
        check(got, want[a:b].sum(0), (slack[a:b] + (b - a + 1) * EPS * want[a:b].abs()).sum(0))
    again, none = lrm.lrm_act_backward(dy, z, act=act, seg_offsets=seg, bias_grad=False, dz=torch.full_like(dz, 7.0),
                                       dev_status=status)
    assert none is None and torch.equal(again, dz)
    _, db2 = lrm.lrm_act_backward(dy, z, act=act, seg_offsets=seg, dev_status=status)
    assert torch.equal(db2, db)  # the sums' order does not depend on scheduling


LINEAR_GRADS = [  # dtype, R, N, K, E, segments
    (BF16, 1, 8, 8, None, None), (F32, 1, 8, 16, None, None), (BF16, 63, 72, 136, None, None),
    (BF16, 65, 264, 64, None, None), (BF16, 300, 128, 520, None, None), (BF16, 1537, 776, 264, None, None),
    (BF16, 5000, 256, 256, None, None), (BF16, 40, 8, 8, None, None), (F32, 3100, 40, 24, None, None),
    (BF16, 4133, 520, 136, None, None), (BF16, 20000, 40, 72, None, None), (F32, 70, 72, 40, None, None),
    (F32, 1500, 136, 264, None, None), (BF16, 8, 72, 64, 12, "ragged"), (BF16, 700, 264, 136, 5, "short"),
    (BF16, 3000, 520, 72, 64, "ragged"), (BF16, 6000, 136, 392, 3, "one"), (BF16, 9000, 72, 328, 2, "ragged"),
    (F32, 900, 72, 136, 9, "short"), (F32, 4000, 40, 264, 4, "ragged"),
    # a popular expert's rows in several runs
    (F32, 9000, 72, 136, 4, "ragged"), (F32, 12000, 136, 264, 10, "short"), (BF16, 40000, 136, 264, 3, "ragged"),
    (F32, 8000, 40, 72, 6, "one"), (BF16, 30000, 72, 40, 2, "short"),
    # dx with few tiles and a long reduction: summed in parts
    (F32, 48, 1232, 288, None, None), (BF16, 300, 4104, 72, None, None), (BF16, 200, 4104, 136, 4, "short"),
    (F32, 130, 2000, 40, 3, "ragged"), (BF16, 33, 8192, 264, None, None),
]


@pytest.mark.parametrize("simt", [False, True], ids=["default", "simt"])
@pytest.mark.parametrize("case", LINEAR_GRADS, ids=str)
def test_linear_backward(case, simt, status):
    import pruned_expert_backward_gb300 as lrm
    dt, R, N, K, E, kind = case
    g = gen(R + N + K)
    seg = segments(kind, R, E, g) if E else None
    x, w, _, _ = linear_inputs(g, dt, R, N, N, K, False, False, E)
    dz = randn(g, R, N, dt=dt)
    n = R if seg is None else int(seg[-1])
    x[n:], dz[n:] = float("nan"), float("nan")
    dx = torch.full((R, K), 7.0, dtype=dt, device="cuda")
    flags = 1 if simt else 0
    _, dw = lrm.lrm_linear_backward(dz, x, w, seg_offsets=seg, dx=dx, flags=flags, dev_status=status)
    assert bool((dx[n:] == 7.0).all())
    for e, a, b in rows_of(seg, R):
        we, xe, de = w.view(-1, N, K)[e].double(), x[a:b].double(), dz[a:b].double()
        check(dx[a:b], de @ we, (N + 1) * EPS * (de.abs() @ we.abs()))
        got, want = dw.view(-1, N, K)[e], de.t() @ xe
        if a == b:
            assert torch.count_nonzero(got) == 0
            continue
        check(got, want, (b - a + 1) * EPS * (de.abs().t() @ xe.abs()))
        # fp32 sums: as near as fp32 arithmetic is, whatever the number of rows
        assert (got.double() - want).norm() <= 5e-6 * want.norm()
    one, none = lrm.lrm_linear_backward(dz, x, w, seg_offsets=seg, need_dw=False, flags=flags, dev_status=status,
                                        dx=torch.full_like(dx, 7.0))
    assert none is None and torch.equal(one, dx)
    none, two = lrm.lrm_linear_backward(dz, x, w, seg_offsets=seg, need_dx=False, flags=flags, dev_status=status)
    assert none is None and torch.equal(two, dw)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("grouped", [False, True], ids=["dense", "experts"])
def test_linear_gradient_against_differences(act, grouped, status):
    """<dy, y> along each gradient's own direction changes at the rate of the gradient's norm.

    Central differences of the fp32 forward: truncation h^2/6 of the third derivative (h = 1e-2 of the
    argument's scale: below 1e-3 relative) and the forward's rounding, 1e-6 |y| per value over a change
    of h: below 1e-3 relative for these sizes; 1e-2 allowed.  Where a step d carries a value z past ReLU's
    corner, the difference of that value is off by up to (|d| - |z|) / 2: summed below and allowed too."""
    import pruned_expert_backward_gb300 as lrm
    R, N, K, E = 48, 40, 64, 4
    NP = 2 * N if act == "swiglu" else N
    g = gen(11)
    seg = torch.tensor([0, 10, 10, 31, R], dtype=torch.int32, device="cuda") if grouped else None
    x, w, b, res = linear_inputs(g, F32, R, NP, N, K, True, True, E if grouped else None)
    dy = randn(g, R, N, dt=F32)
    y, z = lrm.lrm_linear(x, w, bias=b, residual=res, act=act, seg_offsets=seg, save_z=True, dev_status=status)
    dz, db = lrm.lrm_act_backward(dy, z, act=act, seg_offsets=seg, dev_status=status)
    dx, dw = lrm.lrm_linear_backward(dz, x, w, seg_offsets=seg, dev_status=status)

    def loss(x_, w_, b_):
        y_, _ = lrm.lrm_linear(x_, w_, bias=b_, residual=res, act=act, seg_offsets=seg, dev_status=status)
        return (y_.double() * dy.double()).sum().item()

    for i, grad in enumerate((dx, dw, db)):
        args = [x, w, b]
        step = 1e-2 * args[i].norm() * grad / grad.norm()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step, args[i] - step
        size = step.double().norm().item()
        diff = (loss(*up) - loss(*down)) / (2 * size)
        corner = 0.0
        if act == "relu":
            z_up, _ = lrm.lrm_linear(up[0], up[1], bias=up[2], seg_offsets=seg, dev_status=status)
            past = ((z_up - z).abs() - z.abs()).clamp(min=0).double() / 2
            corner = (past * dy.double().abs()).sum().item() / size
        assert abs(diff - grad.double().norm().item()) <= 1e-2 * grad.norm().item() + corner, (act, i)


# ------------------------------------------------------------------------- the layer, refusals --
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_layer_forward_and_backward(dt):
    """The whole layer: forward against a dense 64-bit form, gradients against its differentiation."""
    import pruned_expert_backward_gb300 as lrm
    T, k, E, H, I = 300, 4, 12, 136, 72
    g = gen(3)
    idx, alpha = routing(g, T, k, E, 1.0, 0.1)
    x, residual, dy = randn(g, T, H, dt=dt), randn(g, T, H, dt=dt), randn(g, T, H, dt=dt)
    wg, wd = randn(g, E, 2 * I, H, dt=dt, std=H ** -0.5), randn(g, E, H, I, dt=dt, std=I ** -0.5)
    layer = lrm.MoeLayer(T, k, E, H, I, dtype=dt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a stream other than the tensors' own
        y = layer.forward(x, idx, alpha, wg, wd, residual=residual)
        dx, dalpha, dwg, dwd = layer.backward(dy, alpha, wg, wd)
    torch.cuda.synchronize()
    assert int(layer.dev_status.item()) == 0
    x64, a64, g64, d64 = (t.double().requires_grad_() for t in (x, alpha, wg, wd))
    out = residual.double()
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        out = out.index_add(0, t, a64[t, j, None] * (act64(x64[t] @ g64[e].t(), "swiglu") @ d64[e].t()))
    want = torch.autograd.grad(out, (x64, a64, g64, d64), dy.double())
    # bf16: a handful of intermediates rounded to 2^-9 each; fp32 as the framework's other fp32 results
    tol = 1e-2 if dt == BF16 else 1e-5
    for got, ref in zip((y, dx, dalpha, dwg, dwd), (out, *want)):
        assert (got.double() - ref).norm() <= tol * ref.norm()
    served = lrm.MoeLayer(T, k, E, H, I, dtype=dt, train=False)
    assert torch.equal(served.forward(x, idx, alpha, wg, wd, residual=residual), y)
    with pytest.raises(ValueError):
        served.backward(dy, alpha, wg, wd)


def test_bad_segments_compute_nothing():
    import pruned_expert_backward_gb300 as lrm
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for R, dt, simt in ((8, BF16, 0), (400, BF16, 0), (400, F32, 0), (8, F32, 0), (64, BF16, 1)):
        x, w, _, _ = linear_inputs(gen(R), dt, R, 72, 72, 64, False, False, 3)
        for seg in ([1, 2, 3, R], [0, 5, 4, R], [0, 2, 4, R + 1]):
            s = torch.tensor(seg, dtype=torch.int32, device="cuda")
            y, dx = torch.full((R, 72), 7.0, dtype=dt, device="cuda"), torch.full((R, 64), 7.0, dtype=dt, device="cuda")
            dw = torch.full((3, 72, 64), 7.0, device="cuda")
            for call in (lambda: lrm.lrm_linear(x, w, seg_offsets=s, y=y, flags=simt, dev_status=st),
                         lambda: lrm.lrm_linear_backward(y, x, w, seg_offsets=s, dx=dx, dw=dw, flags=simt,
                                                         dev_status=st),
                         lambda: lrm.lrm_act_backward(y, y, act="silu", seg_offsets=s, dz=y, dev_status=st)):
                st.zero_()
                call()
                assert int(st.item()) == 11
            assert bool((y == 7.0).all()) and bool((dx == 7.0).all()) and bool((dw == 7.0).all())
    # long reductions, summed in parts: the second launch must not write either
    big = torch.full((9000, 72), 7.0, device="cuda")
    wide = torch.full((3, 72, 72), 7.0, device="cuda")
    st.zero_()
    s = torch.tensor([0, 9000, 4, 9000], dtype=torch.int32, device="cuda")
    lrm.lrm_linear_backward(big, big, wide, seg_offsets=s, need_dx=False, dw=wide, dev_status=st)  # (w is not read)
    assert int(st.item()) == 11 and bool((wide == 7.0).all())
    for dt, N, K in ((F32, 72, 2048), (F32, 2048, 72), (BF16, 4096, 72)):
        x, w, _, _ = linear_inputs(gen(N), dt, 200, N, N, K, False, False, 3)
        y, dx = torch.full((200, N), 7.0, dtype=dt, device="cuda"), torch.full((200, K), 7.0, dtype=dt, device="cuda")
        s = torch.tensor([0, 90, 80, 200], dtype=torch.int32, device="cuda")
        for call in (lambda: lrm.lrm_linear(x, w, seg_offsets=s, y=y, dev_status=st),
                     lambda: lrm.lrm_linear_backward(y, x, w, seg_offsets=s, dx=dx, need_dw=False, dev_status=st)):
            st.zero_()
            call()
            assert int(st.item()) == 11
        assert bool((y == 7.0).all()) and bool((dx == 7.0).all())


def test_refusals():
    import pruned_expert_backward_gb300 as lrm
    x, w = torch.zeros(4, 16, device="cuda", dtype=BF16), torch.zeros(24, 16, device="cuda", dtype=BF16)
    seg = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(w=w.float()), dict(w=w[:, :8].contiguous()), dict(act="tanh"), dict(bias=x), dict(residual=x),
                dict(seg_offsets=seg), dict(x=x.cpu()), dict(x=x.half(), w=w.half()), dict(y=x),
                dict(w=torch.zeros(24, 32, device="cuda", dtype=BF16)[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            lrm.lrm_linear(**{"x": x, "w": w, **bad})
    with pytest.raises(lrm.LrmError):  # 20 columns: not a multiple of 8
        lrm.lrm_linear(x, torch.zeros(20, 16, device="cuda", dtype=BF16))
    with pytest.raises(lrm.LrmError):  # a residual needs the type of x
        lrm.lrm_linear(x, w, residual=torch.zeros(4, 24, device="cuda"), out_dtype=F32)
    with pytest.raises(lrm.LrmError):  # misaligned start
        lrm.lrm_linear(torch.zeros(4 * 16 + 1, device="cuda", dtype=BF16)[1:].view(4, 16), w)
    with pytest.raises(lrm.LrmError):
        lrm.lrm_linear(x.float(), w.float(), ws=torch.zeros(0, dtype=torch.uint8, device="cuda"))
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        lrm.lrm_sort_tokens(idx, x[:3], 4)
    with pytest.raises(TypeError):
        lrm.lrm_sort_tokens(idx.long(), x, 4)
    with pytest.raises(lrm.LrmError):  # too many experts
        lrm.lrm_sort_tokens(idx, x, 2000)
    alpha = torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError):
        lrm.lrm_combine(idx.view(-1)[:6].contiguous(), alpha, torch.zeros(8, 16, device="cuda"))
    with pytest.raises(TypeError):
        lrm.lrm_combine(idx.view(-1), alpha.bfloat16(), torch.zeros(8, 16, device="cuda"))
    with pytest.raises(ValueError):
        lrm.lrm_combine_backward(idx.view(-1), alpha, x, None)
    with pytest.raises(ValueError):
        lrm.lrm_act_backward(x, None, act="gelu")
    with pytest.raises(ValueError):
        lrm.lrm_linear_backward(x, x, w)


def test_the_example_runs_and_pruning_nothing_changes_nothing():
    """examples/moe_layer.py: with every pair kept the pruned backward gives the full gradients (bf16 rounding
    of a few intermediates apart); a token alone gives its row of the batch."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.run(tokens=600, hidden=256, inter=128, experts=16, topk=4, keep=(1, 1))
    assert r["kept"] == 1.0
    assert max(r["dx"], r["dw_gate_up"], r["dw_down"]) <= 1e-2
    assert r["token_vs_batch"] <= 2.0 ** -7
    r = example.run(tokens=600, hidden=256, inter=128, experts=16, topk=4, keep=(8, 10))
    assert 0.8 <= r["kept"] <= 0.83 and 0 < r["dw_down"] < 0.5
