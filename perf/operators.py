"""Cases of the MoE layer's forward operators and their gradients, for timing and comparison.

Six calls: the sort of tokens by expert (lrm_sort_tokens), the weighted way back (lrm_combine) and its
gradient (lrm_combine_backward), the product with bias, activation and residual (lrm_linear, dense or
one weight per expert over sorted rows), and its gradient in two steps (lrm_act_backward,
lrm_linear_backward).  With `own` false every call is computed by elementary torch operations in
32 bits; with `own` true by the package's entry points.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "swiglu")


# ------------------------------------------------------------------------------------- cases ----
def _routing(name, op, dtype, T, k, E, H, skew=1.0, masked=0.0, residual=False):
    return {"name": name, "op": op, "dtype": dtype, "T": T, "k": k, "E": E, "H": H, "skew": skew, "masked": masked,
            "residual": residual}


def _dense(name, op, dtype, R, N, K, act="none", bias=False, residual=False, save_z=False, out_f32=False):
    return {"name": name, "op": op, "dtype": dtype, "R": R, "N": N, "K": K, "act": act, "bias": bias,
            "residual": residual, "save_z": save_z, "out_f32": out_f32, "E": 0, "k": 1, "skew": 0.0}


def _experts(name, op, T, k, E, N, K, act="none", bias=False, residual=False, save_z=False, skew=1.0, dtype="bf16"):
    return {"name": name, "op": op, "dtype": dtype, "R": T * k, "N": N, "K": K, "act": act, "bias": bias,
            "residual": residual, "save_z": save_z, "out_f32": False, "E": E, "k": k, "skew": skew}


def listed():
    return [
        # one token being generated, Qwen3-shaped layer: the smallest sort
        _routing("sort_one_token", "sort", "bf16", 1, 8, 128, 2048),
        # sequence 8192 x microbatch 4 through the GLM4.5-shaped layer: the largest sort
        _routing("sort_train_glm45", "sort", "bf16", 32768, 8, 128, 4096),
        # 64 sequences generating, back to tokens with the block's residual
        _routing("combine_decode64", "combine", "bf16", 64, 8, 128, 2048, residual=True),
        # odd fp32 sizes with padding tokens: some pairs, and some whole tokens, are not routed
        _routing("combine_odd_f32", "combine", "f32", 5003, 6, 60, 1032, masked=0.2),
        # sequence 8192 x microbatch 4 through the Qwen3-shaped layer: gradient of the way back
        _routing("combine_bwd_train_qwen3", "combine_bwd", "bf16", 32768, 8, 128, 2048),
        # an expert that every token takes (a dense SwiGLU of the GLM4.5 expert's size), four sequences generating
        _dense("linear_decode4", "linear", "bf16", 4, 1408, 4096, act="swiglu", bias=True),
        # the projection beside the layer at training size: bias, GELU and the residual in one pass
        _dense("linear_train", "linear", "bf16", 32768, 4096, 4096, act="gelu", bias=True, residual=True),
        # odd fp32 sizes: nothing a multiple of a tile
        _dense("linear_odd_f32", "linear", "f32", 1537, 776, 1032, act="silu", bias=True, residual=True),
        # the experts' first product for 64 sequences generating, Qwen3-shaped layer: few rows an expert
        _experts("experts_decode64", "linear", 64, 8, 128, 768, 2048, act="swiglu"),
        # the same for one 8192-token sequence in training: the pre-activation is kept for the backward
        _experts("experts_train_qwen3", "linear", 8192, 8, 128, 768, 2048, act="swiglu", save_z=True),
        # its activation's gradient with the bias gradient of every expert
        _experts("act_bwd_train_qwen3", "act_bwd", 8192, 8, 128, 768, 2048, act="swiglu", bias=True),
        # its product's gradients, both
        _experts("linear_bwd_train_qwen3", "linear_bwd", 8192, 8, 128, 1536, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo=64, hi=4096):
    n = _log(rng, lo, hi) // 8 * 8  # hidden sizes are multiples of 8
    return n - 8 if n in (1536, 3072) else n


def draw(rng):
    op = rng.choice(["sort", "combine", "combine_bwd", "linear", "linear", "act_bwd", "linear_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("sort", "combine", "combine_bwd"):
        E = _log(rng, 2, 256)
        k = rng.randint(1, min(16, E))
        T = _log(rng, 1, 32768)
        H = _width(rng)
        while T * k * H > 32768 * 8 * 2048:
            T = max(1, T // 2)
        c = _routing("", op, dtype, T, k, E, H, skew=rng.choice([0.0, 1.0, 1.5]), masked=rng.choice([0.0, 0.0, 0.3]),
                     residual=op == "combine" and rng.random() < 0.5)
    else:
        act = rng.choice(ACTS) if op != "linear_bwd" else "none"
        N, K = _width(rng), _width(rng)
        bias = rng.random() < 0.6 or (op == "act_bwd" and act == "none")  # that one is the bias gradient alone
        residual, save_z = op == "linear" and rng.random() < 0.5, rng.random() < 0.4
        if rng.random() < 0.5:
            R = _log(rng, 1, 32768)
            while R * N * K > 2 ** 36:
                R = max(1, R // 2)
            c = _dense("", op, dtype, R, N, K, act, bias, residual, op == "linear" and save_z,
                       out_f32=op == "linear" and not residual and rng.random() < 0.2)
        else:
            E = _log(rng, 2, 128)
            k = rng.randint(1, min(8, E))
            T = _log(rng, 1, 8192)
            while E * T * max(2 * N, K) > 2 ** 31 or E * T * N * K > 2 ** 40:
                T = max(1, T // 2)
            c = _experts("", op, T, k, E, N, K, act, bias, residual, op == "linear" and save_z,
                         skew=rng.choice([0.0, 1.0]), dtype=dtype)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs ----
def _route(gen, T, k, E, skew):
    """Top-k experts of each token and their softmax weights, popularity falling as rank ** -skew."""
    logits = torch.randn(T, E, generator=gen, device="cuda")
    logits -= skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    top, idx = torch.topk(logits, k, dim=1)
    return idx.to(torch.int32).contiguous(), torch.softmax(top, 1).contiguous()


def _rows(idx, E):
    """Rows of the pairs sorted by expert (stable), and the segments; a pair of expert -1 has row -1."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    seg = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    seg[1:] = torch.cumsum((key[:, None] == torch.arange(E, device=idx.device)).sum(0), 0)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=idx.device)
    row = torch.where(flat < 0, torch.full_like(row, -1), row)
    return order, row, seg


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op, s = case["op"], {"case": case, "dtype": dt}
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("sort", "combine", "combine_bwd"):
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        idx, s["alpha"] = _route(gen, T, k, E, case["skew"])
        if case["masked"] > 0:
            drop = torch.rand(T, k, generator=gen, device="cuda") < case["masked"]
            drop |= torch.rand(T, 1, generator=gen, device="cuda") < case["masked"] / 2
            idx = torch.where(drop, torch.full_like(idx, -1), idx)
        s["idx"] = idx
        if op == "sort":
            s["x"] = randn(T, H)
        else:
            s["row"] = _rows(idx, E)[1].to(torch.int32)
            s["y_s"] = randn(T * k, H)
            s["residual"] = randn(T, H) if case["residual"] else None
            if op == "combine_bwd":
                s["dy"] = randn(T, H, std=1e-3)
                s["dy_s"] = torch.zeros(T * k, H, dtype=dt, device="cuda")  # rows of no pair stay zero
        return s
    R, N, K, E, act = case["R"], case["N"], case["K"], case["E"], case["act"]
    NP = 2 * N if act == "swiglu" else N  # columns of the product
    s["seg"], s["max_rows"] = None, R
    if E:
        idx, _ = _route(gen, R // case["k"], case["k"], E, case["skew"])
        seg = _rows(idx, E)[2]
        s["seg"], s["max_rows"] = seg.to(torch.int32), int((seg[1:] - seg[:-1]).max())
    lead = (E,) if E else ()
    if op in ("linear", "linear_bwd"):
        s["w"] = randn(*lead, NP, K, std=K ** -0.5)
        s["x"] = randn(R, K)
    if op == "linear":
        s["b"] = randn(*lead, NP, std=0.1) if case["bias"] else None
        s["residual"] = randn(R, N) if case["residual"] else None
    elif op == "act_bwd":
        s["z"], s["dy"] = randn(R, NP), randn(R, N, std=1e-3)
    else:
        s["dz"] = randn(R, NP, std=1e-3)
    return s


# -------------------------------------------------------------------- plain form, in 32 bits ----
def _act(z, act):
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return g / (1 + torch.exp(-g)) * u
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    return torch.maximum(z, torch.zeros_like(z)) if act == "relu" else z


def _act_grad(dy, z, act):
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        sg = 1 / (1 + torch.exp(-g))
        return torch.cat([dy * u * sg * (1 + g * (1 - sg)), dy * g * sg], -1)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return dy * sg * (1 + z * (1 - sg))
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * 0.7071067811865476)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327)
    return dy * (z > 0) if act == "relu" else dy


def _expert_of_row(s, R):
    seg = s["seg"].long()
    r = torch.arange(R, device=seg.device)
    e = torch.searchsorted(seg[1:].contiguous(), r, right=True)
    return e, r - seg[e]


def _padded(s, a):
    """Rows sorted by expert laid out as [experts, most rows of one, columns], zeros between."""
    e, at = _expert_of_row(s, a.shape[0])
    p = torch.zeros(s["case"]["E"], s["max_rows"], a.shape[1], device=a.device)
    p[e, at] = a.float()
    return p, e, at


def _plain(s):
    c, op, dt = s["case"], s["case"]["op"], s["dtype"]
    if op == "sort":
        T, k, E = c["T"], c["k"], c["E"]
        order, row, seg = _rows(s["idx"], E)
        routed = torch.arange(T * k, device="cuda") < seg[E]
        pair = torch.where(routed, order, torch.full_like(order, -1))
        x_s = torch.where(routed[:, None], s["x"][order // k], torch.zeros((), dtype=dt, device="cuda"))
        return {"seg": seg.to(torch.int32), "pair": pair.to(torch.int32), "row": row.to(torch.int32), "x_s": x_s}
    if op in ("combine", "combine_bwd"):
        T, k, H = c["T"], c["k"], c["H"]
        row = s["row"].long()
        live = (row >= 0).float()[:, None]
        rows = s["y_s"][row.clamp(min=0)].float() * live
    if op == "combine":
        y = (rows * s["alpha"].reshape(-1, 1)).view(T, k, H).sum(1)
        return {"y": (y + s["residual"].float() if s["residual"] is not None else y).to(dt)}
    if op == "combine_bwd":
        dy = s["dy"].float()
        dalpha = (rows.view(T, k, H) * dy[:, None]).sum(2)
        scaled = (dy[:, None] * s["alpha"][:, :, None]).view(T * k, H).to(dt)
        dy_s = torch.zeros_like(s["dy_s"])
        at = torch.where(row < 0, torch.full_like(row, T * k), row)
        dy_s = torch.cat([dy_s, dy_s[:1]]).index_copy_(0, at, scaled)[:-1]
        return {"dy_s": dy_s, "dalpha": dalpha}
    act, grouped = c["act"], bool(c["E"])
    if op == "linear":
        if grouped:
            p, e, at = _padded(s, s["x"])
            z = torch.bmm(p, s["w"].float().transpose(1, 2))[e, at]
            z = z + s["b"].float()[e] if s["b"] is not None else z
        else:
            z = s["x"].float() @ s["w"].float().t()
            z = z + s["b"].float() if s["b"] is not None else z
        y = _act(z, act)
        y = y + s["residual"].float() if s["residual"] is not None else y
        return {"y": y.to(torch.float32 if c["out_f32"] else dt), **({"z": z.to(dt)} if c["save_z"] else {})}
    if op == "act_bwd":
        dz = _act_grad(s["dy"].float(), s["z"].float(), act)
        if not c["bias"]:
            return {"dz": dz.to(dt)}
        if not grouped:
            return {"dz": dz.to(dt), "db": dz.sum(0)}
        e, _ = _expert_of_row(s, c["R"])
        mine = (torch.arange(c["E"], device="cuda")[:, None] == e).float()
        return {"dz": dz.to(dt), "db": mine @ dz}
    if grouped:
        p, e, at = _padded(s, s["dz"])
        dx = torch.bmm(p, s["w"].float())[e, at]
        return {"dx": dx.to(dt), "dw": torch.bmm(p.transpose(1, 2), _padded(s, s["x"])[0])}
    return {"dx": (s["dz"].float() @ s["w"].float()).to(dt), "dw": s["dz"].float().t() @ s["x"].float()}


# ------------------------------------------------------------------------- the package's own ----
def _own(s):
    import pruned_expert_backward_gb300 as lrm
    c, op, st = s["case"], s["case"]["op"], s["status"]
    if op == "sort":
        seg, pair, row, x_s = lrm.lrm_sort_tokens(s["idx"], s["x"], c["E"], dev_status=st)
        return {"seg": seg, "pair": pair, "row": row, "x_s": x_s}
    if op == "combine":
        return {"y": lrm.lrm_combine(s["row"], s["alpha"], s["y_s"], residual=s["residual"], dev_status=st)}
    if op == "combine_bwd":
        dy_s, dalpha = lrm.lrm_combine_backward(s["row"], s["alpha"], s["dy"], s["y_s"], dy_s=s["dy_s"], dev_status=st)
        return {"dy_s": dy_s, "dalpha": dalpha}
    if op == "linear":
        y, z = lrm.lrm_linear(s["x"], s["w"], bias=s["b"], residual=s["residual"], act=c["act"], seg_offsets=s["seg"],
                              save_z=c["save_z"], out_dtype=torch.float32 if c["out_f32"] else None, dev_status=st)
        return {"y": y, "z": z} if c["save_z"] else {"y": y}
    if op == "act_bwd":
        dz, db = lrm.lrm_act_backward(s["dy"], s["z"], act=c["act"], seg_offsets=s["seg"], bias_grad=c["bias"],
                                      dev_status=st)
        return {"dz": dz, "db": db} if c["bias"] else {"dz": dz}
    dx, dw = lrm.lrm_linear_backward(s["dz"], s["x"], s["w"], seg_offsets=s["seg"], dev_status=st)
    return {"dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------------- work ----
def _active(c):
    """Experts that have a row, on average over routings with this popularity."""
    w = [(i + 1.0) ** -c["skew"] for i in range(c["E"])]
    top, tokens = c["k"] / sum(w), c["R"] // c["k"]
    return sum(1 - (1 - min(1.0, top * p)) ** tokens for p in w)


def work(case):
    c, op = case, case["op"]
    b = 4 if c["dtype"] == "f32" else 2
    if op in ("sort", "combine", "combine_bwd"):
        T, k, H = c["T"], c["k"], c["H"]
        P = T * k
        L = P * (1 - c["masked"] - c["masked"] / 2 + c["masked"] ** 2 / 2)  # pairs that are routed
        if op == "sort":
            return {"bytes": P * 4 + T * H * b + P * H * b + (2 * P + c["E"] + 1) * 4, "flops": 0}
        if op == "combine":
            return {"bytes": P * 8 + L * H * b + T * H * b * (2 if c["residual"] else 1), "flops": 2 * L * H}
        return {"bytes": P * 12 + T * H * b + 2 * L * H * b, "flops": 3 * L * H}
    R, N, K = c["R"], c["N"], c["K"]
    NP = 2 * N if c["act"] == "swiglu" else N
    weights = (_active(c) if c["E"] else 1) * NP * K
    if op == "linear":
        bytes_ = R * K * b + weights * b + R * N * (4 if c["out_f32"] else b)
        bytes_ += (R * N * b if c["residual"] else 0) + (R * NP * b if c["save_z"] else 0)
        return {"bytes": bytes_, "flops": 2 * R * NP * K}
    if op == "act_bwd":
        reads_z = 0 if c["act"] == "none" else R * NP * b
        return {"bytes": R * N * b + reads_z + R * NP * b, "flops": 8 * R * N}
    every = (c["E"] or 1) * NP * K  # the gradient of an expert without rows is written too
    return {"bytes": R * NP * b + 2 * R * K * b + weights * b + every * 4, "flops": 4 * R * NP * K}


# ----------------------------------------------------------------------------- in 64 bits -------
def _segments(s):
    if s["seg"] is None:
        return [(0, 0, s["case"]["R"])]
    seg = s["seg"].tolist()
    return [(e, seg[e], seg[e + 1]) for e in range(len(seg) - 1)]


def _f64_act(z, act):
    if act == "swiglu":
        n = z.shape[1] // 2
        return z[:, :n] * torch.special.expit(z[:, :n]) * z[:, n:]
    return {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.special.expit(v),
            "gelu": lambda v: v * torch.special.ndtr(v)}[act](z)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("sort", "combine", "combine_bwd"):
        T, k, E, H = c["T"], c["k"], c["E"], c["H"]
        idx = s["idx"].reshape(-1)
        if op == "sort":
            x_s = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
            at = 0
            for e in range(E):
                pairs = torch.nonzero(idx == e).flatten()
                x_s[at:at + pairs.numel()] = s["x"].double()[pairs // k]
                at += pairs.numel()
            return {"seg": None, "pair": None, "row": None, "x_s": x_s}
        row = s["row"].view(T, k).long()
        if op == "combine":
            y = s["residual"].double() if s["residual"] is not None else torch.zeros(T, H, dtype=torch.float64, device="cuda")
            for j in range(k):
                t = torch.nonzero(row[:, j] >= 0).flatten()
                y[t] += s["alpha"][t, j, None].double() * s["y_s"][row[t, j]].double()
            return {"y": y}
        dy = s["dy"].double()
        dy_s = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        dalpha = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(row[:, j] >= 0).flatten()
            dy_s[row[t, j]] = s["alpha"][t, j, None].double() * dy[t]
            dalpha[t, j] = torch.einsum("th,th->t", dy[t], s["y_s"][row[t, j]].double())
        return {"dy_s": dy_s, "dalpha": dalpha}
    R, N, K, E, act = c["R"], c["N"], c["K"], c["E"], c["act"]
    NP = 2 * N if act == "swiglu" else N

    def new(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")

    if op == "linear":
        w = s["w"].view(-1, NP, K)
        y, z = new(R, N), new(R, NP) if c["save_z"] else None
        for e, a, b in _segments(s):
            ze = torch.einsum("rk,nk->rn", s["x"][a:b].double(), w[e].double())
            if s["b"] is not None:
                ze += s["b"].view(-1, NP)[e].double()
            if z is not None:
                z[a:b] = ze
            y[a:b] = _f64_act(ze, act)
        if s["residual"] is not None:
            y += s["residual"].double()
        return {"y": y, "z": z} if c["save_z"] else {"y": y}
    if op == "act_bwd":
        # the derivative of the activation itself, by reverse differentiation of its 64-bit form
        dz, db = new(R, NP), new(*((E,) if E else ()), NP)
        for e, a, b in _segments(s):
            z = s["z"][a:b].double().requires_grad_()
            with torch.enable_grad():
                out = _f64_act(z, act)
            dz[a:b] = torch.autograd.grad(out, z, s["dy"][a:b].double())[0]
            db.view(-1, NP)[e] = dz[a:b].sum(0)
        return {"dz": dz, "db": db} if c["bias"] else {"dz": dz}
    w = s["w"].view(-1, NP, K)
    dx, dw = new(R, K), new(*((E,) if E else ()), NP, K)
    for e, a, b in _segments(s):
        dz = s["dz"][a:b].double()
        dx[a:b] = torch.einsum("rn,nk->rk", dz, w[e].double())
        dw.view(-1, NP, K)[e] = torch.einsum("rn,rk->nk", dz, s["x"][a:b].double())
    return {"dx": dx, "dw": dw}
