"""Cases of the layer's operators in 8 bits and of its optimiser, for timing and comparison.

Four calls, with the values in e4m3 (torch.float8_e4m3fn) and fp32 scales:
  rows     lrm_fp8_quantize: rows in 8 bits with a scale for each 128 columns of a row, sorted by expert or not
  weights  lrm_fp8_quantize_weight: a scale for each block of 128 x 128
  product  lrm_fp8_linear: the product of the two with bias, activation and residual, dense or per expert
  dx       lrm_fp8_linear_backward: the gradient of its rows from the same 8-bit weights
  adamw    AdamW: one step over many tensors, clipped by the norm of all gradients, states in 32 bits or in 8
With `own` false every call is computed by elementary torch operations; with `own` true by the package's
entry points.  SwiGLU weights hold N gate rows, then N up rows, and each half has blocks of its own.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu", "swiglu")
FP8 = torch.float8_e4m3fn
BLOCK = 128       # columns of a row, or rows and columns of a weight, that share a scale
TOP = 448.0       # the largest e4m3 value
LEAST = 2.0 ** -100  # blocks of smaller values are scaled as if this were their largest
STATES = 256      # elements of a tensor whose 8-bit optimiser states share a scale
STATE_LEAST = 2.0 ** -120


# ------------------------------------------------------------------------------------- cases ----
def _rows(name, dtype, T, k, E, K, masked=0.0):
    return {"name": name, "op": "rows", "dtype": dtype, "T": T, "k": k, "E": E, "K": K, "masked": masked}


def _weights(name, dtype, E, N, K, glu=False):
    return {"name": name, "op": "weights", "dtype": dtype, "E": E, "N": N, "K": K, "glu": glu}


def _product(name, op, T, k, E, N, K, act="none", bias=False, residual=False, save_z=False, skew=1.0):
    """E = 0: dense, T rows; else T * k rows sorted by expert."""
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "act": act, "bias": bias,
            "residual": residual, "save_z": save_z, "skew": skew}


def _adamw(name, count, fewest, most, w, g, bits, copy=False, clip=True):
    """count tensors of fewest to most elements; w, g: types of weights and gradients; bits: of the states; copy: a
    bf16 copy of fp32 weights is written too."""
    return {"name": name, "op": "adamw", "count": count, "fewest": fewest, "most": most, "w": w, "g": g, "bits": bits,
            "copy": copy, "clip": clip}


def listed():
    return [
        # the tokens of 64 sequences generating, on their way to the experts of the Qwen3-shaped layer
        _rows("rows_decode64", "bf16", 64, 8, 128, 2048),
        # one 8192-token sequence in training: every token's row goes to eight experts
        _rows("rows_train_qwen3", "bf16", 8192, 8, 128, 2048),
        # odd fp32 rows of a dense product, nothing a multiple of 128
        _rows("rows_odd_f32", "f32", 5003, 0, 0, 1040),
        # the Qwen3-shaped layer's first weights after an optimiser step
        _weights("weights_qwen3", "bf16", 128, 768, 2048, glu=True),
        # an expert that every token takes (GLM4.5's expert size), one sequence generating
        _product("token_dense", "product", 1, 1, 0, 1408, 4096, act="swiglu", bias=True),
        # the experts' first product for 64 sequences generating, Qwen3-shaped layer: few rows an expert
        _product("experts_decode64", "product", 64, 8, 128, 768, 2048, act="swiglu"),
        # a dense projection at training size: bias, GELU and the residual in one pass
        _product("dense_train", "product", 32768, 1, 0, 4096, 4096, act="gelu", bias=True, residual=True),
        # the experts' first product in training: the pre-activation is kept for the backward
        _product("experts_train_qwen3", "product", 8192, 8, 128, 768, 2048, act="swiglu", save_z=True),
        # its rows' gradient
        _product("dx_train_qwen3", "dx", 8192, 8, 128, 768, 2048, act="swiglu"),
        # the same of odd sizes: neither half of the weights nor the hidden size is a multiple of 128
        _product("dx_odd", "dx", 611, 2, 7, 208, 1040, act="swiglu"),
        # the Qwen3-shaped layer's weights after a backward: bf16 weights, fp32 gradients, 8-bit states
        _adamw("adamw_layer_8bit", 3, 262144, 402653184, "bf16", "f32", 8),
        # a model's small tensors (norms, biases, routers): fp32 weights with a bf16 copy, 32-bit states
        _adamw("adamw_small_tensors", 300, 1, 300000, "f32", "bf16", 32, copy=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo=64, hi=4096):
    return _log(rng, lo, hi) // 16 * 16  # 8-bit rows start on 16 bytes


def draw(rng):
    op = rng.choice(["rows", "weights", "product", "product", "product", "dx", "dx", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rows":
        k = rng.choice([0, 1, 2, 6, 8])
        E = _log(rng, max(2, k), 256) if k else 0
        T, K = _log(rng, 1, 32768), _width(rng)
        while T * max(k, 1) * K > 8192 * 8 * 2048:
            T = max(1, T // 2)
        c = _rows("", dtype, T, k, E, K, masked=rng.choice([0.0, 0.3]) if k else 0.0)
    elif op == "weights":
        E, N, K = _log(rng, 1, 128), _width(rng), _width(rng)
        glu = rng.random() < 0.5
        while E * N * K * (2 if glu else 1) > 128 * 1536 * 2048:
            E = max(1, E // 2)
        c = _weights("", dtype, E, N, K, glu)
    elif op == "adamw":
        most = _log(rng, 8, 100000000)
        count = _log(rng, 1, 300)
        while count * most > 600000000:
            count = max(1, count // 2)
        w = rng.choice(["bf16", "f32"])
        c = _adamw("", count, max(1, most // rng.choice([1, 10, 1000])), most, w, rng.choice(["bf16", "f32"]),
                   rng.choice([8, 32]), copy=w == "f32" and rng.random() < 0.5, clip=rng.random() < 0.7)
    else:
        act = rng.choice(ACTS)
        N, K = _width(rng), _width(rng)
        bias, residual, save_z = rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.4
        if op == "dx":
            act, bias, residual, save_z = rng.choice(["none", "swiglu"]), False, False, False
        if rng.random() < 0.4:
            T, k, E = _log(rng, 1, 32768), 1, 0
            while T * N * K > 2 ** 36:
                T = max(1, T // 2)
        else:
            E = _log(rng, 2, 128)
            k = rng.randint(1, min(8, E))
            T = _log(rng, 1, 8192)
            while E * T * max(2 * N, K) > 2 ** 31 or E * T * N * K > 2 ** 40:
                T = max(1, T // 2)
        c = _product("", op, T, k, E, N, K, act, bias, residual, save_z, skew=rng.choice([0.0, 1.0]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs ----
def _sizes(case):
    """Elements of each tensor: spread over their range by the golden ratio, the largest among them."""
    n, lo, hi = case["count"], case["fewest"], case["most"]
    return [int(round(lo * (hi / lo) ** ((i * 0.6180339887498949) % 1.0 if i else 1.0))) for i in range(n)]


def _route(gen, T, k, E, skew):
    """Top-k experts of each token, popularity falling as rank ** -skew."""
    logits = torch.randn(T, E, generator=gen, device="cuda")
    logits -= skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    return torch.topk(logits, k, dim=1).indices.reshape(-1)


def _blocks(a, rows, cols):
    """The largest magnitude of each block of rows x cols of the last two axes."""
    r, c = a.shape[-2:]
    a = torch.nn.functional.pad(a.abs(), (0, -c % cols, 0, -r % rows))
    return a.unflatten(-1, (-1, cols)).unflatten(-3, (-1, rows)).amax((-3, -1))


def _spread(s, rows, cols, like):
    """A scale for each block laid out over the blocks' elements."""
    r, c = like.shape[-2:]
    return s.repeat_interleave(rows, -2)[..., :r, :].repeat_interleave(cols, -1)[..., :c]


def _quantize(a, rows):
    """e4m3 values and scales of blocks of rows x 128, in 32 bits."""
    a = a.float()
    top = _blocks(a, rows, BLOCK).clamp_min(LEAST)
    q = (a * _spread(TOP / top, rows, BLOCK, a)).to(FP8)
    return q, top / TOP


def _halves(a, glu, axis=-2):
    return a.unflatten(axis, (2, -1)) if glu else a


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    c, op = case, case["op"]
    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    types = {"bf16": torch.bfloat16, "f32": torch.float32}
    if op == "rows":
        T, k, E, K = c["T"], c["k"], c["E"], c["K"]
        s["x"], s["row"], s["q"], s["scale"] = randn(T, K, dtype=types[c["dtype"]]), None, None, None
        if k:
            e = _route(gen, T, k, E, 1.0)
            drop = torch.rand(T * k, generator=gen, device="cuda") < c["masked"]
            order = torch.sort(torch.where(drop, torch.full_like(e, E), e), stable=True).indices
            row = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device="cuda"))
            s["row"] = torch.where(drop, torch.full_like(row, -1), row).to(torch.int32)
            # the layer's buffers: rows of no pair stay as they are
            s["q"] = torch.zeros(T * k, K, device="cuda").to(FP8)
            s["scale"] = torch.ones(T * k, -(-K // BLOCK), device="cuda")
    elif op == "weights":
        rows = c["N"] * (2 if c["glu"] else 1)
        s["w"] = randn(c["E"], rows, c["K"], std=c["K"] ** -0.5, dtype=types[c["dtype"]])
    elif op in ("product", "dx"):
        T, k, E, N, K, glu = c["T"], c["k"], c["E"], c["N"], c["K"], c["act"] == "swiglu"
        R, rows, lead = T * k, N * (2 if glu else 1), (E,) if E else ()
        s["seg"], s["max_rows"] = None, R
        if E:
            load = torch.bincount(_route(gen, T, k, E, c["skew"]), minlength=E)
            s["seg"] = torch.nn.functional.pad(load.cumsum(0), (1, 0)).to(torch.int32)
            s["max_rows"] = int(load.max())
        q, scale = _quantize(_halves(randn(*lead, rows, K, std=K ** -0.5), glu), BLOCK)
        s["w"], s["w_scale"] = q.reshape(*lead, rows, K), scale.reshape(*lead, -1, scale.shape[-1])
        if op == "product":
            s["x"], s["x_scale"] = _quantize(randn(R, K), 1)
            s["b"] = randn(*lead, rows, std=0.1) if c["bias"] else None
            s["residual"] = randn(R, N) if c["residual"] else None
        else:
            q, scale = _quantize(_halves(randn(R, rows, std=1e-3), glu, -1), 1)
            s["dz"], s["dz_scale"] = q.reshape(R, rows), scale.reshape(R, -1)
    else:
        # the tensors lie in one buffer of each kind, each on a boundary of 256 elements; a state of some steps ago
        n = _sizes(c)
        at = [0]
        for v in n:
            at.append(at[-1] + -(-v // STATES) * STATES)
        w = randn(at[-1], std=0.02, dtype=types[c["w"]])
        g = randn(at[-1], std=1e-3, dtype=types[c["g"]])
        m = randn(at[-1], std=3e-4, dtype=torch.float32)
        v = (randn(at[-1], std=1e-3, dtype=torch.float32) ** 2 + 1e-8)
        for i, used in enumerate(n):  # nothing lies between the tensors
            for a in (w, g, m, v):
                a[at[i] + used:at[i + 1]] = 0
        s.update(n=n, at=at, w=w, g=g, copy=w.bfloat16() if c["copy"] else None, opt=None)
        if c["bits"] == 8:
            for key, a in (("m", m), ("v", v.sqrt())):
                a = a.view(-1, STATES)
                top = a.abs().amax(1, keepdim=True).clamp_min(STATE_LEAST)
                s[key], s[key + "_scale"] = (a * (TOP / top)).to(FP8).view(-1), (top / TOP).view(-1)
        else:
            s["m"], s["v"] = m, v
        s["hyper"] = {"lr": 3e-4, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1}
        s["max_norm"], s["step"], s["seed"] = 1.0, 7, 1234
    return s


# ----------------------------------------------------------------------------- plain form -------
def _act(z, act):
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return g / (1 + torch.exp(-g)) * u
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    return torch.maximum(z, torch.zeros_like(z)) if act == "relu" else z


def _by_expert(s, a):
    """Rows sorted by expert laid out as [experts, most rows of one, columns], and each row's place in it."""
    seg = s["seg"].long()
    r = torch.arange(a.shape[0], device="cuda")
    e = torch.searchsorted(seg[1:].contiguous(), r, right=True)
    at = r - seg[e]
    p = torch.zeros(s["case"]["E"], s["max_rows"], a.shape[1], device="cuda")
    p[e, at] = a
    return p, e, at


def _values(q, scale, rows, glu, axis):
    """What 8-bit values stand for, in 32 bits."""
    a, t = _halves(q.float(), glu, axis), _halves(scale, glu, axis)
    return (a * _spread(t, rows, BLOCK, a)).flatten(*((-3, -2) if axis == -2 else (-2, -1)) if glu else (-1, -1))


def _mix(h):
    """The 32-bit finaliser of MurmurHash3, in 64-bit integers."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _bits(s, i):
    """32 random bits for each element of tensor i, fixed by seed, step and place."""
    key = _mix(_mix((s["seed"] + 0x9E3779B9 * (i + 1)) & 0xFFFFFFFF) ^ s["step"])
    at = torch.arange(s["n"][i], device="cuda")
    return _mix(((at & 0xFFFFFFFF) * 0x9E3779B1 + key + (at >> 32) * 0xC2B2AE3D) & 0xFFFFFFFF)


def _to_state(a, bits, least):
    """States in 8 bits: the largest magnitude of 256 elements is 448, rounded up or down at random by 16 bits."""
    n = a.numel()
    a = torch.nn.functional.pad(a, (0, -n % STATES)).view(-1, STATES)
    top = a.abs().amax(1, keepdim=True).clamp_min(STATE_LEAST)
    y = (a.abs() * (TOP / top)).view(-1)[:n]
    shift = torch.where(y < 2.0 ** -6, 2.0 ** -6, 0.0)  # values below the normal ones have their spacing
    up = ((y + shift).view(torch.int32) + (bits << 4).to(torch.int32)) & -0x100000
    y = (up.view(torch.float32) - shift).clamp_max(TOP)
    y = torch.where((a.view(-1)[:n] != 0) & (y < least), torch.full_like(y, least), y)
    return torch.copysign(y, a.view(-1)[:n]).to(FP8), (top / TOP).view(-1)


def _norm(s):
    parts = [s["g"][a:a + n].double().square().sum() for a, n in zip(s["at"], s["n"])]
    return torch.stack(parts).sum().sqrt().float()


def _plain_adamw(s):
    c, h = s["case"], s["hyper"]
    b1, b2 = h["betas"]
    out = {}
    factor = 1.0
    if c["clip"]:
        out["norm"] = _norm(s)
        factor = (s["max_norm"] / (out["norm"] + 1e-6)).clamp_max(1.0)
    c1, c2 = 1 - b1 ** s["step"], 1 - b2 ** s["step"]
    for i, n in enumerate(s["n"]):
        at = slice(s["at"][i], s["at"][i] + n)
        blocks = slice(s["at"][i] // STATES, s["at"][i] // STATES + -(-n // STATES))
        g, w = s["g"][at].float() * factor, s["w"][at].float()
        if c["bits"] == 8:
            m = s["m"][at].float() * s["m_scale"][blocks].repeat_interleave(STATES)[:n]
            v = (s["v"][at].float() * s["v_scale"][blocks].repeat_interleave(STATES)[:n]).square()
        else:
            m, v = s["m"][at], s["v"][at]
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        w = w * (1 - h["lr"] * h["weight_decay"]) - h["lr"] / c1 * m / (v.sqrt() / c2 ** 0.5 + h["eps"])
        s["w"][at] = w.to(s["w"].dtype)
        if c["copy"]:
            s["copy"][at] = w.bfloat16()
        if c["bits"] == 8:
            bits = _bits(s, i)
            s["m"][at], s["m_scale"][blocks] = _to_state(m, bits & 0xFFFF, 0.0)
            s["v"][at], s["v_scale"][blocks] = _to_state(v.sqrt(), bits >> 16, 2.0 ** -9)
        else:
            s["m"][at], s["v"][at] = m, v
    return {**out, **{k: s[k] for k in ("w", "m", "v", "m_scale", "v_scale", "copy") if s.get(k) is not None}}


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "rows":
        q, scale = _quantize(s["x"], 1)
        if s["row"] is not None:
            pair = torch.nonzero(s["row"] >= 0).flatten()
            row, token = s["row"][pair].long(), pair // c["k"]
            s["q"].view(torch.uint8)[row], s["scale"][row] = q.view(torch.uint8)[token], scale[token]
            q, scale = s["q"], s["scale"]
        return {"q": q, "scale": scale}
    if op == "weights":
        q, scale = _quantize(_halves(s["w"], c["glu"]), BLOCK)
        return {"q": q.reshape(s["w"].shape), "scale": scale.reshape(c["E"], -1, scale.shape[-1])}
    if op == "adamw":
        return _plain_adamw(s)
    glu = c["act"] == "swiglu"
    w = _values(s["w"], s["w_scale"], BLOCK, glu, -2)
    if op == "dx":
        dz = _values(s["dz"].unsqueeze(-2) if not glu else s["dz"], s["dz_scale"].unsqueeze(-2) if not glu else s["dz_scale"],
                     1, glu, -1).reshape(s["dz"].shape)
        if not c["E"]:
            return {"dx": (dz @ w).bfloat16()}
        p, e, at = _by_expert(s, dz)
        return {"dx": torch.bmm(p, w)[e, at].bfloat16()}
    x = _values(s["x"], s["x_scale"], 1, False, -2)
    if c["E"]:
        p, e, at = _by_expert(s, x)
        z = torch.bmm(p, w.transpose(1, 2))[e, at]
        z = z + s["b"].float()[e] if s["b"] is not None else z
    else:
        z = x @ w.t()
        z = z + s["b"].float() if s["b"] is not None else z
    y = _act(z, c["act"])
    y = y + s["residual"].float() if s["residual"] is not None else y
    return {"y": y.bfloat16(), "z": z.bfloat16()} if c["save_z"] else {"y": y.bfloat16()}


# ------------------------------------------------------------------------- the package's own ----
def _own(s):
    import pruned_expert_backward_gb300 as lrm
    c, op, st = s["case"], s["case"]["op"], s["status"]
    if op == "rows":
        q, scale = lrm.lrm_fp8_quantize(s["x"], row_of_pair=s["row"], k=c["k"] or 1, q=s["q"], scale=s["scale"],
                                        dev_status=st)
        return {"q": q, "scale": scale}
    if op == "weights":
        q, scale = lrm.lrm_fp8_quantize_weight(s["w"], glu=c["glu"])
        return {"q": q, "scale": scale}
    if op == "product":
        y, z = lrm.lrm_fp8_linear(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["b"], residual=s["residual"],
                                  act=c["act"], seg_offsets=s["seg"], save_z=c["save_z"], dev_status=st)
        return {"y": y, "z": z} if c["save_z"] else {"y": y}
    if op == "dx":
        return {"dx": lrm.lrm_fp8_linear_backward(s["dz"], s["dz_scale"], s["w"], s["w_scale"],
                                                  glu=c["act"] == "swiglu", seg_offsets=s["seg"], dev_status=st)}
    if s["opt"] is None:  # a program makes its optimiser once
        def tensors(a):
            return [a[at:at + n] for at, n in zip(s["at"], s["n"])] if a is not None else None

        def scales(a):
            return [a[at // STATES:at // STATES + -(-n // STATES)] for at, n in zip(s["at"], s["n"])]

        state = {"m": tensors(s["m"]), "v": tensors(s["v"])}
        if c["bits"] == 8:
            state.update(m_scale=scales(s["m_scale"]), v_scale=scales(s["v_scale"]))
        s["opt"] = lrm.AdamW(tensors(s["w"]), tensors(s["g"]), copies=tensors(s["copy"]), state_bits=c["bits"], state=state,
                             max_norm=s["max_norm"] if c["clip"] else None, seed=s["seed"], **s["hyper"])
    norm = s["opt"].step(step=s["step"])
    out = {"norm": norm} if c["clip"] else {}
    return {**out, **{k: s[k] for k in ("w", "m", "v", "m_scale", "v_scale", "copy") if s.get(k) is not None}}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------------- work ----
def _active(c):
    """Experts that have a row, on average over routings with this popularity."""
    w = [(i + 1.0) ** -c["skew"] for i in range(c["E"])]
    return sum(1 - (1 - min(1.0, c["k"] / sum(w) * p)) ** c["T"] for p in w)


def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "rows":
        T, K = c["T"], c["K"]
        R = T * max(c["k"], 1)
        rows = R * (1 - c["masked"])  # that a pair names
        read = T * K * size[c["dtype"]] + (4 * R if c["k"] else 0)
        return {"bytes": read + rows * (K + 4 * -(-K // BLOCK)), "flops": T * K}
    if op == "weights":
        n = c["E"] * c["N"] * (2 if c["glu"] else 1) * c["K"]
        return {"bytes": n * (size[c["dtype"]] + 1) + n // 4096, "flops": n}
    if op == "adamw":
        n, b = sum(_sizes(c)), c["bits"] // 8
        each = 2 * size[c["w"]] + size[c["g"]] + 4 * b + (16 / STATES if b == 1 else 0) + (2 if c["copy"] else 0)
        return {"bytes": n * each, "flops": 16 * n}
    R, N, K = c["T"] * c["k"], c["N"], c["K"]
    rows = N * (2 if c["act"] == "swiglu" else 1)
    weights = (_active(c) if c["E"] else 1) * rows * K * (1 + 4 / BLOCK ** 2)
    if op == "dx":
        return {"bytes": R * rows * (1 + 4 / BLOCK) + weights + R * K * 2, "flops": 2 * R * rows * K}
    out = 2 * R * (N + (N if c["residual"] else 0) + (rows if c["save_z"] else 0))
    return {"bytes": R * K * (1 + 4 / BLOCK) + weights + out, "flops": 2 * R * rows * K}


# ----------------------------------------------------------------------------- in 64 bits -------
def _f64_act(z, act):
    if act == "swiglu":
        n = z.shape[1] // 2
        return z[:, :n] * torch.special.expit(z[:, :n]) * z[:, n:]
    return {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.special.expit(v),
            "gelu": lambda v: v * torch.special.ndtr(v)}[act](z)


def _f64_blocks(x, rows):
    """The definition block by block: every value over the block's largest magnitude / 448 (before rounding to
    8 bits), and that scale."""
    R, K = x.shape
    q = torch.empty(R, K, dtype=torch.float64, device="cuda")
    scale = torch.empty(-(-R // rows), -(-K // BLOCK), dtype=torch.float64, device="cuda")
    for b in range(scale.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK].double()
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.stack([t.max() for t in top.split(rows)])
        scale[:, b] = top.clamp(min=LEAST) / 448
        each = scale[:, b] if rows == 1 else scale[:, b].repeat_interleave(rows)[:R]
        q[:, b * BLOCK:(b + 1) * BLOCK] = part / each[:, None]
    return q, scale


def _f64_operand(q, scale, rows):
    """q [a, b] times the scale of its block of rows x 128."""
    a = q.double()
    for i in range(scale.shape[0] if rows > 1 else 1):
        at = slice(i * rows, (i + 1) * rows) if rows > 1 else slice(None)
        for j in range(scale.shape[1]):
            t = scale[i, j].double() if rows > 1 else scale[:, j, None].double()
            a[at, j * BLOCK:(j + 1) * BLOCK] *= t
    return a


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "rows":
        q, scale = _f64_blocks(s["x"], 1)
        if s["row"] is None:
            return {"q": q, "scale": scale}
        row = s["row"].view(c["T"], c["k"]).long()
        q_s, scale_s = s["q"].double(), s["scale"].double()
        for j in range(c["k"]):
            t = torch.nonzero(row[:, j] >= 0).flatten()
            q_s[row[t, j]], scale_s[row[t, j]] = q[t], scale[t]
        return {"q": q_s, "scale": scale_s}
    if op == "weights":
        parts = [_f64_blocks(half, BLOCK) for w in s["w"] for half in (w.chunk(2) if c["glu"] else (w,))]
        q = torch.stack([p[0] for p in parts]).view(s["w"].shape)
        return {"q": q, "scale": torch.stack([p[1] for p in parts]).view(c["E"], -1, parts[0][1].shape[1])}
    if op == "adamw":
        return _exact_adamw(s)
    R, N, K, E, act = c["T"] * c["k"], c["N"], c["K"], c["E"], c["act"]
    glu = act == "swiglu"
    rows = 2 * N if glu else N
    seg = s["seg"].tolist() if E else [0, R]
    w_all, t_all = s["w"].view(-1, rows, K), s["w_scale"].view(len(seg) - 1, -1, s["w_scale"].shape[-1])

    def weight(e):
        halves = zip(w_all[e].chunk(2 if glu else 1), t_all[e].chunk(2 if glu else 1))
        return torch.cat([_f64_operand(q, t, BLOCK) for q, t in halves])

    def new(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")

    if op == "dx":
        halves = zip(s["dz"].chunk(2 if glu else 1, 1), s["dz_scale"].chunk(2 if glu else 1, 1))
        dz, dx = torch.cat([_f64_operand(q, t, 1) for q, t in halves], 1), new(R, K)
        for e, (a, b) in enumerate(zip(seg, seg[1:])):
            if b > a:
                dx[a:b] = torch.einsum("rn,nk->rk", dz[a:b], weight(e))
        return {"dx": dx}
    x, y, z = _f64_operand(s["x"], s["x_scale"], 1), new(R, N), new(R, rows) if c["save_z"] else None
    for e, (a, b) in enumerate(zip(seg, seg[1:])):
        if b > a:
            ze = torch.einsum("rk,nk->rn", x[a:b], weight(e))
            if s["b"] is not None:
                ze += s["b"].view(-1, rows)[e].double()
            if z is not None:
                z[a:b] = ze
            y[a:b] = _f64_act(ze, act)
    if s["residual"] is not None:
        y += s["residual"].double()
    return {"y": y, "z": z} if c["save_z"] else {"y": y}


def _exact_adamw(s):
    """8-bit states are given before their random rounding, over their scales."""
    c, h = s["case"], s["hyper"]
    b1, b2 = h["betas"]
    live = torch.zeros(s["at"][-1], dtype=torch.bool, device="cuda")
    for a, n in zip(s["at"], s["n"]):
        live[a:a + n] = True
    g = torch.where(live, s["g"], torch.zeros_like(s["g"])).double()
    norm = torch.linalg.vector_norm(g)
    if c["clip"]:
        g *= torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    if c["bits"] == 8:
        m = (s["m"].double().view(-1, STATES) * s["m_scale"].double()[:, None]).view(-1)
        v = (s["v"].double().view(-1, STATES) * s["v_scale"].double()[:, None]).view(-1) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m.lerp_(g, 1 - b1)
    v.lerp_(g * g, 1 - b2)
    rate = h["lr"] / -math.expm1(s["step"] * math.log(b1))
    w = s["w"].double() * (1 - h["lr"] * h["weight_decay"])
    w -= rate * m / ((v / -math.expm1(s["step"] * math.log(b2))).sqrt() + h["eps"])
    out = {"norm": norm} if c["clip"] else {}
    out["w"] = w
    if c["bits"] == 8:
        for key, a in (("m", m), ("v", v.sqrt())):
            top = a.view(-1, STATES).abs().amax(1).clamp(min=STATE_LEAST)
            out[key], out[key + "_scale"] = (a.view(-1, STATES) / top[:, None] * 448).view(-1), top / 448
    else:
        out["m"], out["v"] = m, v
    if c["copy"]:
        out["copy"] = w
    return out
