"""Cases of the operators around a mixture-of-experts block with 4-bit experts,
for timing and for comparing results:

* ``norm_fwd`` / ``norm_bwd``: the norms before and after the block with its
  gate and residual scale, N(v; w) = v rsqrt(mean(v^2) + eps) w,
  z = a x + gate N(y; w_post), h = N(z; w_next), and their gradients.
* ``decode4``: the layer for a few tokens from MXFP4 weights (pairs of e2m1
  codes, one E8M0 scale per 32 columns).
* ``grouped4``: the products of expert-sorted rows with their experts' MXFP4
  matrices, y[r] = W_e x[src_of[r] / k] or W_e rows[r], plain or with the
  SwiGLU behind them (a prompt's gate/up and down products).

``own`` selects the framework's kernels; otherwise ``run`` computes the same
in elementary torch operations in float32, rounded once at the end.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def _norm(name, op, T, d, dtype="bf16", block=True, post=True, gate="none", scale=1.0, after=True):
    """block: there is a y (else h = N(x) alone); post, gate and after: its
    norm, its gate ("none", "channel", "token") and the next block's norm."""
    return {"name": name, "op": op, "T": T, "d": d, "dtype": dtype, "block": block, "post": post, "gate": gate,
            "scale": scale, "after": after}


def _decode(name, T, d, E, k, I, logits="bf16", limit=0.0, empty=0.0):
    """logits: dtype of the router logits, or "ids" for ids and weights in
    hand; empty: the share of empty slots (ids form) or of masked experts."""
    return {"name": name, "op": "decode4", "T": T, "d": d, "E": E, "k": k, "I": I, "logits": logits,
            "limit": limit, "empty": empty}


def _grouped(name, T, k, E, K, N, gather=True, swiglu=False, limit=0.0, skew=0.0):
    """T tokens, k experts each; [E, N, K] weights.  skew: exponent of the
    experts' popularity (0: equal)."""
    return {"name": name, "op": "grouped4", "T": T, "k": k, "E": E, "K": K, "N": N, "gather": gather,
            "swiglu": swiglu, "limit": limit, "skew": skew}


def listed():
    return [
        # one request's next token: its residual and the next block's norm
        _norm("norm_fwd_t1", "norm_fwd", 1, 2048, post=False),
        # a training step or long prompt: norms on both sides, channel gate
        _norm("norm_fwd_t16384", "norm_fwd", 16384, 2048, gate="channel", scale=0.7),
        # odd extents in float32, a gate per token, no norm behind
        _norm("norm_fwd_t1001_f32", "norm_fwd", 1001, 1000, dtype="f32", gate="token", after=False),
        # the training step's gradients through all of it
        _norm("norm_bwd_t16384", "norm_bwd", 16384, 2048, gate="channel", scale=0.7),
        # a short batch of wider rows, a gate per token
        _norm("norm_bwd_t333", "norm_bwd", 333, 4096, gate="token"),
        # one request's next token through the layer of 128 experts, top 8
        _decode("decode4_t1", 1, 2048, 128, 8, 768),
        # a batch that touches nearly every expert: the layer's whole weights
        _decode("decode4_t64", 64, 2048, 128, 8, 768),
        # wide experts, ids in hand with empty slots, several rows per expert
        _decode("decode4_t200_ids", 200, 4096, 64, 8, 1024, logits="ids", limit=7.0, empty=0.05),
        # a short prompt's gate/up products: two rows an expert
        _grouped("grouped4_t33", 33, 8, 128, 2048, 1536, swiglu=True),
        # a prompt of ordinary length, few rows per expert, skewed
        _grouped("grouped4_t700_down", 700, 8, 128, 1536, 4096, gather=False, skew=0.6),
        # many prompts at once: the gate/up products of 131072 rows
        _grouped("grouped4_t16384", 16384, 8, 128, 2048, 1536, swiglu=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _unnamed(case):
    del case["name"]
    return case


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "decode4", "decode4", "grouped4", "grouped4"])
    if op.startswith("norm"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = max(8, _log(rng, 64, 8192) // 8 * 8)
        T = _log(rng, 1, min(16384, 16384 * 2048 // d) // (2 if dtype == "f32" else 1))
        block = rng.random() < 0.8
        after = not block or rng.random() < 0.7
        return _unnamed(_norm("", op, T, d, dtype, block, block and rng.random() < 0.7,
                              rng.choice(["none", "channel", "token"]) if block else "none",
                              rng.choice([1.0, rng.uniform(0.2, 2.0)]) if block else 1.0, after))
    if op == "decode4":
        T = _log(rng, 1, 256)
        E = _log(rng, 1, 128)
        k = rng.randint(1, min(E, 8))
        d = max(128, _log(rng, 128, 4096) // 128 * 128)
        I = max(128, _log(rng, 128, 1024) // 128 * 128)
        while E * I * d > 64 * 4096 * 1024:  # no more than the largest listed case
            I = max(128, I // 256 * 128)
            E, k = (E, k) if I > 128 else (E // 2, min(k, E // 2))
        form = rng.choice(["bf16", "f32", "ids"])
        return _unnamed(_decode("", T, d, E, k, I, form, rng.choice([0.0, 0.0, 7.0]),
                                rng.choice([0.0, rng.uniform(0.0, 0.4)])))
    E = _log(rng, 1, 128)
    k = rng.randint(1, min(E, 8))
    T = _log(rng, 1, 16384 * 8 // k)
    K = max(128, _log(rng, 128, 4096) // 128 * 128)
    N = max(16, _log(rng, 128, 4096) // 16 * 16)
    while T * k * K * N > 131072 * 2048 * 1536:  # no more than the largest listed case
        T = T // 2
    return _unnamed(_grouped("", T, k, E, K, N, rng.random() < 0.6, rng.random() < 0.5, rng.choice([0.0, 7.0]),
                             rng.choice([0.0, rng.uniform(0.2, 1.2)])))


def work(case):
    if case["op"].startswith("norm"):
        T, d = case["T"], case["d"]
        es = 4 if case["dtype"] == "f32" else 2
        weights = case["post"] + case["after"] + (case["gate"] == "channel")
        tokens = T if case["gate"] == "token" else 0
        if case["op"] == "norm_fwd":
            rows = 1 + case["after"] + 2 * case["block"]  # x, h, and y, z
            return {"bytes": (rows * T * d + weights * d + tokens) * es, "flops": 4.0 * rows * T * d}
        rows = 3 + case["after"] + 2 * case["block"]  # dz, z, dx; dh; y, dy
        return {"bytes": (rows * T * d + 2 * (weights * d + tokens)) * es, "flops": 5.0 * rows * T * d}
    coded = 0.5 + 1.0 / 32.0
    if case["op"] == "decode4":
        T, d, E, k, I = (case[n] for n in ("T", "d", "E", "k", "I"))
        slots = k * (1.0 - case["empty"]) if case["logits"] == "ids" else k
        pool = E if case["logits"] == "ids" else max(k, E * (1.0 - case["empty"]))
        active = pool * (1.0 - (1.0 - slots / pool) ** T)  # experts that some token takes
        route = 8 * T * k if case["logits"] == "ids" else T * E * (4 if case["logits"] == "f32" else 2) + 8 * T * k
        return {"bytes": active * 3 * I * d * coded + 4 * T * d + route, "flops": 6.0 * T * slots * d * I}
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    R = T * k
    active = sum(1.0 - (1.0 - p) ** T for p in _taken(E, k, case["skew"]))
    rows = min(T, R) if case["gather"] else R
    out = N // 2 if case["swiglu"] else N
    return {"bytes": active * N * K * coded + 2 * rows * K + 2 * R * out + 4 * R + 4 * (E + 1),
            "flops": 2.0 * R * N * K}


def _taken(E, k, skew):
    """About how likely a token takes each expert (for the experts read)."""
    p = [(i + 1.0) ** -skew for i in range(E)]
    return [min(1.0, k * v / sum(p)) for v in p]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _weight4(g, E, N, K):
    """Random [E, N, K] weights of standard deviation K^-1/2 in MXFP4: codes
    [E, N, K/2] (the even column in the low half of a byte) and E8M0 bytes
    [E, N, K/32], the scale the smallest power of two with amax <= 6 of it."""
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (N * K))
    for e in range(0, E, step):
        b = torch.randn((min(step, E - e), N, K // 32, 32), generator=g, device="cuda") * K ** -0.5
        m, x = torch.frexp(b.abs().amax(dim=3))  # amax = m 2^x, m in [0.5, 1); 6 = 0.75 2^3
        x = x - 3 + (m > 0.75)
        v = torch.ldexp(b, -x[..., None])
        a = v.abs()
        unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        a = torch.round(a / unit) * unit
        code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)) + 8 * (v < 0)
        code = code.to(torch.uint8).view(-1, N, K // 2, 2)
        codes[e:e + step] = code[..., 0] | (code[..., 1] << 4)
        scales[e:e + step] = (x + 127).to(torch.uint8)
    return codes, scales


def _choices(g, T, k, E, skew):
    """[T, k] distinct experts a token, popular ones more often with a skew."""
    pop = -skew * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    pop = pop[torch.rand(E, generator=g, device="cuda").argsort()]
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)))
    return (pop + noise).topk(k, dim=1).indices.to(torch.int32).contiguous()


def _sorted_rows(ids, w, E):
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    src = torch.argsort(flat, stable=True)
    row = torch.empty_like(src)
    row[src] = torch.arange(T * k, device="cuda")
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    i32 = torch.int32
    return {"topk_ids": ids, "topk_w": w, "counts": counts.to(i32), "offsets": offsets.to(i32),
            "row_of": row.to(i32), "src_of": src.to(i32)}


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"].startswith("norm"):
        T, d, dt = case["T"], case["d"], _DT[case["dtype"]]
        s["x" if case["op"] == "norm_fwd" else "z"] = _normal(g, (T, d), dt, 2.0)
        s["y"] = _normal(g, (T, d), dt, 0.5) if case["block"] else None
        s["w_post"] = _normal(g, (d,), dt, 0.2, 1.0) if case["post"] else None
        s["w_next"] = _normal(g, (d,), dt, 0.2, 1.0) if case["after"] else None
        s["gate"] = {"none": None, "channel": (d,), "token": (T, 1)}[case["gate"]]
        if s["gate"] is not None:
            s["gate"] = _normal(g, s["gate"], dt, 0.3, 0.5)
        if case["op"] == "norm_bwd":
            s["dz"] = _normal(g, (T, d), dt)
            s["dh"] = _normal(g, (T, d), dt) if case["after"] else None
        return s
    if case["op"] == "decode4":
        T, d, E, k, I = (case[n] for n in ("T", "d", "E", "k", "I"))
        s["x"] = _normal(g, (T, d), torch.bfloat16)
        s["w_gate_up"] = _weight4(g, E, 2 * I, d)
        s["w_down"] = _weight4(g, E, d, I)
        if case["logits"] == "ids":
            ids = _choices(g, T, k, E, 0.0)
            hole = torch.rand((T, k), generator=g, device="cuda") < case["empty"]
            s["ids"] = torch.where(hole, torch.full_like(ids, -1), ids).contiguous()
            s["w"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
        else:
            lg = torch.randn((T, E), generator=g, device="cuda")
            off = torch.rand(E, generator=g, device="cuda").argsort() < int(case["empty"] * E)
            off &= E - int(case["empty"] * E) >= k
            s["logits"] = torch.where(off, torch.full_like(lg, -math.inf), lg).to(_DT[case["logits"]])
        if own:
            from combine_top_route_amd import binding as B
            s["decoder"] = B.MoeDecoder(T, d, E, k, I, weights="mxfp4", device="cuda", swiglu_limit=case["limit"],
                                        logits_dtype=_DT.get(case["logits"], torch.float32))
        return s
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    s["x"] = _normal(g, (T if case["gather"] else T * k, K), torch.bfloat16)
    s["weight"] = _weight4(g, E, N, K)
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
    s["routing"] = _sorted_rows(_choices(g, T, k, E, case["skew"]), w, E)
    s["offsets"] = s["routing"]["offsets"].tolist()
    if own:
        from combine_top_route_amd import binding as B
        s["rows"] = B.Routing(**s["routing"])
    return s


# --------------------------------------------------------------- plain forms
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _matrix4(w, e):
    """Expert e's matrix (e: an index or a tensor of them) in float32."""
    codes, scales = w[0][e], w[1][e]
    lut = torch.tensor(_E2M1 + [-v for v in _E2M1], device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], dim=-1).long()].flatten(-2)
    return torch.ldexp(v.view(*scales.shape, 32), scales[..., None].int() - 127).flatten(-2)


def _act(g, u, limit):
    if limit > 0:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g * torch.sigmoid(g) * u


def _topk(logits, k):
    """Largest k per row, ties to the lower index, and their softmax; -inf
    entries give an empty slot (id -1, weight 0)."""
    v, i = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    none = v == -math.inf
    ex = torch.where(none, torch.zeros_like(v), torch.exp(v - v[:, :1]))
    w = torch.where(none, ex, ex / ex.sum(dim=1, keepdim=True))
    return torch.where(none, torch.full_like(i, -1), i).to(torch.int32).contiguous(), w.contiguous()


def _rstd(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _norm_fwd_plain(s):
    c, dt = s["case"], s["x"].dtype
    z = s["x"].float()
    if c["block"]:
        b = s["y"].float()
        if c["post"]:
            b = b * _rstd(b) * s["w_post"].float()
        if s["gate"] is not None:
            b = b * s["gate"].float()
        z = c["scale"] * z + b
    out = {"z": z.to(dt)} if c["block"] else {}
    if c["after"]:
        out["h"] = (z * _rstd(z) * s["w_next"].float()).to(dt)
    return out


def _norm_bwd_plain(s):
    c, dt = s["case"], s["z"].dtype
    out = {}
    g = s["dz"].float()
    if c["after"]:
        z, dh = s["z"].float(), s["dh"].float()
        r = _rstd(z)
        zh, t = z * r, dh * s["w_next"].float()
        g = g + r * (t - zh * (t * zh).mean(dim=1, keepdim=True))
        out["dw_next"] = (dh * zh).sum(dim=0).to(dt)
    out["dx"] = (c["scale"] * g).to(dt)
    if not c["block"]:
        return out
    y = s["y"].float()
    ry = _rstd(y) if c["post"] else None
    u = y * ry if c["post"] else y
    wp = s["w_post"].float() if c["post"] else 1.0
    gate = s["gate"].float() if s["gate"] is not None else 1.0
    t = g * gate * wp
    if c["post"]:
        out["dw_post"] = (g * gate * u).sum(dim=0).to(dt)
        t = ry * (t - u * (t * u).mean(dim=1, keepdim=True))
    out["dy"] = t.to(dt)
    if c["gate"] == "channel":
        out["dgate"] = (g * u * wp).sum(dim=0).to(dt)
    elif c["gate"] == "token":
        out["dgate"] = (g * u * wp).sum(dim=1, keepdim=True).to(dt)
    return out


def _decode_plain(s):
    c = s["case"]
    T, E, k, I = c["T"], c["E"], c["k"], c["I"]
    ids, w = (s["ids"], s["w"]) if c["logits"] == "ids" else _topk(s["logits"], k)
    x = s["x"].float()
    out = torch.zeros_like(x)
    if T * k <= E:  # fewer slots than experts: fetch each slot's matrices
        for t in range(T):
            e = ids[t].clamp(0, E - 1).long()
            h = torch.matmul(_matrix4(s["w_gate_up"], e), x[t])
            a = _act(h[:, :I], h[:, I:], c["limit"])
            y = torch.matmul(_matrix4(s["w_down"], e), a[:, :, None])[:, :, 0]
            inside = (ids[t] >= 0) & (ids[t] < E)
            out[t] = torch.where(inside[:, None], w[t][:, None] * y, 0.0).sum(dim=0)
    else:
        for e in range(E):
            hit = ids == e
            we = torch.where(hit, w, 0.0).sum(dim=1)
            h = x @ _matrix4(s["w_gate_up"], e).T
            a = _act(h[:, :I], h[:, I:], c["limit"])
            y = we[:, None] * (a @ _matrix4(s["w_down"], e).T)
            out += torch.where(hit.any(dim=1)[:, None], y, 0.0)
    out = out.to(s["x"].dtype)
    return {"out": out} if c["logits"] == "ids" else {"out": out, "topk_ids": ids, "topk_w": w}


def _grouped_plain(s):
    c = s["case"]
    T, k, E, N = c["T"], c["k"], c["E"], c["N"]
    out = torch.empty((T * k, N // 2 if c["swiglu"] else N), dtype=s["x"].dtype, device=s["x"].device)
    token = torch.div(s["routing"]["src_of"], k, rounding_mode="floor").long()
    for e in range(E):
        lo, hi = s["offsets"][e], s["offsets"][e + 1]
        if lo == hi:
            continue
        rows = s["x"][token[lo:hi]] if c["gather"] else s["x"][lo:hi]
        h = rows.float() @ _matrix4(s["weight"], e).T
        out[lo:hi] = _act(h[:, :N // 2], h[:, N // 2:], c["limit"]) if c["swiglu"] else h
    return {"y": out}


# ---------------------------------------------------------------------- run
def run(state):
    c = state["case"]
    if not own:
        return {"norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain, "decode4": _decode_plain,
                "grouped4": _grouped_plain}[c["op"]](state)
    if c["op"] == "decode4":
        dec = state["decoder"]
        if c["logits"] == "ids":
            return {"out": dec.forward(state["x"], state["w_gate_up"], state["w_down"], topk_ids=state["ids"],
                                       topk_w=state["w"])}
        out = dec.forward(state["x"], state["w_gate_up"], state["w_down"], logits=state["logits"])
        return {"out": out, "topk_ids": dec.topk_ids, "topk_w": dec.topk_w}
    from combine_top_route_amd import binding as B
    if c["op"] == "grouped4":
        return {"y": B.grouped_product(state["x"], state["weight"], state["rows"], c["T"], c["k"],
                                       gather=c["gather"], swiglu=c["swiglu"], swiglu_limit=c["limit"])}
    if c["op"] == "norm_fwd":
        z, h = B.norm_residual(state["x"], state["y"], w_post=state["w_post"], gate=state["gate"],
                               res_scale=c["scale"], w_next=state["w_next"], eps=EPS)
        out = {"z": z} if c["block"] else {}
        if c["after"]:
            out["h"] = h
        return out
    grads = B.norm_residual_backward(state["dz"], state["dh"], state["z"], state["y"], w_post=state["w_post"],
                                     gate=state["gate"], res_scale=c["scale"], w_next=state["w_next"], eps=EPS)
    return {n: t for n, t in grads.items() if t is not None}


# -------------------------------------------------------------------- exact
def _m64(w, e):
    codes, scales = w[0][e].long(), w[1][e].double()
    n, half = codes.shape
    nib = torch.empty((n, 2 * half), dtype=torch.int64, device="cuda")
    nib[:, 0::2], nib[:, 1::2] = codes % 16, codes // 16
    mag = nib % 8
    # exponent field 0: halves; else (1 + m / 2) 2^(e - 1)
    val = torch.where(mag < 2, 0.5 * mag, (1.0 + 0.5 * (mag % 2)) * torch.exp2((mag // 2 - 1).double()))
    val = torch.where(nib >= 8, -val, val)
    return (val.view(n, half // 16, 32) * torch.exp2(scales - 127.0)[:, :, None]).view(n, 2 * half)


def _swish64(g, u, limit):
    if limit > 0:
        g, u = torch.minimum(g, g.new_tensor(limit)), torch.maximum(torch.minimum(u, u.new_tensor(limit)),
                                                                    u.new_tensor(-limit))
    return g / (1.0 + torch.exp(-g)) * u


def _exact_norm_fwd(case, s):
    v = s["x"].double()
    if case["block"]:
        b = s["y"].double()
        if case["post"]:
            b = b / (b.square().mean(1, keepdim=True) + EPS).sqrt() * s["w_post"].double()
        v = case["scale"] * v + (b if s["gate"] is None else s["gate"].double() * b)
    res = {"z": v} if case["block"] else {}
    if case["after"]:
        res["h"] = v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * s["w_next"].double()
    return res


def _exact_norm_bwd(case, s):
    """By torch's own differentiation of the formula, in 64 bits: the gradient
    of sum(dz z + dh N(z)) as z moves, and from there that of the block."""
    z = s["z"].double().requires_grad_()
    total = (s["dz"].double() * z).sum()
    wn = None
    if case["after"]:
        wn = s["w_next"].double().requires_grad_()
        total = total + (s["dh"].double() * (z / (z.square().mean(1, keepdim=True) + EPS).sqrt() * wn)).sum()
    grads = torch.autograd.grad(total, [z] + ([wn] if case["after"] else []))
    g = grads[0].detach()
    res = {"dw_next": grads[1]} if case["after"] else {}
    res["dx"] = case["scale"] * g
    if not case["block"]:
        return res
    leaves = {"dy": s["y"].double().requires_grad_()}
    b = leaves["dy"]
    if case["post"]:
        leaves["dw_post"] = s["w_post"].double().requires_grad_()
        b = b / (b.square().mean(1, keepdim=True) + EPS).sqrt() * leaves["dw_post"]
    if s["gate"] is not None:
        leaves["dgate"] = s["gate"].double().requires_grad_()
        b = b * leaves["dgate"]
    for n, t in zip(leaves, torch.autograd.grad((g * b).sum(), list(leaves.values()))):
        res[n] = t
    return res


def _exact_decode(case, s):
    T, E, k, I, L = (case[n] for n in ("T", "E", "k", "I", "limit"))
    if case["logits"] == "ids":
        ids, w = s["ids"].long(), s["w"].double()
    else:
        lg = s["logits"].double()
        left = lg.clone()
        picks = []
        for _ in range(k):  # k times the largest that is left, the first of equals
            top = left.amax(dim=1, keepdim=True)
            first = torch.where(left == top, torch.arange(E, device="cuda"), E).amin(dim=1)
            picks.append(torch.where(top[:, 0] > -math.inf, first, -1))
            left[torch.arange(T, device="cuda"), first.clamp(max=E - 1)] = -math.inf
        ids = torch.stack(picks, dim=1)
        v = torch.where(ids >= 0, lg.gather(1, ids.clamp(min=0)), torch.full_like(lg[:, :k], -math.inf))
        w = torch.nan_to_num(torch.softmax(v, dim=1), nan=0.0)
    out = torch.zeros((T, case["d"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        if not 0 <= e < E:
            continue
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = s["x"][t].double() @ _m64(s["w_gate_up"], e).t()
        y = _swish64(h[:, :I], h[:, I:], L) @ _m64(s["w_down"], e).t()
        out.index_add_(0, t, y * w[t, j][:, None])
    if case["logits"] == "ids":
        return {"out": out}
    return {"out": out, "topk_ids": ids, "topk_w": w}


def _exact_grouped(case, s):
    T, k, N = case["T"], case["k"], case["N"]
    ids = s["routing"]["topk_ids"].reshape(-1)
    src = s["routing"]["src_of"].long()
    out = torch.zeros((T * k, N // 2 if case["swiglu"] else N), dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        r = torch.nonzero(ids[src] == e)[:, 0]
        v = (s["x"][src[r] // k] if case["gather"] else s["x"][r]).double()
        h = torch.mm(v, _m64(s["weight"], e).t())
        out[r] = _swish64(h[:, :N // 2], h[:, N // 2:], case["limit"]) if case["swiglu"] else h
    return {"y": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd, "decode4": _exact_decode,
            "grouped4": _exact_grouped}[case["op"]](case, s)
