"""The operators around and inside the MoE layer, as they are measured.

* block_enter / block_exit: the RMS norm before the layer, and behind it the norm, gate, residual scale and the next
  norm, forward and backward;
* balance: the router's balance loss over ragged sequences with the per-expert counts, forward and backward;
* mx4_quantize: rows to 4-bit floating point with one power-of-two scale per 32 values, and the values read back;
* mx4_product: grouped expert rows times expert weights, both in that format, plain or gate/up with SwiGLU.

With `own` false, run() is plain torch in 32 bits; with `own` true it calls the library.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token of a decode step enters the layer: latency alone
        dict(name="enter_decode_one", op="enter", dir="fwd", T=1, d=2048, dtype="bf16"),
        # a training step of a small fp32 model whose sizes fit no tile
        dict(name="enter_train_odd_f32", op="enter", dir="bwd", T=777, d=1000, dtype="f32"),
        # a decode batch leaves the layer and enters the next one
        dict(name="exit_decode", op="exit", dir="fwd", T=128, d=2048, dtype="bf16", norm=True, gate_c=False, gate_t=True, next=True, a=1.0, b=1.0),
        # prefill of the large layer: every channel has a learned scale, the branch is damped
        dict(name="exit_prefill_large", op="exit", dir="fwd", T=4096, d=7168, dtype="bf16", norm=True, gate_c=True, gate_t=False, next=True, a=1.0, b=0.25),
        # a training step of the usual layer with all of it
        dict(name="exit_train", op="exit", dir="bwd", T=8192, d=2048, dtype="bf16", norm=True, gate_c=True, gate_t=True, next=True, a=1.0, b=0.5),
        # load statistics of a decode batch
        dict(name="balance_decode", op="balance", dir="fwd", T=128, E=128, K=8, S=1, mask=True, kept=False),
        # a large training batch of packed sequences, E = 256
        dict(name="balance_train_packed", op="balance", dir="fwd", T=32768, E=256, K=8, S=13, mask=True, kept=True),
        # the gradient of the usual layer's batch, experts that fill no warp evenly
        dict(name="balance_grad", op="balance", dir="bwd", T=8192, E=60, K=4, S=5, mask=False, kept=False),
        # the token rows of a decode batch's pairs become the product's operand
        dict(name="mx4_rows", op="quantize", rows=1024, cols=2048, dtype="bf16"),
        # one projection of all experts is laid out once
        dict(name="mx4_weights", op="quantize", rows=98304, cols=2048, dtype="bf16"),
        # gate and up of a decode batch of 128 tokens with 15% of its pairs kept
        dict(name="mx4_gate_up_decode", op="product", N=1024, kept=0.15, E=128, n=768, k=2048, swiglu=True, out="bf16", zipf=1.1),
        # the down projection of a prefill batch of 8192 tokens, every pair kept
        dict(name="mx4_down_prefill", op="product", N=65536, kept=1.0, E=128, n=2048, k=768, swiglu=False, out="f32", zipf=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["enter", "exit", "exit", "balance", "balance", "quantize", "product", "product"])
    if op in ("enter", "exit"):
        d = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, min(16384, 29 * 2 ** 20 // d))
        c = dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "exit":
            c.update(norm=rng.random() < 0.7, gate_c=rng.random() < 0.5, gate_t=rng.random() < 0.5, next=rng.random() < 0.7,
                     a=rng.choice([1.0, 1.0, 0.81]), b=rng.choice([1.0, 0.5, 0.22]))
        return c
    if op == "balance":
        E = rng.choice([8, 16, 60, 64, 128, 256, rng.randint(2, 256)])
        T = _log(rng, 1, 32768)
        mask = rng.random() < 0.6
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, E=E, K=rng.randint(1, min(E, 16)), S=_log(rng, 1, min(T, 64)), mask=mask, kept=mask and rng.random() < 0.5)
    if op == "quantize":
        cols = 32 * _log(rng, 1, 224)
        return dict(op=op, rows=_log(rng, 1, min(98304, 98304 * 2048 // cols)), cols=cols, dtype=rng.choice(["bf16", "f32"]))
    E, n, k = rng.choice([8, 16, 60, 64, 128, 256]), 128 * _log(rng, 1, 24), 128 * _log(rng, 1, 24)
    while E * n * k > 128 * 2048 * 768:
        E, n = max(1, E // 2), max(128, n // 256 * 128)
    N = _log(rng, 1, min(65536, 65536 * 2048 * 768 // (n * k)))
    return dict(op=op, N=N, kept=rng.choice([1.0, 0.6, 0.35, 0.15]), E=E, n=n, k=k, swiglu=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]), zipf=rng.choice([0.0, 0.5, 1.1]))


# ---------------------------------------------------------------- inputs --


def _pairs(c):
    return max(1, int(round(c["kept"] * c["N"])))


def _shares(c):
    """The share of each expert, hottest first."""
    p = [1.0 / (i + 1) ** c["zipf"] for i in range(c["E"])]
    t = sum(p)
    return [v / t for v in p]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = dict(c=c, keep={})
    if c["op"] in ("enter", "exit"):
        T, d, dt = c["T"], c["d"], DT[c["dtype"]]
        # a residual stream: a few channels are far larger than the others
        x = normal(T, d)
        x[:, :: max(8, d // 6)] *= 12.0
        if c["op"] == "enter":
            s.update(x=x.to(dt), w=normal(d, std=0.1, mean=1.0, dtype=dt))
            if c["dir"] == "fwd":
                s.update(n=empty(T, d, dtype=dt))
            else:
                s.update(dn=normal(T, d), dskip=normal(T, d, dtype=dt), dx=empty(T, d, dtype=dt), dw=empty(d))
            return s
        s.update(res=x.to(dt), y=normal(T, d, std=0.3, dtype=dt),
                 w=normal(d, std=0.1, mean=1.0, dtype=dt) if c["norm"] else None,
                 gc=normal(d, std=0.2, mean=0.5, dtype=dt) if c["gate_c"] else None,
                 gt=normal(T, dtype=dt) if c["gate_t"] else None,
                 wn=normal(d, std=0.1, mean=1.0, dtype=dt) if c["next"] else None,
                 out=empty(T, d, dtype=dt), n=empty(T, d, dtype=dt) if c["next"] else None)
        if c["dir"] == "bwd":
            s.update(out=(x + 0.3 * normal(T, d)).to(dt), dout=normal(T, d, dtype=dt), dn=normal(T, d) if c["next"] else None,
                     dres=empty(T, d, dtype=dt), dy=empty(T, d, dtype=dt), dw=empty(d) if c["norm"] else None,
                     dgc=empty(d) if c["gate_c"] else None, dgt=empty(T) if c["gate_t"] else None, dwn=empty(d) if c["next"] else None)
        return s
    if c["op"] == "balance":
        T, E, S = c["T"], c["E"], c["S"]
        lg = normal(T, 2 * E if c["mask"] else E)
        # the router prefers some experts: a Zipf prior over their rank
        lg[:, :E] -= 1.1 * torch.log(torch.randperm(E, generator=g, device="cuda").float() + 1.0)
        cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")).values
        begin = torch.cat([torch.zeros(1, device="cuda"), cuts, torch.full((1,), T, device="cuda")]).to(torch.int32)
        s.update(logits=lg, begin=begin, loss=empty(1), prob=empty(S, E), cand=empty(S, E, dtype=torch.int32), kept=empty(S, E, dtype=torch.int32) if c["mask"] else None)
        if c["dir"] == "bwd":
            s.update(counts=_candidates(lg, c)[0] if not c["kept"] else _candidates(lg, c)[1], dloss=normal(1, std=0.1, mean=1.0), dlogits=empty(T, E))
            s["counts"] = _per_sequence(s["counts"], begin, c)
        return s
    if c["op"] == "quantize":
        x = normal(c["rows"], c["cols"], std=1.0 / math.sqrt(c["cols"]))
        x *= torch.exp(0.5 * normal(c["rows"], 1))
        s.update(x=x.to(DT[c["dtype"]]), codes=empty(c["rows"], c["cols"] // 2, dtype=torch.uint8), scales=empty(c["rows"], c["cols"] // 32, dtype=torch.uint8),
                 values=empty(c["rows"], c["cols"], dtype=torch.bfloat16))
        return s
    N, E, n, k = c["N"], c["E"], c["n"], c["k"]
    p = torch.tensor(_shares(c), device="cuda")[torch.randperm(E, generator=g, device="cuda")]
    counts = torch.bincount(torch.multinomial(p, _pairs(c), replacement=True, generator=g), minlength=E)
    s.update(counts=counts.to(torch.int32), most=int(counts.max()), out=torch.zeros(N, n, dtype=DT[c["out"]], device="cuda"))
    s["a"] = _encode(normal(N, k))
    s["w"] = _encode(normal(E * n, k, std=1.0 / math.sqrt(k)))
    s["w3"] = _encode(normal(E * n, k, std=1.0 / math.sqrt(k))) if c["swiglu"] else None
    # a program lays its weights' scales out once, as the product reads them
    s["tiles"] = [_tiled(v[1]) for v in (s["w"], s["w3"]) if v is not None]
    return s


# ------------------------------------------------------- the plain forms --


def _rstd(x):
    return torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS)


def _enter(s):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    r = _rstd(x)
    if s["c"]["dir"] == "fwd":
        return (x * r * w).to(dt)
    h, dn = x * r, s["dn"]
    dh = dn * w
    dx = s["dskip"].float() + r * (dh - h * (dh * h).mean(dim=1, keepdim=True))
    return dx.to(dt), (dn * h).sum(dim=0)


def _exit(s):
    c, dt = s["c"], s["y"].dtype
    y = s["y"].float()
    ry = _rstd(y) if c["norm"] else 1.0
    h = y * ry
    m = torch.ones(c["d"], device=y.device)
    if c["norm"]:
        m = m * s["w"].float()
    if c["gate_c"]:
        m = m * s["gc"].float()
    sig = torch.sigmoid(s["gt"].float())[:, None] if c["gate_t"] else 1.0
    if c["dir"] == "fwd":
        out = (c["a"] * s["res"].float() + c["b"] * sig * m * h).to(dt)
        if not c["next"]:
            return (out,)
        o = out.float()
        return out, (o * _rstd(o) * s["wn"].float()).to(dt)
    grad, dwn = s["dout"].float(), None
    if c["next"]:
        o = s["out"].float()
        r = _rstd(o)
        ho, dho = o * r, s["dn"] * s["wn"].float()
        grad = grad + r * (dho - ho * (dho * ho).mean(dim=1, keepdim=True))
        dwn = (s["dn"] * ho).sum(dim=0)
    dz = c["b"] * grad * sig
    dh = dz * m
    col = (dz * h).sum(dim=0)
    dot = (dh * h).sum(dim=1, keepdim=True)
    dy = ry * (dh - h * dot / c["d"]) if c["norm"] else dh
    dw = dgc = dgt = None
    if c["norm"]:
        dw = col * s["gc"].float() if c["gate_c"] else col
    if c["gate_c"]:
        dgc = col * s["w"].float() if c["norm"] else col
    if c["gate_t"]:
        dgt = ((1.0 - sig) * dot).reshape(-1)
    return (c["a"] * grad).to(dt), dy.to(dt), [v for v in (dw, dgc, dgt, dwn) if v is not None]


COEF = 0.01


def _candidates(lg, c):
    """[T, E] whole numbers: which experts are a token's K largest (ties to the lower index), and which of them its mask keeps."""
    E = c["E"]
    order = torch.sort(lg[:, :E], dim=1, descending=True, stable=True).indices[:, : c["K"]]
    cand = torch.zeros(lg.shape[0], E, dtype=torch.int32, device=lg.device).scatter_(1, order, 1)
    return cand, cand * (lg[:, E:] >= 0) if c["mask"] else cand


def _sequence_of(begin, T):
    return torch.searchsorted(begin[1:].long(), torch.arange(T, device=begin.device), right=True)


def _per_sequence(v, begin, c):
    zero = torch.zeros(c["S"], c["E"], dtype=v.dtype, device=v.device)
    return zero.index_add_(0, _sequence_of(begin, c["T"]), v)


def _balance(s):
    c, lg = s["c"], s["logits"]
    E = c["E"]
    p = torch.exp(lg[:, :E] - lg[:, :E].max(dim=1, keepdim=True).values)
    p = p / p.sum(dim=1, keepdim=True)
    length = (s["begin"][1:] - s["begin"][:-1]).float()[:, None].clamp(min=1.0)
    if c["dir"] == "fwd":
        cand, kept = (_per_sequence(v, s["begin"], c) for v in _candidates(lg, c))
        # the mean probability is a long sum: 64 bits
        P = _per_sequence(p.double(), s["begin"], c) / length
        f = (kept if c["kept"] else cand) * E / (c["K"] * length)
        loss = ((COEF / c["S"]) * (f * P).sum()).float().reshape(1)
        return (loss, P.float(), cand, kept) if c["mask"] else (loss, P.float(), cand)
    f = s["counts"] * E / (c["K"] * length)
    q = (f / length)[_sequence_of(s["begin"], c["T"])]
    return s["dloss"] * (COEF / c["S"]) * p * (q - (q * p).sum(dim=1, keepdim=True))


def _exponent_and_digits(x):
    """Per 32 values: the shared exponent, the largest one's less 2; and each value's multiple of half of that scale on the 4-bit grid."""
    v = x.float().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(min=-127)  # frexp's fraction lies in [1/2, 1)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    u = torch.ldexp(torch.ldexp(v, -(e // 2)), -(e - e // 2))
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return e, torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)


def _encode(x):
    """(codes [rows, cols / 2], two values a byte, the even one low; scales [rows, cols / 32], exponent + 127)."""
    e, q = _exponent_and_digits(x)
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    code = code.reshape(x.shape[0], -1, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), (e + 127).to(torch.uint8).reshape(x.shape[0], -1)


def _tiled(scales):
    """The scales in tiles of 128 rows by 4 blocks, as the product reads its weights'."""
    t = scales.reshape(scales.shape[0] // 128, 4, 32, scales.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).contiguous().reshape(scales.shape)


def _decode(codes, scales):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], dim=2).reshape(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int()[:, :, None] - 127).reshape(codes.shape[0], -1)


def _quantize(s):
    e, q = _exponent_and_digits(s["x"])
    return torch.ldexp(q, e).reshape(s["x"].shape).to(torch.bfloat16), (e.reshape(e.shape[0], -1) + 127).to(torch.uint8)


def _grouped(a, w, idx, c, most):
    x = torch.zeros(c["E"] * most + 1, c["k"], device=a.device).index_copy_(0, idx, a)
    return torch.bmm(x[:-1].view(c["E"], most, c["k"]), w.view(c["E"], c["n"], c["k"]).transpose(1, 2)).view(-1, c["n"])


def _product(s):
    c, most = s["c"], s["most"]
    end = s["counts"].long().cumsum(0)
    row = torch.arange(c["N"], device=end.device)
    e = torch.searchsorted(end, row, right=True)
    live = e < c["E"]
    first = (end - s["counts"])[e.clamp(max=c["E"] - 1)]
    idx = torch.where(live, e * most + row - first, torch.full_like(e, c["E"] * most))
    a = _decode(*s["a"])
    y = _grouped(a, _decode(*s["w"]), idx, c, most)
    if c["swiglu"]:
        y = y / (1.0 + torch.exp(-y)) * _grouped(a, _decode(*s["w3"]), idx, c, most)
    at = idx.clamp(max=c["E"] * most - 1)
    return torch.where(live[:, None], y[at], torch.zeros((), device=y.device)).to(DT[c["out"]])


# ------------------------------------------------ the library's own calls --


def _own(s):
    from dynamic_expert_routing_router_b200 import abi

    c, keep = s["c"], s["keep"]
    if c["op"] in ("enter", "exit"):
        if not keep:
            keep["dsc"] = abi.block_desc(c["T"], c["d"], c["dtype"], eps=EPS, res_scale=c.get("a", 1.0), branch_scale=c.get("b", 1.0))
            keep["ws"] = abi.alloc_block_workspace(keep["dsc"]) if c["dir"] == "bwd" else None
        dsc, ws = keep["dsc"], keep["ws"]
        if c["op"] == "enter" and c["dir"] == "fwd":
            abi.block_enter(dsc, s["x"], s["w"], s["n"])
            return s["n"]
        if c["op"] == "enter":
            abi.block_enter_backward(dsc, s["x"], s["w"], s["dn"], s["dx"], s["dw"], ws, dskip=s["dskip"])
            return s["dx"], s["dw"]
        if c["dir"] == "fwd":
            abi.block_exit(dsc, s["res"], s["y"], s["out"], w_out=s["w"], gate_c=s["gc"], gate_t=s["gt"], w_next=s["wn"], n_next=s["n"])
            return (s["out"], s["n"]) if c["next"] else (s["out"],)
        abi.block_exit_backward(dsc, s["y"], s["dout"], s["dres"], s["dy"], ws, out=s["out"] if c["next"] else None, dn_next=s["dn"], w_out=s["w"], gate_c=s["gc"],
                                gate_t=s["gt"], w_next=s["wn"], dw_out=s["dw"], dgate_c=s["dgc"], dgate_t=s["dgt"], dw_next=s["dwn"])
        return s["dres"], s["dy"], [v for v in (s["dw"], s["dgc"], s["dgt"], s["dwn"]) if v is not None]
    if c["op"] == "balance":
        if not keep:
            keep["dsc"] = abi.balance_desc(c["T"], c["E"], c["K"], n_seq=c["S"], coef=COEF, has_mask=c["mask"], count_kept=c["kept"])
            keep["ws"] = abi.alloc_balance_workspace(keep["dsc"])
        if c["dir"] == "fwd":
            abi.balance(keep["dsc"], s["logits"], s["loss"], s["cand"], keep["ws"], kept_counts=s["kept"], mean_prob=s["prob"], seq_begin=s["begin"])
            return (s["loss"], s["prob"], s["cand"], s["kept"]) if c["mask"] else (s["loss"], s["prob"], s["cand"])
        abi.balance_backward(keep["dsc"], s["logits"], s["counts"], s["dlogits"], seq_begin=s["begin"], dloss=s["dloss"])
        return s["dlogits"]
    if c["op"] == "quantize":
        abi.mx4_quantize(s["x"], s["codes"], s["scales"])
        abi.mx4_dequantize(s["codes"], s["scales"], s["values"])
        return s["values"], s["scales"]
    if not keep:
        keep["dsc"] = abi.mx4_desc(c["N"], c["E"], c["n"], c["k"], swiglu=c["swiglu"], out=c["out"])
        keep["ws"] = abi.alloc_mx4_workspace(keep["dsc"])
    w3, t3 = (s["w3"][0], s["tiles"][1]) if c["swiglu"] else (None, None)
    abi.mx4_expert_product(keep["dsc"], s["a"][0], s["a"][1], s["counts"], s["w"][0], s["tiles"][0], s["out"], keep["ws"], w3_codes=w3, w3_scales=t3)
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"enter": _enter, "exit": _exit, "balance": _balance, "quantize": _quantize, "product": _product}[state["c"]["op"]](state)


# ------------------------------------------------------------------ work --


def work(case):
    c = case
    if c["op"] in ("enter", "exit"):
        b, v = (2 if c["dtype"] == "bf16" else 4), c["T"] * c["d"]
        if c["op"] == "enter":
            if c["dir"] == "fwd":
                return {"bytes": 2 * b * v + b * c["d"], "flops": 5 * v}
            return {"bytes": (3 * b + 4) * v + (b + 4) * c["d"], "flops": 12 * v}
        cols = sum(c[k] for k in ("norm", "gate_c", "next"))
        if c["dir"] == "fwd":
            return {"bytes": (3 + c["next"]) * b * v + b * (cols * c["d"] + c["gate_t"] * c["T"]), "flops": (6 + 4 * c["norm"] + 4 * c["next"]) * v}
        return {"bytes": (4 * b + (b + 4) * c["next"]) * v + (b + 4) * (cols * c["d"] + c["gate_t"] * c["T"]), "flops": (10 + 6 * c["norm"] + 10 * c["next"]) * v}
    if c["op"] == "balance":
        v, se = c["T"] * c["E"], c["S"] * c["E"]
        if c["dir"] == "fwd":
            return {"bytes": 4 * v * (2 if c["mask"] else 1) + 4 * se * (3 if c["mask"] else 2), "flops": 4 * v + c["T"] * c["K"]}
        return {"bytes": 8 * v + 4 * se, "flops": 8 * v}
    if c["op"] == "quantize":
        v = c["rows"] * c["cols"]
        # the values, then codes and scales out, and the values they stand for
        return {"bytes": v * (2 if c["dtype"] == "bf16" else 4) + v // 2 + v // 32 + 2 * v, "flops": 4 * v}
    P = _pairs(c)
    touched = sum(1.0 - (1.0 - p) ** P for p in _shares(c))
    mats = 2 if c["swiglu"] else 1
    weights = touched * c["n"] * c["k"] * (0.5 + 1 / 32) * mats
    return {"bytes": int(weights + P * c["k"] * (0.5 + 1 / 32) + P * c["n"] * (2 if c["out"] == "bf16" else 4)), "flops": 2 * P * c["n"] * c["k"] * mats}


# ----------------------------------------------------------------- exact --


def _x_norm(x):
    rms = (x.pow(2).sum(1) / x.shape[1] + EPS).sqrt()
    return x / rms[:, None], rms


def _x_norm_grad(hat, rms, g):
    """The gradient of the rows from that of the normed rows."""
    return (g - hat * ((g * hat).sum(1) / g.shape[1])[:, None]) / rms[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    D = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    if c["op"] == "enter":
        hat, rms = _x_norm(D["x"])
        if c["dir"] == "fwd":
            return hat * D["w"]
        return D["dskip"] + _x_norm_grad(hat, rms, D["dn"] * D["w"]), torch.einsum("td,td->d", D["dn"], hat)
    if c["op"] == "exit":
        one = torch.ones((), dtype=torch.float64, device="cuda")
        hat, rms = _x_norm(D["y"]) if c["norm"] else (D["y"], None)
        w = D["w"] if c["norm"] else one
        gc = D["gc"] if c["gate_c"] else one
        gate = (1 / (1 + (-D["gt"]).exp()))[:, None] if c["gate_t"] else one
        if c["dir"] == "fwd":
            full = c["a"] * D["res"] + c["b"] * (gate * gc) * (w * hat)
            if not c["next"]:
                return (full,)
            # the next norm reads the rows as they are stored
            return full, _x_norm(full.to(s["out"].dtype).double())[0] * D["wn"]
        up, more = D["dout"], []
        if c["next"]:
            nh, nr = _x_norm(D["out"])
            up = up + _x_norm_grad(nh, nr, D["dn"] * D["wn"])
            more = [torch.einsum("td,td->d", D["dn"], nh)]
        branch = c["b"] * up
        to_hat = branch * gate * gc * w
        dy = _x_norm_grad(hat, rms, to_hat) if c["norm"] else to_hat
        grads = [(branch * gate * gc * hat).sum(0)] if c["norm"] else []
        grads += [(branch * gate * w * hat).sum(0)] if c["gate_c"] else []
        grads += [(branch * gc * w * hat).sum(1) * (gate * (1 - gate))[:, 0]] if c["gate_t"] else []
        return c["a"] * up, dy, grads + more
    if c["op"] == "balance":
        E, b = c["E"], [int(v) for v in s["begin"]]
        lg = D["logits"][:, :E]
        prob = torch.softmax(lg, dim=1)
        if c["dir"] == "fwd":
            loss, P = 0.0, torch.zeros(c["S"], E, dtype=torch.float64, device="cuda")
            ranked = torch.argsort(lg, dim=1, descending=True, stable=True)[:, : c["K"]]
            used = torch.zeros_like(lg, dtype=torch.bool).scatter_(1, ranked, True)
            if c["kept"]:
                used &= D["logits"][:, E:] >= 0
            for q, (lo, hi) in enumerate(zip(b[:-1], b[1:])):
                if hi > lo:
                    P[q] = prob[lo:hi].mean(0)
                    loss = loss + (P[q] * used[lo:hi].double().mean(0) * E / c["K"]).sum()
            loss = (COEF * loss / c["S"]).reshape(1)
            return (loss, P, None, None) if c["mask"] else (loss, P, None)
        out = torch.zeros_like(lg)
        for q, (lo, hi) in enumerate(zip(b[:-1], b[1:])):
            if hi > lo:
                f = s["counts"][q].double() * E / (c["K"] * (hi - lo))
                p = prob[lo:hi]
                out[lo:hi] = D["dloss"] * COEF / c["S"] / (hi - lo) * (p * f - p * (p @ f)[:, None])
        return out
    if c["op"] == "quantize":
        x = D["x"].view(c["rows"], -1, 32)
        top = x.abs().max(2, keepdim=True).values
        scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2)
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        mid = (grid[1:] + grid[:-1]) / 2
        a = (x / scale).abs().contiguous()
        # to the nearest of the grid; a tie goes to the even digit
        up, down = torch.bucketize(a, mid, right=True), torch.bucketize(a, mid, right=False)
        near = torch.where(up % 2 == 0, up, down)
        return (grid[near] * scale * torch.sign(x)).view(c["rows"], c["cols"]), None
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def matrix(pair):
        codes, scales = pair
        nib = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.long, device="cuda")
        nib[:, 0::2], nib[:, 1::2] = codes % 16, codes // 16
        v = torch.where(nib < 8, 1.0, -1.0).double() * grid[nib % 8]
        return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)

    out = torch.zeros(c["N"], c["n"], dtype=torch.float64, device="cuda")
    a, w = matrix(s["a"]), matrix(s["w"]).view(c["E"], c["n"], c["k"])
    w3 = matrix(s["w3"]).view(c["E"], c["n"], c["k"]) if c["swiglu"] else None
    row = 0
    for e, m in enumerate(s["counts"].tolist()):
        if m:
            y = a[row:row + m] @ w[e].T
            out[row:row + m] = y * torch.sigmoid(y) * (a[row:row + m] @ w3[e].T) if c["swiglu"] else y
            row += m
    return out
