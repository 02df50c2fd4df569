"""The residual block's operators (norm in front of the layer, norm, gates,
residual and next norm behind it) on the GPU, forward and backward, against
the formulas in 64 bits, and their gradients against differences.

Bars, with u = 2^-24 (half a step of fp32) and h = eps/2 of the stored type
(half a step: bf16 2^-8, fp32 2^-24).  A row sum of squares runs over at most
32 terms per thread, 5 shuffles and 16 warps, so it is off by at most 54 u of
itself and its root by half of that; the reciprocal root adds 4 u (2 ulp) and
each product u: 40 u for a normed value.  Signed row sums are off by 54 u of
the sum of magnitudes.  The logistic function adds 10 u (exp 2 ulp = 4 u, a
sum, a quotient).  Every result is then stored with one rounding, h.  Sums of
over T rows add a chain of at most T / 148 + 15 + 8 + 19 further terms.
"""
import pytest
import torch

from dynamic_expert_routing_router_b200 import abi

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IDS = ["bf16", "f32"]


def half_step(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def draw(T, d, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def r(*s, std=1.0, mean=0.0, dt=None):
        return (torch.randn(*s, generator=g, device=DEV) * std + mean).to(dt or TYPES[dtype])
    f32 = torch.float32
    return dict(x=r(T, d) * 3, y=r(T, d, std=0.3), w=r(d, std=0.2, mean=1), gc=r(d, std=0.3, mean=0.5),
                gt=r(T, std=2), wn=r(d, std=0.2, mean=1), dout=r(T, d), dn=r(T, d, dt=f32))


def full(*s, dt=torch.float32):
    return torch.full(s, float("nan"), dtype=dt, device=DEV)


def near(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all() == torch.isfinite(ref).all(), what
    bad = (got - ref).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           float(((got - ref).abs() / tol.clamp(min=1e-300)).max()))


def D(v):
    return v.double()


def rms(x, eps=EPS):
    return (x.square().mean(1, keepdim=True) + eps).sqrt()


SIZES = [(1, 8), (3, 256), (150, 1000), (17, 2048), (9, 4104), (5, 8192), (3, 16384), (700, 2048)]
PARTS = [(1, 1, 1, 1), (1, 0, 0, 1), (0, 0, 0, 1), (0, 1, 0, 0), (1, 0, 1, 0), (0, 0, 0, 0)]


@pytest.mark.parametrize("dtype", IDS)
@pytest.mark.parametrize("T,d", SIZES)
def test_enter_and_its_gradient(T, d, dtype):
    s, h = draw(T, d, dtype, T + d), half_step(dtype)
    dsc = abi.block_desc(T, d, dtype, eps=EPS)
    n, dx, dw = full(T, d, dt=TYPES[dtype]), full(T, d, dt=TYPES[dtype]), full(d)
    abi.block_enter(dsc, s["x"], s["w"], n)
    x, w = D(s["x"]), D(s["w"])
    r = rms(x)
    ref = x / r * w
    near(n, ref, (h + 41 * U) * ref.abs() * 1.01 + 1e-37, "n")
    ws = abi.alloc_block_workspace(dsc)
    for dskip in (None, s["dout"]):
        abi.block_enter_backward(dsc, s["x"], s["w"], s["dn"], dx, dw, ws, dskip=dskip)
        p, o = D(s["dn"]) * w, x / r
        ref = (p - o * (p * o).mean(1, keepdim=True)) / r
        mag = (p.abs() + o.abs() * (p * o).abs().mean(1, keepdim=True)) / r
        if dskip is not None:
            ref, mag = ref + D(dskip), mag + D(dskip).abs()
        near(dx, ref, h * ref.abs() * 1.01 + 160 * U * mag, "dx")
        terms = D(s["dn"]) * o
        near(dw, terms.sum(0), (100 + T / 148) * U * terms.abs().sum(0), "dw")


def exit_reference(s, parts, a, b, out):
    """(out, tol), gradients and their tolerances in 64 bits."""
    norm, gate_c, gate_t, nxt = parts
    y, d = D(s["y"]), s["y"].shape[1]
    ry = rms(y) if norm else torch.ones(y.shape[0], 1, dtype=torch.float64, device=DEV)
    hat = y / ry
    m = torch.ones(d, dtype=torch.float64, device=DEV)
    m = m * D(s["w"]) if norm else m
    m = m * D(s["gc"]) if gate_c else m
    sig = torch.sigmoid(D(s["gt"]))[:, None] if gate_t else torch.ones_like(ry)
    branch = b * sig * m * hat
    ref = dict(out=a * D(s["x"]) + branch)
    tol = dict(out=60 * U * ((a * D(s["x"])).abs() + branch.abs()))
    g, mag = D(s["dout"]), D(s["dout"]).abs()
    if nxt:
        o = D(out)
        ro = rms(o)
        oh, p = o / ro, D(s["dn"]) * D(s["wn"])
        ref["n"] = oh * D(s["wn"])
        tol["n"] = 41 * U * ref["n"].abs()
        g = g + (p - oh * (p * oh).mean(1, keepdim=True)) / ro
        mag = mag + (p.abs() + oh.abs() * (p * oh).abs().mean(1, keepdim=True)) / ro
        ref["dwn"], tol["dwn"] = (D(s["dn"]) * oh).sum(0), (D(s["dn"]) * oh).abs().sum(0)
    ref["dres"], tol["dres"] = a * g, 160 * U * abs(a) * mag
    dz, magz = b * sig * g, abs(b) * sig * mag
    dot = (dz * m * hat).sum(1, keepdim=True)
    adot = (magz * (m * hat).abs()).sum(1, keepdim=True)
    ref["dy"] = (dz * m - hat * dot / d) / ry if norm else dz * m
    tol["dy"] = 320 * U * (magz * m.abs() + (hat.abs() * adot / d if norm else 0.0)) / ry
    terms, aterms = dz * hat, magz * hat.abs()
    one = torch.ones((), dtype=torch.float64, device=DEV)
    if norm:
        c = D(s["gc"]) if gate_c else one
        ref["dw"], tol["dw"] = c * terms.sum(0), c.abs() * aterms.sum(0)
    if gate_c:
        c = D(s["w"]) if norm else one
        ref["dgc"], tol["dgc"] = c * terms.sum(0), c.abs() * aterms.sum(0)
    if gate_t:
        rest = torch.sigmoid(-D(s["gt"]))
        ref["dgt"], tol["dgt"] = rest * dot[:, 0], 320 * U * rest * adot[:, 0]
    chain = (320 + s["y"].shape[0] / 148) * U
    for k in ("dw", "dgc", "dwn"):
        if k in tol:
            tol[k] = tol[k] * chain
    return ref, tol


def run_exit(s, parts, a, b, dtype, stream=None):
    norm, gate_c, gate_t, nxt = parts
    T, d = s["y"].shape
    dt, dsc = TYPES[dtype], abi.block_desc(T, d, dtype, eps=EPS, res_scale=a, branch_scale=b)
    pick = dict(w_out=s["w"] if norm else None, gate_c=s["gc"] if gate_c else None,
                gate_t=s["gt"] if gate_t else None, w_next=s["wn"] if nxt else None)
    out, n = full(T, d, dt=dt), full(T, d, dt=dt) if nxt else None
    abi.block_exit(dsc, s["x"], s["y"], out, n_next=n, stream=stream, **pick)
    g = dict(dres=full(T, d, dt=dt), dy=full(T, d, dt=dt), dw=full(d) if norm else None,
             dgc=full(d) if gate_c else None, dgt=full(T) if gate_t else None,
             dwn=full(d) if nxt else None)
    abi.block_exit_backward(dsc, s["y"], s["dout"], g["dres"], g["dy"],
                            abi.alloc_block_workspace(dsc), out=out if nxt else None,
                            dn_next=s["dn"] if nxt else None, dw_out=g["dw"], dgate_c=g["dgc"],
                            dgate_t=g["dgt"], dw_next=g["dwn"], stream=stream, **pick)
    return dict(g, out=out, n=n)


@pytest.mark.parametrize("dtype", IDS)
@pytest.mark.parametrize("parts", PARTS, ids=["".join(map(str, p)) for p in PARTS])
@pytest.mark.parametrize("T,d", SIZES)
def test_exit_and_its_gradients(T, d, parts, dtype):
    s, h = draw(T, d, dtype, 7 * T + d), half_step(dtype)
    a, b = (1.0, 1.0) if T % 2 else (0.81, -0.25)
    got = run_exit(s, parts, a, b, dtype)
    ref, tol = exit_reference(s, parts, a, b, got["out"])
    assert {k for k, v in got.items() if v is not None} == set(ref)
    for k in ref:
        stored = h * ref[k].abs() * 1.01 if k in ("out", "n", "dres", "dy") else 0.0
        near(got[k], ref[k], stored + 1.01 * tol[k] + 1e-37, k)


def test_gradients_are_the_differences_of_the_forward():
    """<gradient, direction> against the central difference of
    <dout, out> + <dn, n> along it, the outputs of fp32 rows.

    Bar: outputs are off by 101 u of their magnitudes (above), at each end;
    with step t the difference quotient is off by that over t, and by t^2
    times a third derivative; the directions are of the inputs' own size and
    the functions smooth on that scale (the third derivative is of the order
    of the function's magnitude): t = 2^-8 gives 2 * 101 * 2^-24 * 2^8 + 2^-16
    = 0.31 % of sum |dout| |out| + |dn| |n|."""
    T, d, dtype = 6, 256, "f32"
    s = draw(T, d, dtype, 3)
    parts, a, b = (1, 1, 1, 1), 0.9, 0.7
    got = run_exit(s, parts, a, b, dtype)
    grads = dict(x=got["dres"], y=got["dy"], w=got["dw"], gc=got["dgc"], gt=got["dgt"], wn=got["dwn"])
    gen = torch.Generator(device=DEV).manual_seed(9)
    size = float((D(s["dout"]) * D(got["out"])).abs().sum() + (D(s["dn"]) * D(got["n"])).abs().sum())
    t = 2.0 ** -8
    for k, grad in grads.items():
        v = torch.randn(s[k].shape, generator=gen, device=DEV) * s[k].abs().mean()
        ends = []
        for sign in (1, -1):
            e = run_exit(dict(s, **{k: s[k] + sign * t * v}), parts, a, b, dtype)
            ends.append(float((D(s["dout"]) * D(e["out"])).sum() + (D(s["dn"]) * D(e["n"])).sum()))
        diff, want = (ends[0] - ends[1]) / (2 * t), float((D(grad) * D(v)).sum())
        assert abs(diff - want) <= 0.0031 * size, (k, diff, want, size)


def test_saturated_gates_keep_their_gradient():
    """A gate's slope s (1 - s) where s is 1 up to fp32's last bit, and where
    it is almost 0: relative to itself (320 u, as in the bars above)."""
    T, d = 8, 64
    s = draw(T, d, "f32", 1)
    s["gt"] = torch.tensor([12.0, 17.0, 30.0, -12.0, -30.0, 80.0, -80.0, 0.0], device=DEV)
    got = run_exit(s, (1, 0, 1, 0), 1.0, 1.0, "f32")
    ref, tol = exit_reference(s, (1, 0, 1, 0), 1.0, 1.0, None)
    near(got["dgt"], ref["dgt"], 1.01 * tol["dgt"], "dgt")
    assert (got["dgt"][:3] != 0).all()


@pytest.mark.parametrize("scale", [0.0, 1e-13, 1e15], ids=["zero", "tiny", "huge"])
def test_rows_far_from_one(scale):
    """Rows of zeros (r = 1 / sqrt(eps)), rows whose square sum is far below
    eps, and rows whose squares are large: finite, and as the formula."""
    T, d = 4, 512
    s = draw(T, d, "f32", 2)
    s["x"] = s["x"] * scale
    dsc = abi.block_desc(T, d, "f32", eps=1e-30)
    n, dx, dw = full(T, d), full(T, d), full(d)
    abi.block_enter(dsc, s["x"], s["w"], n)
    abi.block_enter_backward(dsc, s["x"], s["w"], s["dn"], dx, dw, abi.alloc_block_workspace(dsc))
    x, w = D(s["x"]), D(s["w"])
    r = (x.square().mean(1, keepdim=True) + D(torch.tensor(1e-30, device=DEV))).sqrt()
    o, p = x / r, D(s["dn"]) * w
    near(n, o * w, 42 * U * (o * w).abs() + 1e-37, "n")
    ref = (p - o * (p * o).mean(1, keepdim=True)) / r
    mag = (p.abs() + o.abs() * (p * o).abs().mean(1, keepdim=True)) / r
    near(dx, ref, 162 * U * mag + 1e-37, "dx")


def test_a_bad_row_stays_in_its_row():
    s = draw(40, 1024, "bf16", 5)
    clean = run_exit(s, (1, 1, 1, 1), 1.0, 0.5, "bf16")
    s2 = dict(s, y=s["y"].clone(), x=s["x"].clone())
    s2["y"][7, 3], s2["x"][11, 1000] = float("nan"), float("inf")
    got = run_exit(s2, (1, 1, 1, 1), 1.0, 0.5, "bf16")
    rows = [t for t in range(40) if t not in (7, 11)]
    for k in ("out", "n", "dres", "dy", "dgt"):
        assert torch.equal(got[k][rows], clean[k][rows]), k
    assert torch.isnan(got["out"][7]).all() and torch.isnan(got["n"][11, 1000])


@pytest.mark.parametrize("dtype", IDS)
def test_outputs_over_inputs_accumulation_and_repetition(dtype):
    """Every output in an input's buffer gives the same bits, accumulate adds,
    and a second run repeats the first."""
    T, d, dt = 333, 1536, TYPES[dtype]
    s = draw(T, d, dtype, 8)
    parts = (1, 1, 1, 1)
    one = run_exit(s, parts, 1.0, 0.5, dtype)
    two = run_exit(s, parts, 1.0, 0.5, dtype)
    for k in one:
        assert torch.equal(one[k], two[k]), k
    dsc = abi.block_desc(T, d, dtype, eps=EPS, branch_scale=0.5, accumulate=True)
    res, y = s["x"].clone(), s["y"].clone()
    pick = dict(w_out=s["w"], gate_c=s["gc"], gate_t=s["gt"], w_next=s["wn"])
    abi.block_exit(dsc, res, y, res, n_next=y, **pick)
    assert torch.equal(res, one["out"]) and torch.equal(y, one["n"])
    y, dout = s["y"].clone(), s["dout"].clone()
    acc = dict(dw_out=one["dw"].clone(), dgate_c=one["dgc"].clone(), dw_next=one["dwn"].clone())
    dgt = full(T)
    abi.block_exit_backward(dsc, y, dout, dout, y, abi.alloc_block_workspace(dsc), out=one["out"],
                            dn_next=s["dn"], dgate_t=dgt, **acc, **pick)
    assert torch.equal(dout, one["dres"]) and torch.equal(y, one["dy"]) and torch.equal(dgt, one["dgt"])
    for k, g in (("dw_out", "dw"), ("dgate_c", "dgc"), ("dw_next", "dwn")):
        assert torch.equal(acc[k], 2 * one[g]), k
    x, dskip, dw = s["x"].clone(), s["dout"].clone(), torch.zeros(d, device=DEV)
    n, dx = full(T, d, dt=dt), full(T, d, dt=dt)
    ws = abi.alloc_block_workspace(dsc)
    abi.block_enter(dsc, s["x"], s["w"], n)
    abi.block_enter_backward(dsc, s["x"], s["w"], s["dn"], dx, dw, ws, dskip=s["dout"])
    abi.block_enter_backward(dsc, s["x"], s["w"], s["dn"], dskip, dw, ws, dskip=dskip)
    assert torch.equal(dskip, dx)
    abi.block_enter(dsc, x, s["w"], x)
    assert torch.equal(x, n)


def test_no_rows():
    d = 256
    for acc in (False, True):
        dsc = abi.block_desc(0, d, "bf16", accumulate=acc)
        z = torch.empty(0, d, dtype=torch.bfloat16, device=DEV)
        z32, zt = torch.empty(0, d, device=DEV), torch.empty(0, device=DEV)
        w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
        ws = abi.alloc_block_workspace(dsc)
        g = [torch.full((d,), 3.0, device=DEV) for _ in range(3)]
        abi.block_enter(dsc, z, w, z)
        abi.block_exit(dsc, z, z, z, w_out=w, gate_t=zt.to(torch.bfloat16), w_next=w, n_next=z)
        abi.block_enter_backward(dsc, z, w, z32, z, g[0], ws)
        abi.block_exit_backward(dsc, z, z, z, z, ws, out=z, dn_next=z32, w_out=w, dw_out=g[1],
                                w_next=w, dw_next=g[2], gate_t=zt.to(torch.bfloat16), dgate_t=zt)
        assert all((v == (3.0 if acc else 0.0)).all() for v in g)


def test_another_stream_and_a_captured_graph():
    """The calls follow the stream they are given, and a captured pair of them
    replays on new data."""
    T, d = 64, 2048
    s = draw(T, d, "bf16", 4)
    want = run_exit(s, (1, 1, 1, 1), 1.0, 1.0, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_exit(s, (1, 1, 1, 1), 1.0, 1.0, "bf16")
    side.synchronize()
    got2 = run_exit(s, (1, 1, 1, 1), 1.0, 1.0, "bf16", stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]) and torch.equal(got2[k], want[k]), k
    dsc, ws = abi.block_desc(T, d), abi.alloc_block_workspace(abi.block_desc(T, d))
    n, dx, dw = full(T, d, dt=torch.bfloat16), full(T, d, dt=torch.bfloat16), full(d)
    x = s["x"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.block_enter(dsc, x, s["w"], n)
        abi.block_enter_backward(dsc, x, s["w"], s["dn"], dx, dw, ws)
    x.copy_(s["y"])
    graph.replay()
    e = [full(T, d, dt=torch.bfloat16), full(T, d, dt=torch.bfloat16), full(d)]
    abi.block_enter(dsc, s["y"], s["w"], e[0])
    abi.block_enter_backward(dsc, s["y"], s["w"], s["dn"], e[1], e[2], abi.alloc_block_workspace(dsc))
    torch.cuda.synchronize()
    for a, b in zip((n, dx, dw), e):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows are those of a small call."""
    T, d = 270_000, 8192
    s = draw(3, d, "bf16", 4)
    x = torch.ones(T, d, dtype=torch.bfloat16, device=DEV)
    x[-3:] = s["x"]
    n = torch.empty_like(x)
    abi.block_enter(abi.block_desc(T, d), x, s["w"], n)
    ref = torch.empty_like(s["x"])
    abi.block_enter(abi.block_desc(3, d), s["x"], s["w"], ref)
    assert torch.equal(n[-3:], ref)
    dsc = abi.block_desc(T, d)
    dn = torch.zeros(T, d, device=DEV)
    dn[-3:] = s["dn"]
    dw, ws = full(d), abi.alloc_block_workspace(dsc)
    abi.block_enter_backward(dsc, x, s["w"], dn, n, dw, ws)
    small, dws = abi.block_desc(3, d), full(d)
    abi.block_enter_backward(small, s["x"], s["w"], s["dn"], ref, dws, abi.alloc_block_workspace(small))
    assert torch.equal(n[-3:], ref) and (n[:-3] == 0).all()
    # the same three rows' terms, all others zeros, in another order: 3 roundings
    assert ((dw - dws).abs() <= 3 * U * (s["dn"] * 100).abs().sum(0)).all()
