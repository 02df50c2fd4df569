"""The residual block as it is used: norm, layer, balance loss, gates, residual
and next norm, forward and backward, and served with 4-bit experts.

The pieces have tests of their own; here they run together.  Forward: every
stage against the formula in 64 bits from the block's own input of that stage.
Gradients: against differences of the whole forward.
"""
import numpy as np
import pytest
import torch

from dynamic_expert_routing_router_b200 import abi, block, inputs

from _parity import gpu_forward, gpu_route
from test_gpu_mx4 import plain_quantize, plain_values, tile_scales

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16 = torch.bfloat16


def parts(T, sh, dtype, masked, seed, **kw):
    t = BF16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device=DEV).manual_seed(seed)

    def r(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g, device=DEV) * std + mean).to(t)
    W = [w.to(t) for w in inputs.make_experts(sh, seed=seed, device=DEV)]
    Wg = inputs.make_gate(sh, seed=seed, device=DEV).to(t)
    Wm = inputs.make_mask(sh, 0.5, seed=seed, device=DEV).to(t) if masked else None
    v = dict(x=r(T, sh.d, std=2.0), dout=r(T, sh.d), gt=r(T), w_next=r(sh.d, std=0.1, mean=1),
             dn=torch.randn(T, sh.d, generator=g, device=DEV),
             w_in=r(sh.d, std=0.1, mean=1), w_out=r(sh.d, std=0.1, mean=1), gc=r(sh.d, std=0.2, mean=0.7))
    b = block.MoeBlock(T, sh.d, sh.E, sh.I, sh.K, sh.renorm, Wg, Wm, *W, v["w_in"], v["w_out"], v["gc"],
                       dtype=dtype, **kw)
    return b, v, (Wg, Wm, *W)


def step(b, v, w, loss_grad=None, seq=None, back=True):
    """One forward (and backward) with every part; fresh outputs."""
    out, n = torch.empty_like(v["x"]), torch.empty_like(v["x"])
    b.forward(v["x"], out, gate_t=v["gt"], w_next=v["w_next"], n_next=n, seq_begin=seq)
    got = dict(out=out, n_next=n, loss=b.loss.clone())
    if back:
        b.zero_grad()
        dx, dgt = torch.empty_like(v["x"]), torch.empty(v["x"].shape[0], device=DEV)
        dwn = torch.zeros(v["x"].shape[1], device=DEV)
        b.backward(v["x"], out, v["dout"], dx, gate_t=v["gt"], dgate_t=dgt, w_next=v["w_next"], dn_next=v["dn"],
                   dw_next=dwn, seq_begin=seq, dloss=loss_grad)
        got.update(dx=dx, dgt=dgt, dwn=dwn, **{"d" + k: g.clone() for k, g in b.grads.items() if g is not None})
    b.check()
    return got


def rms(x, eps=1e-6):
    return (x.square().mean(1, keepdim=True) + eps).sqrt()


@pytest.mark.parametrize("T", [1, 5, 130])
def test_forward_is_its_stages(T):
    """enter, the layer on its rows, exit: one rounding (2^-8) each and 60 u."""
    sh = inputs.Shape(256, 16, 4, 256, 1, "bf16")
    b, v, W = parts(T, sh, "bf16", True, T, res_scale=0.9, branch_scale=0.5)
    got = step(b, v, W, back=False)
    x, h = v["x"].double(), 2.0 ** -8
    n = x / rms(x) * v["w_in"].double()
    assert ((b.n.double() - n).abs() <= (h + 42 * U) * n.abs() + 1e-37).all()
    layer, _ = gpu_forward(abi.desc(T, sh.d, sh.E, sh.I, sh.K, "bf16", 1), b.n, *W)
    assert torch.equal(layer, b.y)  # the layer keeps its results
    y = b.y.double()
    branch = 0.5 * torch.sigmoid(v["gt"].double())[:, None] * v["gc"].double() * v["w_out"].double() * y / rms(y)
    out = 0.9 * x + branch
    tol = h * out.abs() * 1.01 + 60 * U * (x.abs() + branch.abs()) + 1e-37
    assert ((got["out"].double() - out).abs() <= tol).all()
    o = got["out"].double()
    nn = o / rms(o) * v["w_next"].double()
    assert ((got["n_next"].double() - nn).abs() <= (h + 42 * U) * nn.abs() + 1e-37).all()


def test_gradients_are_the_differences_of_the_block():
    """An fp32 block without a mask (whose estimator is no derivative): the
    change of <dout, out> + <dn, n_next> + dloss loss along the gradient's own
    signs, per input and weight.

    Bar: outputs are off by at most (d + I + 500) u of their magnitudes' sum M
    (dot products over d = 128 and I = 128 and the norms' bars), so the quotient
    by 2 t with t = 2^-9 s, s the input's mean magnitude, by 756 u 2^9 M = 2.4 %
    of M, against a change of sum |g| s that is larger than M for the rows and
    of its order for the weights; the third derivative's share is of the order
    of t^2 = 2^-18.  No candidate changes over the step (checked)."""
    sh = inputs.Shape(128, 8, 2, 128, 1, "f32")
    T, seq = 12, torch.tensor([0, 5, 12], dtype=torch.int32, device=DEV)
    b, v, W = parts(T, sh, "f32", False, 3, balance=0.5, n_seq=2, train=True)
    dl = torch.tensor([2.0], device=DEV)
    base = step(b, v, W, dl, seq)
    cand = b.cand.clone()

    def total(g):
        return float((v["dout"].double() * g["out"].double()).sum() + (v["dn"].double() * g["n_next"].double()).sum()
                     + 2.0 * g["loss"].double().sum())
    M = float((v["dout"].double() * base["out"].double()).abs().sum()
              + (v["dn"].double() * base["n_next"].double()).abs().sum())
    tensors = dict(dx=v["x"], dgt=v["gt"], dwn=v["w_next"], dw_in=b.w_in, dw_out=b.w_out, dgate_c=b.gate_c,
                   dW_gate=b.layer[0], dW1=b.layer[2], dW3=b.layer[3], dW2=b.layer[4])
    for k, t in tensors.items():
        g, keep = base[k].double(), t.clone()
        s = float(keep.abs().mean())
        h = 2.0 ** -9 * s
        ends = []
        for sign in (1.0, -1.0):
            t.copy_(keep + sign * h * torch.sign(g).to(t.dtype))
            ends.append(total(step(b, v, W, dl, seq, back=False)))
            assert torch.equal(b.cand, cand), k
        t.copy_(keep)
        diff, want = (ends[0] - ends[1]) / (2 * h), float(g.abs().sum())
        assert abs(diff - want) * s <= 0.024 * M + 1e-4 * want * s, (k, diff * s, want * s, M)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step_is_its_pieces_and_replays(dtype):
    """Masked, with the kept experts' balance loss: the gradients are those of
    the pieces called one by one, two runs agree bit for bit, gradients add up
    over steps, and a captured step replays on new rows."""
    sh = inputs.Shape(256, 16, 4, 256, 1, dtype)
    T, seq = 40, torch.tensor([0, 1, 40], dtype=torch.int32, device=DEV)
    b, v, W = parts(T, sh, dtype, True, 5, balance=0.1, n_seq=2, count_kept=True, beta=0.01, train=True)
    dl = torch.tensor([0.7], device=DEV)
    one, two = step(b, v, W, dl, seq), step(b, v, W, dl, seq)
    for k in one:
        assert torch.equal(one[k], two[k]), k
    assert int(b.cand.sum()) == T * sh.K and int(b.kept.sum()) < T * sh.K
    # the pieces
    e = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    z = lambda w: torch.zeros(w.shape, device=DEV)  # noqa: E731
    dres, dy, dgt = torch.empty_like(v["x"]), torch.empty_like(v["x"]), e(T)
    bd = abi.block_desc(T, sh.d, dtype)
    bw = abi.alloc_block_workspace(bd)
    gw, gc, gn = e(sh.d), e(sh.d), e(sh.d)
    abi.block_exit_backward(bd, b.y, v["dout"], dres, dy, bw, out=one["out"], dn_next=v["dn"], w_out=b.w_out,
                            gate_c=b.gate_c, gate_t=v["gt"], w_next=v["w_next"], dw_out=gw, dgate_c=gc, dgate_t=dgt,
                            dw_next=gn)
    rt = gpu_route(abi.desc(T, sh.d, sh.E, sh.I, sh.K, dtype, 1), b.n, W[0], W[1])
    lg = torch.as_tensor(rt["logits"], device=DEV)
    dlog = e(T, sh.E)
    abi.balance_backward(b.bal, lg, b.kept, dlog, seq_begin=seq, dloss=dl)
    dn, dW = e(T, sh.d), [z(w) for w in W]
    ld = abi.desc(T, sh.d, sh.E, sh.I, sh.K, dtype, 1)
    abi.backward(ld, b.n, *W, dy, 0.01, dn, *dW, abi.alloc_backward_workspace(ld, DEV), dlogits=dlog)
    dx, gi = torch.empty_like(v["x"]), e(sh.d)
    abi.block_enter_backward(bd, v["x"], b.w_in, dn, dx, gi, bw, dskip=dres)
    for k, want in dict(dx=dx, dgt=dgt, dwn=gn, dw_out=gw, dgate_c=gc, dw_in=gi, dW_gate=dW[0], dW_mask=dW[1],
                        dW1=dW[2], dW3=dW[3], dW2=dW[4]).items():
        assert torch.equal(one[k], want), k
    # two steps without zeroing: twice the gradients
    sink = torch.empty_like(v["x"])
    b.backward(v["x"], one["out"], v["dout"], sink, gate_t=v["gt"], dgate_t=dgt, w_next=v["w_next"], dn_next=v["dn"],
               dw_next=gn, seq_begin=seq, dloss=dl)
    for k, g in b.grads.items():
        assert torch.equal(g, 2 * one["d" + k]), k
    # a captured step on other rows
    keep = v["x"].clone()
    out, n, dx2 = (torch.empty_like(keep) for _ in range(3))
    b.zero_grad()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(v["x"], out, gate_t=v["gt"], w_next=v["w_next"], n_next=n, seq_begin=seq)
        b.backward(v["x"], out, v["dout"], dx2, gate_t=v["gt"], dgate_t=dgt, w_next=v["w_next"], dn_next=v["dn"],
                   dw_next=gn, seq_begin=seq, dloss=dl)
    v["x"].copy_(keep.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    replayed = dict(out=out.clone(), n_next=n.clone(), dx=dx2.clone(), **{"d" + k: g.clone() for k, g in b.grads.items()})
    eager = step(b, v, W, dl, seq)
    for k, want in replayed.items():
        assert torch.equal(eager[k], want), k


@pytest.mark.parametrize("T,masked", [(1, True), (7, True), (130, True), (33, False)])
def test_served_with_4_bit_experts(T, masked):
    """Every stage from the one before it: the rows and activations quantised
    bit for bit, each product against 64 bits (the bars of the products' own
    test), the combine in fp32; then the block around it, captured and
    replayed."""
    sh = inputs.Shape(256, 16, 4, 384, 1, "bf16")
    b, v, W = parts(T, sh, "bf16", masked, 9)
    ex = block.Mx4Experts(T, sh.d, sh.E, sh.I, sh.K, 1, *W)
    b = block.MoeBlock(T, sh.d, sh.E, sh.I, sh.K, 1, *W, v["w_in"], v["w_out"], v["gc"], experts=ex)
    got = step(b, v, W, back=False)
    rt = gpu_route(ex.dsc, b.n, W[0], W[1])
    assert np.array_equal(ex.idx.cpu().numpy(), rt["idx"])
    counts = rt["counts"]
    P = int(counts.sum())
    assert int(ex.kept[0]) == P and (not masked or P < T * sh.K)

    def values(pair):
        return plain_values(pair[0][:P].cpu().numpy(), pair[1][:P].cpu().numpy())
    wv = []
    for w, got4 in ((W[2], ex.w1), (W[3], ex.w3), (W[4], ex.w2)):
        c, s = plain_quantize(w.reshape(-1, w.shape[2]))
        assert np.array_equal(got4[0].cpu().numpy(), c)
        assert torch.equal(got4[1], tile_scales(torch.as_tensor(s, device=DEV)))
        wv.append(plain_values(c, s).reshape(w.shape))
    rows = np.repeat(np.arange(sh.E), counts)
    tok = ex.pair[:P].cpu().numpy() // sh.K
    assert torch.equal(ex.x_rows[:P], b.n[torch.as_tensor(tok, device=DEV).long()])
    for src, dst in ((ex.x_rows, ex.x4), (ex.h, ex.h4)):
        c, s = plain_quantize(src[:P])
        assert np.array_equal(dst[0][:P].cpu().numpy(), c) and np.array_equal(dst[1][:P].cpu().numpy(), s)
    a, hv = values(ex.x4), values(ex.h4)
    dot = lambda A, Wt: np.einsum("rk,rnk->rn", A, Wt[rows])  # noqa: E731
    g, u = dot(a, wv[0]), dot(a, wv[1])
    eps = sh.d * 2.0 ** -23
    dg, du = (eps * dot(np.abs(a), np.abs(w)) for w in wv[:2])
    ref = g / (1 + np.exp(-g)) * u
    tol = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 8 * U * np.abs(ref)
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 1e-37
    assert (np.abs(ex.h[:P].double().cpu().numpy() - ref) <= tol).all()
    y, ty = dot(hv, wv[2]), sh.I * 2.0 ** -23 * dot(np.abs(hv), np.abs(wv[2])) + 1e-37
    yg = ex.y_rows[:P].double().cpu().numpy()
    assert (np.abs(yg - y) <= ty).all()
    # the combine of these rows: K products and sums in fp32, one rounding
    ref, mag = np.zeros((T, sh.d)), np.zeros((T, sh.d))
    for r, pair in enumerate(ex.pair[:P].cpu().numpy()):
        term = float(ex.w.reshape(-1)[pair]) * yg[r]
        ref[pair // sh.K] += term
        mag[pair // sh.K] += np.abs(term)
    assert (np.abs(b.y.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * sh.K * U * mag + 1e-37).all()
    out, n = torch.empty_like(v["x"]), torch.empty_like(v["x"])
    graph = torch.cuda.CUDAGraph()
    keep = v["x"].clone()
    with torch.cuda.graph(graph):
        b.forward(v["x"], out, gate_t=v["gt"], w_next=v["w_next"], n_next=n)
    v["x"].copy_(keep.flip(0) * 1.5)
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone(), n.clone()
    eager = step(b, v, W, back=False)
    assert torch.equal(eager["out"], replayed[0]) and torch.equal(eager["n_next"], replayed[1])
    assert not torch.equal(eager["out"], got["out"])


def test_refusals():
    sh = inputs.Shape(128, 8, 2, 128, 1, "bf16")
    b, v, W = parts(3, sh, "bf16", True, 1)
    with pytest.raises(ValueError):
        b.backward(v["x"], v["x"], v["dout"], v["x"])
    ex = block.Mx4Experts(3, sh.d, sh.E, sh.I, sh.K, 1, *W)
    with pytest.raises(ValueError):
        block.MoeBlock(3, sh.d, sh.E, sh.I, sh.K, 1, *W, v["w_in"], train=True, experts=ex)


def test_check_before_the_first_calls():
    """In memory that an earlier tensor left full, check() before any call and
    between the first forward and the first backward reports nothing."""
    sh = inputs.Shape(128, 8, 2, 128, 1, "bf16")
    torch.cuda.empty_cache()
    dirty = [torch.full((1 << k,), 255, dtype=torch.uint8, device=DEV) for k in range(12, 25)]
    dirty += [torch.full((1 << k,), 255, dtype=torch.uint8, device=DEV) for k in range(12, 25)]
    torch.cuda.synchronize()
    del dirty
    b, v, W = parts(6, sh, "bf16", True, 1, balance=0.1, train=True)
    b.check()
    step(b, v, W, back=False)  # checks behind the forward
    block.Mx4Experts(6, sh.d, sh.E, sh.I, sh.K, 1, *W).check()


def gradients_in_64_bits(b, v, W, seq, renorm, dl, dout, dn, scales=(1.0, 1.0)):
    """Autograd of the unmasked block's formula in 64 bits, with the block's own
    candidates and counts."""
    leaf = {k: t.double().requires_grad_() for k, t in
            dict(dx=v["x"], dgt=v["gt"], dwn=v["w_next"], dw_in=b.w_in, dw_out=b.w_out, dgate_c=b.gate_c, dW_gate=W[0],
                 dW1=W[2], dW3=W[3], dW2=W[4]).items()}
    x, idx = leaf["dx"], b.idx.long()
    n = x / rms(x) * leaf["dw_in"]
    logits = n @ leaf["dW_gate"].T
    p = torch.softmax(logits, 1)
    g = torch.softmax(logits.gather(1, idx), 1) if renorm else p.gather(1, idx)
    y = torch.zeros_like(x)
    for k in range(idx.shape[1]):
        e = idx[:, k]
        h = torch.nn.functional.silu(torch.einsum("td,tid->ti", n, leaf["dW1"][e])) \
            * torch.einsum("td,tid->ti", n, leaf["dW3"][e])
        y = y + g[:, k:k + 1] * torch.einsum("ti,tdi->td", h, leaf["dW2"][e])
    branch = torch.sigmoid(leaf["dgt"])[:, None] * leaf["dgate_c"] * leaf["dw_out"] * y / rms(y)
    out = scales[0] * x + scales[1] * branch
    n_next = out / rms(out) * leaf["dwn"]
    loss, S, E = 0.0, len(seq) - 1, W[0].shape[0]
    for s, (lo, hi) in enumerate(zip(seq[:-1], seq[1:])):
        f = b.cand[s].double() * E / (idx.shape[1] * (hi - lo))
        loss = loss + b.bal.coef / S * (f * p[lo:hi].mean(0)).sum()
    ((dout.double() * out).sum() + (dn.double() * n_next).sum() + dl * loss).backward()
    return {k: t.grad for k, t in leaf.items()}


@pytest.mark.parametrize("upstream", [1.0, 0.0], ids=["all", "balance_alone"])
@pytest.mark.parametrize("T,sh", [(12, inputs.Shape(128, 8, 2, 128, 1, "f32")), (40, inputs.Shape(256, 16, 4, 128, 0, "f32"))],
                         ids=["T12", "T40_all_softmax"])
def test_gradients_are_those_of_the_formula_in_64_bits(T, sh, upstream):
    """An fp32 block without a mask against autograd in 64 bits, with the
    rows' upstream gradients and with the balance loss's alone, which then hides
    behind nothing.

    Bar, normwise: forward values are off by at most (d + I + 500) u of their
    magnitudes' sum, each gradient by the same once more on its way back, and
    magnitudes add up to at most sqrt(d) = 16 times what the signed sums of
    random terms come to: 2 x 884 x 16 u = 1.7e-3 of the largest entry.  A part
    that is missing changes it by a share of one."""
    seq = [0, 5, T]
    b, v, W = parts(T, sh, "f32", False, 3, balance=0.5, n_seq=2, train=True, res_scale=0.9, branch_scale=0.5)
    for k in ("dout", "dn"):
        v[k] *= upstream
    got = step(b, v, W, torch.tensor([2.0], device=DEV), torch.tensor(seq, dtype=torch.int32, device=DEV))
    want = gradients_in_64_bits(b, v, W, seq, sh.renorm, 2.0, v["dout"], v["dn"], (0.9, 0.5))
    for k, w in want.items():
        if w is None or not w.abs().max() > 0:
            assert upstream == 0.0 and k not in ("dx", "dw_in", "dW_gate") and (got[k] == 0).all(), k
            continue
        assert float((got[k].double() - w).abs().max()) <= 1.7e-3 * float(w.abs().max()), k


def test_two_blocks_train_on_two_streams_at_once():
    """Blocks share no buffer: steps of two of them that overlap give what they
    give one after the other."""
    sh, T = inputs.Shape(256, 16, 4, 256, 1, "bf16"), 200
    seq = torch.tensor([0, 90, T], dtype=torch.int32, device=DEV)
    dl = torch.tensor([0.7], device=DEV)
    made = [parts(T, sh, "bf16", True, s, balance=0.1, n_seq=2, beta=0.01, train=True) for s in (11, 12)]
    want = [step(*m, dl, seq) for m in made]
    streams = [torch.cuda.Stream() for _ in made]
    own = [dict(out=torch.empty_like(v["x"]), n=torch.empty_like(v["x"]), dx=torch.empty_like(v["x"]),
                dgt=torch.empty(T, device=DEV), dwn=torch.zeros(sh.d, device=DEV)) for _, v, _ in made]
    torch.cuda.synchronize()
    for _ in range(4):
        for (b, v, _), o, s in zip(made, own, streams):
            with torch.cuda.stream(s):
                b.zero_grad()
                o["dwn"].zero_()
                b.forward(v["x"], o["out"], gate_t=v["gt"], w_next=v["w_next"], n_next=o["n"], seq_begin=seq)
                b.backward(v["x"], o["out"], v["dout"], o["dx"], gate_t=v["gt"], dgate_t=o["dgt"], w_next=v["w_next"],
                           dn_next=v["dn"], dw_next=o["dwn"], seq_begin=seq, dloss=dl)
    torch.cuda.synchronize()
    for (b, _, _), o, w in zip(made, own, want):
        b.check()
        for k, t in dict(out=o["out"], n_next=o["n"], loss=b.loss, dx=o["dx"], dgt=o["dgt"], dwn=o["dwn"],
                         **{"d" + k: g for k, g in b.grads.items()}).items():
            assert torch.equal(t, w[k]), k


def test_no_tokens_and_rows_of_another_number():
    """A block of no tokens runs and leaves the gradients as they were; rows of
    another number than the block's or the experts' are refused."""
    sh = inputs.Shape(128, 8, 2, 128, 1, "bf16")
    b, v, W = parts(0, sh, "bf16", True, 1, balance=0.1, n_seq=2, train=True)
    seq = torch.zeros(3, dtype=torch.int32, device=DEV)
    out, n, dx = (torch.empty_like(v["x"]) for _ in range(3))
    for g in b.grads.values():
        g.fill_(3.0)
    b.forward(v["x"], out, w_next=v["w_next"], n_next=n, seq_begin=seq)
    dwn = torch.full((sh.d,), 3.0, device=DEV)
    b.backward(v["x"], out, v["dout"], dx, w_next=v["w_next"], dn_next=v["dn"], dw_next=dwn, seq_begin=seq)
    b.check()
    assert float(b.loss) == 0.0 and all((g == 3.0).all() for g in (dwn, *b.grads.values()))
    ex = block.Mx4Experts(6, sh.d, sh.E, sh.I, sh.K, 1, *W)
    rows = torch.zeros(7, sh.d, dtype=BF16, device=DEV)
    for x, y in ((rows[:5], rows[:5]), (rows[:6], rows[:5]), (rows, rows[:6])):
        with pytest.raises(abi.BeamError):
            ex.forward(x, y)
    served = block.MoeBlock(6, sh.d, sh.E, sh.I, sh.K, 1, *W, v["w_in"], experts=ex)
    for x, y in ((rows[:5], rows[:5]), (rows[:6], rows)):
        with pytest.raises(abi.BeamError):
            served.forward(x, y)
    assert ex.forward(rows[:6], torch.empty_like(rows[:6])).isfinite().all()
