"""The router's balance loss, its counts and its gradient on the GPU against
the formula in 64 bits and against differences, and the gradient's way through
the layer's backward.

Bars, with u = 2^-24: a probability's exponent r - max is off by u of itself
(|r - max| < 40 here), exp by 4 u, the sum of at most 8 values a lane and 5
shuffles by 13 u, the quotient by 2 u: 60 u.  Means and the loss add positive
terms in a fixed order, at most chunks + tokens per warp + 16 of them in a row
(fewer than the sequence's tokens, and fewer than 600 + 16 + T / 592).
"""
import pytest
import torch

import oracle
from dynamic_expert_routing_router_b200 import abi, inputs

from _parity import gpu_route, host

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def logits_of(T, E, seed, mask, ld=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    width = (2 * E if mask else E) if ld is None else ld
    lg = torch.randn(T, width, generator=g, device=DEV)
    lg[:, :E] -= torch.log(torch.arange(1, E + 1, device=DEV).float())
    return lg


def counts_of(lg, E, K, thr=None):
    """[T, E] candidates (K largest, ties to the lower id) and kept ones."""
    r = lg[:, :E].double()
    order = torch.sort(r, dim=1, descending=True, stable=True).indices[:, :K]
    c = torch.zeros_like(r).scatter_(1, order, 1.0)
    return c, None if thr is None else c * (lg[:, E:2 * E] >= thr)


def reference(lg, E, K, begin, coef, counted, counts=None):
    """loss, P [S, E], f [S, E] and dloss/dlogits for the counts given (or
    those of `counted` [T, E])."""
    S = len(begin) - 1
    p = torch.softmax(lg[:, :E].double(), 1)
    P, f, grad = torch.zeros(S, E).double().to(DEV), torch.zeros(S, E).double().to(DEV), torch.zeros_like(p)
    for s in range(S):
        lo, hi = begin[s], begin[s + 1]
        if hi == lo:
            continue
        P[s] = p[lo:hi].mean(0)
        n = counted[lo:hi].sum(0) if counts is None else counts[s].double()
        f[s] = n * E / (K * (hi - lo))
        grad[lo:hi] = coef / (S * (hi - lo)) * p[lo:hi] * (f[s] - (p[lo:hi] * f[s]).sum(1, keepdim=True))
    return coef / S * (f * P).sum(), P, f, grad


CASES = [  # T, E, K, boundaries, mask, count kept
    (1, 8, 2, [0, 1], False, False), (7, 60, 4, [0, 3, 3, 7], True, False),
    (128, 128, 8, [0, 128], True, True), (1000, 256, 16, [0, 1, 17, 900, 1000], True, True),
    (333, 33, 1, [0, 333], False, False), (500, 2, 2, [0, 250, 500], True, False),
    (2048, 64, 6, list(range(0, 2049, 32)), True, True), (20000, 128, 8, [0, 19999, 20000], False, False),
    (40000, 16, 2, [0, 40000], True, False)]


@pytest.mark.parametrize("T,E,K,begin,mask,kept", CASES, ids=[f"T{c[0]}E{c[1]}K{c[2]}S{len(c[3]) - 1}" for c in CASES])
def test_loss_counts_and_gradient(T, E, K, begin, mask, kept):
    lg, S, coef = logits_of(T, E, T + E, mask), len(begin) - 1, 0.02
    dsc = abi.balance_desc(T, E, K, n_seq=S, coef=coef, has_mask=mask, count_kept=kept, tau=0.4)
    b = torch.tensor(begin, dtype=torch.int32, device=DEV)
    cand_t, kept_t = counts_of(lg, E, K, dsc.mask_logit_threshold if mask else None)
    loss, prob = torch.full((1,), float("nan"), device=DEV), torch.full((S, E), float("nan"), device=DEV)
    cand = torch.full((S, E), -7, dtype=torch.int32, device=DEV)
    kc = torch.full((S, E), -7, dtype=torch.int32, device=DEV) if mask else None
    ws = abi.alloc_balance_workspace(dsc)
    abi.balance(dsc, lg, loss, cand, ws, kept_counts=kc, mean_prob=prob, seq_begin=b)
    rl, rP, rf, _ = reference(lg, E, K, begin, coef, kept_t if kept else cand_t)
    for got, per_token in ((cand, cand_t), (kc, kept_t)):
        if got is not None:
            want = torch.stack([per_token[lo:hi].sum(0) for lo, hi in zip(begin[:-1], begin[1:])])
            assert torch.equal(got.double(), want)
    chain = min(T, 616 + T / 592)
    assert ((prob.double() - rP).abs() <= (60 + chain) * U * rP + 1e-38).all()
    assert abs(float(loss) - float(rl)) <= (80 + chain + S) * U * float(rl)
    # the loss alone, without the outputs that may be left out, bit for bit
    again = torch.full((1,), float("nan"), device=DEV)
    abi.balance(dsc, lg, again, cand, ws, seq_begin=b)
    assert torch.equal(again, loss)
    up = torch.tensor([-1.5], device=DEV)
    for dloss in (None, up):
        dl = torch.full((T, E), float("nan"), device=DEV)
        abi.balance_backward(dsc, lg, kc if kept else cand, dl, seq_begin=b, dloss=dloss)
        _, _, _, g = reference(lg, E, K, begin, coef * (1.0 if dloss is None else -1.5),
                               kept_t if kept else cand_t)
        p = torch.softmax(lg[:, :E].double(), 1)
        seq = torch.bucketize(torch.arange(T, device=DEV), b[1:].long(), right=True)
        length = (b[1:] - b[:-1]).double().clamp(min=1)[seq][:, None]
        ft = rf[seq]
        mag = coef * 1.5 / (S * length) * p * (ft + (p * ft).sum(1, keepdim=True))
        assert ((dl.double() - g).abs() <= 150 * U * mag + 1e-38).all()


def test_gradient_is_the_difference_of_the_loss():
    """Central differences of the 64-bit loss with the counts held, along one
    direction per case; their error is h^2 / 6 of the third derivative, below
    1e-7 of the loss for h = 1e-3, and the gradient's own 150 u."""
    T, E, K, begin = 60, 16, 3, [0, 25, 60]
    lg = logits_of(T, E, 3, False)
    dsc = abi.balance_desc(T, E, K, n_seq=2)
    b = torch.tensor(begin, dtype=torch.int32, device=DEV)
    loss, cand = torch.empty(1, device=DEV), torch.empty(2, E, dtype=torch.int32, device=DEV)
    abi.balance(dsc, lg, loss, cand, abi.alloc_balance_workspace(dsc), seq_begin=b)
    dl = torch.empty(T, E, device=DEV)
    abi.balance_backward(dsc, lg, cand, dl, seq_begin=b)
    v = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).double()
    h = 1e-3
    ends = [float(reference(lg.double() + s * h * v, E, K, begin, 1.0, None, counts=cand)[0]) for s in (1, -1)]
    want = (ends[0] - ends[1]) / (2 * h)
    assert abs(float((dl.double() * v).sum()) - want) <= 1e-5 * float(loss)


def test_gradient_where_it_almost_cancels():
    """Every expert a candidate (f = 1 everywhere: the gradient is 0 but
    for the second order), and one
    expert with nearly all of the probability: relative to p_e |f_e - f_e'| p_e'
    summed over e', not to f itself.  (The reference is that sum with signs: f -
    <f, p> in 64 bits is off by f 2^-53 = 9e-16, against 2e-12 here.)"""
    T, E = 9, 16
    lg = logits_of(T, E, 5, False)
    cand = torch.full((1, E), T, dtype=torch.int32, device=DEV)
    dl = torch.full((T, E), float("nan"), device=DEV)
    abi.balance_backward(abi.balance_desc(T, E, E), lg, cand, dl)
    # <f, p> is off by 60 u, and what is left of it by its own 73 u
    assert (dl.abs().double() <= 60 * 133 * U * U * torch.softmax(lg.double(), 1) / T).all()
    lg[:, 3] += 30.0
    dsc = abi.balance_desc(T, E, 2)
    abi.balance(dsc, lg, torch.empty(1, device=DEV), cand, abi.alloc_balance_workspace(dsc))
    abi.balance_backward(dsc, lg, cand, dl)
    f, p = cand[0].double() * E / (2 * T), torch.softmax(lg.double(), 1)
    apart = p[:, None, :] * (f[:, None] - f[None, :])
    g, spread = apart.sum(2) * p / T, apart.abs().sum(2) * p / T
    assert ((dl.double() - g).abs() <= 150 * U * spread + 1e-38).all()


@pytest.mark.parametrize("copies", [1, 100])  # one launch, and chunks
def test_ties_infinities_and_rows_without_a_softmax(copies):
    """Equal logits count for the lower ids, -inf logits weigh nothing, a row
    of -inf counts its lowest ids and adds no probability, z = NaN is not kept."""
    T, E, K = 6, 40, 3
    lg = torch.zeros(T, 2 * E, device=DEV)
    ninf = float("-inf")
    lg[1, :E] = ninf
    lg[2, :38] = ninf
    lg[3, 5], lg[3, 6] = -0.0, 1.0
    lg[4, E:] = float("nan")
    lg[5, 39] = 3e38
    lg, T = lg.repeat(copies, 1), T * copies
    dsc = abi.balance_desc(T, E, K, has_mask=True)
    loss, prob = torch.empty(1, device=DEV), torch.empty(1, E, device=DEV)
    cand, kept = (torch.empty(1, E, dtype=torch.int32, device=DEV) for _ in range(2))
    abi.balance(dsc, lg, loss, cand, abi.alloc_balance_workspace(dsc), kept_counts=kept, mean_prob=prob)
    want = torch.zeros(E, dtype=torch.int32)
    for ids in ((0, 1, 2), (0, 1, 2), (38, 39, 0), (6, 0, 1), (0, 1, 2), (39, 0, 1)):
        want[list(ids)] += 1
    assert torch.equal(cand[0].cpu(), copies * want)
    want[[0, 1, 2]] -= 1
    assert torch.equal(kept[0].cpu(), copies * want)
    p = torch.softmax(lg[:, :E].double(), 1).nan_to_num(0.0).mean(0)
    assert ((prob[0].double() - p).abs() <= 170 * U * p + 1e-38).all() and torch.isfinite(loss).all()
    dl = torch.empty(T, E, device=DEV)
    abi.balance_backward(dsc, lg, cand, dl)
    assert torch.isfinite(dl).all() and (dl[1] == 0).all()


@pytest.mark.parametrize("f", [1, 20])  # one launch, and chunks
def test_sequences_that_leave_tokens_out_and_bad_boundaries(f):
    T, E, K = 50 * f, 24, 2
    lg = logits_of(T, E, 9, False)
    dsc = abi.balance_desc(T, E, K, n_seq=2)
    ws, loss = abi.alloc_balance_workspace(dsc), torch.empty(1, device=DEV)
    cand = torch.empty(2, E, dtype=torch.int32, device=DEV)
    b = torch.tensor([10 * f, 30 * f, 45 * f], dtype=torch.int32, device=DEV)
    abi.balance(dsc, lg, loss, cand, ws, seq_begin=b)
    c, _ = counts_of(lg, E, K)
    rl, _, _, g = reference(lg, E, K, [10 * f, 30 * f, 45 * f], 1.0, c)
    assert abs(float(loss) - float(rl)) <= (150 + T) * U * float(rl)
    dl = torch.full((T, E), float("nan"), device=DEV)
    abi.balance_backward(dsc, lg, cand, dl, seq_begin=b)
    assert (dl[:10 * f] == 0).all() and (dl[45 * f:] == 0).all()
    assert ((dl.double() - g).abs() <= 1e-6).all() and (dl[10 * f:45 * f] != 0).any()
    for bad in ([0, 40, 30], [-1, 20, 50], [0, 25, T + 1], [T, 0, T]):
        b = torch.tensor(bad, dtype=torch.int32, device=DEV)
        abi.balance(dsc, lg, loss, cand, ws, seq_begin=b)
        assert torch.isnan(loss).all(), bad


def test_wide_rows_no_tokens_streams_and_graphs():
    T, E, K = 200, 60, 4
    lg = logits_of(T, E, 2, True)
    wide = torch.full((T, 200), float("nan"), device=DEV)
    wide[:, :2 * E] = lg
    got = []
    side = torch.cuda.Stream()
    for x, ld, stream in ((lg, None, None), (wide, 200, None), (lg, None, side)):
        dsc = abi.balance_desc(T, E, K, logits_ld=ld, has_mask=True, count_kept=True)
        o = dict(loss=torch.empty(1, device=DEV), c=torch.empty(1, E, dtype=torch.int32, device=DEV),
                 k=torch.empty(1, E, dtype=torch.int32, device=DEV), p=torch.empty(1, E, device=DEV),
                 d=torch.empty(T, E, device=DEV))
        ws = abi.alloc_balance_workspace(dsc)
        side.wait_stream(torch.cuda.current_stream())
        abi.balance(dsc, x, o["loss"], o["c"], ws, kept_counts=o["k"], mean_prob=o["p"], stream=stream)
        abi.balance_backward(dsc, x, o["k"], o["d"], stream=stream)
        torch.cuda.synchronize()
        got.append(o)
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros_like(lg)
    g = {k: torch.empty_like(v) for k, v in got[0].items()}
    dsc = abi.balance_desc(T, E, K, has_mask=True, count_kept=True)
    ws = abi.alloc_balance_workspace(dsc)
    with torch.cuda.graph(graph):
        abi.balance(dsc, x, g["loss"], g["c"], ws, kept_counts=g["k"], mean_prob=g["p"])
        abi.balance_backward(dsc, x, g["k"], g["d"])
    x.copy_(lg)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for o in got[1:] + [g]:
        for k in o:
            assert torch.equal(o[k], got[0][k]), k
    none = abi.balance_desc(0, E, K, n_seq=3)
    loss, c = torch.full((1,), 5.0, device=DEV), torch.full((3, E), 9, dtype=torch.int32, device=DEV)
    z = torch.zeros(4, dtype=torch.int32, device=DEV)
    abi.balance(none, torch.empty(0, E, device=DEV), loss, c, abi.alloc_balance_workspace(none), seq_begin=z)
    abi.balance_backward(none, torch.empty(0, E, device=DEV), c, torch.empty(0, E, device=DEV), seq_begin=z)
    assert float(loss) == 0.0 and (c == 0).all()


@pytest.mark.parametrize("renorm", [1, 0])
def test_counts_are_the_routers_own(renorm):
    """The layer's own logits give the router's kept counts."""
    sh = inputs.Shape(2048, 128, 8, 768, renorm, "bf16")
    T = 100
    x = inputs.make_tokens(sh, T, seed=4, device=DEV)
    Wg, Wm = inputs.make_gate(sh, seed=1, device=DEV), inputs.make_mask(sh, 0.35, seed=1, device=DEV)
    rt = gpu_route(abi.desc(T, sh.d, sh.E, sh.I, sh.K, "bf16", renorm), x, Wg, Wm)
    lg = torch.as_tensor(rt["logits"], device=DEV).contiguous()
    dsc = abi.balance_desc(T, sh.E, sh.K, has_mask=True)
    c, k = (torch.empty(1, sh.E, dtype=torch.int32, device=DEV) for _ in range(2))
    abi.balance(dsc, lg, torch.empty(1, device=DEV), c, abi.alloc_balance_workspace(dsc), kept_counts=k)
    assert torch.equal(k[0].cpu(), torch.as_tensor(rt["counts"]).to(torch.int32).reshape(-1))
    assert int(c.sum()) == T * sh.K


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-4), ("bf16", 1e-2)])
def test_gradient_through_the_layer(dtype, tol):
    """backward(dlogits=...) adds dlogits W_gate to dx and dlogits^T x to
    dW_gate; the oracle's gradients and these products in 64 bits, with the
    bars of the layer's own backward (normwise).  Without dlogits, and with
    zeros, nothing changes by a bit."""
    sh = inputs.Shape(256, 16, 4, 256, 1, dtype)
    T, beta = 48, 0.01
    x = inputs.make_tokens(sh, T, seed=3, device=DEV)
    Wg, Wm = inputs.make_gate(sh, seed=4, device=DEV), inputs.make_mask(sh, 0.35, seed=4, device=DEV)
    W = inputs.make_experts(sh, seed=4, device=DEV)
    dy = inputs.make_upstream_grad(sh, T, seed=9, device=DEV)
    dsc = abi.desc(T, sh.d, sh.E, sh.I, sh.K, dtype, 1)
    rt = gpu_route(dsc, x, Wg, Wm)
    dl = torch.randn(T, sh.E, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)

    def run(dlogits):
        z = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
        g = dict(dx=z(T, sh.d), dWg=z(sh.E, sh.d), dWm=z(sh.E, sh.d), dW1=z(sh.E, sh.I, sh.d),
                 dW3=z(sh.E, sh.I, sh.d), dW2=z(sh.E, sh.d, sh.I))
        ws = abi.alloc_backward_workspace(dsc, DEV)
        abi.backward(dsc, x, Wg, Wm, *W, dy, beta, *g.values(), ws, dlogits=dlogits)
        abi.check(dsc, ws)
        return g
    plain, zero, got = run(None), run(torch.zeros_like(dl)), run(dl)
    for k in plain:
        assert torch.equal(plain[k], zero[k]), k
    for k in ("dWm", "dW1", "dW3", "dW2"):
        assert torch.equal(plain[k], got[k]), k
    ref = oracle.backward(host(x), host(Wg), host(Wm), *[host(w) for w in W], host(dy), sh.K, 1, dtype,
                          beta=beta, logits=rt["logits"])
    for k, r, add in (("dx", "dx", dl.double() @ Wg.double()), ("dWg", "dW_gate", dl.double().T @ x.double())):
        want = torch.as_tensor(ref[r], device=DEV) + add
        assert float((got[k].double() - want).abs().max()) <= tol * float(want.abs().max()), k
        assert float((plain[k].double() - want).abs().max()) > tol * float(want.abs().max()), k


def test_offsets_past_32_bits_and_many_sequences():
    """More than 2^31 logits, and one sequence per three tokens: counts add up,
    the last rows' gradient is that of a small call."""
    T, E, K = 8_500_000, 256, 4
    lg = torch.zeros(T, E, device=DEV)
    lg[:, 3], lg[:, 100], lg[:, 200], lg[:, 255] = 4.0, 3.0, 2.0, 1.0
    dsc = abi.balance_desc(T, E, K)
    loss, cand = torch.empty(1, device=DEV), torch.empty(1, E, dtype=torch.int32, device=DEV)
    abi.balance(dsc, lg, loss, cand, abi.alloc_balance_workspace(dsc))
    p = torch.softmax(lg[0].double(), 0)
    assert cand[0, [3, 100, 200, 255]].tolist() == [T] * 4 and int(cand.long().sum()) == 4 * T
    want = float((p[[3, 100, 200, 255]]).sum() * E / K)
    # a chunk's warp adds T / (8 * 444) equal terms one by one
    assert abs(float(loss) - want) <= (T / 3552 + 700) * U * want
    dl = torch.empty(T, E, device=DEV)
    abi.balance_backward(dsc, lg, cand, dl)
    assert torch.equal(dl[-5:], dl[:5]) and torch.isfinite(dl[-1]).all()
    del lg, dl
    T, E, S = 9000, 20, 3000
    lg = logits_of(T, E, 1, False)
    b = torch.arange(0, T + 1, 3, dtype=torch.int32, device=DEV)
    dsc = abi.balance_desc(T, E, 2, n_seq=S)
    cand = torch.empty(S, E, dtype=torch.int32, device=DEV)
    abi.balance(dsc, lg, loss, cand, abi.alloc_balance_workspace(dsc), seq_begin=b)
    c, _ = counts_of(lg, E, 2)
    assert torch.equal(cand.double(), c.view(S, 3, E).sum(1))
    dl = torch.empty(T, E, device=DEV)
    abi.balance_backward(dsc, lg, cand, dl, seq_begin=b)
    rl, _, _, g = reference(lg, E, 2, list(range(0, T + 1, 3)), 1.0, c)
    assert abs(float(loss) - float(rl)) <= (80 + S) * U * float(rl)
    assert ((dl.double() - g).abs() <= 150 * U * E).all()


def test_many_sequences_entry_by_entry():
    """3000 sequences of three tokens, where a gradient's entry is of the order
    of 1e-5: each within 150 u of its own terms' magnitudes."""
    T, E, K, S = 9000, 20, 2, 3000
    lg, begin = logits_of(T, E, 1, False), list(range(0, 9001, 3))
    b = torch.tensor(begin, dtype=torch.int32, device=DEV)
    dsc = abi.balance_desc(T, E, K, n_seq=S)
    cand, dl = torch.empty(S, E, dtype=torch.int32, device=DEV), torch.full((T, E), float("nan"), device=DEV)
    abi.balance(dsc, lg, torch.empty(1, device=DEV), cand, abi.alloc_balance_workspace(dsc), seq_begin=b)
    abi.balance_backward(dsc, lg, cand, dl, seq_begin=b)
    p = torch.softmax(lg.double(), 1)
    f = counts_of(lg, E, K)[0].view(S, 3, E).sum(1).repeat_interleave(3, 0) * E / (K * 3)
    dot = (p * f).sum(1, keepdim=True)
    g, mag = p * (f - dot) / (3 * S), p * (f + dot) / (3 * S)
    assert ((dl.double() - g).abs() <= 150 * U * mag + 1e-38).all()
