"""The 4-bit floating point operators on the GPU: rows to MXFP4 and back
against a plain implementation of the format in 64 bits, the grouped product
against fp64 products of the values the codes stand for, and refusals.

Bars, from the arithmetic: quantising and reading back round nothing but the
4-bit digits, so codes, scales and values are equal bit for bit.  The product
accumulates exact products in fp32: each of the k terms adds at most 2^-24 of
the running sum, bounded by sum |a w|, and some tensor core sums cut rather
than round, hence k 2^-23 sum|a w|; the bf16 output adds half a step, 2^-9
relative to a power of two above, 2^-8 of the value.  SwiGLU: SiLU's slope is
at most 1.1, so an error of dg in the gate and du in the up value moves
g s(g) u by at most 1.1 dg |u| + |g| du, plus 8 2^-24 of the result for the
exponential, division and products.
"""
import time

import numpy as np
import pytest
import torch

from dynamic_expert_routing_router_b200 import abi

pytestmark = pytest.mark.gpu
DEV = "cuda"
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def plain_quantize(x):
    """(digits' codes, scale bytes) in 64 bits, straight from the format."""
    x = x.double().cpu().numpy()
    rows, cols = x.shape
    v = x.reshape(rows, cols // 32, 32)
    top = np.abs(v).max(axis=2)
    bad = ~np.isfinite(top)
    with np.errstate(divide="ignore"):
        X = np.where((top > 0) & ~bad, np.floor(np.log2(np.where(bad | (top == 0), 1.0, top))), -125) - 2
    X = np.maximum(X, -127)
    a = np.abs(np.where(bad[:, :, None], 0.0, v)) / np.exp2(X)[:, :, None]
    mid = (GRID[1:] + GRID[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    code = np.where(hi % 2 == 0, hi, lo)  # they differ on a tie: the even digit
    code = code + 8 * np.signbit(v)
    code = np.where(bad[:, :, None], 0, code).reshape(rows, cols // 2, 2)
    return ((code[:, :, 0] | (code[:, :, 1] << 4)).astype(np.uint8),
            np.where(bad, 255, X + 127).astype(np.uint8))


def plain_values(codes, scales):
    c = np.stack([codes & 15, codes >> 4], axis=2).reshape(codes.shape[0], -1)
    v = np.where(c < 8, 1.0, -1.0) * GRID[c & 7]
    f = np.exp2(scales.astype(np.float64) - 127)
    f[scales == 255] = np.nan
    return v * np.repeat(f, 32, axis=1)


def tile_scales(scales):
    t = scales.reshape(scales.shape[0] // 128, 4, 32, scales.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).contiguous().reshape(scales.shape)


def quantize(x, **kw):
    codes = torch.full((x.shape[0], x.shape[1] // 2), 0xEE, dtype=torch.uint8, device=DEV)
    scales = torch.full((x.shape[0], x.shape[1] // 32), 0xEE, dtype=torch.uint8, device=DEV)
    abi.mx4_quantize(x, codes, scales, **kw)
    return codes, scales


def rows_of(rows, cols, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=DEV)
    return (x * torch.exp(3 * torch.randn(rows, 1, generator=g, device=DEV))).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (129, 2048), (1000, 160)])
def test_quantize_is_the_format_bit_for_bit(rows, cols, dtype):
    x = rows_of(rows, cols, dtype, rows + cols)
    codes, scales = quantize(x)
    c, s = plain_quantize(x)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    for out in (torch.bfloat16, torch.float32):
        v = torch.empty(rows, cols, dtype=out, device=DEV)
        abi.mx4_dequantize(codes, scales, v)
        assert np.array_equal(v.double().cpu().numpy(), plain_values(c, s))


def test_quantize_ties_zeros_extremes_and_non_finite():
    x = torch.zeros(9, 32, device=DEV)
    # every digit's neighbourhood and both ties, with 6 (or 4) as the largest
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2499, 0.2501, 5.0001, 6.0, 7.9],
                     device=DEV)
    x[0, :12] = t
    x[0, 12:24] = -t
    x[1, :5] = torch.tensor([1e-45, -1e-45, 1e-40, 0.0, -0.0], device=DEV)  # subnormals
    x[2, 7] = 3.4e38
    x[2, 8] = -3.0e38
    x[3, 3] = float("inf")
    x[4, 31] = float("nan")
    x[4, 0] = 1.0
    x[5, 0] = -0.0
    x[6, :] = 2.0 ** -126
    x[7, :] = 2.0 ** -124 * 1.5
    x[8, 0], x[8, 1] = float("-inf"), float("nan")
    codes, scales = quantize(x)
    c, s = plain_quantize(x)
    assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), c)
    v = torch.empty_like(x)
    abi.mx4_dequantize(codes, scales, v)
    assert np.array_equal(v.double().cpu().numpy(), plain_values(c, s), equal_nan=True)
    assert torch.isnan(v[3]).all() and torch.isnan(v[4]).all() and (v[5] == 0).all()


def test_tiled_scales_and_row_limit():
    x = rows_of(256, 384, torch.bfloat16, 5)
    codes, scales = quantize(x)
    codes_t, scales_t = quantize(x, tiled=True)
    assert torch.equal(codes, codes_t) and torch.equal(scales_t, tile_scales(scales))
    v, vt = torch.empty_like(x), torch.empty_like(x)
    abi.mx4_dequantize(codes, scales, v)
    abi.mx4_dequantize(codes_t, scales_t, vt, tiled=True)
    assert torch.equal(v, vt)
    for n in (0, 1, 77, 256, 1000, -3):
        c, s = quantize(x, n_rows=torch.tensor([n], dtype=torch.int32, device=DEV))
        m = min(max(n, 0), 256)
        assert torch.equal(c[:m], codes[:m]) and torch.equal(s[:m], scales[:m])
        assert (c[m:] == 0xEE).all() and (s[m:] == 0xEE).all()


# ------------------------------------------------------------- product --

def operands(counts, n, k, seed, swiglu=False, tail=0):
    E, P = len(counts), sum(counts)
    a = quantize(rows_of(P + tail, k, torch.float32, seed)) if P + tail else (
        torch.empty(0, k // 2, dtype=torch.uint8, device=DEV),
        torch.empty(0, k // 32, dtype=torch.uint8, device=DEV))
    ws = [quantize(rows_of(E * n, k, torch.float32, seed + 1 + i)) for i in range(2 if swiglu else 1)]
    return a, ws


def product(counts, n, k, a, ws, out="f32", stream=None, N=None):
    E, N = len(counts), a[0].shape[0] if N is None else N
    dsc = abi.mx4_desc(N, E, n, k, swiglu=len(ws) == 2, out=out)
    wk = abi.alloc_mx4_workspace(dsc)
    y = torch.full((N, n), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device=DEV)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    kw = dict(w3_codes=ws[1][0], w3_scales=tile_scales(ws[1][1])) if len(ws) == 2 else {}
    abi.mx4_expert_product(dsc, *a, c, ws[0][0], tile_scales(ws[0][1]), y, wk, **kw)
    return y, dsc, wk


def assert_product(y, counts, n, k, a, ws, out):
    A = plain_values(a[0].cpu().numpy(), a[1].cpu().numpy())
    W = [plain_values(w[0].cpu().numpy(), w[1].cpu().numpy()).reshape(len(counts), n, k) for w in ws]
    y = y.double().cpu().numpy()
    r = 0
    eps = k * 2.0 ** -23
    for e, m in enumerate(counts):
        if m == 0:
            continue
        rows = A[r:r + m]
        g, dg = rows @ W[0][e].T, eps * (np.abs(rows) @ np.abs(W[0][e]).T)
        ref, tol = g, dg
        if len(ws) == 2:
            u, du = rows @ W[1][e].T, eps * (np.abs(rows) @ np.abs(W[1][e]).T)
            ref = g / (1 + np.exp(-g)) * u
            tol = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 8 * 2.0 ** -24 * np.abs(ref)
        if out == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        bad = np.abs(y[r:r + m] - ref) > tol + 1e-37
        assert not bad.any(), (e, m, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                               float(np.abs(y[r:r + m] - ref).max()))
        r += m
    assert (y[r:] == 7.0).all(), "rows behind the last expert's were written"


SIZES = [([1], 128, 128), ([5, 0, 3], 128, 256), ([0, 17, 1, 33], 256, 384), ([130, 2], 384, 640),
         ([300], 128, 1024), ([0, 0, 0, 0, 9], 640, 768),
         # several units per SM with more stages than the ring has, small and large tiles
         ([2] * 40, 768, 1280), ([150] * 9, 512, 1152), ([701, 0, 390], 384, 640)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("counts,n,k", SIZES, ids=[f"{sum(c)}x{n}x{k}" for c, n, k in SIZES])
def test_product_matches_fp64(counts, n, k, swiglu, out):
    a, ws = operands(counts, n, k, seed=n + k, swiglu=swiglu, tail=3)
    if swiglu:  # keep exp(-g) far from overflow: the bound above is relative
        a = (a[0], a[1].clamp(max=127))
    y, dsc, wk = product(counts, n, k, a, ws, out)
    abi.mx4_check(dsc, wk)
    assert_product(y, counts, n, k, a, ws, out)


# ---------------------------------------------- what is there besides values --

def small(counts=(3, 0, 20), n=128, k=256, seed=1, tail=4, swiglu=False):
    return (list(counts), n, k) + operands(list(counts), n, k, seed, swiglu=swiglu, tail=tail)


def test_not_a_number_stays_in_its_row_and_column():
    """A token row's block that stands for NaN makes its row NaN, a weight's its
    column of its expert; rows behind the last expert's and other experts'
    do not see them."""
    counts, n, k, a, ws = small()
    clean, _, _ = product(counts, n, k, a, ws)
    a = (a[0], a[1].clone())
    a[1][5, 1] = 255           # a row of expert 2
    a[1][23:] = 255            # rows nobody owns
    w = (ws[0][0], ws[0][1].clone())
    w[1][7, 0] = 255           # expert 0, column 7
    w[1][n + 9] = 255          # expert 1, without rows
    y, dsc, wk = product(counts, n, k, a, [w])
    abi.mx4_check(dsc, wk)
    bad = torch.zeros(27, n, dtype=torch.bool, device=DEV)
    bad[5], bad[:3, 7] = True, True
    bad[23:] = False
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
def test_no_rows_and_no_capacity(swiglu):
    counts, n, k, a, ws = small((0, 0, 0), tail=5, swiglu=swiglu)
    y, dsc, wk = product(counts, n, k, a, ws)
    abi.mx4_check(dsc, wk)
    assert (y == 7.0).all()
    empty = (a[0][:0], a[1][:0])
    y, dsc, wk = product(counts, n, k, empty, ws)
    abi.mx4_check(dsc, wk)
    assert y.shape == (0, n)


@pytest.mark.parametrize("counts", [[3, -2, 20], [30, 0, 0], [20, 5, 20], [2 ** 31 - 1, 2 ** 31 - 1, 5]])
def test_counts_that_do_not_fit_are_cut_and_reported(counts):
    """Negative counts and sums past N: an error, nothing written past N, rows
    of the experts before the fault as they are; the next call is clean."""
    good, n, k, a, ws = small()
    N = a[0].shape[0]
    guard = torch.full((N + 8, n), 7.0, device=DEV)
    dsc = abi.mx4_desc(N, 3, n, k, out="f32")
    wk = abi.alloc_mx4_workspace(dsc)
    args = (*a,), (ws[0][0], tile_scales(ws[0][1]))
    abi.mx4_expert_product(dsc, *args[0], torch.tensor(counts, dtype=torch.int32, device=DEV), *args[1], guard[:N], wk)
    with pytest.raises(abi.BeamError) as e:
        abi.mx4_check(dsc, wk)
    assert e.value.status == 6 and (guard[N:] == 7.0).all()
    abi.mx4_expert_product(dsc, *args[0], torch.tensor(good, dtype=torch.int32, device=DEV), *args[1], guard[:N], wk)
    abi.mx4_check(dsc, wk)
    clean, _, _ = product(good, n, k, a, ws)
    assert torch.equal(guard[:23], clean[:23])


def test_streams_graphs_and_two_calls_at_once():
    """A captured product follows the counts and rows of its replay, two calls
    on two streams with a workspace each do not meet, and results repeat."""
    counts, n, k, a, ws = small((40, 0, 200), n=384, k=512, tail=16, swiglu=True)
    want, _, _ = product(counts, n, k, a, ws)
    N, E = a[0].shape[0], 3
    dsc = abi.mx4_desc(N, E, n, k, swiglu=True, out="f32")
    scales = [tile_scales(w[1]) for w in ws]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    wks = [abi.alloc_mx4_workspace(dsc) for _ in range(2)]
    torch.cuda.synchronize()
    for s, wk in zip(streams, wks):
        with torch.cuda.stream(s):
            y = torch.full((N, n), 7.0, device=DEV)
        for _ in range(3):
            abi.mx4_expert_product(dsc, *a, c, ws[0][0], scales[0], y, wk, w3_codes=ws[1][0], w3_scales=scales[1],
                                   stream=s)
        outs.append(y)
    torch.cuda.synchronize()
    for y, wk in zip(outs, wks):
        abi.mx4_check(dsc, wk)
        assert torch.equal(y, want)
    codes, sc = torch.zeros_like(a[0]), torch.zeros_like(a[1])
    cg = torch.zeros(E, dtype=torch.int32, device=DEV)
    y = torch.full((N, n), 7.0, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.mx4_expert_product(dsc, codes, sc, cg, ws[0][0], scales[0], y, wks[0], w3_codes=ws[1][0],
                               w3_scales=scales[1])
    codes.copy_(a[0])
    sc.copy_(a[1])
    for trial in (counts, [200, 40, 0], [0, 1, 0]):
        cg.copy_(torch.tensor(trial, dtype=torch.int32))
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        ref, _, _ = product(trial, n, k, a, ws)
        assert torch.equal(y, ref)


def test_expired_wait_is_reported_and_the_next_call_is_clean():
    """A stage that never fills (the library's test switch): a timeout, and the
    workspace serves the next call."""
    counts, n, k, a, ws = small((150, 3, 20), n=256, k=4096)
    want, dsc, wk = product(counts, n, k, a, ws)
    try:
        abi.set_fault_injection(abi.FAULT_MX4_STAGE, 20_000_000)
        _, dsc, wk = product(counts, n, k, a, ws)
        with pytest.raises(abi.BeamError) as e:
            abi.mx4_check(dsc, wk)
        assert e.value.status == 5
    finally:
        abi.set_fault_injection(abi.FAULT_NONE, 0)
    y, dsc, wk = product(counts, n, k, a, ws)
    abi.mx4_check(dsc, wk)
    assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """More than 2^31 values of rows and of outputs: the last rows are those of
    a small call."""
    rows, cols = 1_100_000, 2048
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[:-3] = 0.5
    x[-3:] = rows_of(3, cols, torch.bfloat16, 4)
    codes, scales = quantize(x)
    c, s = quantize(x[-3:].clone())
    assert torch.equal(codes[-3:], c) and torch.equal(scales[-3:], s)
    abi.mx4_dequantize(codes, scales, x)
    v = torch.empty(3, cols, dtype=torch.bfloat16, device=DEV)
    abi.mx4_dequantize(c, s, v)
    assert torch.equal(x[-3:], v) and (x[:-3] == 0.5).all()
    del x, codes, scales
    N, n, k = 70_000, 32768, 128
    a, ws = operands([N], n, k, 2)
    y, dsc, wk = product([N], n, k, a, ws)
    abi.mx4_check(dsc, wk)
    last = (a[0][-100:].clone(), a[1][-100:].clone())
    ref, _, _ = product([100], n, k, last, ws)
    assert torch.equal(y[-100:], ref)


@pytest.mark.parametrize("k", [1024, 8192])
def test_a_call_that_gives_up_waits_for_its_copies_and_for_nothing_else(k):
    """A stage that never fills, with every other stage issued before the wait
    runs out (k = 1024: four stages in all) and with more stages than the ring
    holds: one wait limit passes, not another one for the stage that never
    comes, and the next call is clean."""
    counts, n, k, a, ws = small((20,), k=k)
    want, dsc, wk = product(counts, n, k, a, ws)
    limit = 0.2
    c = torch.tensor(counts, dtype=torch.int32, device=DEV)
    y, tiled = torch.empty_like(want), tile_scales(ws[0][1])
    torch.cuda.synchronize()
    try:
        abi.set_fault_injection(abi.FAULT_MX4_STAGE, int(limit * 1e9))
        begin = time.perf_counter()
        abi.mx4_expert_product(dsc, *a, c, ws[0][0], tiled, y, wk)
        torch.cuda.synchronize()
        took = time.perf_counter() - begin
    finally:
        abi.set_fault_injection(abi.FAULT_NONE, 0)
    with pytest.raises(abi.BeamError) as e:
        abi.mx4_check(dsc, wk)
    assert e.value.status == 5 and limit <= took < 1.8 * limit, took
    y.fill_(7.0)
    abi.mx4_expert_product(dsc, *a, c, ws[0][0], tiled, y, wk)
    abi.mx4_check(dsc, wk)
    assert torch.equal(y, want)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("counts", [[40, 0, 64, 23, 1], [100, 0, 3, 65, 20], [64] * 30])
def test_tiles_of_64_rows_match_fp64(counts, swiglu, out):
    """17 to 64 rows of capacity per expert: full, unfilled and several tiles."""
    n, k = 256, 640
    a, ws = operands(counts, n, k, sum(counts), swiglu=swiglu, tail=3)
    y, dsc, wk = product(counts, n, k, a, ws, out)
    abi.mx4_check(dsc, wk)
    assert_product(y, counts, n, k, a, ws, out)
