"""What the block, balance and 4-bit operators refuse, before anything is
launched (these tests run without a GPU): the library on descriptors, pointers
and workspaces, the binding on tensors."""
import pytest
import torch

from dynamic_expert_routing_router_b200 import abi

BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def ptrs(n):
    return [4096 * (i + 1) for i in range(n)]  # never dereferenced


def block(**kw):
    return abi.block_desc(**{**dict(T=4, d=2048, dtype="bf16"), **kw})


def with_fields(dsc, **kw):
    for k, v in kw.items():
        setattr(dsc, k, v)
    return dsc


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(d=-8), 1), (dict(dtype=2), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(eps=9e-31), 1), (dict(res_scale=NAN), 1),
    (dict(branch_scale=INF), 1), (dict(accumulate=2), 1), (dict(d=100), 2), (dict(d=16392), 2)])
def test_block_descriptors(bad, code):
    dsc = with_fields(block(), **bad)
    assert abi.block_workspace_size(dsc) == 0
    L, p = abi.lib(), ptrs(16)
    assert L.beam_block_enter(dsc, *p[:3], None) == code
    assert L.beam_block_exit(dsc, *p[:8], None) == code
    assert L.beam_block_enter_backward(dsc, *p[:7], BIG, None) == code
    assert L.beam_block_exit_backward(dsc, *p[:15], BIG, None) == code
    if code == 1:
        with pytest.raises(abi.BeamError):
            abi.alloc_block_workspace(dsc, "cpu")


def test_block_pointers_and_workspaces():
    L, dsc = abi.lib(), block()
    need = abi.block_workspace_size(dsc)
    assert need >= 4 * 2 * 2048 * 4 and need % 256 == 0
    for i in range(3):
        for v in (0, 4104):
            p = ptrs(3)
            p[i] = v
            assert L.beam_block_enter(dsc, *p, None) == 1
    for i, may_be_null in enumerate((0, 0, 1, 1, 1, 0, 0, 0)):  # res y w gc gt out w_next n_next
        p = ptrs(8)
        p[i] += 8
        assert L.beam_block_exit(dsc, *p, None) == 1
        p[i] = 0
        if not may_be_null:
            assert L.beam_block_exit(dsc, *p, None) == 1
    for i in (0, 1, 2, 4, 5):  # x w dn . dx dw
        p = ptrs(7)
        p[i] = 0
        assert L.beam_block_enter_backward(dsc, *p, need, None) == 1
    for i in range(15 - 1):  # y out w gc gt wn dout dn dres dy dw dgc dgt dwn: each alone
        p = ptrs(15)
        p[i] = 0
        assert L.beam_block_exit_backward(dsc, *p, need, None) == 1, i
        p[i] = 4104
        assert L.beam_block_exit_backward(dsc, *p, need, None) == 1, i
    for ws, size in ((0, need), (4096 + 16, need), (4096, need - 1)):
        assert L.beam_block_enter_backward(dsc, *ptrs(6), ws, size, None) == 3
        assert L.beam_block_exit_backward(dsc, *ptrs(14), ws, size, None) == 3


def balance(**kw):
    base = dict(T=16, E=128, K=8, n_seq=2, has_mask=True)
    fields = {k: kw.pop(k) for k in list(kw) if k not in base}
    return with_fields(abi.balance_desc(**{**base, **kw}), **fields)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(E=257), 1), (dict(K=0), 1), (dict(K=17), 1),
    (dict(E=4), 1), (dict(n_seq=0), 1), (dict(logits_ld=255), 1), (dict(has_mask=False, logits_ld=127), 1),
    (dict(has_mask=False, count_kept=1, logits_ld=256), 1), (dict(count_kept=2), 1),
    (dict(mask_logit_threshold=NAN), 1), (dict(coef=INF), 1), (dict(coef=NAN), 1),
    (dict(n_seq=(1 << 20) + 1), 2), (dict(T=1 << 30), 2)])
def test_balance_descriptors(bad, code):
    dsc = balance(**bad)
    assert abi.balance_workspace_size(dsc) == 0
    L, p = abi.lib(), ptrs(7)
    assert L.beam_moe_balance(dsc, *p, BIG, None) == code
    assert L.beam_moe_balance_backward(dsc, *p[:5], None) == code


def test_balance_pointers_and_workspaces():
    L, dsc = abi.lib(), balance()
    need = abi.balance_workspace_size(dsc)
    for i in range(6):  # logits seq loss cand kept prob
        p = ptrs(7)
        p[i] += 4
        assert L.beam_moe_balance(dsc, *p, need, None) == 1
        p[i] = 0
        if i < 4:
            assert L.beam_moe_balance(dsc, *p, need, None) == 1
    for i in range(5):  # logits seq counts dloss dlogits
        p = ptrs(5)
        p[i] += 4
        assert L.beam_moe_balance_backward(dsc, *p, None) == 1
        p[i] = 0
        if i != 3:
            assert L.beam_moe_balance_backward(dsc, *p, None) == 1
    assert L.beam_moe_balance(balance(has_mask=False), *ptrs(7), need, None) == 1  # kept, no mask
    for ws, size in ((0, need), (4096 + 16, need), (4096, need - 1)):
        assert L.beam_moe_balance(dsc, *ptrs(6), ws, size, None) == 3


def test_backward_aux_checks_its_gradient():
    dsc = abi.desc(8, 2048, 128, 768, 8, "bf16", 1)
    L, p = abi.lib(), ptrs(16)

    def call(dlogits, beta=0.1):
        return L.beam_moe_backward_aux(dsc, *p[:7], dlogits, beta, *p[7:14], BIG, None)
    assert call(4100) == 1 and call(4096, NAN) == 1
    with pytest.raises(abi.BeamError) as e:
        abi.backward(dsc, *[None] * 7, 0.0, *[None] * 6, None, dlogits=torch.zeros(8, 64))
    assert e.value.status == 1


@pytest.mark.parametrize("bad,code", [
    (dict(N=-1), 1), (dict(E=0), 1), (dict(E=257), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(swiglu=2), 1),
    (dict(out_dtype=3), 1), (dict(n=64), 2), (dict(k=96), 2), (dict(E=256, n=1 << 24), 2), (dict(N=1 << 30), 2)])
def test_product_descriptors(bad, code):
    dsc = with_fields(abi.mx4_desc(64, 8, 256, 512, swiglu=True), **bad)
    assert abi.mx4_workspace_size(dsc) == 0
    L, p = abi.lib(), ptrs(9)
    assert L.beam_mx4_expert_product(dsc, *p, BIG, None) == code
    assert L.beam_mx4_check(dsc, p[0], None) == code


def test_product_pointers_and_workspaces():
    L = abi.lib()
    dsc, plain = abi.mx4_desc(64, 8, 256, 512, swiglu=True), abi.mx4_desc(64, 8, 256, 512)
    need = abi.mx4_workspace_size(dsc)
    for i in range(8):  # a, its scales, counts, w, its scales, w3, its scales, out
        for v in (0, 4104):
            p = ptrs(9)
            p[i] = v
            assert L.beam_mx4_expert_product(dsc, *p, need, None) == 1, (i, v)
    assert L.beam_mx4_expert_product(plain, *ptrs(9), need, None) == 1  # w3 without swiglu
    for ws, size in ((0, need), (4096 + 16, need), (4096, need - 1)):
        assert L.beam_mx4_expert_product(dsc, *ptrs(8), ws, size, None) == 3
    assert L.beam_mx4_check(dsc, 0, None) == 3


def test_quantize_arguments():
    L, p = abi.lib(), ptrs(4)  # x, n_rows, codes, scales

    def q(dtype=0, rows=4, cols=64, x=p[0], n=None, codes=p[2], scales=p[3], tiled=0):
        return L.beam_mx4_quantize(dtype, rows, cols, x, n, codes, scales, tiled, None)

    def dq(dtype=0, rows=4, cols=64, codes=p[2], scales=p[3], tiled=0, out=p[0]):
        return L.beam_mx4_dequantize(dtype, rows, cols, codes, scales, tiled, out, None)
    for f in (q, dq):
        assert f(dtype=2) == 1 and f(rows=-1) == 1 and f(cols=0) == 1 and f(tiled=2) == 1
        assert f(cols=48) == 2 and f(tiled=1) == 2 and f(rows=128, cols=64, tiled=1) == 2
        assert f(rows=1 << 50, cols=1 << 20) == 2
        for k in ("codes", "scales"):
            assert f(**{k: 0}) == 1 and f(**{k: 4104}) == 1
        assert f(rows=0) == 0
    assert q(x=0) == 1 and q(x=4104) == 1 and dq(out=0) == 1 and dq(out=4104) == 1
    assert q(n=4098) == 1 and q(rows=128, cols=128, tiled=1, n=4096) == 1


def test_the_binding_refuses_what_the_library_cannot_see():
    """Another dtype, shape, stride or device: an error that names the tensor."""
    dsc, bf = block(T=4, d=64), torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)

    def says(text, status, f, *a, **kw):
        with pytest.raises(abi.BeamError) as e:
            f(*a, **kw)
        assert text in str(e.value) and e.value.status == status, e.value
    says("x has to be", 1, abi.block_enter, dsc, x.float(), w, x)
    says("x has to be", 1, abi.block_enter, dsc, x[:3], w, x)
    says("x has to be", 1, abi.block_enter, dsc, torch.zeros(64, 4, dtype=bf).t(), w, x)
    says("not the current CUDA device", 1, abi.block_enter, dsc, x, w, x)
    says("is missing", 1, abi.block_enter, dsc, None, w, x)
    with pytest.raises(TypeError):
        abi.block_enter(None, x, w, x)
    says("go together", 1, abi.block_exit, dsc, x, x, x, w_next=w)
    says("go together", 1, abi.block_exit_backward, dsc, x, x, x, x, x, w_out=w)
    says("workspace is missing", 3, abi.block_exit_backward, dsc, x, x, x, x, None)
    says("workspace has to be", 1, abi.block_enter_backward, dsc, x, w, x.float(), x, w.float(), x)
    b = balance(T=4, n_seq=2, has_mask=False)
    lg, i32 = torch.zeros(4, 128), torch.int32
    u8 = torch.zeros(64, dtype=torch.uint8)
    table = torch.zeros(2, 128, dtype=i32)
    seq = torch.zeros(3, dtype=i32)
    says("not the current", 1, abi.balance, b, lg, torch.zeros(1), table, u8, seq_begin=seq)
    says("seq_begin has to be", 1, abi.balance, b, lg, torch.zeros(1), table, u8, seq_begin=seq[1:])
    says("workspace is missing", 3, abi.balance, b, lg, torch.zeros(1), table, None)
    says("without a mask", 1, abi.balance, b, lg, lg, lg, u8, kept_counts=lg)
    says("logits has to be", 1, abi.balance_backward, b, lg[:, :64], lg, lg)
    says("logits has to be", 1, abi.balance_backward, b, lg.double(), torch.zeros(2, 128, dtype=i32), lg)
    says("a bf16 or f32 matrix", 1, abi.mx4_quantize, x.double(), u8, u8)
    says("no multiple of 32", 2, abi.mx4_quantize, x[:, :40].contiguous(), u8, u8)
    m = abi.mx4_desc(4, 2, 128, 128)
    a, s, c = torch.zeros(4, 64).byte(), torch.zeros(4, 4).byte(), torch.zeros(2, dtype=i32)
    says("second weight without swiglu", 1, abi.mx4_expert_product, m, a, s, c, a, s, x, u8, w3_codes=a)
    says("workspace is missing", 3, abi.mx4_expert_product, m, a, s, c, a, s, x, None)
    says("a_codes has to be", 1, abi.mx4_expert_product, m, a[:, :32], s, c, a, s, x, u8)
