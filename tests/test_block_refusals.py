"""What the residual block's classes refuse before anything is launched (these
tests run without a GPU): the calls below them take addresses and sizes, so a
batch of another size would be read or written past its end."""
import pytest
import torch

from dynamic_expert_routing_router_b200 import abi, block

T, D, E, I, K = 6, 128, 8, 256, 2
BF16 = torch.bfloat16


def weights(dtype=BF16, **other):
    shapes = dict(Wg=(E, D), Wm=(E, D), W1=(E, I, D), W3=(E, I, D), W2=(E, D, I))
    return {k: other.get(k, torch.zeros(s, dtype=dtype)) for k, s in shapes.items()}


@pytest.fixture
def no_launches(monkeypatch):
    """CPU tensors count as the current device's; every launch fails the test
    (but for the weights' quantisation)."""
    monkeypatch.setattr(abi, "_current_device", lambda: -1)
    monkeypatch.setattr(abi, "mx4_quantize", lambda *a, **kw: None)
    launches = []
    for f in ("route", "ep_dispatch", "mx4_expert_product", "ep_combine", "forward", "block_enter"):
        monkeypatch.setattr(abi, f, lambda *a, f=f, **kw: launches.append(f))
    return launches


def refused(text, f, *a, **kw):
    with pytest.raises(abi.BeamError) as e:
        f(*a, **kw)
    assert e.value.status == 1 and text in str(e.value), e.value


def test_experts_take_rows_of_their_own_size(no_launches):
    ex = block.Mx4Experts(T, D, E, I, K, 1, *weights().values())
    x, out, lg = torch.zeros(T, D, dtype=BF16), torch.zeros(T, D, dtype=BF16), torch.zeros(T, 2 * E)
    for bad in (x[:4], torch.zeros(T + 1, D, dtype=BF16), x.float(), x[:, :64], torch.zeros(D, T, dtype=BF16).t()):
        refused("x has to be", ex.forward, bad, out)
        refused("out has to be", ex.forward, x, bad)
    for bad in (lg[:, :E], lg[:5], lg.to(BF16)):
        refused("logits has to be", ex.forward, x, out, logits=bad)
    refused("x is missing", ex.forward, None, out)
    refused("tensors on cpu and meta", ex.forward, x.to("meta"), out.to("meta"))
    assert no_launches == []
    assert ex.forward(x, out) is out and "ep_combine" in no_launches


def test_experts_take_rows_on_the_current_device(monkeypatch):
    monkeypatch.setattr(abi, "mx4_quantize", lambda *a, **kw: None)
    ex = block.Mx4Experts(T, D, E, I, K, 1, *weights().values())
    x = torch.zeros(T, D, dtype=BF16)
    refused("not the current CUDA device", ex.forward, x, x.clone())


@pytest.mark.parametrize("name,shape", [("Wg", (E, D - 8)), ("Wm", (E + 8, D)), ("W1", (E, D, I)), ("W3", (E - 1, I, D)),
                                        ("W2", (E, I, D))])
def test_experts_weights(no_launches, name, shape):
    refused("has to be", block.Mx4Experts, T, D, E, I, K, 1, *weights(**{name: torch.zeros(shape, dtype=BF16)}).values())
    if name in ("Wg", "Wm"):
        refused("has to be", block.Mx4Experts, T, D, E, I, K, 1, *weights(**{name: torch.zeros(E, D)}).values())
    refused("tensors on", block.Mx4Experts, T, D, E, I, K, 1,
            *weights(**{name: weights()[name].to("meta")}).values())
    assert no_launches == []


def norms(dtype=BF16):
    return [torch.ones(D, dtype=dtype)] * 2


def test_a_block_takes_experts_of_its_own_size_and_type(no_launches):
    ex = block.Mx4Experts(T, D, E, I, K, 1, *weights().values())
    for t, d, e in ((T - 1, D, E), (T + 1, D, E), (T, 2 * D, E), (T, D, 2 * E)):
        with pytest.raises(ValueError):
            block.MoeBlock(t, d, e, I, K, 1, *weights().values(), *norms(), experts=ex)
    with pytest.raises(ValueError):
        block.MoeBlock(T, D, E, I, K, 1, *weights(torch.float32).values(), *norms(torch.float32), dtype="f32",
                       experts=ex)
    refused("tensors on", block.MoeBlock, T, D, E, I, K, 1, torch.zeros(E, D, dtype=BF16, device="meta"), None, None,
            None, None, *norms(), experts=ex)
    # the layer's own weights may be gone
    b = block.MoeBlock(T, D, E, I, K, 1, weights()["Wg"], None, None, None, None, *norms(), experts=ex)
    assert b.experts is ex and no_launches == []


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("name,shape", [("Wg", (E, D - 8)), ("Wm", (E + 8, D)), ("W1", (E, D, I)), ("W3", (E - 1, I, D)),
                                        ("W2", (E, I, D))])
def test_a_blocks_weights(no_launches, name, shape, train):
    f = lambda dtype="bf16", **w: block.MoeBlock(T, D, E, I, K, 1, *weights(**w).values(), *norms(),  # noqa: E731
                                                 dtype=dtype, train=train, balance=0.1)
    f()
    refused("has to be", f, **{name: torch.zeros(shape, dtype=BF16)})
    refused("has to be", f, **{name: weights(torch.float32)[name]})
    refused("has to be", f, **{name: weights()[name].transpose(0, 1).contiguous().transpose(0, 1)})
    refused("tensors on", f, **{name: weights()[name].to("meta")})
    refused("has to be", f, dtype="f32")
    assert no_launches == []


def test_workspaces_start_without_an_error(no_launches):
    """check() before the first backward (or forward) reads the words that no
    call has written yet."""
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)  # fills what torch.empty returns
    try:
        assert (torch.empty(64, dtype=torch.uint8) != 0).all()
        ex = block.Mx4Experts(T, D, E, I, K, 1, *weights().values())
        b = block.MoeBlock(T, D, E, I, K, 1, *weights().values(), *norms(), train=True, balance=0.1)
    finally:
        torch.use_deterministic_algorithms(before)
    for ws in (ex.ws, ex.ws_up, ex.ws_down, b.ws, b.route_ws, b.bwd_ws):
        assert (ws == 0).all()
