"""The MLP block on inputs of any layout and with some of its parameters frozen."""
import pytest

pytestmark = pytest.mark.gpu

WIDTH, HIDDEN = 64, 96


def block():
    import torch
    from gradient_compression_ddp_amd.mlp_block import MlpBlock8
    torch.manual_seed(1)
    b = MlpBlock8(WIDTH, HIDDEN, device="cuda")
    with torch.no_grad():
        b.ln_w.uniform_(0.5, 1.5)
        b.ln_b.normal_(0, 0.2)
    return b


LAYOUTS = {
    "one sequence, transposed": lambda g: g(1, WIDTH, 5).transpose(1, 2),
    "two sequences, transposed": lambda g: g(2, WIDTH, 5).transpose(1, 2),
    "transposed matrix": lambda g: g(WIDTH, 7).t(),
    "every second column": lambda g: g(6, 2 * WIDTH)[:, ::2],
    "columns of wider rows": lambda g: g(6, WIDTH + 3)[:, 2:2 + WIDTH],
    "one row repeated": lambda g: g(1, WIDTH).expand(9, WIDTH),
    "one value repeated": lambda g: g(4, 1).expand(4, WIDTH),
    "one row, strided": lambda g: g(WIDTH, 3).t()[:1],
    "a vector": lambda g: g(WIDTH),
}


@pytest.mark.parametrize("layout", LAYOUTS)
def test_any_strides(layout):
    """The layout changes nothing but where the values lie: the same bits as with a copy without gaps."""
    import torch
    b = block()
    leaf = []

    def g(*shape):
        leaf.append(torch.randn(*shape, device="cuda", requires_grad=True))
        return leaf[0]
    x = LAYOUTS[layout](g)
    plain = x.detach().contiguous().requires_grad_()
    d = torch.randn(plain.shape, device="cuda")
    y, want = b(x), b(plain)
    assert y.shape == x.shape and torch.equal(y, want)
    want.backward(d)
    grads = [p.grad for p in b.parameters()]
    b.zero_grad(set_to_none=True)
    y.backward(d)
    assert all(torch.equal(p.grad, q) for p, q in zip(b.parameters(), grads))
    # the leaf's gradient is what its views make of the plain one's
    again, = torch.autograd.grad(x, leaf[0], plain.grad, retain_graph=True) if x is not leaf[0] else (plain.grad,)
    assert torch.equal(leaf[0].grad, again)
    # and the incoming gradient may have any layout
    b.zero_grad(set_to_none=True)
    plain.grad = None
    b(plain).backward(torch.ones(1, device="cuda").expand(plain.shape))
    assert all(torch.isfinite(p.grad).all() for p in b.parameters())


@pytest.fixture
def calls(monkeypatch):
    """What the block asks of the operators: {name: number of calls}, and the checkpoints that it has made."""
    from gradient_compression_ddp_amd import mlp_block as m
    seen = {"linear_wgrad": 0, "act_backward": 0, "layernorm_backward": 0, "packs": 0}

    def counted(name):
        f = getattr(m, name)

        def call(*a, **k):
            if name in seen:
                seen[name] += 1
            seen["packs"] += k.get("pack_x", False) + k.get("pack_y", False)
            return f(*a, **k)
        monkeypatch.setattr(m, name, call)
    for name in ("linear_wgrad", "act_backward", "layernorm_backward", "layernorm_forward", "act_forward"):
        counted(name)
    return seen


NAMES = ("ln_w", "ln_b", "w1", "b1", "w2", "b2")
# what needs a gradient: checkpoints packed, and calls of linear_wgrad, act_backward and layernorm_backward
NEEDS = {
    ("x",) + NAMES: (4, 2, 1, 1),
    NAMES: (4, 2, 1, 1),
    ("x",): (2, 0, 1, 1),
    ("ln_b",): (2, 0, 1, 1),
    ("w1", "b1"): (2, 1, 1, 0),
    ("b1",): (2, 1, 1, 0),
    ("w2",): (1, 1, 0, 0),
    ("b2",): (1, 1, 0, 0),
    ("w1", "w2"): (3, 2, 1, 0),
    ("x", "w2", "b2"): (3, 1, 1, 1),
    (): (0, 0, 0, 0),
}


@pytest.mark.parametrize("needs", NEEDS, ids="+".join)
def test_only_needed_gradients(calls, needs):
    """Frozen parameters cost no product and no checkpoint, and leave the other gradients as they are."""
    import torch
    b = block()
    x = torch.randn(20, WIDTH, device="cuda")
    d = torch.randn(20, WIDTH, device="cuda")
    full = x.clone().requires_grad_()
    b(full).backward(d)
    want = {"x": full.grad, **{n: getattr(b, n).grad for n in NAMES}}
    calls.update(dict.fromkeys(calls, 0))
    b.zero_grad(set_to_none=True)
    for n in NAMES:
        getattr(b, n).requires_grad_(n in needs)
    y = b(x.requires_grad_("x" in needs))
    assert y.requires_grad == bool(needs)
    if needs:
        y.backward(d)
    for n in ("x",) + NAMES:
        got = x.grad if n == "x" else getattr(b, n).grad
        assert (got is None) == (n not in needs), n
        assert got is None or torch.equal(got, want[n]), n
    assert (calls["packs"], calls["linear_wgrad"], calls["act_backward"], calls["layernorm_backward"]) == NEEDS[needs]


def test_no_grad_packs_nothing(calls):
    import torch
    b = block()
    x = torch.randn(20, WIDTH, device="cuda", requires_grad=True)
    want = b(x).detach()
    calls["packs"] = 0
    with torch.no_grad():
        assert torch.equal(b(x), want)
    assert calls["packs"] == 0


def test_part_of_the_gradients_asked_for():
    """torch.autograd.grad for one of the parameters, and the rest later."""
    import torch
    b = block()
    x = torch.randn(20, WIDTH, device="cuda", requires_grad=True)
    d = torch.randn(20, WIDTH, device="cuda")
    y = b(x)
    w2, = torch.autograd.grad(y, b.w2, d, retain_graph=True)
    y.backward(d)
    assert torch.equal(w2, b.w2.grad)
