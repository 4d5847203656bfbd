"""The training-step operators where their arithmetic, their row walks and their arguments have edges, against the
float64 oracle.  u = 2^-24 is fp32's rounding; the hardware's exp2 and reciprocal are off by 2 u each."""
import numpy as np
import pytest

from oracle import train as o
from test_gpu_train import U, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gc():
    import gradient_compression_ddp_amd as lib
    return lib


# --- the activations' own roundings ---------------------------------------------------------

def p_bound(p, arg, arg_rel):
    """Relative error of p = 1 / (1 + exp(-arg)) in units of u, arg itself off by arg_rel u: the exponent's
    rounding and its constant (1.25 u of arg), exp2 (2), of which p sees the share 1 - p; sum (1), reciprocal (2)."""
    return (1 - p) * (2 + (1.25 + arg_rel) * np.abs(arg)) + 3


@pytest.mark.parametrize("kind,arg_rel", [("silu", 0), ("gelu_tanh", 6)])
@pytest.mark.parametrize("top", [1, 6, 100])
def test_sigmoid_kinds_are_as_exact_as_fp32(gc, kind, arg_rel, top):
    """gelu_tanh's argument: two constants' product (3), the square (1), the sum and the last product (1 each)."""
    import torch
    x = torch.from_numpy(np.linspace(-top, top, 40003)).float().cuda()[None]
    dy = torch.full_like(x, 0.75)
    v, d = host(x), 0.75
    p, s = o.act_parts(v, kind)
    c = np.clip(v, -32, 32)
    arg = v if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (c + 0.044715 * c ** 3)
    e = p_bound(p, arg, arg_rel)
    off = np.abs(host(gc.act_forward(x, kind)[0]) - v * p)
    # 2^-149: the least fp32 number, which p and the result are rounded to at their smallest
    assert (off <= 1.01 * U * (e + 1) * np.abs(v * p) + (1 + np.abs(v)) * 2.0 ** -149).all(), (off / (U * np.abs(v * p) + 1e-300)).max()
    # 1 - p is off by p's error and its own rounding
    rest = e * p + (1 - p)
    if kind == "silu":           # p (1 + x (1 - p))
        b = e * np.abs(p + s) + p * (np.abs(v) * rest + np.abs(1 + v * (1 - p))) + np.abs(p + s)
    else:                        # p + (c u') (p (1 - p)), c u' off by 7 u
        cdu = c * 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * c * c)
        b = e * p + np.abs(s) * (8 + e) + np.abs(cdu) * p * rest + np.abs(p + s)
    got = host(gc.act_backward(dy, kind, x=x))
    off = np.abs(got - d * (p + s))
    assert (off <= 1.01 * U * d * (b + np.abs(p + s)) + (1 + np.abs(v)) ** 3 * 2.0 ** -148).all()


def test_gelu_tail_is_as_exact_as_stated(gc):
    """x Phi(x) for x < 0, in units of u: the exponent z^2/2 (its square, its constant and their product: 2.25 of it), exp2
    (2); t = 1 / (1 + 0.23 z) (4, and R goes at most as t); R's eight steps and constants (6), its fit (1), the two
    last products (2).  Past z = 13.2, where exp(-z^2/2) < 2^-126, 0 is allowed."""
    import torch
    x = torch.from_numpy(np.linspace(-16, 0, 40003)).float().cuda()[None]
    v = host(x)
    want = o.act_forward(v, "gelu")
    off = np.abs(host(gc.act_forward(x, "gelu")[0]) - want)
    bound = 1.01 * U * (15 + 2.25 * v * v / 2) * np.abs(want)
    assert (off <= np.where(v < -13.2, np.abs(want), bound)).all(), (off / (U * np.abs(want) + 1e-300)).max()
    p, s = o.act_parts(v, "gelu")
    # f' = Q - z phi: each by its own bound (phi: the exponent's, its constant and two roundings)
    off = np.abs(host(gc.act_backward(torch.ones_like(x), "gelu", x=x)) - (p + s))
    bound = 1.01 * U * ((15 + 2.25 * v * v / 2) * p + (6 + 2.25 * v * v / 2) * np.abs(s) + np.abs(p + s))
    assert (off <= np.where(v < -13.2, np.abs(p + s), bound)).all()


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_every_bf16_value(gc, kind):
    """All finite bfloat16 inputs: the result is the 64-bit one's nearest bfloat16, wherever it is above the flushed tail."""
    import torch
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x)][None]
    want = torch.from_numpy(o.act_forward(x.double().numpy(), kind))
    got = gc.act_forward(x.cuda(), kind)[0].cpu()
    off = (got != want.bfloat16()) & (want.abs() >= 2.0 ** -100)
    assert not off.any(), (x[off].tolist(), want[off].tolist(), got[off].tolist())
    tail = want.abs() < 2.0 ** -100
    assert (got[tail].double() - want[tail]).abs().max() < 2.0 ** -99


# --- layer norm -----------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("cols", [1, 7, 96, 100, 600, 1025, 2056, 4095, 5000, 8200, 8201, 12300, 16001, 16390])
def test_layernorm_backward_of_rows_far_from_zero(gc, name, cols):
    """|mean| rstd past the largest fp32 number: the columns that exist have no deviation, so every xh is 0 and
    dx = rstd (t - mean(t)); columns past the row's end add nothing.  Sums of t: a chain of at most 16 + 6 terms and
    the team's, as rows / 8192 columns more for the widest; the result's own rounding on top."""
    import torch
    rows = 5
    dt = getattr(torch, name)
    x = torch.full((rows, cols), 2.0 ** 120, device="cuda", dtype=dt)
    g = torch.Generator(device="cuda").manual_seed(cols)
    dy = torch.randn(rows, cols, device="cuda", generator=g).to(dt)
    mean = torch.full((rows,), 2.0 ** 120, device="cuda")
    rstd = torch.full((rows,), 1e-5 ** -0.5, device="cuda")
    t, r = host(dy), host(rstd)[0]
    want = r * (t - t.mean(1, keepdims=True))
    bound = r * (U * (50 * np.abs(t).mean(1, keepdims=True) + 8 * np.abs(t))) + torch.finfo(dt).eps / 2 * np.abs(want)
    for kw in (dict(x=x), dict(ckpt=gc.ckpt_pack(x))):
        dx, dw, db = gc.layernorm_backward(dy, mean, rstd, **kw)
        assert (np.abs(host(dx) - want) <= bound).all(), list(kw)
        assert not dw.any() and torch.isfinite(db).all()
    # and the statistics themselves, where the sum of the row is a number
    if cols < 256:
        y, m, s, _, _ = gc.layernorm_forward(x)
        assert not y.any() and torch.equal(m, mean) and np.abs(host(s) - r).max() <= 4 * U * r


def test_layernorm_backward_of_the_widest_rows(gc):
    """More columns than one launch has threads for: one row of 2^28 + 40, its far end included, and no rows."""
    import torch
    cols = 2 ** 28 + 40
    none, st = torch.zeros(0, cols, device="cuda", dtype=torch.bfloat16), torch.zeros(0, device="cuda")
    dw, db = torch.ones(cols, device="cuda"), torch.ones(cols, device="cuda")
    gc.layernorm_backward(none, st, st, x=none, dw=dw, db=db)
    assert not dw.any() and not db.any()
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(1, cols, device="cuda", generator=g).bfloat16()
    dy = torch.randn(1, cols, device="cuda", generator=g).bfloat16()
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 1.5, device="cuda")
    dx, dw, db = gc.layernorm_backward(dy, mean, rstd, x=x, dw=dw, db=db)
    t = dy[0].double()
    assert torch.equal(db.double(), t)                               # one row: the values themselves
    xh = (x[0].double() - 0.25) * 1.5
    assert ((dw.double() - t * xh).abs() <= 4 * U * (t * xh).abs()).all()
    # a thread's chain of chunk sums: one per 8192 columns, its own and the team's 40 more; the two means enter every column
    chain = (40 + cols / 8192) * U
    want = 1.5 * (t - t.mean() - xh * (t * xh).mean())
    off = (dx[0].double() - want).abs() - 2.0 ** -8 * want.abs()
    assert (off <= 1.5 * (chain * (t.abs().mean() + xh.abs() * (t * xh).abs().mean()) + 16 * U * (t.abs() + xh.abs() + 1))).all()


# --- outputs and inputs in one memory ---------------------------------------------------------

def test_slices_beside_each_other(gc):
    """Every operand a run of columns of one wider matrix: the same bits as apart."""
    import torch
    rows, cols = 37, 101
    wide = torch.randn(rows, 4 * cols + 3, device="cuda").bfloat16()
    x, dy, y, dx = (wide[:, k * cols + 1:(k + 1) * cols + 1] for k in range(4))
    xa, dya = x.clone(), dy.clone()
    w = torch.rand(cols, device="cuda")
    edge = wide[:, [0, -2, -1]].clone()
    gc.act_forward(x, "silu", y=y)
    assert torch.equal(y, gc.act_forward(xa, "silu")[0])
    gc.act_backward(dy, "silu", x=x, dx=dx)
    assert torch.equal(dx, gc.act_backward(dya, "silu", x=xa))
    _, mean, rstd, _, _ = gc.layernorm_forward(x, w, y=y)
    assert torch.equal(y, gc.layernorm_forward(xa, w)[0])
    gc.layernorm_backward(dy, mean, rstd, w, x=x, dx=dx)
    assert torch.equal(dx, gc.layernorm_backward(dya, mean, rstd, w, x=xa)[0])
    assert torch.equal(x, xa) and torch.equal(dy, dya) and torch.equal(wide[:, [0, -2, -1]], edge)


def test_in_place_is_refused(gc):
    import torch
    x = torch.randn(37, 101, device="cuda")
    dy, w = torch.randn_like(x), torch.rand(101, device="cuda")
    _, mean, rstd, ckpt, _ = gc.layernorm_forward(x, pack_x=True)
    wide = torch.randn(37, 150, device="cuda")
    was = [t.clone() for t in (x, dy, wide)]
    for call in (lambda: gc.act_forward(x, y=x), lambda: gc.act_backward(dy, x=x, dx=dy), lambda: gc.act_backward(dy, x=x, dx=x),
                 lambda: gc.act_forward(wide[:, :101], y=wide[:, 49:]), lambda: gc.layernorm_forward(x, y=x),
                 lambda: gc.layernorm_backward(dy, mean, rstd, x=x, dx=dy), lambda: gc.layernorm_backward(dy, mean, rstd, ckpt=ckpt, dx=dy),
                 lambda: gc.layernorm_backward(dy, mean, rstd, w, x=x, dw=w), lambda: gc.layernorm_backward(dy, mean, rstd, x=x, dw=w, db=w),
                 lambda: gc.linear_wgrad(x[:, :30], *ckpt, 101, dw=x[:30])):
        with pytest.raises(gc.GCError, match="overlap"):
            call()
    assert all(torch.equal(a, b) for a, b in zip((x, dy, wide), was))


# --- more rows than blocks, and rows that are not numbers -------------------------------------

# The forward pass gives a block a second row past 8192 rows (teams of 64 threads), 2048 (256) or 1024 (512); the backward
# pass a second and third one past 256 blocks, with several partial sums to join.  Whole and ragged widths of each team.
WALKS = [(8300, 100), (8300, 520), (2100, 1032), (2100, 2049), (2100, 4096), (1100, 8192), (1100, 8201), (1100, 12296), (1100, 16383),
         (600, 16384), (40, 16385)]


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols", WALKS)
def test_layernorm_row_walk(gc, name, rows, cols):
    """Bounds as for one row a block: a thread's chain of at most 16 terms (one more per 8192 columns) and the team's tree."""
    import torch
    dt = getattr(torch, name)
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    x = (rand(rows, cols) * torch.exp(0.5 * rand(cols)) + 0.3 * rand(rows, 1)).to(dt)
    dy = (rand(rows, cols) * rand(rows, 1).abs()).to(dt)
    w, b = 1 + 0.2 * rand(cols), 0.1 * rand(cols)
    y, mean, rstd, xc, yc = gc.layernorm_forward(x, w, b, pack_x=True, pack_y=True)
    # row by row the same as in calls that give every row a team of its own
    some = 500
    for r in range(0, rows, some):
        part = gc.layernorm_forward(x[r:r + some], w, b, pack_x=True, pack_y=True)
        assert torch.equal(part[0], y[r:r + some]) and torch.equal(part[1], mean[r:r + some]) and torch.equal(part[2], rstd[r:r + some])
        for p, q in ((part[3], xc), (part[4], yc)):
            assert torch.equal(p[0], q[0][r:r + some]) and torch.equal(p[1], q[1][r:r + some])
    again = gc.layernorm_forward(x, w, b, pack_x=True, pack_y=True)
    assert all(torch.equal(p, q) for p, q in zip(again[:3], (y, mean, rstd)))
    xv, half = x.double(), torch.finfo(dt).eps / 2
    m = xv.mean(1)
    r = 1 / torch.sqrt((xv - m[:, None]).square().mean(1) + 1e-5)
    chain = 40 + cols / 8192
    dm = chain * U * xv.abs().mean(1) + U * m.abs()
    dr = 0.5 * (2 * chain * U + (dm * r) ** 2) + 4 * U
    assert ((mean.double() - m).abs() <= dm + U * m.abs()).all() and ((rstd.double() - r).abs() <= (dr + U) * r).all()
    xh = (xv - m[:, None]) * r[:, None]
    want = xh * w.double() + b.double()
    bound = w.double().abs() * ((dm * r)[:, None] + xh.abs() * (dr[:, None] + 4 * U)) + (4 * U + half) * want.abs()
    assert ((y.double() - want).abs() <= bound).all()
    # backward, from the statistics as stored
    m, r, dv, wv = mean.double()[:, None], rstd.double()[:, None], dy.double(), w.double()
    for kw, kept in ((dict(ckpt=xc), gc.ckpt_unpack(*xc, cols, dt).double()), (dict(x=x), xv)):
        dx, dw, db = gc.layernorm_backward(dy, mean, rstd, w, **kw)
        xh, t = (kept - m) * r, dv * wv
        want = r * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
        bound = r * U * (8 * t.abs() + (chain + 8) * t.abs().mean(1, keepdim=True) + (chain + 16) * xh.abs() * (t * xh).abs().mean(1, keepdim=True))
        assert ((dx.double() - want).abs() <= bound + half * want.abs()).all(), list(kw)
        assert ((dw.double() - (dv * xh).sum(0)).abs() <= (rows + 8) * U * (dv * xh).abs().sum(0)).all(), list(kw)
        assert ((db.double() - dv.sum(0)).abs() <= rows * U * dv.abs().sum(0)).all(), list(kw)
        for _ in range(3):
            assert all(torch.equal(p, q) for p, q in zip(gc.layernorm_backward(dy, mean, rstd, w, **kw), (dx, dw, db)))


@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("cols", [5, 100, 512, 2049, 4096, 9000, 16390])
def test_layernorm_non_finite_rows(gc, name, cols):
    """A row with an Inf or a NaN has no finite statistics, result or dx, and dw none where it enters; every other
    row, and db, are as without it.  An Inf of dy stays in its row of dx and its column of dw and db."""
    import torch
    dt = getattr(torch, name)
    g = torch.Generator(device="cuda").manual_seed(cols)
    rows, bad = 23, [3, 7, 22]
    x, dy = (torch.randn(rows, cols, device="cuda", generator=g).to(dt) for _ in range(2))
    w, b = torch.rand(cols, device="cuda", generator=g) + 0.5, torch.rand(cols, device="cuda", generator=g)
    fine = [i for i in range(rows) if i not in bad]
    odd = x.clone()
    for i, v in zip(bad, ("inf", "nan", "-inf")):
        odd[i, (i * 37) % cols] = float(v)
    want, got = (gc.layernorm_forward(v, w, b, pack_x=True) for v in (x, odd))
    assert got[0][bad].isnan().all() and got[2][bad].isnan().all() and not torch.isfinite(got[1][bad]).any()
    for p, q in zip(got[:3], want):
        assert torch.equal(p[fine], q[fine])
    for kw, kw_odd in ((dict(x=x), dict(x=odd)), (dict(ckpt=want[3]), dict(ckpt=got[3]))):
        dx, dw, db = gc.layernorm_backward(dy, want[1], want[2], w, **kw)
        dx2, dw2, db2 = gc.layernorm_backward(dy, got[1], got[2], w, **kw_odd)
        assert torch.equal(dx2[fine], dx[fine]) and dx2[bad].isnan().all()
        assert torch.equal(db2, db) and dw2.isnan().all()
        c = 11 % cols
        far = dy.clone()
        far[9, c] = float("inf")
        dx3, dw3, db3 = gc.layernorm_backward(far, want[1], want[2], w, **kw)
        rest, cut = [i for i in range(rows) if i != 9], [i for i in range(cols) if i != c]
        assert torch.equal(dx3[rest], dx[rest]) and not torch.isfinite(dx3[9]).any()
        assert torch.equal(dw3[cut], dw[cut]) and torch.equal(db3[cut], db[cut])
        assert db3[c] == float("inf") and not torch.isfinite(dw3[c])
