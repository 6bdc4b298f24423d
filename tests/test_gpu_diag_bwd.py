"""GPU parity of the diagonal scan's and the conv's gradients: against autograd
through the float64 definitions of diag_ref (themselves checked against
differences in test_diag_host), and directly against differences of the
float64 loss along random directions."""
import pytest
import torch

import diag_ref as R
import ssd_selective_scan_b200 as ssd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])

SCANS = {   # b, L, E, N, G
    "one_token": (3, 1, 64, 16, 1),
    "short": (2, 5, 40, 16, 1),
    "eight": (1, 8, 64, 16, 1),
    "nine": (1, 9, 72, 16, 3),
    "tile_and_one": (2, 17, 136, 16, 1),
    "tiles": (2, 70, 64, 16, 1),
    "n4": (2, 19, 264, 4, 1),
    "n8": (1, 70, 144, 8, 2),
    "n12": (2, 45, 24, 12, 1),
    "n24": (1, 67, 48, 24, 2),
    "n32": (2, 33, 16, 32, 1),
    "n64": (2, 35, 24, 64, 3),
    "cut": (1, 600, 16, 16, 1),
    "cut_batch": (2, 390, 24, 8, 1),
    "cut_n64": (1, 300, 16, 64, 2),
}
ROWS = ("u", "dt_raw", "B", "C", "z")


def case(name, full, dtype, seed):
    b, L, E, N, G = SCANS[name]
    p = R.scan_inputs((b, L), E, N, G, dtype, seed=seed, z=full, bias=full, D=full, device="cuda", pad=int(full))
    g = torch.Generator().manual_seed(seed + 1)
    init = 0.5 * torch.randn(b, E, N, generator=g) if full else None
    dfinal = torch.randn(b, E, N, generator=g) if full else None
    dy = torch.randn(b, L, E, generator=g).to(dtype)
    return p, init, dfinal, dy


def loss(d, init, dfinal, dy):
    """sum(y dy) + sum(final dfinal) of float64 inputs."""
    total = 0.0
    E, N = d["A"].shape
    for i in range(dy.shape[0]):
        one = {k: (v[i] if v is not None and k in ROWS else v) for k, v in d.items()}
        y, h = R.scan(one, torch.zeros(E, N, dtype=torch.float64) if init is None else init[i])
        total = total + (y * dy[i]).sum()
        if dfinal is not None:
            total = total + (h[-1] * dfinal[i]).sum()
    return total


NAMES = dict(u="du", dt_raw="ddt_raw", z="dz", B="dB", C="dC", A="dA", D="dD", dt_bias="ddt_bias")


@DTYPES
@pytest.mark.parametrize("name", sorted(SCANS))
@pytest.mark.parametrize("full", [True, False], ids=["all", "bare"])
def test_scan_bwd(name, full, dtype):
    p, init, dfinal, dy = case(name, full, dtype, seed=len(name))
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    r = ssd.diag_scan_bwd(**p, dy=on(dy), init_state=on(init), dfinal=on(dfinal), want_dinit=full)
    d = R.f64(p)
    b, L, E = dy.shape
    if not full:    # D and dt_bias default to zero and still have gradients
        d |= dict(D=torch.zeros(E, dtype=torch.float64), dt_bias=torch.zeros(E, dtype=torch.float64))
        assert r["dz"] is None and r["dinit"] is None
    leaves = {k: v.requires_grad_() for k, v in d.items() if v is not None}
    init64 = None if init is None else init.double().requires_grad_()
    total = loss(leaves | {k: None for k in d if d[k] is None}, init64, None if dfinal is None else dfinal.double(), dy.double())
    wrt = list(leaves.items()) + ([("init", init64)] if full else [])
    for (k, _), ref in zip(wrt, torch.autograd.grad(total, [v for _, v in wrt])):
        got = r["dinit"] if k == "init" else r[NAMES[k]]
        R.close(got, ref.reshape(got.shape), NAMES.get(k, "dinit"))


def test_scan_bwd_against_differences():
    """The loss along a random direction of every input at once: the central
    difference of the float64 loss, step 1e-5 (its own error is below 1e-8 of
    the slope), against the gradients' product with the direction."""
    p, init, dfinal, dy = case("nine", True, F32, seed=77)
    r = ssd.diag_scan_bwd(**p, dy=dy.cuda(), init_state=init.cuda(), dfinal=dfinal.cuda())
    d, g = R.f64(p) | dict(init=init.double()), torch.Generator().manual_seed(5)
    for k in d:
        way = {q: torch.zeros_like(v) for q, v in d.items()}
        way[k] = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        at = lambda s: {q: v + s * way[q] for q, v in d.items()}  # noqa: E731
        f = lambda s: loss({q: v for q, v in at(s).items() if q != "init"}, at(s)["init"], dfinal.double(), dy.double())  # noqa: E731
        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        got = r["dinit"] if k == "init" else r[NAMES[k]]
        terms = got.double().cpu().reshape(way[k].shape) * way[k]
        assert abs(terms.sum() - slope) <= R.C_SCAN * terms.abs().sum(), k


def test_scan_bwd_handed_over_state():
    """The gradient of two halves, dinit of the second being dfinal of the
    first, is that of the whole."""
    p, init, dfinal, dy = case("tiles", True, F32, seed=21)
    dyd, init, dfinal = dy.cuda(), init.cuda(), dfinal.cuda()
    whole = ssd.diag_scan_bwd(**p, dy=dyd, init_state=init, dfinal=dfinal)
    cut = lambda a, b: {k: (v[:, a:b].contiguous() if v is not None and k in ROWS else v) for k, v in p.items()}  # noqa: E731
    _, mid = ssd.diag_scan_fwd(**cut(0, 29), init_state=init)
    two = ssd.diag_scan_bwd(**cut(29, 70), dy=dyd[:, 29:].contiguous(), init_state=mid, dfinal=dfinal)
    one = ssd.diag_scan_bwd(**cut(0, 29), dy=dyd[:, :29].contiguous(), init_state=init, dfinal=two["dinit"])
    for k in ("du", "ddt_raw", "dz", "dB", "dC"):
        R.close(torch.cat([one[k], two[k]], 1), whole[k].double(), k)
    for k in ("dA", "dD", "ddt_bias"):
        R.close(one[k] + two[k], whole[k].double(), k)
    R.close(one["dinit"], whole["dinit"].double(), "dinit")


def test_scan_bwd_empty_and_repeated():
    p, init, dfinal, dy = case("cut", True, BF16, seed=4)
    on = dict(dy=dy.cuda(), init_state=init.cuda(), dfinal=dfinal.cuda())
    a, b = ssd.diag_scan_bwd(**p, **on), ssd.diag_scan_bwd(**p, **on)
    assert all(torch.equal(a[k], b[k]) for k in a)
    none = {k: (v[:, :0] if v is not None and k in ROWS else v) for k, v in p.items()}
    r = ssd.diag_scan_bwd(**none, dy=on["dy"][:, :0].contiguous(), init_state=on["init_state"], dfinal=on["dfinal"])
    assert (r["dA"] == 0).all() and (r["dD"] == 0).all() and (r["ddt_bias"] == 0).all() and torch.equal(r["dinit"], on["dfinal"])


def test_scan_bwd_masked_rows():
    """dt_raw = -inf: the row passes the state and its gradient on unchanged."""
    p, init, dfinal, dy = case("tiles", True, F32, seed=8)
    p["dt_raw"][:, 20:50] = -float("inf")
    p["B"][:, 20:50] = p["C"][:, 20:50] = 0
    r = ssd.diag_scan_bwd(**p, dy=dy.cuda(), init_state=init.cuda(), dfinal=dfinal.cuda())
    keep = [*range(20), *range(50, 70)]
    less = {k: (v[:, keep] if v is not None and k in ROWS else v) for k, v in p.items()}
    less |= {k: less[k].contiguous() for k in ("u", "dt_raw", "z", "B", "C")}
    want = ssd.diag_scan_bwd(**less, dy=dy[:, keep].contiguous().cuda(), init_state=init.cuda(), dfinal=dfinal.cuda())
    for k in ("du", "ddt_raw", "dz", "dB", "dC"):
        R.close(r[k][:, keep], want[k].double(), k)
    R.close(r["dA"], want["dA"].double(), "dA")
    R.close(r["dinit"], want["dinit"].double(), "dinit")
    assert (r["ddt_raw"][:, 20:50] == 0).all()


# ---------------------------------------------------------------------------
# conv

CONVS = [(1, 1, 8, True), (2, 2, 40, True), (2, 3, 24, False), (1, 4, 520, True), (3, 63, 16, True), (1, 64, 16, False), (2, 65, 24, True),
         (1, 66, 16, True), (1, 200, 1032, True)]


@DTYPES
@pytest.mark.parametrize("k", [2, 3, 4])
@pytest.mark.parametrize("b,L,E,full", CONVS)
def test_conv_bwd(b, L, E, full, k, dtype):
    g = torch.Generator().manual_seed(L + k)
    x, dout = torch.randn(b, L, E, generator=g).to(dtype), torch.randn(b, L, E, generator=g).to(dtype)
    w, bias = 0.5 * torch.randn(E, k, generator=g), 0.3 * torch.randn(E, generator=g) if full else None
    st = torch.randn(b, E, k, generator=g).to(dtype) if full else None
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    r = ssd.conv1d_silu_bwd(on(x), on(w), on(dout), on(bias), on(st))
    leaf = lambda t, like: (torch.zeros(like, dtype=torch.float64) if t is None else t.double()).requires_grad_()  # noqa: E731
    lx, lw, lb, ls = leaf(x, None), leaf(w, None), leaf(bias, (E,)), leaf(st, (b, E, k))
    total = sum((R.conv(torch.cat([ls[i].t(), lx[i]]), lw, lb) * dout[i].double()).sum() for i in range(b))
    gx, gw, gb, gs = torch.autograd.grad(total, [lx, lw, lb, ls])
    # 4 products of rounded float32 terms, SiLU' and its exponential: as C_CONV,
    # doubled for the second factor; the sums over rows add sqrt(600) 2^-24
    R.close(r["dx"], gx, "dx", c=2 * R.C_CONV)
    R.close(r["dw"], gw, "dw", c=1e-5)
    if full:
        R.close(r["dbias"], gb, "dbias", c=1e-5)
        R.close(r["dconv_state"], gs, "dconv_state", c=2 * R.C_CONV)
        assert (r["dconv_state"][:, :, 0] == 0).all()
    else:
        assert r["dbias"] is None and r["dconv_state"] is None


def test_conv_bwd_long_tiles():
    """Enough channels and rows for the 256-row tiles, the last one short."""
    test_conv_bwd(10, 270, 7608, True, 4, BF16)


def test_conv_bwd_empty():
    w = torch.randn(16, 4, device="cuda")
    x = torch.zeros(2, 0, 16, device="cuda")
    r = ssd.conv1d_silu_bwd(x, w, x, torch.zeros(16, device="cuda"), torch.ones(2, 16, 4, device="cuda"))
    assert (r["dw"] == 0).all() and (r["dbias"] == 0).all() and (r["dconv_state"] == 0).all() and r["dx"].shape == (2, 0, 16)


def test_conv_and_scan_bwd_in_a_graph():
    """A training step's gradients, captured and replayed on new inputs."""
    b, L, E, N = 2, 40, 64, 16
    p, init, dfinal, dy = R.scan_inputs((b, L), E, N, 1, F32, seed=3, device="cuda"), None, None, None
    x, w, dy = torch.randn(b, L, E, device="cuda"), torch.randn(E, 4, device="cuda"), torch.randn(b, L, E, device="cuda")
    rest = {k: v for k, v in p.items() if k != "u"}

    def step():
        u = ssd.conv1d_silu(x, w)
        r = ssd.diag_scan_bwd(u=u, dy=dy, **rest)
        return ssd.conv1d_silu_bwd(x, w, r["du"])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn(b, L, E))
        dy.copy_(torch.randn(b, L, E))
        graph.replay()
        got = {k: out[k].clone() for k in ("dx", "dw")}
        want = step()
        assert all(torch.equal(got[k], want[k]) for k in got)
