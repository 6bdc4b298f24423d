"""The diagonal scan's calls on paths that only some sizes take (dense batches
that are not cut, packed ones taken longest first, long gradient pieces, pools
past 2^32 elements), from several threads and on other streams, and what NaN in
one row reaches in the gradients."""
import threading

import pytest
import torch

import diag_ref as R
import ssd_selective_scan_b200 as ssd
import test_gpu_diag as fwd
import test_gpu_diag_bwd as bwd
import test_gpu_diag_edges as edges

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def test_dense_scan_that_is_not_cut_takes_no_workspace():
    """16384 sequences of one token, and 600 of 100: results, and what the call
    allocates beside them."""
    for b, L, E in ((16384, 1, 128), (600, 100, 64)):
        p = R.scan_inputs((b, L), E, 16, 1, F32, seed=b, device="cuda")
        init = 0.5 * torch.randn(b, E, 16, device="cuda")
        y, fs = torch.empty(b, L, E, device="cuda"), torch.empty_like(init)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        held = torch.cuda.memory_allocated()
        ssd.diag_scan_fwd(**p, init_state=init, y=y, final_state=fs)
        assert torch.cuda.max_memory_allocated() == held
        some = [0, 1, b // 2, b - 1]
        ry, rf = fwd.dense_ref({k: (v[some] if v is not None and k in ("u", "dt_raw", "B", "C", "z") else v) for k, v in p.items()}, init[some])
        R.close(y[some], ry, "y")
        R.close(fs[some], rf, "final state")


# Enough channel tiles that one sequence alone fills the device (no cut), and
# at least 128 rows to a request on average (longest first): lens, ctx, block, E, N, G
WIDE = {
    "n16": ([400, 0, 129, 260, 1, 130], [0, 3, 70, 64, 9, 0], 64, 6400, 16, 1),
    "n64": ([129, 257, 3, 258], [5, 0, 0, 33], 100, 1600, 64, 2),
    "equal_lengths": ([130, 130, 130], [0, 1, 2], 100000, 6400, 16, 1),
}


@DTYPES
@pytest.mark.parametrize("name", sorted(WIDE))
def test_packed_scan_longest_first_and_whole(name, dtype, monkeypatch):
    lens, _, _, E, N, G = WIDE[name]
    rows = sum(lens) + 5      # with those behind the last request
    assert rows >= 128 * len(lens) and ssd.diag_scan_workspace_bytes(len(lens), rows, E, N, G) == 0
    monkeypatch.setitem(fwd.PACKED, name, WIDE[name])
    fwd.test_scan_packed(name, dtype)


@DTYPES
def test_scan_bwd_long_pieces(dtype):
    """24 sequences x 40 tiles of 64 channels, 600 rows: 960 CTAs, pieces of 512
    rows and a short last one.  Only 16 channels have a dy, in tiles far apart,
    so that the definition is that of those alone, dB and dC among it."""
    b, L, E, N = 24, 600, 2560, 16
    p = R.scan_inputs((b, L), E, N, 1, dtype, seed=31, device="cuda")
    some = torch.tensor([*range(0, 4), *range(62, 66), *range(1300, 1304), *range(2556, 2560)])
    g = torch.Generator().manual_seed(32)
    dy, dfinal = torch.zeros(b, L, E, dtype=dtype), torch.zeros(b, E, N)
    dy[:, :, some] = torch.randn(b, L, len(some), generator=g).to(dtype)
    dfinal[:, some] = torch.randn(b, len(some), N, generator=g)
    init = 0.5 * torch.randn(b, E, N, generator=g)
    r = ssd.diag_scan_bwd(**p, dy=dy.cuda(), init_state=init.cuda(), dfinal=dfinal.cuda())
    d = R.f64(p)
    d |= {k: d[k][..., some] for k in ("u", "dt_raw", "z", "dt_bias", "D")} | dict(A=d["A"][some])
    d = {k: v.clone().requires_grad_() for k, v in d.items()}
    di = init[:, some].double().requires_grad_()
    # all sequences side by side: step() takes one, so its formulas, with a leading axis
    dt = R.softplus(d["dt_raw"] + d["dt_bias"])
    h, total = di, 0.0
    for t in range(L):
        h = torch.exp(dt[:, t, :, None] * d["A"]) * h + (dt[:, t] * d["u"][:, t])[..., None] * d["B"][:, t]
        y = ((h * d["C"][:, t]).sum(-1) + d["D"] * d["u"][:, t]) * R.silu(d["z"][:, t])
        total = total + (y * dy[:, t, some].double()).sum()
    (total + (h * dfinal[:, some].double()).sum()).backward()
    for k, name in bwd.NAMES.items():
        got = r[name] if k in ("B", "C") else r[name][some] if k == "A" else r[name][..., some]
        R.close(got, d[k].grad, name)
    R.close(r["dinit"][:, some], di.grad, "dinit")
    rest = torch.ones(E, dtype=torch.bool)
    rest[some] = False
    assert all((r[k][..., rest] == 0).all() for k in ("du", "ddt_raw", "dz", "dD", "ddt_bias"))
    assert (r["dA"][rest] == 0).all() and (r["dinit"][:, rest] == 0).all()


# What a NaN in row 30 of channel 5 of the last sequence reaches, by the
# formulas at the head of diag_scan_bwd.cu: rows of the channel (du, ddt_raw,
# dz) and of its group (dB, dC); the sums and the state gradient of the channel.
# h is NaN from the row on where x or a is; g is NaN before it where a is, and
# up to it where p is.
BEFORE, AT, FROM, UPTO, ALL, NONE = (slice(0, 30), slice(30, 31), slice(30, None), slice(0, 31), slice(0, None), slice(0, 0))
NAN = {
    "u": dict(du=NONE, ddt_raw=FROM, dz=FROM, dB=AT, dC=FROM, dA=True, dD=True, ddt_bias=True, dinit=False),
    "dy": dict(du=UPTO, ddt_raw=UPTO, dz=AT, dB=UPTO, dC=AT, dA=True, dD=True, ddt_bias=True, dinit=True),
    "dt_raw": dict(du=UPTO, ddt_raw=ALL, dz=FROM, dB=UPTO, dC=FROM, dA=True, dD=False, ddt_bias=True, dinit=True),
}


@DTYPES
@pytest.mark.parametrize("what", sorted(NAN))
@pytest.mark.parametrize("name", ["tiles", "n8", "n12", "n64", "cut"])
def test_scan_bwd_nan_in_one_row(name, what, dtype):
    p, init, dfinal, dy = bwd.case(name, True, dtype, seed=14)
    G = bwd.SCANS[name][4]
    p["dy"], at = dy.cuda(), (-1, 30, 5)
    on = dict(init_state=init.cuda(), dfinal=dfinal.cuda())
    p[what] = p[what].clone()
    p[what][at] = 0
    clean = ssd.diag_scan_bwd(**p, **on)
    p[what][at] = float("nan")
    r = ssd.diag_scan_bwd(**p, **on)
    for k, v in r.items():
        want = torch.zeros(v.shape, dtype=torch.bool)
        reach = NAN[what][k]
        if k in ("du", "ddt_raw", "dz"):
            want[-1, reach, 5] = True
        elif k in ("dB", "dC"):
            want[-1, reach, 5 // (dy.shape[2] // G)] = True
        elif k == "dinit":
            want[-1, 5] = reach
        else:
            want[5] = reach
        got = torch.isnan(v).cpu()
        assert torch.equal(got, want), k
        if what in ("u", "dy"):     # (a dt_raw of 0 is no neutral value)
            assert torch.equal(v.cpu()[~want], clean[k].cpu()[~want]), k


# ---------------------------------------------------------------------------
# pools past 2^32 elements


def test_state_offsets_past_32_bits_unsigned():
    """Slots from 32768 on, of 8192 x 16 states each."""
    assert 32768 * 8192 * 16 == 1 << 32
    edges.test_offsets_beyond_32_bits(8, 33000)


@pytest.mark.parametrize("lens", [[1, 1, 1], [40, 3, 70]], ids=["tokens", "prompts"])
def test_conv_cache_offsets_past_32_bits(lens):
    """Caches of 8192 channels x 4 columns in slots from 131072 on: the same
    as in a small pool."""
    E, k, bs, ctx = 8192, 4, 16, [0, 30, 8]
    assert 131072 * E * k == 1 << 32
    g = torch.Generator().manual_seed(6)
    x, w = torch.randn(sum(lens), E, generator=g).to(BF16).cuda(), (0.5 * torch.randn(E, k, generator=g)).cuda()
    q = R.batch(lens, ctx, bs, seed=2)
    held = 0.5 * torch.randn(q["nslots"], E, k, generator=g).to(BF16)

    def run(far):
        cache = torch.empty(far + q["nslots"], E, k, dtype=BF16, device="cuda")
        cache[far:] = held.cuda()
        table = q["table"].copy()
        table[table >= 0] += far
        st = fwd.zero_status()
        m = fwd.call_map(q | dict(table=table, free=q["free"] + far, nslots=far + q["nslots"]), sum(lens), st)
        out = ssd.conv1d_silu_varlen(x, w, cache, m, status=st)
        assert st.item() == 0
        return out, cache[far:].clone()

    for a, b in zip(run(131072), run(0)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# other buffers, threads, streams, modes


@pytest.mark.parametrize("before,now", [(2, 5), (5, 2)])
def test_state_map_out_of_another_batch(before, now):
    """Refused on the host, before anything is launched."""
    q = R.batch([1] * before, [3] * before, 4, spare=9, max_blocks=4)
    old = fwd.call_map(q, 8)
    new = R.batch([1] * now, [3] * now, 4, spare=9, max_blocks=4)
    with pytest.raises(ValueError, match="requests"):
        fwd.call_map(new, 8, out=old._replace(table=fwd.up(new["table"])))
    fwd.assert_map(fwd.call_map(q, 8, out=old), R.ref_map(q, 8))


def every_call(stream=None):
    """A map, a prompt step, a token step and both gradients; all they give."""
    E, N, k, bs, lens = 64, 16, 4, 16, [40, 0, 300, 7]
    q = R.batch(lens, [0, 5, 16, 3], bs, seed=4, spare=8)
    T = sum(lens)
    on = dict(stream=stream)
    g = torch.Generator().manual_seed(8)
    states, cache = torch.randn(q["nslots"], E, N, generator=g).cuda(), torch.randn(q["nslots"], E, k, generator=g).cuda()
    w = torch.randn(E, k, generator=g).cuda()
    p, one = (R.scan_inputs((n,), E, N, 1, F32, seed=n, device="cuda") for n in (T, len(lens)))
    d = R.scan_inputs((2, 700), E, N, 1, F32, seed=5, device="cuda")
    x, dy = torch.randn(2, 700, E, generator=g).cuda(), torch.randn(2, 700, E, generator=g).cuda()
    lens_d, ones, ctx = fwd.up(lens), fwd.up([1] * len(lens)), fwd.up(q["ctx"])
    table, free, head, after, st = fwd.up(q["table"]), fwd.up(q["free"]), fwd.up([0]), ctx + lens_d, fwd.zero_status()
    cur = torch.cuda.current_stream()
    if stream is not None:
        stream.wait_stream(cur)
    m = ssd.state_map(lens_d, ctx, table, free, head, T, bs, q["nslots"], status=st, **on)
    u = ssd.conv1d_silu_varlen(p["u"], w, cache, m, status=st, **on)
    y = ssd.diag_scan_fwd_varlen(**(p | dict(u=u)), states=states, m=m, status=st, **on)
    m2 = ssd.state_map(ones, after, m.table, free, m.free_head, len(lens), bs, q["nslots"], status=st, **on)
    u2 = ssd.conv1d_silu_varlen(one["u"], w, cache, m2, status=st, **on)
    y2 = ssd.diag_state_update(states, u2, one["dt_raw"], one["A"], one["B"], one["C"], m2, dt_bias=one["dt_bias"], D=one["D"], z=one["z"],
                               status=st, **on)
    yd, fs = ssd.diag_scan_fwd(**d, **on)
    r = ssd.diag_scan_bwd(**d, dy=dy, **on)
    c = ssd.conv1d_silu_bwd(x, w, dy, **on)
    if stream is not None:
        cur.wait_stream(stream)
    cur.synchronize()
    assert st.item() == 0
    return [*m[:7], u, y, *m2[:7], u2, y2, yd, fs, *r.values(), c["dx"], c["dw"], states, cache]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(v, w) for v, w in zip(a, b))


def test_every_call_on_another_stream():
    want = every_call()
    for _ in range(3):
        assert same(every_call(torch.cuda.Stream()), want)


def test_every_call_in_inference_mode():
    want = every_call()
    with torch.inference_mode():
        assert same(every_call(), want)


def test_every_call_from_threads():
    """Four threads at once, each with a stream of its own as the current one."""
    want, wrong = every_call(), []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    if not same(every_call(), want):
                        wrong.append("results differ")
        except Exception as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
