"""GPU parity of the diagonal scan's forward calls, the packed conv, the state
map and the single-token update with the float64 definitions of diag_ref,
and what the calls do with odd batches, bad maps, streams and graphs."""
import numpy as np
import pytest
import torch

import diag_ref as R
import ssd_selective_scan_b200 as ssd
from ssd_selective_scan_b200 import SsdError, StateMap

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def up(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a))).to(dtype).cuda()


def zero_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def call_map(q, T, status=None, **kw):
    return ssd.state_map(up(q["lens"]), up(q["ctx"]), up(q["table"]), up(q["free"]), up([q["head"]]), T, q["bs"], q["nslots"],
                         status=status, **kw)


def dev_map(m, bs):
    return StateMap(up(m["cu_seqlens"]), up(m["seq_of"]), up(m["pos_of"]), up(m["slot_of"], torch.int64), up(m["init_slot"]), None, None, bs)


def cuda(p):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}


# ---------------------------------------------------------------------------
# state map


def assert_map(m, ref):
    for k in ("cu_seqlens", "seq_of", "pos_of", "slot_of", "init_slot", "table", "free_head"):
        assert np.array_equal(getattr(m, k).cpu().numpy().reshape(-1), np.asarray(ref[k]).reshape(-1)), k


MAPS = {
    "one_token": ([1], [0], 4),
    "decode": ([1] * 37, list(range(37)), 4),
    "prompts": ([5, 0, 17, 1, 64, 3], [0, 9, 8, 7, 0, 64], 8),
    "block_of_one": ([3, 1, 2], [0, 4, 1], 1),
    "one_block_per_request": ([300, 20, 1], [0, 1, 999], 4096),
    "more_than_a_block_of_threads": ([i % 3 for i in range(2500)], [(7 * i) % 40 for i in range(2500)], 16),
    "many_rows": ([4000, 1, 0, 9000, 12], [0, 100, 5, 33, 0], 100),
    "nothing_new": ([0, 0, 0], [5, 0, 16], 8),
}


@pytest.mark.parametrize("name", sorted(MAPS))
@pytest.mark.parametrize("pad", [0, 5])
def test_state_map(name, pad):
    lens, ctx, bs = MAPS[name]
    q = R.batch(lens, ctx, bs, seed=len(name))
    T = int(sum(lens)) + pad
    st = zero_status()
    m = call_map(q, T, st)
    assert_map(m, R.ref_map(q, T))
    assert st.item() == 0


def test_state_map_without_requests_or_rows():
    st = zero_status()
    m = call_map(dict(lens=[], ctx=[], table=np.zeros((0, 3)), free=[4, 2], head=1, bs=8, nslots=6), 5, st)
    assert m.cu_seqlens.tolist() == [0] and m.seq_of.tolist() == [-1] * 5 and m.slot_of.tolist() == [-1] * 5 and m.free_head.item() == 1
    m = call_map(R.batch([0, 0], [3, 0], 8), 0, st)
    assert m.cu_seqlens.tolist() == [0, 0, 0] and m.seq_of.numel() == 0 and st.item() == 0


def test_state_map_in_place_over_steps():
    """A scheduler's loop: table and free_head are updated in place, step by
    step, as the reference's are."""
    bs = 4
    q = R.batch([6, 1, 9], [0, 3, 8], bs, spare=40, max_blocks=12)
    table, head = up(q["table"]), up([q["head"]])
    free = up(q["free"])
    st = zero_status()
    for lens in ([6, 1, 9], [1, 1, 1], [1, 0, 1], [4, 5, 1]):
        q["lens"] = np.array(lens)
        T = sum(lens) + 2
        e = lambda *s, dtype=torch.int32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        out = StateMap(e(4), e(T), e(T), e(T, dtype=torch.int64), e(3), table, head, bs)
        m = ssd.state_map(up(lens), up(q["ctx"]), table, free, head, T, bs, q["nslots"], out=out, status=st)
        ref = R.ref_map(q, T)
        assert_map(m, ref)
        q |= dict(table=ref["table"], head=ref["free_head"][0], ctx=q["ctx"] + q["lens"])
    assert st.item() == 0


def test_state_map_shared_prefix():
    """Two requests that begin with the same whole blocks read one slot."""
    q = R.batch([3, 2], [8, 8], 4, spare=4)
    q["table"][1, :2] = q["table"][0, :2]
    st = zero_status()
    assert_map(call_map(q, 5, st), R.ref_map(q, 5))
    assert st.item() == 0


def _bad_maps():
    yield "negative length", lambda q: q["lens"].__setitem__(1, -1)
    yield "negative context", lambda q: q["ctx"].__setitem__(1, -1)
    yield "too many rows", lambda q: q["lens"].__setitem__(0, 7)
    yield "sum beyond int32", lambda q: q.__setitem__("lens", np.array([2 ** 31 - 100] * 3))
    yield "table too narrow", lambda q: q.__setitem__("table", q["table"][:, :2])
    yield "free list short", lambda q: q.__setitem__("head", len(q["free"]))
    yield "free head negative", lambda q: q.__setitem__("head", -1)
    yield "held slot outside the pool", lambda q: q["table"].__setitem__((2, 1), q["nslots"])
    yield "free slot outside the pool", lambda q: q["free"].__setitem__(0, -3)
    yield "unfinished block twice", lambda q: q["table"].__setitem__((0, 0), q["table"][2, 1])
    yield "free slot twice", lambda q: q["free"].__setitem__(1, q["free"][0])
    yield "free slot in use", lambda q: q["free"].__setitem__(0, q["table"][2, 1])
    yield "free slot read by another", lambda q: q["free"].__setitem__(0, q["table"][1, 0])


@pytest.mark.parametrize("what,spoil", list(_bad_maps()), ids=[w.replace(" ", "_") for w, _ in _bad_maps()])
def test_state_map_refuses(what, spoil):
    # request 0 continues an unfinished block, 1 a whole one, 2 an unfinished one
    q = R.batch([4, 4, 4], [1, 4, 6], 4, spare=6)
    q["free"], q["table"] = q["free"].copy(), q["table"].copy()
    T = 14
    spoil(q)
    st = zero_status()
    m = call_map(q, T, st)
    assert st.item() == 1, what
    assert m.cu_seqlens.tolist() == [0] * 4 and m.init_slot.tolist() == [-1] * 3
    for k in ("seq_of", "pos_of", "slot_of"):
        assert (getattr(m, k) == -1).all()
    assert np.array_equal(m.table.cpu().numpy(), q["table"]) and m.free_head.item() == q["head"]


# ---------------------------------------------------------------------------
# conv over packed requests

CONV_BATCHES = {
    "decode": ([1] * 9, [0, 1, 2, 3, 4, 5, 6, 7, 8], 4),
    "short": ([1, 2, 3, 4, 5, 0, 6], [0, 5, 1, 2, 0, 3, 8], 4),
    "cuts": ([31, 1, 33, 64, 2, 30, 95, 3], [0, 3, 0, 17, 1, 0, 40, 6], 16),
    "block_of_one": ([5, 1, 40], [0, 2, 3], 1),
    "block_of_two": ([37, 66], [1, 0], 2),
    "odd_blocks": ([100, 29, 31], [3, 0, 50], 7),
    "in_one_block": ([100, 200, 1], [30, 0, 7], 100000),
    # fewer rows than requests: single tokens, none, and a few longer ones
    "mostly_empty": ([0] * 11 + [1, 0, 7, 0, 1, 1] + [0] * 9 + [2] + [0] * 6, [(5 * i) % 13 for i in range(33)], 4),
}


@DTYPES
@pytest.mark.parametrize("k", [2, 3, 4])
@pytest.mark.parametrize("name", sorted(CONV_BATCHES))
def test_conv_varlen(name, k, dtype):
    lens, ctx, bs = CONV_BATCHES[name]
    E = 40 if k != 4 else 520     # a partial and more than one channel block
    q = R.batch(lens, ctx, bs, seed=3)
    T = sum(lens) + 3
    m = R.ref_map(q, T)
    g = torch.Generator().manual_seed(5 + k)
    x = torch.randn(T, E + 8, generator=g).to(dtype)
    w, bias = 0.5 * torch.randn(E, k, generator=g), (0.3 * torch.randn(E, generator=g) if k != 3 else None)
    cache = torch.randn(q["nslots"], E, k, generator=g).to(dtype)
    out = torch.full((T, E + 16), 7.0, dtype=dtype, device="cuda")
    xd, cd = x.cuda(), cache.cuda()
    xd[sum(lens):] = float("nan")      # rows behind the last request are not read
    st = zero_status()
    ssd.conv1d_silu_varlen(xd[:, :E], w.cuda(), cd, dev_map(m, bs), bias=None if bias is None else bias.cuda(), out=out[:, :E], status=st)
    ref, pool = torch.zeros(T, E, dtype=torch.float64), cache.double()
    cu, ext = m["cu_seqlens"], {}
    for r in range(len(lens)):
        left = cache[m["init_slot"][r]].double().t() if m["init_slot"][r] >= 0 else torch.zeros(k, E, dtype=torch.float64)
        ext[r] = torch.cat([left, x[cu[r]:cu[r + 1], :E].double()])
        ref[cu[r]:cu[r + 1]] = R.conv(ext[r], w.double(), None if bias is None else bias.double())
    for t, r, slot in R.kept_rows(m, bs):
        at = t - cu[r] + 1
        pool[slot] = ext[r][at:at + k].t()
    assert st.item() == 0
    R.close(out[:sum(lens), :E], ref[:sum(lens)], "conv", c=R.C_CONV)
    assert (out[sum(lens):] == 7).all() and (out[:, E:] == 7).all()
    assert torch.equal(cd.double().cpu(), pool), "caches"


# ---------------------------------------------------------------------------
# the scan, dense

DENSE = {   # b, L, E, N, G
    "one_token": (3, 1, 64, 16, 1),
    "short": (2, 5, 40, 16, 1),
    "tile": (1, 32, 32, 16, 1),
    "tile_and_one": (2, 33, 72, 16, 3),
    "n4": (2, 19, 264, 4, 1),
    "n8": (1, 70, 144, 8, 2),
    "n12": (2, 45, 24, 12, 1),
    "n24": (1, 67, 48, 24, 2),
    "n32": (2, 33, 16, 32, 1),
    "n48": (1, 40, 24, 48, 1),
    "n64": (2, 35, 24, 64, 3),
    "cut": (1, 1500, 16, 16, 1),
    "cut_batch": (2, 700, 24, 8, 1),
    "cut_n64": (1, 500, 16, 64, 2),
}


def dense_ref(p, init):
    d = R.f64(p)
    b = p["u"].shape[0]
    E, N = p["A"].shape
    ys, hs = [], []
    for i in range(b):
        one = {k: (v[i] if v is not None and k in ("u", "dt_raw", "B", "C", "z") else v) for k, v in d.items()}
        y, h = R.scan(one, torch.zeros(E, N, dtype=torch.float64) if init is None else init[i].double().cpu())
        ys.append(y)
        hs.append(h[-1])
    return torch.stack(ys), torch.stack(hs)


@DTYPES
@pytest.mark.parametrize("name", sorted(DENSE))
@pytest.mark.parametrize("full", [True, False], ids=["all", "bare"])
def test_scan_dense(name, full, dtype):
    b, L, E, N, G = DENSE[name]
    p = R.scan_inputs((b, L), E, N, G, dtype, seed=len(name), z=full, bias=full, D=full, device="cuda", pad=int(full))
    init = 0.5 * torch.randn(b, E, N, device="cuda") if full else None
    y, fs = ssd.diag_scan_fwd(**p, init_state=init)
    ry, rf = dense_ref(p, init)
    R.close(y, ry, "y")
    R.close(fs, rf, "final state")


@pytest.mark.parametrize("L,E", [(1500, 16), (40, 64)], ids=["cut", "whole"])
def test_scan_dense_state_in_place_and_handed_over(L, E):
    """final_state may be init_state; two halves with the state handed over
    are the whole."""
    p = R.scan_inputs((2, L), E, 16, 1, F32, seed=9, device="cuda")
    init = 0.5 * torch.randn(2, E, 16, device="cuda")
    ry, rf = dense_ref(p, init)
    st = init.clone()
    y, fs = ssd.diag_scan_fwd(**p, init_state=st, final_state=st)
    assert fs is st
    R.close(st, rf, "state in place")
    cut = L // 3
    half = lambda a, c: {k: (v[:, a:c].contiguous() if v is not None and k in ("u", "dt_raw", "z") else v[:, a:c] if k in ("B", "C") else v)  # noqa: E731
                         for k, v in p.items()}
    pb = lambda h: h | dict(B=h["B"].contiguous(), C=h["C"].contiguous())  # noqa: E731
    y1, s1 = ssd.diag_scan_fwd(**pb(half(0, cut)), init_state=init)
    y2, s2 = ssd.diag_scan_fwd(**pb(half(cut, L)), init_state=s1)
    R.close(torch.cat([y1, y2], 1), ry, "y of two halves")
    R.close(s2, rf, "state of two halves")


def test_scan_dense_empty():
    p = R.scan_inputs((2, 0), 16, 16, 1, F32, seed=1, device="cuda")
    init = torch.randn(2, 16, 16, device="cuda")
    y, fs = ssd.diag_scan_fwd(**p, init_state=init)
    assert y.shape == (2, 0, 16) and torch.equal(fs, init)
    assert (ssd.diag_scan_fwd(**p)[1] == 0).all()
    p = R.scan_inputs((0, 4), 16, 16, 1, F32, seed=1, device="cuda")
    assert ssd.diag_scan_fwd(**p)[1].shape == (0, 16, 16)


@DTYPES
def test_scan_masked_and_extreme_rows(dtype):
    """dt_raw = -inf leaves the state as it was; dt_raw large with A < 0
    forgets it; a NaN row spoils its own sequence from there on only."""
    p = R.scan_inputs((3, 50), 32, 16, 1, dtype, seed=4, device="cuda", bias=False)
    p["dt_raw"][0, 10:40] = -float("inf")
    p["dt_raw"][1, 20] = 100.0
    p["u"][2, 30] = float("nan")
    y, fs = ssd.diag_scan_fwd(**p)
    q = dict(p)
    q["u"] = p["u"].clone()
    q["u"][2, 30] = 0
    ry, rf = dense_ref(q, None)
    R.close(y[:2], ry[:2], "y")
    R.close(fs[:2], rf[:2], "final state")
    R.close(y[2, :30], ry[2, :30], "y before the NaN")
    assert torch.isnan(y[2, 30:]).all() and torch.isnan(fs[2]).all()


# ---------------------------------------------------------------------------
# the scan over packed requests

PACKED = {   # lens, ctx, block, E, N, G
    "decode": ([1] * 9, list(range(9)), 4, 64, 16, 1),
    "short": ([1, 2, 3, 4, 5, 0, 6], [0, 5, 1, 2, 0, 3, 8], 4, 40, 16, 1),
    "tiles": ([31, 1, 33, 64, 2, 30, 95, 3], [0, 3, 0, 17, 1, 0, 40, 6], 16, 48, 16, 2),
    "block_of_one": ([5, 1, 40], [0, 2, 3], 1, 16, 8, 1),
    "odd_blocks": ([100, 29, 31], [3, 0, 50], 7, 24, 24, 1),
    "cut": ([700, 3, 0, 300, 1, 150], [0, 20, 4, 100, 0, 64], 64, 16, 16, 1),
    "cut_in_one_block": ([900, 200], [30, 0], 100000, 16, 16, 1),
    "cut_n4": ([513, 600], [0, 129], 128, 16, 4, 1),
}


@DTYPES
@pytest.mark.parametrize("name", sorted(PACKED))
def test_scan_packed(name, dtype):
    lens, ctx, bs, E, N, G = PACKED[name]
    q = R.batch(lens, ctx, bs, seed=3)
    used = sum(lens)
    T = used + 5
    m = R.ref_map(q, T)
    p = R.scan_inputs((T,), E, N, G, dtype, seed=len(name), device="cuda")
    for k in ("u", "dt_raw", "z", "B", "C"):
        p[k][used:] = float("nan")      # rows behind the last request are not read
    states = 0.5 * torch.randn(q["nslots"], E, N, generator=torch.Generator().manual_seed(2))
    ref_states = states.double()
    taken = {s for _, _, s in R.kept_rows(m, bs)} | set(m["init_slot"])
    loose = [s for s in range(q["nslots"]) if s not in taken]
    states[loose] = float("nan")        # nor are slots that no request names
    dev = states.cuda()
    y = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    st = zero_status()
    ssd.diag_scan_fwd_varlen(**p, states=dev, m=dev_map(m, bs), y=y, status=st)
    d, cu = R.f64(p), m["cu_seqlens"]
    kept = {t: s for t, _, s in R.kept_rows(m, bs)}
    ry, start = torch.zeros(used, E, dtype=torch.float64), ref_states.clone()
    for r in range(len(lens)):
        if lens[r]:
            h = start[m["init_slot"][r]] if m["init_slot"][r] >= 0 else torch.zeros(E, N, dtype=torch.float64)
            yy, hs = R.scan(R.rows(d, cu[r], cu[r + 1]), h)
            ry[cu[r]:cu[r + 1]] = yy
            for i, h in enumerate(hs):
                if cu[r] + i in kept:
                    ref_states[kept[cu[r] + i]] = h
    assert st.item() == 0
    R.close(y[:used], ry, "y")
    assert (y[used:] == 7).all()
    sure = [s for s in range(q["nslots"]) if s not in loose]
    R.close(dev[sure], ref_states[sure], "states")
    assert torch.isnan(dev[loose]).all()


# ---------------------------------------------------------------------------
# single tokens


@DTYPES
@pytest.mark.parametrize("E,N,G", [(64, 16, 1), (40, 4, 1), (136, 8, 1), (48, 12, 2), (72, 32, 3), (24, 64, 1), (16, 40, 1)])
@pytest.mark.parametrize("mapped", [True, False])
def test_state_update(E, N, G, mapped, dtype):
    n, bs = 21, 4
    lens, ctx = [1] * n, [i % 11 for i in range(n)]
    lens[4] = lens[20] = 0          # requests that bring no token
    q = R.batch(lens, ctx, bs, seed=3)
    T = sum(lens) + 2 if mapped else n
    m = R.ref_map(q, T) if mapped else None
    p = R.scan_inputs((T,), E, N, G, dtype, seed=E + N, device="cuda")
    states = 0.5 * torch.randn(q["nslots"] if mapped else n, E, N, generator=torch.Generator().manual_seed(2))
    dev = states.cuda()
    y = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    st = zero_status()
    ssd.diag_state_update(dev, **p, m=dev_map(m, bs) if mapped else None, y=y, status=st)
    d, ref = R.f64(p), states.double()
    for i in range(sum(lens) if mapped else n):
        frm, to = (m["init_slot"][m["seq_of"][i]], m["slot_of"][i] // bs) if mapped else (i, i)
        h = states[frm].double() if frm >= 0 else torch.zeros(E, N, dtype=torch.float64)
        yy, hs = R.scan(R.rows(d, i, i + 1), h)
        R.close(y[i:i + 1], yy, f"y of row {i}", scale=4.0)
        ref[to] = hs[0]
    assert st.item() == 0
    R.close(dev, ref, "states", c=1e-5)
    if mapped:
        assert (y[sum(lens):] == 7).all()


# ---------------------------------------------------------------------------
# the calls together


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_serving_run(graph):
    """Prompts, then decode steps, then more prompt for some: map, conv,
    projections, scan or update on one set of buffers, against the whole
    sequences in float64.  As a captured graph the decode step is replayed on
    new lengths and inputs in the same buffers."""
    E, N, k, bs, n, rank = 64, 16, 4, 16, 5, 5
    g = torch.Generator().manual_seed(11)
    w, cb = 0.5 * torch.randn(E, k, generator=g), 0.2 * torch.randn(E, generator=g)
    proj = torch.randn(rank + 2 * N, E, generator=g) / E ** 0.5
    dtw, dtb = torch.randn(E, rank, generator=g) * 0.2, torch.full((E,), -2.0)
    A, D = -(0.3 + torch.rand(E, N, generator=g) * 3), torch.randn(E, generator=g)
    plan = [[20, 0, 33, 7, 16]] + [[1, 1, 1, 1, 1], [1, 1, 0, 1, 1], [1, 1, 1, 1, 1]] + [[0, 40, 3, 1, 17]]
    total = np.sum(plan, 0)
    x = [torch.randn(int(t), E, generator=g) for t in total]
    z = [torch.randn(int(t), E, generator=g) for t in total]

    # the whole sequences
    want = []
    for r in range(n):
        u = R.conv(torch.cat([torch.zeros(k, E), x[r]]).double(), w.double(), cb.double())
        pr = u @ proj.double().t()
        p = dict(u=u, dt_raw=pr[:, :rank] @ dtw.double().t(), A=A.double(), B=pr[:, None, rank:rank + N], C=pr[:, None, rank + N:],
                 dt_bias=dtb.double(), D=D.double(), z=z[r].double())
        want.append(R.scan(p, torch.zeros(E, N, dtype=torch.float64))[0] if total[r] else u)

    nslots = int(sum(-(-t // bs) for t in total)) + 2
    mb = int(max(-(-t // bs) for t in total))
    table, head = torch.full((n, mb), -1, dtype=torch.int32, device="cuda"), up([0])
    free = up(np.random.default_rng(0).permutation(nslots))
    states, cache = torch.full((nslots, E, N), float("nan"), device="cuda"), torch.full((nslots, E, k), float("nan"), device="cuda")
    wd, cbd, projd, dtwd, dtbd, Ad, Dd = (t.cuda() for t in (w, cb, proj, dtw, dtb, A, D))
    status = zero_status()
    got = [[] for _ in range(n)]
    ctx = np.zeros(n, np.int64)
    e = lambda *s, dtype=torch.int32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731

    def one(lens_d, ctx_d, xt, zt, y, out, single):
        m = ssd.state_map(lens_d, ctx_d, table, free, head, xt.shape[0], bs, nslots, out=out, status=status)
        u = ssd.conv1d_silu_varlen(xt, wd, cache, m, bias=cbd, status=status, out=torch.zeros_like(xt))
        pr = u @ projd.t()
        par = dict(dt_bias=dtbd, D=Dd, z=zt, y=y, status=status)
        B, C = pr[:, rank:rank + N].unflatten(1, (1, N)), pr[:, rank + N:].unflatten(1, (1, N))
        if single:
            ssd.diag_state_update(states, u, pr[:, :rank] @ dtwd.t(), Ad, B, C, m, **par)
        else:
            ssd.diag_scan_fwd_varlen(u, pr[:, :rank] @ dtwd.t(), Ad, B, C, states, m, **par)

    torch.backends.cuda.matmul.allow_tf32 = False
    bufs = replay = None
    for lens in plan:
        T = sum(lens) if max(lens) > 1 else n      # decode batches are padded to n rows
        at = [int(c) for c in ctx]
        xt = torch.zeros(T, E)
        zt = torch.zeros(T, E)
        rows = torch.cat([x[r][at[r]:at[r] + lens[r]] for r in range(n)])
        xt[:len(rows)], zt[:len(rows)] = rows, torch.cat([z[r][at[r]:at[r] + lens[r]] for r in range(n)])
        single = max(lens) == 1
        if single and graph:
            if bufs is None:
                bufs = (up(lens), up(ctx), xt.cuda(), zt.cuda(), torch.zeros(T, E, device="cuda"))
                out = StateMap(e(n + 1), e(T), e(T), e(T, dtype=torch.int64), e(n), table, head, bs)
                projd @ projd.t()          # the library's workspace exists before the capture
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                keep = [t.clone() for t in (table, head, states, cache)]
                with torch.cuda.stream(side):
                    one(*bufs, out, True)  # warm-up of the library products
                torch.cuda.current_stream().wait_stream(side)
                for t, v in zip((table, head, states, cache), keep):
                    t.copy_(v)
                replay = torch.cuda.CUDAGraph()
                with torch.cuda.graph(replay):
                    one(*bufs, out, True)
            for b, v in zip(bufs, (up(lens), up(ctx), xt.cuda(), zt.cuda(), torch.zeros(T, E, device="cuda"))):
                b.copy_(v)
            replay.replay()
            y = bufs[4].clone()
        else:
            y = torch.zeros(T, E, device="cuda")
            one(up(lens), up(ctx), xt.cuda(), zt.cuda(), y, StateMap(e(n + 1), e(T), e(T), e(T, dtype=torch.int64), e(n), table, head, bs), single)
        cu = np.concatenate([[0], np.cumsum(lens)])
        for r in range(n):
            got[r].append(y[cu[r]:cu[r + 1]].cpu())
        ctx += np.array(lens)
    assert status.item() == 0
    for r in range(n):
        # the float32 products before the scan add their own rounding
        R.close(torch.cat(got[r]), want[r][:int(total[r])], f"request {r}", c=2e-4)


def test_prefix_reuse():
    """A request that begins with another's whole blocks starts from the state
    kept at their end."""
    E, N, bs = 32, 16, 32
    p = R.scan_inputs((100,), E, N, 1, F32, seed=6, device="cuda")
    states = torch.zeros(8, E, N, device="cuda")
    st = zero_status()
    whole = R.batch([100], [0], bs)
    whole |= dict(nslots=8, free=np.arange(8, dtype=np.int32))
    m = call_map(whole, 100, st)
    y = ssd.diag_scan_fwd_varlen(**p, states=states, m=m, status=st)
    again = dict(lens=np.array([36]), ctx=np.array([64]), bs=bs, nslots=8, table=m.table.cpu().numpy().copy(), free=np.arange(4, 8, dtype=np.int32), head=0)
    m2 = call_map(again, 36, st)
    tail = {k: (v[64:].contiguous() if k in ("u", "dt_raw", "z", "B", "C") else v) for k, v in p.items()}
    y2 = ssd.diag_scan_fwd_varlen(**tail, states=states, m=m2, status=st)
    assert st.item() == 0
    R.close(y2, y[64:].double(), "the tail from the kept state")


def test_calls_on_another_stream():
    p = R.scan_inputs((2, 1500), 16, 16, 1, F32, seed=3, device="cuda")
    want = ssd.diag_scan_fwd(**p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, fs = ssd.diag_scan_fwd(**p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0]) and torch.equal(fs, want[1])


def test_results_repeat():
    """The same inputs give the same bits, cut rows included."""
    p = R.scan_inputs((1, 3000), 32, 16, 1, BF16, seed=3, device="cuda")
    a, b = ssd.diag_scan_fwd(**p), ssd.diag_scan_fwd(**p)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------
# maps that are not sound: reported, nothing outside the buffers is touched


def _spoilt():
    def put(key, i, v):
        return lambda m: m[key].__setitem__(i, v)
    yield "cu negative", put("cu_seqlens", 1, -5), False
    yield "cu beyond the rows", put("cu_seqlens", 3, 10 ** 6), False
    yield "cu falls", put("cu_seqlens", 2, 30), False
    yield "init outside the pool", put("init_slot", 0, 10 ** 6), False
    yield "slot outside the pool", put("slot_of", 39, 10 ** 12), False
    yield "slot negative", put("slot_of", 39, -2), False
    yield "request out of range", put("seq_of", 32, 99), True
    yield "request of other rows", put("seq_of", 32, 2), True
    yield "no request for a row", put("seq_of", 32, -1), True


@pytest.mark.parametrize("what,spoil,by_row", list(_spoilt()), ids=[w[0].replace(" ", "_") for w in _spoilt()])
def test_unsound_maps_are_reported(what, spoil, by_row):
    lens, ctx, bs, E = [40, 40, 40], [5, 0, 8], 8, 16
    q = R.batch(lens, ctx, bs)
    m = R.ref_map(q, 120)
    spoil(m)
    d = dev_map(m, bs)
    p = R.scan_inputs((120,), E, 16, 1, F32, seed=1, device="cuda")
    states, cache = torch.zeros(q["nslots"] + 2, E, 16, device="cuda"), torch.zeros(q["nslots"] + 2, E, 4, device="cuda")
    st = zero_status()
    if not by_row:   # seq_of is read where a piece starts, which a short whole sequence has none of
        ssd.diag_scan_fwd_varlen(**p, states=states[1:-1], m=d, status=st)
        assert st.item() == 1, what
    st.zero_()
    ssd.conv1d_silu_varlen(p["u"].contiguous(), torch.ones(E, 4, device="cuda"), cache[1:-1], d, status=st)
    assert st.item() == 1, what
    for pool in (states, cache):
        assert (pool[0] == 0).all() and (pool[-1] == 0).all()


def test_cut_scan_reports_rows_without_their_request():
    """Pieces of a cut sequence are found by their first row's request."""
    q = R.batch([900], [0], 64)
    m = R.ref_map(q, 900)
    m["seq_of"][256:] = [-1] * 644
    p = R.scan_inputs((900,), 16, 16, 1, F32, seed=1, device="cuda")
    states, st = torch.zeros(q["nslots"], 16, 16, device="cuda"), zero_status()
    ssd.diag_scan_fwd_varlen(**p, states=states, m=dev_map(m, 64), status=st)
    assert st.item() == 1


def test_state_update_refuses_two_rows_of_a_request():
    q = R.batch([1, 2, 1], [4, 0, 1], 8)
    m = R.ref_map(q, 4)
    p = R.scan_inputs((4,), 16, 16, 1, F32, seed=1, device="cuda")
    states, st = torch.zeros(q["nslots"], 16, 16, device="cuda"), zero_status()
    y = torch.full((4, 16), 7.0, device="cuda")
    ssd.diag_state_update(states, **p, m=dev_map(m, 8), y=y, status=st)
    assert st.item() == 1 and (y[1:3] == 7).all() and (y[0] != 7).all() and (y[3] != 7).all()


def test_python_refusals():
    p = R.scan_inputs((2, 8), 16, 16, 1, F32, seed=1, device="cuda")
    with pytest.raises(ValueError):
        ssd.diag_scan_fwd(**(p | dict(A=p["A"].double())))
    with pytest.raises(ValueError):
        ssd.diag_scan_fwd(**(p | dict(z=p["z"].bfloat16())))
    with pytest.raises(ValueError):
        ssd.diag_scan_fwd(**(p | dict(dt_raw=p["dt_raw"].transpose(0, 1).contiguous().transpose(0, 1))))
    with pytest.raises(ValueError):
        ssd.diag_scan_fwd(**(p | dict(C=p["C"].contiguous())))
    with pytest.raises(ValueError):
        ssd.diag_scan_fwd(**p, init_state=torch.zeros(2, 16, 8, device="cuda"))
    with pytest.raises(ValueError):
        ssd.diag_scan_fwd(**{k: (v.cpu() if v is not None else None) for k, v in p.items()})
    big = R.scan_inputs((1, 4), 16, 68, 1, F32, seed=1, device="cuda")
    with pytest.raises(SsdError, match="UNSUPPORTED"):
        ssd.diag_scan_fwd(**big)
    odd = R.scan_inputs((1, 4), 16, 6, 1, F32, seed=1, device="cuda")
    with pytest.raises(SsdError, match="INVALID_ARG"):
        ssd.diag_scan_fwd(**odd)
    with pytest.raises(SsdError, match="INVALID_ARG"):
        ssd.diag_scan_fwd(**p, y=p["dt_raw"])
