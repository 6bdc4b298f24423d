"""The diagonal scan's calls where they meet the rest of a program: memory that
another stream still uses, prompts among single tokens, states that forget at
once, slots of earlier states given back."""
import numpy as np
import pytest
import torch

import diag_ref as R
import ssd_selective_scan_b200 as ssd
import test_gpu_diag as fwd
import test_gpu_diag_bwd as bwd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])

# At most two rows to a request, some with many more than one.
MIXED = {
    "a_prompt": ([1] * 70 + [100] + [1] * 9 + [0] * 12 + [1] * 5, 16),
    "prompts": ([0] * 60 + [33, 1, 64, 2, 32] + [0] * 20, 7),
    "in_one_block": ([1] * 100 + [95], 4096),
    "block_of_one": ([1] * 40 + [35] + [0] * 8, 1),
}


@DTYPES
@pytest.mark.parametrize("k", [2, 3, 4])
@pytest.mark.parametrize("name", sorted(MIXED))
def test_conv_prompts_among_single_tokens(name, k, dtype, monkeypatch):
    lens, bs = MIXED[name]
    assert sum(lens) + 3 <= 2 * len(lens)
    monkeypatch.setitem(fwd.CONV_BATCHES, name, (lens, [(5 * i) % 37 for i in range(len(lens))], bs))
    fwd.test_conv_varlen(name, k, dtype)


def test_results_do_not_take_memory_in_use():
    """A result on another stream is not laid into a block that was freed on
    the current one while work there still reads it."""
    p = R.scan_inputs((2, 600), 64, 16, 1, F32, seed=3, device="cuda")
    want, _ = ssd.diag_scan_fwd(**p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.ones_like(want) for _ in range(8)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)              # about 0.1 s
    copies = [h.clone() for h in held]          # waits behind it
    del held
    results = [ssd.diag_scan_fwd(**p, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    for c in copies:
        assert (c == 1).all()
    for y, _ in results:
        assert torch.equal(y, want)


NOW = -1e5     # exp(dt A) is 0 in float64 as in float32 (dt >= 0.007: e^-700)


def forgetful(p):
    """(p with every third decay -inf, p with a finite decay of the same effect)"""
    a, b = dict(p), dict(p)
    a["A"], b["A"] = p["A"].clone(), p["A"].clone()
    a["A"].view(-1)[::3] = -float("inf")
    b["A"].view(-1)[::3] = NOW
    return a, b


@pytest.mark.parametrize("name", ["short", "tile_and_one", "n12", "n64", "cut"])
def test_scan_forgets_at_once(name):
    b, L, E, N, G = fwd.DENSE[name]
    p, q = forgetful(R.scan_inputs((b, L), E, N, G, F32, seed=2, device="cuda"))
    init = 0.5 * torch.randn(b, E, N, device="cuda")
    y, fs = ssd.diag_scan_fwd(**p, init_state=init)
    ry, rf = fwd.dense_ref(q, init)
    R.close(y, ry, "y")
    R.close(fs, rf, "final state")
    one = {k: (v[:, 0] if v is not None and k in bwd.ROWS else v) for k, v in p.items()}
    st = init.clone()
    y1 = ssd.diag_state_update(st, one["u"], one["dt_raw"], one["A"], one["B"], one["C"], dt_bias=one["dt_bias"], D=one["D"], z=one["z"])
    R.close(y1, ry[:, 0], "y of one token")


@pytest.mark.parametrize("name", ["short", "tile_and_one", "n12", "n64", "cut"])
def test_scan_bwd_forgets_at_once(name):
    p, init, dfinal, dy = bwd.case(name, True, F32, seed=3)
    p, q = forgetful(p)
    r = ssd.diag_scan_bwd(**p, dy=dy.cuda(), init_state=init.cuda(), dfinal=dfinal.cuda())
    d = {k: (v.requires_grad_() if v is not None else None) for k, v in R.f64(q).items()}
    di = init.double().requires_grad_()
    bwd.loss(d, di, dfinal.double(), dy.double()).backward()
    for k, name in bwd.NAMES.items():
        R.close(r[name], d[k].grad, name)
    R.close(r["dinit"], di.grad, "dinit")


def test_state_map_reads_the_last_state_only():
    """The slots of a request's earlier blocks may be given back and used anew."""
    q = R.batch([4, 6], [9, 3], 4, seed=1, spare=4)
    old = q["table"][0, :2].copy()
    q["free"] = np.concatenate([old[:1], q["free"]])      # block 0's slot is the first to be taken
    q["table"][0, 1] = -1                                   # block 1's belongs to nobody
    T = 11
    st = fwd.zero_status()
    m = fwd.call_map(q, T, st)
    fwd.assert_map(m, R.ref_map(q, T))
    assert st.item() == 0


def _serve(q, E, N, k, states, cache, dtype):
    """A step of prompts and one of single tokens over these pools; (y, the
    slots that hold each request's last state)."""
    g = torch.Generator().manual_seed(12)
    st = fwd.zero_status()
    n = len(q["lens"])
    w, ctx, ys = (0.5 * torch.randn(E, k, generator=g)).cuda(), fwd.up(q["ctx"]), []
    table, free, head = fwd.up(q["table"]), fwd.up(q["free"]), fwd.up([q["head"]])
    for lens in (q["lens"], [1] * n):
        T = int(sum(lens))
        p = fwd.cuda(R.scan_inputs((T,), E, N, 1, dtype, seed=T))
        m = ssd.state_map(fwd.up(lens), ctx, table, free, head, T, q["bs"], q["nslots"], status=st)
        p["u"] = ssd.conv1d_silu_varlen(p["u"], w, cache, m, status=st)
        call = ssd.diag_scan_fwd_varlen if T > n else None
        ys.append(call(**p, states=states, m=m, status=st) if call else
                  ssd.diag_state_update(states, p["u"], p["dt_raw"], p["A"], p["B"], p["C"], m, dt_bias=p["dt_bias"], D=p["D"], z=p["z"], status=st))
        table, head, ctx = m.table, m.free_head, ctx + fwd.up(lens)
    assert st.item() == 0
    last = table.gather(1, ((ctx.long() - 1) // q["bs"])[:, None])[:, 0]
    return torch.cat(ys), last


@pytest.mark.parametrize("bs,pool", [(1 << 28, None), (8, 17000), (1 << 18, 17000)], ids=["long_blocks", "large_pool", "both"])
def test_offsets_beyond_32_bits(bs, pool):
    """Places of tokens (slot * block_tokens) and of states (slot * E * N) past
    2^32: what a small pool of short blocks' slots gives."""
    E, N, k = 8192, 16, 4
    lens, ctx = [20, 1, 7], [0, 30, 8]

    def run(bs, pool):
        q = R.batch(lens, ctx, bs, seed=2, spare=40)
        if pool is not None:     # the slots at the pool's far end
            far = pool - q["nslots"]
            held = q["table"] >= 0
            q["table"][held] += far
            q["free"] = q["free"] + far
            q["nslots"] = pool
        states = torch.empty(q["nslots"], E, N, device="cuda")
        cache = torch.empty(q["nslots"], E, k, dtype=BF16, device="cuda")
        g = torch.Generator().manual_seed(5)
        for r in range(3):
            if ctx[r]:
                slot = q["table"][r, (ctx[r] - 1) // bs]
                states[slot] = torch.randn(E, N, generator=g).cuda()
                cache[slot] = torch.randn(E, k, generator=g).to(BF16).cuda()
        y, last = _serve(q, E, N, k, states, cache, BF16)
        if bs > 1 << 16 or pool:
            assert int(last.max()) * max(bs, E * N) > 1 << (31 if pool else 32)
        return y, states[last], cache[last]

    want, got = run(8, None), run(bs, pool)
    assert torch.equal(got[2], want[2]), "caches"
    for a, b, what in zip(got, want, ("y", "states")):
        R.close(a, b.double(), what)
