"""Cases of the diagonal selective scan and what serves it: state maps built
from request lengths, the short causal convolution (packed prompts and single
tokens by cache slots; its gradient), the scan (dense, packed, backward) and
the single-token state update.

Every case is a dict; ``op`` names the operator:

  map    block tables and slot maps of a batch of requests
  conv   causal depthwise conv + SiLU; ``dir`` fwd (packed, by slots) or bwd
  scan   h_t = exp(dt_t A) h_{t-1} + dt_t u_t B_t, y_t = (h_t C_t + D u_t) SiLU(z_t);
         ``dir`` fwd or bwd, ``packed`` for requests packed along one token
         dimension with states in slots, else a dense [b, L] batch
  step   one token per request of the same recurrence

``run`` computes them in plain torch operations, or with ``own`` through the
framework's calls.
"""
import math

import numpy as np
import torch

own = False

_IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of a small server: 24 running requests, a new slot block here and there
        dict(name="map_decode", op="map", n=24, kind="decode", total=24, pad=8, lo=1, hi=1, ctx=6000, block=256),
        # a full batch of prompts with prefix-cached beginnings, state blocks of 256 tokens
        dict(name="map_prompts", op="map", n=700, kind="prompts", total=262144, pad=1000, lo=16, hi=4096, ctx=8192, block=256),
        # the decode step's conv: 256 requests, the 8B layer's inner channels
        dict(name="conv_tokens", op="conv", dir="fwd", n=256, kind="decode", total=256, pad=0, lo=1, hi=1, ctx=2048, block=512,
             E=8192, k=4, dtype="bf16", bias=True),
        # a prefill batch of unequal prompts in float32, one of them empty, rows behind the last
        dict(name="conv_prompts", op="conv", dir="fwd", n=0, kind="prompts", total=16384, pad=77, lo=64, hi=4096, ctx=1500, block=512,
             E=2560, k=4, dtype="f32", bias=True),
        # the conv's gradient in training: the 3B layer's conv channels
        dict(name="conv_grad", op="conv", dir="bwd", b=8, L=2048, E=4608, k=4, dtype="bf16", bias=True, state=False),
        # training forward: 8 sequences of 2048 tokens, 3B inner width
        dict(name="scan_train", op="scan", dir="fwd", packed=False, b=8, L=2048, E=2560, N=16, G=1, dtype="bf16", z=True, state=False),
        # one long prompt of a narrow layer: few rows, a long axis
        dict(name="scan_long", op="scan", dir="fwd", packed=False, b=1, L=32768, E=1024, N=16, G=1, dtype="bf16", z=True, state=True),
        # a serving prefill batch: unequal prompts, states kept every 512 tokens
        dict(name="scan_prompts", op="scan", dir="fwd", packed=True, n=0, kind="prompts", total=16384, pad=77, lo=64, hi=4096,
             ctx=1500, block=512, E=4096, N=16, G=1, dtype="bf16", z=True),
        # a small odd float32 gradient: two groups, 24 states, a state handed over
        dict(name="scan_grad_odd", op="scan", dir="bwd", packed=False, b=2, L=517, E=784, N=24, G=2, dtype="f32", z=False, state=True),
        # training backward at the forward's size
        dict(name="scan_grad", op="scan", dir="bwd", packed=False, b=8, L=2048, E=2560, N=16, G=1, dtype="bf16", z=True, state=False),
        # one decode token for a handful of requests, float32
        dict(name="step_few", op="step", n=5, kind="decode", total=5, pad=3, lo=1, hi=1, ctx=900, block=256, E=2560, N=16, G=1,
             dtype="f32", z=True),
        # one decode token for 256 requests, the 8B layer's inner channels
        dict(name="step_many", op="step", n=256, kind="decode", total=256, pad=0, lo=1, hi=1, ctx=4096, block=1024, E=8192, N=16, G=1,
             dtype="bf16", z=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["map", "conv", "conv_bwd", "scan", "packed", "scan_bwd", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    block = rng.choice([64, 100, 256, 512, 1024])
    E = 8 * _log(rng, 16, 1024)
    N = rng.choice([16, 16, 16, 8, 12, 32, 64])
    G = rng.choice([1, 1, 1, 2]) if E % 16 == 0 else 1
    if kind == "map":
        if rng.random() < 0.5:
            n = _log(rng, 1, 2000)
            return dict(op="map", n=n, kind="decode", total=n, pad=rng.randrange(9), lo=1, hi=1, ctx=_log(rng, 1, 16000), block=block)
        return dict(op="map", n=0, kind="prompts", total=_log(rng, 64, 262144), pad=rng.randrange(300), lo=rng.choice([1, 16, 200]),
                    hi=rng.choice([512, 4096, 10000]), ctx=_log(rng, 1, 8000), block=block)
    if kind == "conv":
        if rng.random() < 0.4:
            n = _log(rng, 1, 512)
            return dict(op="conv", dir="fwd", n=n, kind="decode", total=n, pad=rng.randrange(5), lo=1, hi=1, ctx=_log(rng, 1, 4000),
                        block=block, E=E, k=rng.choice([4, 4, 3, 2]), dtype=dtype, bias=rng.random() < 0.7)
        return dict(op="conv", dir="fwd", n=0, kind="prompts", total=_log(rng, 16, 16384), pad=rng.randrange(100), lo=rng.choice([1, 3, 64]),
                    hi=rng.choice([300, 4096]), ctx=_log(rng, 1, 3000), block=block, E=min(E, 4096), k=rng.choice([4, 4, 3, 2]),
                    dtype=dtype, bias=rng.random() < 0.7)
    if kind == "conv_bwd":
        b = rng.choice([1, 2, 3, 8])
        return dict(op="conv", dir="bwd", b=b, L=max(1, min(_log(rng, 1, 8192), 16384 // b)), E=min(E, 4608), k=rng.choice([4, 4, 3, 2]),
                    dtype=dtype, bias=rng.random() < 0.7, state=rng.random() < 0.5)
    if kind == "step":
        n = _log(rng, 1, 256)
        return dict(op="step", n=n, kind="decode", total=n, pad=rng.randrange(5), lo=1, hi=1, ctx=_log(rng, 1, 4000), block=block, E=E,
                    N=N if n * E * N <= 1 << 25 else 16, G=G, dtype=dtype, z=rng.random() < 0.7)
    if kind == "packed":
        total = _log(rng, 16, 16384)
        return dict(op="scan", dir="fwd", packed=True, n=0, kind="prompts", total=total, pad=rng.randrange(100), lo=rng.choice([1, 30, 200]),
                    hi=rng.choice([512, 4096]), ctx=_log(rng, 1, 3000), block=block, E=min(E, 4096, 8 * max(2, (1 << 22) // total)),
                    N=rng.choice([16, 16, 8, 12, 32]), G=1, dtype=dtype, z=rng.random() < 0.7)
    most = 1 << (21 if kind == "scan_bwd" else 22)   # channels x tokens, in eights
    b = rng.choice([1, 1, 2, 4, 8])
    L = _log(rng, 1, 16384 if kind == "scan" else 4096)
    E = 16 * max(1, min(E // 16, most // 2 // (b * L)))
    N = rng.choice([16, 16, 8, 12, 32])
    return dict(op="scan", dir="fwd" if kind == "scan" else "bwd", packed=False, b=b, L=L, E=E, N=N if b * L * E * N <= 1 << 29 else 16,
                G=rng.choice([1, 1, 2]), dtype=dtype, z=rng.random() < 0.7, state=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# what a batch of requests looks like, on the host


def _lengths(case):
    """New tokens and held tokens of the case's requests (their order is the
    seed's): the buffers of a case have one size."""
    r = np.random.default_rng([case["total"], case["ctx"], case["block"], case["hi"]])
    if case["kind"] == "decode":
        lens = np.ones(case["n"], np.int64)
    else:
        lens, left = [], case["total"]
        while left > 0:
            m = int(round(math.exp(r.uniform(math.log(case["lo"]), math.log(case["hi"])))))
            m = min(m, left)
            lens.append(m)
            left -= m
        if len(lens) > 3:
            lens.insert(len(lens) // 2, 0)   # a request that brings no token
        lens = np.array(lens, np.int64)
    n = len(lens)
    ctx = np.floor(np.exp(r.uniform(0, math.log(case["ctx"] + 1), n))).astype(np.int64)
    if case["kind"] == "prompts":
        ctx[r.uniform(size=n) < 0.5] = 0         # new requests
        whole = r.uniform(size=n) < 0.3          # a cached prefix of whole blocks
        ctx[whole] = ctx[whole] // case["block"] * case["block"]
    return lens, ctx


def _requests(case, seed):
    """lens, ctx, table, free list and head: what a scheduler holds."""
    r = np.random.default_rng(seed)
    lens, ctx = _lengths(case)
    order = r.permutation(len(lens))
    lens, ctx = lens[order], ctx[order]
    bs, n = case["block"], len(lens)
    held, need = -(-ctx // bs), -(-(ctx + lens) // bs)
    fresh = int((need - held).sum())
    head = int(r.integers(0, 5))
    first = int(held.sum())
    nslots = first + fresh + 8
    order = r.permutation(nslots).astype(np.int32)
    most = int(need.max()) + 1
    table = np.full((n, most), -1, np.int32)
    at = np.arange(most)[None, :] < held[:, None]
    table[at] = order[:first]
    return dict(lens=lens, ctx=ctx, table=table, free=order[first:], head=head, nslots=nslots, T=int(lens.sum()) + case["pad"], bs=bs)


def _host_map(q):
    """The map of a batch, token by token arithmetic in numpy: the plan that
    the conv, scan and step cases start from."""
    lens, ctx, bs = q["lens"], q["ctx"], q["bs"]
    n, used, T = len(lens), int(lens.sum()), q["T"]
    held, need = -(-ctx // bs), -(-(ctx + lens) // bs)
    table = q["table"].copy()
    j = np.arange(table.shape[1])[None, :]
    new = (j >= held[:, None]) & (j < need[:, None])
    base = q["head"] + np.cumsum(need - held) - (need - held)
    table[new] = q["free"][(base[:, None] + j - held[:, None])[new]]
    cu = np.concatenate([[0], np.cumsum(lens)])
    seq = np.repeat(np.arange(n), lens)
    pos = np.arange(used) - cu[seq] + ctx[seq]
    slot = table[seq, pos // bs].astype(np.int64) * bs + pos % bs
    behind = np.full(T - used, -1)
    init = np.where(ctx > 0, table[np.arange(n), np.maximum(ctx - 1, 0) // bs], -1)
    last = np.arange(used) + 1 == cu[seq + 1]
    ends = np.nonzero(last | (pos % bs == bs - 1))[0]
    return dict(cu_seqlens=cu.astype(np.int32), seq_of=np.concatenate([seq, behind]).astype(np.int32),
                pos_of=np.concatenate([pos, behind]).astype(np.int32), slot_of=np.concatenate([slot, behind]),
                init_slot=init.astype(np.int32), table=table, free_head=np.array([q["head"] + int((need - held).sum())], np.int32),
                ends=ends)


def _up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _weights(g, E, N):
    """A around -1 .. -N per channel, dt_bias 0 mean, D near 1: a layer's
    parameters."""
    A = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.3 * _randn(g, E, N))
    return dict(A=A.contiguous(), dt_bias=0.3 * _randn(g, E), D=1.0 + 0.3 * _randn(g, E))


def _rows(g, rows, case, io):
    """u, dt_raw, z and B, C of `rows` tokens: z is the second half of the
    in-projection's rows, B and C are columns of the x-projection's rows
    behind its dt part."""
    E, N, G = case["E"], case["N"], case["G"]
    rank = max(8, E // 32)
    u = _randn(g, rows, E).to(io)
    dt_raw = (_rand(g, rows, E) * 3.0 - 4.0).to(io)
    z = _randn(g, rows, 2 * E).to(io)[:, E:] if case["z"] else None
    proj = (_randn(g, rows, rank + 2 * G * N) / math.sqrt(N)).to(io)
    B = proj[:, rank:rank + G * N].unflatten(1, (G, N))
    C = proj[:, rank + G * N:].unflatten(1, (G, N))
    return u, dt_raw, z, B, C


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if "kind" in case:
        q = _requests(case, seed)
        if case["op"] == "map":
            return s | dict(lens=_up(q["lens"], torch.int32), ctx=_up(q["ctx"], torch.int32), table=_up(q["table"]),
                            free_list=_up(q["free"]), free_head=_up(np.array([q["head"]], np.int32)), T=q["T"],
                            nslots=q["nslots"], status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        m = _host_map(q)
        used = int(q["lens"].sum())
        s |= {k: _up(v) for k, v in m.items()}
        s |= dict(used=used, T=q["T"], nslots=q["nslots"], status=torch.zeros(1, dtype=torch.int32, device="cuda"),
                  ends_slot=s["slot_of"][s["ends"]] // case["block"], table=None)
    io, E = _IO[case["dtype"]], case["E"]
    if case["op"] == "conv":
        k = case["k"]
        s |= dict(w=0.5 * _randn(g, E, k), bias=0.3 * _randn(g, E) if case["bias"] else None)
        if case["dir"] == "bwd":
            b, L = case["b"], case["L"]
            return s | dict(x=_randn(g, b, L, E).to(io), dout=_randn(g, b, L, E).to(io),
                            conv_state=_randn(g, b, E, k).to(io) if case["state"] else None)
        # the conv's input is the first part of the in-projection's rows
        wide = _randn(g, s["T"], 2 * E).to(io)
        return s | dict(x=wide[:, :E], out=torch.zeros(s["T"], E, dtype=io, device="cuda"), pool=_randn(g, s["nslots"], E, k).to(io))
    N = case["N"]
    s |= _weights(g, E, N)
    if "kind" in case:   # packed scan, step
        u, dt_raw, z, B, C = _rows(g, s["T"], case, io)
        return s | dict(u=u, dt_raw=dt_raw, z=z, B=B, C=C, y=torch.zeros(s["T"], E, dtype=io, device="cuda"),
                        states=0.3 * _randn(g, s["nslots"], E, N))
    b, L = case["b"], case["L"]
    u, dt_raw, z, B, C = (None if t is None else t.unflatten(0, (b, L)) for t in _rows(g, b * L, case, io))
    s |= dict(u=u, dt_raw=dt_raw, z=z, B=B, C=C, init_state=0.3 * _randn(g, b, E, N) if case["state"] else None)
    if case["dir"] == "bwd":
        s |= dict(dy=_randn(g, b, L, E).to(io), dfinal=_randn(g, b, E, N) if case["state"] else None)
    return s


# ---------------------------------------------------------------------------
# one pass


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    with torch.no_grad():
        if c["op"] == "map":
            return _plain_map(s)
        if c["op"] == "conv":
            return _plain_conv_bwd(s) if c["dir"] == "bwd" else _plain_conv(s)
        if c["op"] == "step":
            return _plain_step(s)
        return _plain_scan_bwd(s) if c["dir"] == "bwd" else _plain_packed(s) if c["packed"] else _plain_scan(s)


def _own(s):
    import ssd_selective_scan_b200 as ssd
    c = s["case"]
    if c["op"] == "map":
        m = ssd.state_map(s["lens"], s["ctx"], s["table"], s["free_list"], s["free_head"], s["T"], c["block"], s["nslots"],
                          status=s["status"])
        return dict(cu_seqlens=m.cu_seqlens, seq_of=m.seq_of, pos_of=m.pos_of, slot_of=m.slot_of, init_slot=m.init_slot,
                    table=m.table, free_head=m.free_head)
    if "kind" in c:
        m = ssd.StateMap(s["cu_seqlens"], s["seq_of"], s["pos_of"], s["slot_of"], s["init_slot"], None, None, c["block"])
    if c["op"] == "conv":
        if c["dir"] == "bwd":
            r = ssd.conv1d_silu_bwd(s["x"], s["w"], s["dout"], s["bias"], s["conv_state"])
            return {k: v for k, v in r.items() if v is not None}
        ssd.conv1d_silu_varlen(s["x"], s["w"], s["pool"], m, bias=s["bias"], out=s["out"], status=s["status"])
        return dict(out=s["out"], pool=s["pool"])
    par = dict(dt_bias=s["dt_bias"], D=s["D"], z=s["z"])
    if c["op"] == "step":
        ssd.diag_state_update(s["states"], s["u"], s["dt_raw"], s["A"], s["B"], s["C"], m, y=s["y"], status=s["status"], **par)
        return dict(y=s["y"], states=s["states"])
    if c["dir"] == "bwd":
        r = ssd.diag_scan_bwd(s["u"], s["dt_raw"], s["A"], s["B"], s["C"], s["dy"], init_state=s["init_state"], dfinal=s["dfinal"],
                              want_dinit=c["state"], **par)
        return {k: v for k, v in r.items() if v is not None}
    if c["packed"]:
        ssd.diag_scan_fwd_varlen(s["u"], s["dt_raw"], s["A"], s["B"], s["C"], s["states"], m, y=s["y"], status=s["status"], **par)
        return dict(y=s["y"], states=s["states"])
    y, final = ssd.diag_scan_fwd(s["u"], s["dt_raw"], s["A"], s["B"], s["C"], init_state=s["init_state"], **par)
    return dict(y=y, final_state=final)


def _plain_map(s):
    bs, T = s["case"]["block"], s["T"]
    lens, ctx, table = s["lens"].long(), s["ctx"].long(), s["table"].long()
    n = lens.numel()
    held, need = (ctx + bs - 1) // bs, (ctx + lens + bs - 1) // bs
    fresh = need - held
    base = s["free_head"].long() + torch.cumsum(fresh, 0) - fresh
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    new = (j >= held[:, None]) & (j < need[:, None])
    pick = (base[:, None] + j - held[:, None]).clamp(0, s["free_list"].numel() - 1)
    table = torch.where(new, s["free_list"].long()[pick], table)
    cu = torch.cat([lens.new_zeros(1), torch.cumsum(lens, 0)])
    t = torch.arange(T, device=table.device)
    live = t < cu[-1]
    seq = torch.searchsorted(cu, t, right=True).sub(1).clamp(max=n - 1)
    pos = t - cu[seq] + ctx[seq]
    slot = table[seq, (pos // bs).clamp(max=table.shape[1] - 1)] * bs + pos % bs
    init = torch.where(ctx > 0, table.gather(1, ((ctx - 1).clamp(min=0) // bs)[:, None])[:, 0], -1)
    i32 = torch.int32
    return dict(cu_seqlens=cu.to(i32), seq_of=torch.where(live, seq, -1).to(i32), pos_of=torch.where(live, pos, -1).to(i32),
                slot_of=torch.where(live, slot, -1), init_slot=init.to(i32), table=table.to(i32),
                free_head=(s["free_head"].long() + fresh.sum()).to(i32))


def _plain_conv(s):
    k, used, x = s["case"]["k"], s["used"], s["x"].float()
    seq = s["seq_of"][:used].long()
    off = torch.arange(used, device=x.device) - s["cu_seqlens"].long()[seq]            # place in its request
    back = torch.arange(k, device=x.device)[None, :] - (k - 1) + off[:, None]          # place of each tap, < 0: cached
    rows = (torch.arange(used, device=x.device)[:, None] + torch.arange(k, device=x.device)[None, :] - (k - 1)).clamp(min=0)
    init = s["init_slot"].long()[seq]
    cached = s["pool"].float()[init.clamp(min=0)[:, None], :, (back + k).clamp(0, k - 1)]
    cached = torch.where((init >= 0)[:, None, None], cached, 0.0)
    win = torch.where((back < 0)[:, :, None], cached, x[rows])                         # [used, k, E]
    v = (win * s["w"].t()[None]).sum(1)
    if s["bias"] is not None:
        v = v + s["bias"]
    s["out"][:used] = (v / (1.0 + torch.exp(-v))).to(s["out"].dtype)
    s["pool"][s["ends_slot"]] = win[s["ends"]].transpose(1, 2).to(s["pool"].dtype)
    return dict(out=s["out"], pool=s["pool"])


def _plain_conv_bwd(s):
    c, x, w = s["case"], s["x"].float(), s["w"]
    b, L, E, k = c["b"], c["L"], c["E"], c["k"]
    left = s["conv_state"].float().transpose(1, 2) if c["state"] else x.new_zeros(b, k, E)
    ext = torch.cat([left, x], 1)                                   # times -k .. L-1
    win = ext[:, 1:].unfold(1, k, 1)                                # [b, L, E, k]
    v = (win * w).sum(-1)
    if s["bias"] is not None:
        v = v + s["bias"]
    sg = 1.0 / (1.0 + torch.exp(-v))
    dv = s["dout"].float() * sg * (1.0 + v * (1.0 - sg))
    dext = torch.cat([x.new_zeros(b, k, E), dv, x.new_zeros(b, k - 1, E)], 1).unfold(1, k, 1)   # [b, L+k, E, k]
    dext = (dext * w.flip(1)).sum(-1)
    out = dict(dx=dext[:, k:].to(s["x"].dtype), dw=(win * dv[..., None]).sum((0, 1)))
    if s["bias"] is not None:
        out["dbias"] = dv.sum((0, 1))
    if c["state"]:
        out["dconv_state"] = dext[:, :k].transpose(1, 2).to(s["x"].dtype).contiguous()
    return out


def _softplus(v):
    return v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _recurrence(a, x):
    """h_t = a_t h_{t-1} + x_t along dim 1, by doubling; x is overwritten."""
    step = 1
    while step < a.shape[1]:
        x[:, step:] += a[:, step:] * x[:, :-step]
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return x


def _per_channel(t, E):
    """[b, L, G, N] -> [b, L, E, N], channel e reading group e // (E / G)."""
    return t.float().repeat_interleave(E // t.shape[2], dim=2) if t.shape[2] > 1 else t.float()


def _plain_scan(s):
    c = s["case"]
    u, E = s["u"].float(), c["E"]
    dt = _softplus(s["dt_raw"].float() + s["dt_bias"])
    a = torch.exp(dt[..., None] * s["A"])
    x = (dt * u)[..., None] * _per_channel(s["B"], E)
    if s["init_state"] is not None:
        x[:, 0] += a[:, 0] * s["init_state"]
    h = _recurrence(a, x)
    y = (h * _per_channel(s["C"], E)).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1.0 + torch.exp(-z))
    return dict(y=y.to(s["u"].dtype), final_state=h[:, -1].clone())


def _plain_packed(s):
    c, used = s["case"], s["used"]
    u, E = s["u"][:used].float(), c["E"]
    dt = _softplus(s["dt_raw"][:used].float() + s["dt_bias"])
    a = torch.exp(dt[..., None] * s["A"])
    x = (dt * u)[..., None] * _per_channel(s["B"][None, :used], E)[0]
    # a request's first token: its state from the slot goes into the input,
    # and the decay over the border is zero
    seq = s["seq_of"][:used].long()
    first = torch.arange(used, device=u.device) == s["cu_seqlens"].long()[seq]
    init = s["init_slot"].long()[seq]
    held = torch.where((first & (init >= 0))[:, None, None], s["states"][init.clamp(min=0)], 0.0)
    x += a * held
    del held
    a = torch.where(first[:, None, None], 0.0, a)
    h = _recurrence(a[None], x[None])[0]
    del a
    y = (h * _per_channel(s["C"][None, :used], E)[0]).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"][:used].float()
        y = y * z / (1.0 + torch.exp(-z))
    s["y"][:used] = y.to(s["y"].dtype)
    s["states"][s["ends_slot"]] = h[s["ends"]]
    return dict(y=s["y"], states=s["states"])


def _plain_step(s):
    used, E = s["used"], s["case"]["E"]
    seq = s["seq_of"][:used].long()
    init = s["init_slot"].long()[seq]
    slot = s["slot_of"][:used] // s["case"]["block"]
    u = s["u"][:used].float()
    dt = _softplus(s["dt_raw"][:used].float() + s["dt_bias"])
    h = torch.where((init >= 0)[:, None, None], s["states"][init.clamp(min=0)], 0.0)
    h = torch.exp(dt[..., None] * s["A"]) * h + (dt * u)[..., None] * _per_channel(s["B"][None, :used], E)[0]
    y = (h * _per_channel(s["C"][None, :used], E)[0]).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"][:used].float()
        y = y * z / (1.0 + torch.exp(-z))
    s["y"][:used] = y.to(s["y"].dtype)
    s["states"][slot] = h
    return dict(y=s["y"], states=s["states"])


def _plain_scan_bwd(s):
    c = s["case"]
    b, L, E, N, G = c["b"], c["L"], c["E"], c["N"], c["G"]
    u, A = s["u"].float(), s["A"]
    v = s["dt_raw"].float() + s["dt_bias"]
    dt = _softplus(v)
    a = torch.exp(dt[..., None] * A)
    x = (dt * u)[..., None] * _per_channel(s["B"], E)
    first = s["init_state"] if s["init_state"] is not None else u.new_zeros(b, E, N)
    x[:, 0] += a[:, 0] * first
    h = _recurrence(a.clone(), x)
    dy = s["dy"].float()
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = 1.0 / (1.0 + torch.exp(-z))
        y = (h * _per_channel(s["C"], E)).sum(-1) + s["D"] * u
        out["dz"] = (dy * y * sg * (1.0 + z * (1.0 - sg))).to(s["z"].dtype)
        dy = dy * z * sg
    g = dy[..., None] * _per_channel(s["C"], E)
    if s["dfinal"] is not None:
        g[:, -1] += s["dfinal"]
    # g_t = C_t dy_t + a_{t+1} g_{t+1}: the same recurrence, from the end
    back = torch.cat([torch.zeros_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    g = _recurrence(back, g.flip(1)).flip(1)
    del back
    grouped = lambda t: t.unflatten(2, (G, E // G)).sum(3)  # noqa: E731
    io = s["u"].dtype
    out["dC"] = grouped(h * dy[..., None]).to(io)
    out["dB"] = grouped(g * (dt * u)[..., None]).to(io)
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    del h, x
    wide = g * a * before
    del before
    gb = (g * _per_channel(s["B"], E)).sum(-1)
    ddt = (gb * u + (wide * A).sum(-1)) / (1.0 + torch.exp(-v))
    out |= dict(du=(s["D"] * dy + dt * gb).to(io), ddt_raw=ddt.to(io), dA=(wide * dt[..., None]).sum((0, 1)), dD=(u * dy).sum((0, 1)),
                ddt_bias=ddt.sum((0, 1)))
    if c["state"]:
        out["dinit"] = a[:, 0] * g[:, 0]
    return out


# ---------------------------------------------------------------------------


def work(case):
    """Bytes and operations that a pass cannot do without: every input once,
    every output once; exp counted as one operation."""
    c = case
    if c["op"] == "map":
        q = _requests(c, 1)
        n, bs = len(q["lens"]), q["bs"]
        fresh = int((-(-(q["ctx"] + q["lens"]) // bs) + (-q["ctx"] // bs)).sum())
        return dict(bytes=4 * (2 * n + q["table"].size + fresh + 1) + 4 * (2 * n + 1 + q["table"].size + 1) + 16 * q["T"], flops=0)
    e, E = (2 if c["dtype"] == "bf16" else 4), c["E"]
    if "kind" in c:
        q = _requests(c, 1)
        m = _host_map(q)
        T, reads, ends = int(q["lens"].sum()), int((m["init_slot"] >= 0).sum()), len(m["ends"])
        idx = 16 * T
    if c["op"] == "conv":
        k = c["k"]
        if c["dir"] == "bwd":
            rows = c["b"] * c["L"]
            return dict(bytes=rows * E * 3 * e + E * (2 * k + 2) * 4 + (2 * c["b"] * E * k * e if c["state"] else 0), flops=rows * E * (6 * k + 8))
        return dict(bytes=T * E * 2 * e + (reads + ends) * E * k * e + E * (k + 1) * 4 + idx, flops=T * E * (2 * k + 4))
    N, G = c["N"], c["G"]
    par = E * (N + 2) * 4
    if "kind" in c:
        return dict(bytes=T * (E * (4 if c["z"] else 3) + 2 * G * N) * e + (reads + ends) * E * N * 4 + par + idx, flops=T * E * (7 * N + 10))
    rows, st = c["b"] * c["L"], c["b"] * E * N * 4
    if c["dir"] == "fwd":
        return dict(bytes=rows * (E * (4 if c["z"] else 3) + 2 * G * N) * e + par + st * (2 if c["state"] else 1), flops=rows * E * (7 * N + 10))
    return dict(bytes=rows * (E * (7 if c["z"] else 5) + 4 * G * N) * e + 2 * par + st * (3 if c["state"] else 0), flops=rows * E * (22 * N + 20))


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "map":
        return None
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    silu = lambda v: v * torch.sigmoid(v)  # noqa: E731
    if c["op"] == "conv":
        k = c["k"]
        bias = 0.0 if s["bias"] is None else s["bias"]
        if c["dir"] == "bwd":
            b, L, E = c["b"], c["L"], c["E"]
            st = s["conv_state"] if c["state"] else torch.zeros(b, E, k, dtype=torch.float64, device="cuda")
            with torch.enable_grad():
                x, w, st = s["x"].requires_grad_(), s["w"].requires_grad_(), st.requires_grad_()
                bt = (torch.zeros(E, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"]).requires_grad_()
                ext = torch.cat([st.transpose(1, 2), x], 1)
                v = bt + sum(w[:, j] * ext[:, 1 + j:1 + j + L] for j in range(k))
                grads = torch.autograd.grad((silu(v) * s["dout"]).sum(), [x, w, bt, st])
            out = dict(dx=grads[0], dw=grads[1])
            if s["bias"] is not None:
                out["dbias"] = grads[2]
            if c["state"]:
                out["dconv_state"] = grads[3]
            return out
        pool, out = s["pool"].clone(), s["out"].clone()
        cu, init = s["cu_seqlens"].tolist(), s["init_slot"].tolist()
        pieces = []
        for r in range(len(init)):
            left = s["pool"][init[r]].t() if init[r] >= 0 else torch.zeros(k, c["E"], dtype=torch.float64, device="cuda")
            pieces.append(torch.cat([left, s["x"][cu[r]:cu[r + 1]]]))
        for r, ext in enumerate(pieces):
            m = cu[r + 1] - cu[r]
            if m:
                out[cu[r]:cu[r + 1]] = silu(bias + sum(s["w"][:, j] * ext[1 + j:1 + j + m] for j in range(k)))
        for t, slot in zip(s["ends"].tolist(), s["ends_slot"].tolist()):
            r = int(np.searchsorted(cu, t, side="right")) - 1
            at = t - cu[r] + 1
            pool[slot] = pieces[r][at:at + k].t()
        return dict(out=out, pool=pool)
    N, G, E = c["N"], c["G"], c["E"]
    A, D = s["A"], s["D"]
    v = s["dt_raw"] + s["dt_bias"]
    dt = torch.where(v > 30, v, torch.log1p(torch.exp(v.clamp(max=30))))
    group = torch.arange(E, device="cuda") // (E // G)
    gate = torch.ones_like(s["u"]) if s["z"] is None else silu(s["z"])
    if "kind" in c:
        states, y = s["states"].clone(), s["y"].clone()
        cu, init = s["cu_seqlens"].tolist(), s["init_slot"].tolist()
        keep = dict(zip(s["ends"].tolist(), s["ends_slot"].tolist()))
        zero = torch.zeros(E, N, dtype=torch.float64, device="cuda")
        live = [r for r in range(len(init)) if cu[r + 1] > cu[r]]
        h = torch.stack([s["states"][init[r]] if init[r] >= 0 else zero for r in live])
        longest = max(cu[r + 1] - cu[r] for r in live)
        # the requests walk side by side; one that has ended keeps its last row
        start = torch.tensor([cu[r] for r in live], device="cuda")
        stop = torch.tensor([cu[r + 1] for r in live], device="cuda")
        for i in range(longest):
            t = torch.minimum(start + i, stop - 1)
            h = torch.exp(dt[t][..., None] * A) * h + (dt[t] * s["u"][t])[..., None] * s["B"][t][:, group]
            now = [(p, cu[r] + i) for p, r in enumerate(live) if cu[r] + i < cu[r + 1]]
            if len(now) < len(live):
                t = torch.tensor([q for _, q in now], device="cuda")
                hh = h[torch.tensor([p for p, _ in now], device="cuda")]
            else:
                hh = h
            y[t] = ((hh * s["C"][t][:, group]).sum(-1) + D * s["u"][t]) * gate[t]
            for (_, at), row in zip(now, hh):
                if at in keep:
                    states[keep[at]] = row
        return dict(y=y, states=states)
    b, L = c["b"], c["L"]
    h = torch.zeros(b, E, N, dtype=torch.float64, device="cuda") if s["init_state"] is None else s["init_state"]
    if c["dir"] == "fwd":
        y = torch.empty_like(s["u"])
        for t in range(L):
            h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * s["u"][:, t])[..., None] * s["B"][:, t][:, group]
            y[:, t] = (h * s["C"][:, t][:, group]).sum(-1)
        return dict(y=(y + D * s["u"]) * gate, final_state=h)
    hs = [h]
    pre = torch.empty_like(s["u"])
    for t in range(L):
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * s["u"][:, t])[..., None] * s["B"][:, t][:, group]
        pre[:, t] = (h * s["C"][:, t][:, group]).sum(-1) + D * s["u"][:, t]
        hs.append(h)
    dpre = s["dy"] * gate
    g = torch.zeros_like(h) if s["dfinal"] is None else s["dfinal"]
    dA, zero = torch.zeros_like(A), torch.zeros(b, L, G, N, dtype=torch.float64, device="cuda")
    dB, dC, dx, ddt = zero.clone(), zero.clone(), torch.empty_like(pre), torch.empty_like(pre)
    for t in reversed(range(L)):
        Bt, Ct = s["B"][:, t][:, group], s["C"][:, t][:, group]
        g = g + dpre[:, t, :, None] * Ct
        dC[:, t] = (hs[t + 1] * dpre[:, t, :, None]).unflatten(1, (G, E // G)).sum(2)
        dB[:, t] = (g * (dt[:, t] * s["u"][:, t])[..., None]).unflatten(1, (G, E // G)).sum(2)
        dx[:, t] = (g * Bt).sum(-1)
        g = g * torch.exp(dt[:, t, :, None] * A)
        flow = g * hs[t]
        ddt[:, t] = (flow * A).sum(-1)
        dA += (flow * dt[:, t, :, None]).sum(0)
    draw_ = (ddt + dx * s["u"]) * torch.sigmoid(v)
    out = dict(du=D * dpre + dt * dx, ddt_raw=draw_, dA=dA, dB=dB, dC=dC, dD=(dpre * s["u"]).sum((0, 1)), ddt_bias=draw_.sum((0, 1)))
    if s["z"] is not None:
        sg = torch.sigmoid(s["z"])
        out["dz"] = s["dy"] * pre * sg * (1 + s["z"] * (1 - sg))
    if c["state"]:
        out["dinit"] = g
    return out
