"""float64 definitions of the diagonal scan and what serves it, token by token
on the CPU (torch), written from the formulas and sharing nothing with the
kernels, and the batches and tolerances of their tests.

Tolerances, derived before any run.  An output element is held to
    |got - ref| <= r |ref| + c scale,   scale = max |ref|,
r = half a step of its type (bf16: 2^-8, float32: 2^-24, doubled for the
rounding of the reference's own inputs to nothing else), and c the float32
arithmetic inside.  A step of the recurrence multiplies by exp(dt A) with a
relative error of at most 2 ulp of the hardware exponential (2^-22) plus the
rounding of its argument (|dt A log2 e| <= 8 here: 8 * 2^-24) and three
roundings (3 * 2^-24): 1e-6.  Errors carry on with the state, so they pile up
over 1 / (1 - exp(dt A)) steps; dt >= softplus(-4.9) = 0.007 and |A| >= 0.3
give at most 470 steps, all errors of one sign: 4.7e-4.  Errors of random sign
over that horizon give sqrt(470) 1e-6 = 2.2e-5.  The tests draw |A| >= 0.3 and
take C_SCAN = 1e-4, between the two.  The conv has at most 4 products
(8 * 2^-24) and SiLU's exponential and divide (6 * 2^-24, arguments to 8
adding 8 * 2^-24): C_CONV = 2e-6.  Sums over R rows of a gradient add
sqrt(R) 2^-24 in random sign, R <= 20000: 1e-5 on top, inside C_SCAN.
"""
import numpy as np
import torch

R_IO = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8}
C_SCAN = 1e-4
C_CONV = 2e-6


def close(got, ref, what, c=C_SCAN, scale=None):
    r = R_IO[got.dtype]
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    if not ref.numel():
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    scale = ref.abs().max().item() if scale is None else scale
    off = (got - ref).abs() - (r * ref.abs() + c * scale)
    assert off.max().item() <= 0, f"{what}: {(got - ref).abs().max().item():.3e} off at scale {scale:.3e}"


def softplus(v):
    return torch.where(v > 40, v, torch.log1p(torch.exp(v.clamp(max=40.0))))


def silu(v):
    return v * torch.sigmoid(v)


# ---------------------------------------------------------------------------
# the recurrence


def step(h, u, dt_raw, A, B, C, dt_bias, D, z):
    """One token: h [E, N], u, dt_raw, z [E], B, C [G, N]; -> (h, y)."""
    E = u.shape[0]
    v = dt_raw if dt_bias is None else dt_raw + dt_bias
    dt = softplus(v)
    Bc, Cc = B.repeat_interleave(E // B.shape[0], 0), C.repeat_interleave(E // C.shape[0], 0)
    h = torch.exp(dt[:, None] * A) * h + (dt * u)[:, None] * Bc
    y = (h * Cc).sum(-1)
    if D is not None:
        y = y + D * u
    if z is not None:
        y = y * silu(z)
    return h, y


def scan(p, h):
    """A sequence's rows, p = dict of float64 u, dt_raw, A, B, C, dt_bias, D, z
    with a leading token axis; -> (y [L, E], states after each token)."""
    ys, hs = [], []
    for t in range(p["u"].shape[0]):
        h, y = step(h, p["u"][t], p["dt_raw"][t], p["A"], p["B"][t], p["C"][t], p["dt_bias"], p["D"], None if p["z"] is None else p["z"][t])
        ys.append(y)
        hs.append(h)
    return torch.stack(ys), hs


def rows(p, a, b):
    return {k: (v[a:b] if v is not None and k in ("u", "dt_raw", "B", "C", "z") else v) for k, v in p.items()}


def f64(p):
    return {k: (v.double().cpu() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}


def scan_inputs(lead, E, N, G, dtype, seed, z=True, bias=True, D=True, device="cpu", pad=0):
    """Random rows: u and z views of wider rows, B and C columns of a
    projection's rows at an odd offset where the type allows it."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    lo = 0.3
    A = -(lo + torch.rand(E, N, generator=g) * torch.linspace(1.0, 6.0, N))
    wide = torch.zeros(*lead, 2 * E)
    wide[..., E:] = rn(*lead, E)
    off = 3 + pad
    proj = torch.zeros(*lead, off + 2 * G * N)
    proj[..., off:] = rn(*lead, 2 * G * N) / N ** 0.5
    proj = proj.to(dtype).to(device)
    uw = torch.zeros(*lead, E + 8)
    uw[..., :E] = rn(*lead, E)
    p = dict(u=uw.to(dtype).to(device)[..., :E], dt_raw=(torch.rand(*lead, E, generator=g) * 3 - 4).to(dtype).to(device), A=A.to(device),
             B=proj[..., off:off + G * N].unflatten(-1, (G, N)), C=proj[..., off + G * N:].unflatten(-1, (G, N)),
             dt_bias=(0.3 * rn(E)).to(device) if bias else None, D=rn(E).to(device) if D else None,
             z=wide.to(dtype).to(device)[..., E:] if z else None)
    return p


# ---------------------------------------------------------------------------
# the conv


def conv(ext, w, bias):
    """ext [k + L, E]: k cached rows, then the tokens; -> silu outputs [L, E]."""
    k = w.shape[1]
    L = ext.shape[0] - k
    v = sum(w[:, j] * ext[1 + j:1 + j + L] for j in range(k))
    return silu(v if bias is None else v + bias)


# ---------------------------------------------------------------------------
# batches of requests


def batch(lens, ctx, bs, seed=0, spare=3, max_blocks=None):
    """What a scheduler holds for requests of these lengths: every held block
    in a slot of its own, the rest in the free list."""
    r = np.random.default_rng(seed)
    lens, ctx = np.asarray(lens, np.int64), np.asarray(ctx, np.int64)
    held, need = -(-ctx // bs), -(-(ctx + lens) // bs)
    nslots = int(held.sum() + (need - held).sum()) + spare
    order = r.permutation(nslots).astype(np.int32)
    mb = int(need.max(initial=0)) + 1 if max_blocks is None else max_blocks
    table = np.full((len(lens), mb), -7, np.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        at += h
    return dict(lens=lens, ctx=ctx, bs=bs, nslots=nslots, table=table, free=order[at:], head=0)


def ref_map(q, T):
    """The map of a batch, request by request and row by row."""
    n, bs = len(q["lens"]), q["bs"]
    table, head = q["table"].copy(), q["head"]
    cu, seq, pos, slot, init = [0], [-1] * T, [-1] * T, [-1] * T, []
    for r in range(n):
        ctx, m = int(q["ctx"][r]), int(q["lens"][r])
        init.append(int(q["table"][r, (ctx - 1) // bs]) if ctx else -1)
        for j in range(-(-ctx // bs), -(-(ctx + m) // bs)):
            table[r, j] = q["free"][head]
            head += 1
        for i in range(m):
            t, p = cu[-1] + i, ctx + i
            seq[t], pos[t], slot[t] = r, p, int(table[r, p // bs]) * bs + p % bs
        cu.append(cu[-1] + m)
    return dict(cu_seqlens=cu, seq_of=seq, pos_of=pos, slot_of=slot, init_slot=init, table=table, free_head=[head])


def kept_rows(m, bs):
    """(row, request, slot) of every row whose state a packed call keeps."""
    cu = list(m["cu_seqlens"])
    out = []
    for t, s in enumerate(m["slot_of"]):
        if s >= 0:
            r = m["seq_of"][t]
            if t + 1 == cu[r + 1] or s % bs == bs - 1:
                out.append((t, r, s // bs))
    return out
