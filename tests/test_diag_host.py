"""The C boundary of include/ssd_diag.h on the host (no GPU): exports, argument
validation, workspace sizes; and the float64 references of the GPU tests
against differences.

Pointer arguments are fake addresses that are never dereferenced: every call
below fails validation or is empty work."""
import os
import re
import subprocess

import pytest
import torch

import diag_ref as R
from ssd_selective_scan_b200 import binding as libssd
from ssd_selective_scan_b200 import build as ssd_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INV, UNS = libssd.SSD_OK, libssd.SSD_ERR_INVALID_ARG, libssd.SSD_ERR_UNSUPPORTED
F32, BF16 = libssd.SSD_F32, libssd.SSD_BF16


@pytest.fixture(scope="module", autouse=True)
def built():
    ssd_build.build()
    libssd.load()


def fake(i, off=0):
    return 0x7f0000000000 + i * (1 << 36) + off


def test_header_binding_and_exports_agree():
    txt = open(os.path.join(ROOT, "include", "ssd_diag.h")).read()
    declared = set(re.findall(r"SSD_API\s+[\w\s\*]+?\b(ssd_\w+)\s*\(", txt))
    assert declared == set(libssd.DIAG_SIGNATURES)
    out = subprocess.check_output(["nm", "-D", "--defined-only", libssd.LIB_PATH], text=True)
    assert declared <= {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    for name in declared:
        assert callable(getattr(libssd, name))


def smap(**kw):
    a = dict(lens=fake(1), ctx=fake(2), table=fake(3), free_list=fake(4), free_head=fake(5), n=4, max_blocks=8, nfree=16, T=64,
             block_tokens=16, nslots=64, cu_seqlens=fake(6), seq_of=fake(7), pos_of=fake(8), slot_of=fake(9), init_slot=fake(10),
             table_out=fake(11), free_head_out=fake(12), workspace=fake(13), workspace_bytes=1 << 20, status=fake(14), stream=None)
    a.update(kw)
    return libssd.ssd_state_map(**a)


def test_state_map_validation():
    for k in ("lens", "ctx", "table", "free_list", "free_head", "cu_seqlens", "seq_of", "pos_of", "slot_of", "init_slot", "table_out",
              "free_head_out", "workspace", "status"):
        assert smap(**{k: None}) == INV, k
    for k in ("n", "max_blocks", "nfree", "T", "nslots"):
        assert smap(**{k: -1}) == INV, k
    assert smap(block_tokens=0) == INV
    assert smap(workspace_bytes=libssd.ssd_state_map_workspace_bytes(4) - 1) == INV
    assert smap(seq_of=fake(7, 4)) == INV and smap(slot_of=fake(9, 8)) == INV and smap(lens=fake(1, 2)) == INV
    assert smap(cu_seqlens=fake(1)) == INV and smap(table_out=fake(3, 16)) == INV and smap(pos_of=fake(7, 16)) == INV
    assert smap(free_head_out=fake(3)) == INV and smap(status=fake(13)) == INV
    assert smap(nslots=1500001) == UNS and smap(n=1 << 25, workspace_bytes=1 << 30) == UNS
    assert libssd.ssd_state_map_workspace_bytes(-1) == 0 and libssd.ssd_state_map_workspace_bytes(0) > 0


def conv(**kw):
    a = dict(x=fake(1), x_stride=128, out=fake(2), out_stride=64, w=fake(3), bias=None, cache=fake(4), cu_seqlens=fake(5), seq_of=fake(6),
             slot_of=fake(7), init_slot=fake(8), nseq=3, T=20, E=64, k=4, block_tokens=8, nslots=9, dtype=BF16, status=fake(9), stream=None)
    a.update(kw)
    return libssd.ssd_conv1d_silu_varlen(**a)


def test_conv_varlen_validation():
    for k in ("x", "out", "w", "cache", "cu_seqlens", "seq_of", "slot_of", "init_slot", "status"):
        assert conv(**{k: None}) == INV, k
    assert conv(T=0) == OK and conv(T=0, x=None, out=None, seq_of=None, slot_of=None) == OK and conv(nseq=0, init_slot=None) == OK
    assert conv(T=-1) == INV and conv(nseq=-1) == INV and conv(nslots=-1) == INV and conv(block_tokens=0) == INV and conv(E=60) == INV
    assert conv(x_stride=56) == INV and conv(x_stride=130) == INV and conv(out_stride=60) == INV and conv(dtype=5) == INV
    assert conv(x=fake(1, 8)) == INV and conv(cache=fake(4, 2)) == INV and conv(slot_of=fake(7, 4)) == INV and conv(w=fake(3, 1)) == INV
    assert conv(out=fake(1, 64)) == INV and conv(cache=fake(1)) == INV and conv(out=fake(6)) == INV and conv(status=fake(4, 4)) == INV
    assert conv(k=1) == UNS and conv(k=5) == UNS


def cbwd(**kw):
    a = dict(x=fake(1), w=fake(2), bias=None, conv_state=None, dout=fake(3), dx=fake(4), dw=fake(5), dbias=fake(6), dconv_state=fake(7),
             b=2, L=20, E=64, k=4, dtype=BF16, workspace=fake(8), workspace_bytes=1 << 20, stream=None)
    a.update(kw)
    return libssd.ssd_conv1d_silu_bwd(**a)


def test_conv_bwd_validation():
    for k in ("x", "w", "dout", "dx", "dw", "workspace"):
        assert cbwd(**{k: None}) == INV, k
    assert cbwd(b=-1) == INV and cbwd(L=-1) == INV and cbwd(E=62) == INV and cbwd(k=0) == INV and cbwd(dtype=2) == INV
    assert cbwd(workspace_bytes=libssd.ssd_conv1d_silu_bwd_workspace_bytes(2, 20, 64, 4) - 1) == INV
    assert cbwd(dx=fake(1)) == INV and cbwd(dw=fake(2)) == INV and cbwd(workspace=fake(3)) == INV and cbwd(dconv_state=fake(4, 16)) == INV
    assert cbwd(x=fake(1, 8)) == INV and cbwd(dw=fake(5, 2)) == INV
    assert cbwd(k=1) == UNS and cbwd(k=5) == UNS
    assert libssd.ssd_conv1d_silu_bwd_workspace_bytes(0, 5, 64, 4) == 0


def scan(**kw):
    a = dict(u=fake(1), u_stride=64, dt_raw=fake(2), dt_stride=72, z=fake(3), z_stride=128, B=fake(4), C=fake(4, 64), bc_stride=64, A=fake(5),
             dt_bias=None, D=None, init_state=fake(6), y=fake(7), final_state=fake(8), b=2, L=30, E=64, N=16, G=2, dtype=BF16,
             workspace=fake(9), workspace_bytes=1 << 24, stream=None)
    a.update(kw)
    return libssd.ssd_diag_scan_fwd(**a)


def test_scan_validation():
    for k in ("u", "dt_raw", "B", "C", "A", "y"):
        assert scan(**{k: None}) == INV, k
    assert scan(b=0, u=None, y=None) == OK and scan(L=0, final_state=None, u=None, y=None) == OK
    assert scan(L=0, final_state=fake(6)) == OK                     # in place: nothing to copy
    assert scan(b=-1) == INV and scan(L=-1) == INV and scan(E=0) == INV and scan(G=3) == INV and scan(dtype=9) == INV
    assert scan(E=72, G=2, u_stride=128, dt_stride=128, bc_stride=32) == INV    # 36 channels a group
    assert scan(N=6) == INV and scan(N=0) == INV
    assert scan(u_stride=56) == INV and scan(dt_stride=68) == INV and scan(z_stride=8) == INV and scan(bc_stride=31) == INV
    assert scan(u=fake(1, 8)) == INV and scan(A=fake(5, 4)) == INV and scan(init_state=fake(6, 8)) == INV and scan(B=fake(4, 1)) == INV
    assert scan(y=fake(1, 64)) == INV and scan(y=fake(3)) == INV and scan(final_state=fake(7)) == INV and scan(y=fake(6)) == INV
    assert scan(final_state=fake(6, 64)) == INV                     # partly over init_state
    assert scan(N=68, bc_stride=136) == UNS and scan(b=1 << 16, L=1 << 16) == UNS


def test_scan_workspace():
    need = libssd.ssd_diag_scan_workspace_bytes(1, 4096, 64, 16, 1)
    assert need > 0 and libssd.ssd_diag_scan_workspace_bytes(1, 100, 64, 16, 1) == 0      # a short one is not cut
    assert libssd.ssd_diag_scan_workspace_bytes(64, 64 * 2048, 8192, 16, 1) == 0          # nor one that fills the device
    assert scan(b=1, L=4096, G=1, workspace_bytes=need - 1) == INV and scan(b=1, L=4096, G=1, workspace=None) == INV
    assert scan(b=1, L=4096, G=1, workspace=fake(9, 8)) == INV and scan(b=1, L=4096, G=1, workspace=fake(1)) == INV
    for bad in ((0, 5, 64, 16, 1), (1, 0, 64, 16, 1), (1, 5, 64, 80, 1), (1, 5, 64, 16, 0)):
        assert libssd.ssd_diag_scan_workspace_bytes(*bad) == 0


def packed(fn="ssd_diag_scan_fwd_varlen", **kw):
    a = dict(u=fake(1), u_stride=64, dt_raw=fake(2), dt_stride=72, z=None, z_stride=64, B=fake(4), C=fake(4, 64), bc_stride=64, A=fake(5),
             dt_bias=None, D=None, states=fake(6), y=fake(7), cu_seqlens=fake(8), seq_of=fake(9), slot_of=fake(10), init_slot=fake(11),
             nseq=3, T=30, E=64, N=16, G=2, block_tokens=8, nslots=9, dtype=BF16, workspace=fake(12), workspace_bytes=1 << 24,
             status=fake(13), stream=None)
    a.update(kw)
    if fn == "ssd_diag_state_update":
        a["rows"] = a.pop("T")
        del a["workspace"], a["workspace_bytes"]
    return getattr(libssd, fn)(**a)


@pytest.mark.parametrize("fn", ["ssd_diag_scan_fwd_varlen", "ssd_diag_state_update"])
def test_packed_validation(fn):
    call = lambda **kw: packed(fn, **kw)  # noqa: E731
    for k in ("u", "dt_raw", "B", "C", "A", "y", "states", "cu_seqlens", "seq_of", "slot_of", "init_slot", "status"):
        assert call(**{k: None}) == INV, k
    assert call(T=0) == OK
    assert call(T=-1) == INV and call(nseq=-1) == INV and call(nslots=-1) == INV and call(block_tokens=0) == INV and call(N=10) == INV
    assert call(y=fake(6)) == INV and call(states=fake(1)) == INV and call(y=fake(10)) == INV and call(status=fake(7)) == INV
    assert call(slot_of=fake(10, 4)) == INV and call(seq_of=fake(9, 2)) == INV and call(u_stride=60) == INV and call(states=fake(6, 4)) == INV
    assert call(N=128, bc_stride=256) == UNS


def test_update_without_a_map():
    none = dict(cu_seqlens=None, seq_of=None, slot_of=None, init_slot=None, nseq=0, status=None)
    assert packed("ssd_diag_state_update", T=0, **none) == OK
    assert packed("ssd_diag_state_update", nslots=29, **none) == INV      # fewer states than rows


def bwd(**kw):
    a = dict(u=fake(1), u_stride=64, dt_raw=fake(2), dt_stride=72, z=fake(3), z_stride=128, B=fake(4), C=fake(4, 64), bc_stride=64, A=fake(5),
             dt_bias=None, D=None, init_state=fake(6), dy=fake(7), dfinal=fake(8), du=fake(9), ddt_raw=fake(10), dz=fake(11), dB=fake(12),
             dC=fake(13), dA=fake(14), dD=fake(15), ddt_bias=fake(16), dinit=fake(17), b=2, L=30, E=64, N=16, G=2, dtype=BF16,
             workspace=fake(18), workspace_bytes=1 << 24, stream=None)
    a.update(kw)
    return libssd.ssd_diag_scan_bwd(**a)


def test_scan_bwd_validation():
    for k in ("u", "dt_raw", "B", "C", "A", "dy", "du", "ddt_raw", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "workspace"):
        assert bwd(**{k: None}) == INV, k
    assert bwd(b=-1) == INV and bwd(L=-1) == INV and bwd(G=3) == INV and bwd(N=2) == INV and bwd(dtype=7) == INV
    need = libssd.ssd_diag_scan_bwd_workspace_bytes(2, 30, 64, 16, 2)
    assert need > 0 and bwd(workspace_bytes=need - 1) == INV and bwd(workspace=fake(18, 8)) == INV
    assert bwd(du=fake(1)) == INV and bwd(dA=fake(5)) == INV and bwd(dinit=fake(6)) == INV and bwd(dB=fake(9, 32)) == INV
    assert bwd(workspace=fake(7)) == INV and bwd(dy=fake(7, 8)) == INV and bwd(dz=fake(11, 2)) == INV
    assert bwd(N=68, bc_stride=136) == UNS
    assert libssd.ssd_diag_scan_bwd_workspace_bytes(2, 0, 64, 16, 2) == 0 and libssd.ssd_diag_scan_bwd_workspace_bytes(2, 5, 64, 68, 2) == 0


def test_row_numbers_stay_ints():
    """Calls whose last rows lie a tile's step from the end of int are refused
    (the kernels' row counters would run over)."""
    T = 2 ** 31 - 9
    tiny = dict(E=8, N=4, G=1, u_stride=8, dt_stride=8, z_stride=8, bc_stride=4, workspace_bytes=1 << 50)
    assert smap(T=T) == UNS
    assert conv(T=T, E=8, x_stride=8, out_stride=8) == UNS
    assert cbwd(b=1, L=T, E=8, workspace_bytes=1 << 50) == UNS
    assert scan(b=1, L=T, **tiny) == UNS
    assert packed(T=T, C=fake(14), **tiny) == UNS
    assert packed("ssd_diag_state_update", T=T, C=fake(14), **tiny) == UNS
    assert bwd(b=1, L=T, **tiny) == UNS


# ---------------------------------------------------------------------------
# the references themselves


def test_reference_gradients_against_differences():
    """Autograd through the float64 definitions, which the GPU gradients are
    held to, against central differences (torch.autograd.gradcheck)."""
    p = R.f64(R.scan_inputs((5,), 8, 4, 1, torch.float32, seed=3))
    keys = list(p)
    leaves = [p[k].clone().requires_grad_() for k in keys] + [torch.randn(8, 4, dtype=torch.float64, requires_grad=True)]

    def run(*v):
        y, h = R.scan(dict(zip(keys, v[:-1])), v[-1])
        return y, h[-1]
    assert torch.autograd.gradcheck(run, leaves)
    w = torch.randn(3, 4, dtype=torch.float64, requires_grad=True)
    ext = torch.randn(9, 3, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(lambda e, v, b: R.conv(e, v, b), (ext, w, torch.randn(3, dtype=torch.float64, requires_grad=True)))


def test_reference_step_by_hand():
    """One channel, one state: the formula on paper."""
    one = torch.ones(1, dtype=torch.float64)
    h, y = R.step(2 * one[:, None], 3 * one, 0 * one, -one[:, None], 0.5 * one[:, None], 4 * one[:, None], None, 10 * one, 0 * one + 1)
    dt = torch.log(torch.tensor(2.0, dtype=torch.float64))               # softplus(0)
    want = torch.exp(-dt) * 2 + dt * 3 * 0.5
    assert abs(h.item() - want.item()) < 1e-15
    assert abs(y.item() - ((4 * want + 30) / (1 + torch.exp(-one)))).item() < 1e-13


def test_reference_map_by_hand():
    q = dict(lens=[3, 1], ctx=[2, 4], bs=4, table=torch.tensor([[5, -1, -1], [7, -1, -1]]).numpy(), free=[9, 8], head=0, nslots=10)
    m = R.ref_map(q, 6)
    assert m["cu_seqlens"] == [0, 3, 4] and m["seq_of"] == [0, 0, 0, 1, -1, -1] and m["pos_of"] == [2, 3, 4, 4, -1, -1]
    assert m["slot_of"] == [22, 23, 36, 32, -1, -1] and m["init_slot"] == [5, 7] and m["free_head"] == [2]
    assert m["table"].tolist() == [[5, 9, -1], [7, 8, -1]]
    assert R.kept_rows(m, 4) == [(1, 0, 5), (2, 0, 9), (3, 1, 8)]
