"""diag.py's calls on the host (no GPU): tensors on the CPU, and in the place of
the extension's entry points ones that note their arguments and launch nothing."""
import pytest
import torch

from ssd_selective_scan_b200 import StateMap, diag
from ssd_selective_scan_b200 import binding as libssd
from ssd_selective_scan_b200 import build as ssd_build

I32 = torch.int32


@pytest.fixture(scope="module")
def ext():
    ssd_build.build()
    return libssd.load_pycall()


class HostOn(diag._On):
    """A call's device and stream, on the CPU."""

    def __init__(self, like, stream):
        self.device, self.handle, self.switch, self.other = like.device, 0, None, None


@pytest.fixture
def calls(ext, monkeypatch):
    """(name, arguments) of the entry points called, all of which answer SSD_OK."""
    made = []

    class Noting:
        def __getattr__(self, name):
            if not name.startswith("ssd_") or name.endswith("_bytes"):
                return getattr(ext, name)
            return lambda *a: made.append((name, a)) or libssd.SSD_OK

    diag._load()
    monkeypatch.setattr(diag, "_native", Noting())
    monkeypatch.setattr(diag, "_On", HostOn)
    return made


def requests(n, blocks=3):
    i = lambda *s: torch.zeros(*s, dtype=I32)  # noqa: E731
    return dict(lens=i(n), ctx=i(n), table=i(n, blocks), free_list=i(8), free_head=i(1))


@pytest.mark.parametrize("before,now", [(2, 5), (5, 2), (0, 3), (3, 0)])
def test_state_map_out_of_another_batch(calls, before, now):
    """A map made for fewer requests would be written past its end, one for
    more would keep the old batch's last entries: both are refused, whatever
    table and free_head stand in it."""
    old = diag.state_map(**requests(before), T=7, block_tokens=4, nslots=9)
    new = requests(now)
    del calls[:]
    with pytest.raises(ValueError, match=f"out is the map of {before} requests"):
        diag.state_map(**new, T=7, block_tokens=4, nslots=9, out=old._replace(table=new["table"], free_head=new["free_head"]))
    assert not calls
    same = requests(before)
    assert diag.state_map(**same, T=7, block_tokens=4, nslots=9, out=old) is old
    (name, a), = calls
    assert name == "ssd_state_map" and a[5] == before and a[11] == old.cu_seqlens.data_ptr()


def test_state_map_out_of_other_rows(calls):
    old = diag.state_map(**requests(3), T=7, block_tokens=4, nslots=9)
    for T in (6, 8):
        with pytest.raises(ValueError):
            diag.state_map(**requests(3), T=T, block_tokens=4, nslots=9, out=old)
    with pytest.raises(ValueError, match="another block size"):
        diag.state_map(**requests(3), T=7, block_tokens=8, nslots=9, out=old)
    assert len(calls) == 1 and isinstance(old, StateMap)


def test_first_use_from_two_threads(ext, monkeypatch):
    """Another thread takes the extension for loaded when it sees `_native`:
    the checks that it then calls have to be there."""
    seen = []

    class Slow:
        def __getattr__(self, name):
            seen.append((name, diag._native))     # what another thread would find now
            return getattr(ext, name)

    for name in ("_native", "_dense", "_rows", "_bc"):
        monkeypatch.setattr(diag, name, None)
    monkeypatch.setattr(libssd, "load_pycall", Slow)
    diag._load()
    assert {n for n, _ in seen} == {"dense", "rows", "bc"}
    assert all(native is None for _, native in seen)
    assert diag._native is not None and None not in (diag._dense, diag._rows, diag._bc)


def dense(b, L, E, N=16, G=1):
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    return dict(u=f(b, L, E), dt_raw=f(b, L, E), A=f(E, N), B=f(b, L, G, N), C=f(b, L, G, N))


@pytest.mark.parametrize("b,L,E,cut", [(16384, 1, 128, False), (512, 100, 64, False), (40, 128, 64, False), (40, 129, 64, True), (1, 4096, 64, True),
                                       (1, 100, 64, False), (64, 300, 8192, False)])
def test_dense_scan_asks_for_what_it_uses(calls, b, L, E, cut):
    """Sequences no longer than a piece are not cut, however many they are:
    the call takes no workspace for them."""
    need = libssd.ssd_diag_scan_fwd_workspace_bytes(b, L, E, 16, 1)
    assert (need > 0) == cut
    assert need == (libssd.ssd_diag_scan_workspace_bytes(b, b * L, E, 16, 1) if cut else 0)
    if b * L * E < 1 << 23:
        diag.diag_scan_fwd(**dense(b, L, E))
        (name, a), = calls
        assert name == "ssd_diag_scan_fwd" and a[-2] == need and (a[-3] is None) == (need == 0)


def test_dense_scan_workspace_of_no_call():
    for bad in ((0, 5, 64, 16, 1), (1, 0, 64, 16, 1), (1, 5, 64, 80, 1), (1, 5, 64, 16, 0), (1 << 16, 1 << 16, 64, 16, 1)):
        assert libssd.ssd_diag_scan_fwd_workspace_bytes(*bad) == 0
