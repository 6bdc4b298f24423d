"""The extension behind diag.py on the host (no GPU): its checks of tensors
give what the entry points take or say what is wrong, and its calls convert
arguments as the header declares them."""
import pytest
import torch

from ssd_selective_scan_b200 import binding as libssd
from ssd_selective_scan_b200 import build as ssd_build
from test_diag_host import INV, fake, packed

F32, BF16 = torch.float32, torch.bfloat16
CPU = torch.device("cpu")


@pytest.fixture(scope="module")
def ext():
    ssd_build.build()
    return libssd.load_pycall()


def test_covers_the_header(ext):
    for name in libssd.DIAG_SIGNATURES:
        assert callable(getattr(ext, name))


def test_dense(ext):
    t = torch.zeros(3, 4)
    assert ext.dense(t, "t", F32, (3, 4), CPU) == t.data_ptr()
    assert ext.dense(t[1:], "t", F32, torch.Size((2, 4)), CPU) == t[1:].data_ptr()
    assert ext.dense(None, "t", F32, (3, 4), CPU) is None
    assert ext.dense(torch.nn.Parameter(t), "t", F32, (3, 4), CPU) == t.data_ptr()
    assert ext.dense(torch.zeros(0, 4), "t", F32, (0, 4), CPU) == 0
    for bad in ((t, "t", BF16, (3, 4), CPU), (t, "t", F32, (4, 3), CPU), (t, "t", F32, (12,), CPU), (t.t(), "t", F32, (4, 3), CPU),
                (t[:, :2], "t", F32, (3, 2), CPU), (t, "t", F32, (3, 4), torch.device("cuda:0")), (t.to_sparse(), "t", F32, (3, 4), CPU)):
        with pytest.raises(ValueError, match="t must be a contiguous"):
            ext.dense(*bad)
    with pytest.raises(ValueError, match=r"torch.float32 tensor of shape \(2, 4\) on cpu"):
        ext.dense(t, "t", F32, torch.Size((2, 4)), CPU)
    with pytest.raises(TypeError, match="t must be a tensor"):
        ext.dense([1.0], "t", F32, (1,), CPU)
    with pytest.raises(TypeError):
        ext.dense(t, "t", F32, (3, 4))
    with pytest.raises(TypeError):
        ext.dense(t, "t", "float32", (3, 4), CPU)
    with pytest.raises(TypeError):
        ext.dense(t, "t", F32, [3, 4], CPU)


def test_rows(ext):
    w = torch.zeros(2, 5, 24)
    v = w[..., 8:16]
    assert ext.rows(v, "v", (2, 5), 8, w) == (v.data_ptr(), 24)
    assert ext.rows(v[0], "v", (5,), 8, w) == (v.data_ptr(), 24)
    assert ext.rows(v[:, :1], "v", (2, 1), 8, w) == (v.data_ptr(), 120)      # one row each: the sequences' spacing
    assert ext.rows(v[:1, :1], "v", (1, 1), 8, w) == (v.data_ptr(), 8)       # a single row has none
    assert ext.rows(v[0, :1], "v", (1,), 8, w) == (v.data_ptr(), 8)
    assert ext.rows(v[:, :0], "v", (2, 0), 8, w)[1] == 8
    assert ext.rows(None, "v", (2, 5), 8, w) == (None, 8)
    assert ext.rows(w[0, :1].expand(5, 24), "v", (5,), 24, w)[1] == 0        # the entry points refuse it
    for bad, why in (((v, "v", (2, 4), 8, w), "tensor of shape"), ((v.double(), "v", (2, 5), 8, w), "torch.float32 tensor"),
                     ((w[:, ::2, :8].flatten(0, 1)[:, ::2], "v", (6,), 4, w), "dense rows"),
                     ((w[..., ::3], "v", (2, 5), 8, w), "dense rows"), ((w[:, :4, :8], "v", (2, 4), 8, w), "evenly spaced")):
        with pytest.raises(ValueError, match=why):
            ext.rows(*bad)
    with pytest.raises(TypeError):
        ext.rows(3, "v", (2, 5), 8, w)
    with pytest.raises(TypeError):
        ext.rows(v, "v", (1, 2, 5), 8, w)


def test_bc(ext):
    p = torch.zeros(2, 5, 40)
    B, C = p[..., 3:19].unflatten(-1, (2, 8)), p[..., 19:35].unflatten(-1, (2, 8))
    assert ext.bc(B, C, (2, 5), p) == (B.data_ptr(), C.data_ptr(), 40, 2, 8)
    assert ext.bc(B[0], C[0], (5,), p) == (B.data_ptr(), C.data_ptr(), 40, 2, 8)
    assert ext.bc(B[:, :0], C[:, :0], (2, 0), p)[2:] == (16, 2, 8)
    for b, c, lead in ((B, C[..., :4], (2, 5)), (B, C, (2, 4)), (B, C.contiguous(), (2, 5)), (B.double(), C.double(), (2, 5)),
                       (B.transpose(2, 3).contiguous().transpose(2, 3), C, (2, 5)), (B[0], C[0], (2, 5))):
        with pytest.raises(ValueError):
            ext.bc(b, c, lead, p)
    with pytest.raises(TypeError):
        ext.bc(B, None, (2, 5), p)


def test_empty_and_part(ext):
    e = ext.empty((3, 0, 2), BF16, CPU)
    assert e.shape == (3, 0, 2) and e.dtype == BF16
    whole = torch.arange(20, dtype=torch.int32)
    p = ext.part(whole, (2, 3), 5)
    assert p.tolist() == [[5, 6, 7], [8, 9, 10]] and p.is_contiguous() and p.untyped_storage().data_ptr() == whole.data_ptr()
    p[0, 0] = -1
    assert whole[5] == -1
    assert ext.part(whole, (4, 0), 20).shape == (4, 0) and ext.part(whole, (20,), 0).numel() == 20
    for shape, off in (((21,), 0), ((1,), 20), ((3, 3), 12), ((1,), -1), ((-1,), 0)):
        with pytest.raises(ValueError):
            ext.part(whole, shape, off)


def test_arguments(ext):
    a = [fake(6), fake(1), 64, fake(2), 72, None, 64, fake(4), fake(4, 64), 64, fake(5), None, None, fake(7), fake(8), fake(9), fake(10),
         fake(11), 3, 30, 64, 16, 2, 8, 9, libssd.SSD_BF16, fake(13), None]
    assert len(a) == len(libssd.DIAG_SIGNATURES["ssd_diag_state_update"][1])
    a[19] = 0
    assert ext.ssd_diag_state_update(*a) == libssd.SSD_OK == packed("ssd_diag_state_update", T=0)
    a[23] = 0
    assert ext.ssd_diag_state_update(*a) == INV == packed("ssd_diag_state_update", T=0, block_tokens=0)
    with pytest.raises(TypeError, match="28 arguments"):
        ext.ssd_diag_state_update(*a[:-1])
    with pytest.raises(OverflowError):
        ext.ssd_diag_state_update(*a[:18], 2 ** 31, *a[19:])
    with pytest.raises(TypeError):
        ext.ssd_diag_state_update("here", *a[1:])
    for args in ((1, 4096, 64, 16, 1), (64, 64 * 2048, 8192, 16, 1)):
        assert ext.ssd_diag_scan_workspace_bytes(*args) == libssd.ssd_diag_scan_workspace_bytes(*args)
