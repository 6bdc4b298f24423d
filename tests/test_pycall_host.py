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


def test_empty(ext):
    e = ext.empty((3, 0, 2), BF16, CPU)
    assert e.shape == (3, 0, 2) and e.dtype == BF16


@pytest.mark.parametrize("n,blocks,T", [(3, 2, 7), (0, 0, 0), (1, 0, 5), (5, 4, 0), (9, 3, 16)])
def test_map_out(ext, n, blocks, T):
    *parts, end = ext.map_out(n, blocks, T, 11, CPU)
    shapes = [(n + 1,), (T,), (T,), (T,), (n,), (n, blocks), (1,)]
    assert [tuple(p.shape) for p in parts] == shapes and all(p.is_contiguous() for p in parts)
    assert [p.dtype for p in parts] == [torch.int32] * 3 + [torch.int64] + [torch.int32] * 3
    # no part overlaps another, the last 11 entries neither; each on 16 bytes
    whole = parts[0].untyped_storage()
    assert end + 44 == whole.data_ptr() + whole.nbytes()
    spans = sorted((p.data_ptr(), p.data_ptr() + p.element_size() * p.numel()) for p in parts if p.numel())
    assert all(hi <= lo for (_, hi), (lo, _) in zip(spans, spans[1:] + [(end, 0)]))
    assert all((p.data_ptr() - whole.data_ptr()) % 16 == 0 for p in parts if p.numel())
    for i, p in enumerate(parts):
        p.fill_(i)
    assert all((p == i).all() for i, p in enumerate(parts))
    with pytest.raises(ValueError):
        ext.map_out(-1, blocks, T, 0, CPU)
    with pytest.raises(ValueError):
        ext.map_out(n, blocks, 2 ** 31, 0, CPU)


def test_map_in(ext):
    i32, i64 = torch.int32, torch.int64
    m = [torch.zeros(4, dtype=i32), torch.zeros(7, dtype=i32), torch.zeros(7, dtype=i64), torch.zeros(3, dtype=i32)]
    assert ext.map_in(*m, 7, CPU) == (*(t.data_ptr() for t in m), 3)
    for i, bad in ((1, torch.zeros(6, dtype=i32)), (2, torch.zeros(7, dtype=i32)), (3, torch.zeros(4, dtype=i32)), (0, torch.zeros(0, dtype=i32)),
                   (0, torch.zeros(2, 2, dtype=i32)), (1, torch.zeros(14, dtype=i32)[::2])):
        with pytest.raises(ValueError):
            ext.map_in(*m[:i], bad, *m[i + 1:], 7, CPU)
    with pytest.raises(ValueError, match=r"seq_of must be a contiguous torch.int32 tensor of shape \(8,\) on cpu"):
        ext.map_in(*m, 8, CPU)
    with pytest.raises(TypeError, match="init_slot must be a tensor"):
        ext.map_in(*m[:3], None, 7, CPU)


def test_where_wants_a_cuda_tensor(ext):
    with pytest.raises(ValueError, match="CUDA tensors expected"):
        ext.where(torch.zeros(3))
    with pytest.raises(TypeError):
        ext.where(3)


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
