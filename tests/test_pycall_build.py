"""The extension _pycall.so reads tensors by torch's own headers: one that was
built for another torch or Python is rebuilt, and is not used (no GPU)."""
import sysconfig

import pytest
import torch

from ssd_selective_scan_b200 import binding as libssd
from ssd_selective_scan_b200 import build as ssd_build

config_var = sysconfig.get_config_var


def other_torch(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")


def other_python(monkeypatch):
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-27-other" if name == "SOABI" else config_var(name))


@pytest.fixture
def builds(monkeypatch):
    """The builds of the extension that build() starts; none is made."""
    ssd_build.build()
    made = []
    monkeypatch.setattr(ssd_build, "_build_pycall", lambda verbose: made.append(1))
    return made


@pytest.mark.parametrize("change", [other_torch, other_python])
def test_rebuilt_for_another(change, builds, monkeypatch):
    ssd_build.build()
    assert not builds
    change(monkeypatch)
    ssd_build.build()
    assert builds


@pytest.mark.parametrize("change", [other_torch, other_python])
def test_not_used_with_another(change, monkeypatch):
    ssd_build.build()
    assert libssd.load_pycall() is libssd.load_pycall()
    change(monkeypatch)
    with pytest.raises(RuntimeError, match="built for .* build it with"):
        libssd.load_pycall()
