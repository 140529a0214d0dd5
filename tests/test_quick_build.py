"""The quick form of the binding is built with the library, and one that is
missing, old or another torch's does not go unnoticed (no GPU needed)."""
import os
import types

import pytest
import torch

import kalman_filter_linear_b200 as package
from kalman_filter_linear_b200 import build, kdn


@pytest.fixture(scope='module', autouse=True)
def built():
    if build.is_stale():
        build.build()


def test_a_missing_or_old_module_is_stale(monkeypatch, tmp_path):
    assert not build.is_stale()
    quick = tmp_path / '_kdn_quick.so'
    monkeypatch.setattr(build, 'QUICK', str(quick))
    assert build.is_stale()
    quick.write_bytes(b'')
    assert not build.is_stale()
    os.utime(quick, (0, 0))
    assert build.is_stale()
    # where it cannot be built, the library alone counts
    monkeypatch.setattr(build.importlib.util, 'find_spec', lambda name: None)
    assert not build.is_stale()


def test_the_module_knows_its_torch():
    assert kdn._load_quick().torch_version == torch.__version__.partition('+')[0]


@pytest.mark.parametrize("module", [types.SimpleNamespace(torch_version='1.0'),
                                    types.SimpleNamespace()])   # (one from before it knew)
def test_a_module_of_another_torch_is_not_used(monkeypatch, module):
    monkeypatch.setattr(kdn, '_quick', None)
    monkeypatch.setattr(package, '_kdn_quick', module, raising=False)
    with pytest.warns(RuntimeWarning, match='built against torch'):
        assert kdn._load_quick() is kdn._NoQuick
    with pytest.raises(TypeError, match='CUDA tensor'):
        kdn.kdn_linear_scan_step(torch.zeros(2, 4), torch.zeros(2, 4), torch.zeros(2, 4))
