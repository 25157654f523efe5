"""libflce_torch.so is built for one PyTorch: another one is noticed, by the build and by the load."""
import json

import pytest
import torch

from linear_cross_entropy_vocab_gb300 import native_build, norm


@pytest.fixture
def stamp(tmp_path, monkeypatch):
    native_build.build()
    path = tmp_path / "stamp.json"
    path.write_text(open(native_build.TORCH_STAMP).read())
    monkeypatch.setattr(native_build, "TORCH_STAMP", str(path))
    monkeypatch.setattr(norm, "_ops", None)
    return path


def test_the_installed_one_is_current(stamp):
    assert native_build.torch_mismatch() is None and native_build.up_to_date()
    assert json.loads(stamp.read_text())["version"] == str(torch.__version__)


@pytest.mark.parametrize("key,value", [("version", "2.0.0"), ("git", "0" * 40),
                                       ("cxx11_abi", None)])
def test_another_one_is_stale(stamp, key, value):
    stamp.write_text(json.dumps({**json.loads(stamp.read_text()), key: value}))
    assert not native_build.up_to_date()
    with pytest.raises(RuntimeError, match=f"another PyTorch.*{key}"):
        norm._operators()


@pytest.mark.parametrize("text", ["", "[]", "{}"])
def test_a_missing_or_broken_stamp_is_stale(stamp, text):
    stamp.write_text(text)
    assert not native_build.up_to_date()
    stamp.unlink()
    assert not native_build.up_to_date()
    with pytest.raises(RuntimeError, match="another PyTorch"):
        norm._operators()
