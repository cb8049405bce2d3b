"""The native module is rebuilt for another torch or Python, and not loaded if it was
built for one."""
import pytest

from attention_learnable_head_gb300 import binding
from attention_learnable_head_gb300 import build as B


def test_a_module_of_another_torch_is_rebuilt(monkeypatch, tmp_path):
    B.build()
    started = []

    class Stop(Exception):
        pass

    def start(cmd, verbose):
        started.append(cmd)
        raise Stop

    monkeypatch.setattr(B, "_start", start)
    B.build()                              # up to date: nothing is compiled
    assert not started
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(B, "FAST_STAMP", str(stamp))
    for text in (None, "torch 1.0, cpython-30"):
        if text is not None:
            stamp.write_text(text)
        with pytest.raises(Stop):
            B.build()
        assert started.pop()[-1] == "-lc10_cuda" and not started


def test_a_module_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    B.build()
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(B, "FAST_STAMP", str(stamp))
    monkeypatch.setattr(binding, "_FAST", None)
    stamp.write_text("torch 1.0, cpython-30")
    with pytest.raises(RuntimeError, match="not built for torch"):
        binding._fast()
    stamp.write_text(B.fast_target())
    assert hasattr(binding._fast(), "page_plan")
