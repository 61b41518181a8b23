"""The C marshalling of the block calls is optional: one that was built for another interpreter is not found, and one that
does not load leaves the calls to ctypes (no GPU)."""
import os
import sysconfig

import pytest
import torch

from test_block_refusals import m  # noqa: F401


def test_name_carries_the_interpreter(m):  # noqa: F811
    from nvfp4_w4a4_mixture_gb300 import build

    assert build.CALLS == m.CALLS_PATH
    assert os.path.basename(m.CALLS_PATH) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")


def test_broken_file_leaves_the_calls_to_ctypes(m, monkeypatch, tmp_path):  # noqa: F811
    broken = tmp_path / os.path.basename(m.CALLS_PATH)
    broken.write_bytes(b"no shared object")
    monkeypatch.setattr(m, "CALLS_PATH", str(broken))
    monkeypatch.setattr(m, "_calls", m._calls)
    m._load_calls(m.lib())
    assert m._calls is None
    with pytest.raises(TypeError, match="CUDA"):
        m.moe_select_experts(torch.zeros(4, 8), 2)
