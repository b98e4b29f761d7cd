"""The compiled Python module is bound to the PyTorch it was compiled against."""
import os

import diffusion_transformer_mlp_gb300 as fc2
from diffusion_transformer_mlp_gb300 import build


def test_module_of_another_pytorch_is_made_again(monkeypatch):
    build.build()
    assert build.binding_is_current()
    before = os.stat(build.BINDING).st_mtime_ns
    build.build()
    assert os.stat(build.BINDING).st_mtime_ns == before
    monkeypatch.setattr(build, "_torch_stamp", lambda: "another version")
    assert not build.binding_is_current()
    made = []
    monkeypatch.setattr(build, "_binding_job", lambda: made.append(1) or ["cp", build.BINDING, f"{build.BINDING}.tmp{os.getpid()}"])
    build.build()
    assert made and build.binding_is_current()
    monkeypatch.undo()
    assert not build.binding_is_current()
    build.build()
    assert build.binding_is_current() and fc2.mxfp4_padded_cols(5) == 128


def test_module_without_its_record_is_not_current(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_mxfp4.so"))
    assert not build.binding_is_current()
    (tmp_path / "_mxfp4.so").write_bytes(b"")
    assert not build.binding_is_current()
    (tmp_path / "_mxfp4.so.torch").write_text(build._torch_stamp())
    assert build.binding_is_current()
