"""The binding's short way, without a GPU: it is built, loads beside the
library, and leaves every call that it cannot take to the Python way."""
import pytest
import torch


def test_leaves_what_it_cannot_take():
    from mla_decode_attention_05_gb300 import build
    build.build()
    import mla_decode_attention_05_gb300 as mla
    mla.lib()
    f = mla._fast
    if f is None:
        pytest.skip("fastcall.so was not built here")
    t = torch.zeros((2, 3, 512), dtype=torch.bfloat16)
    for args in ((), (None, None, None), (t, t, None), (t, t, 3), ("x", t, None)):
        assert f.value_project(*args) is None
    assert f.prefill(*[t] * 11) is None and f.kv_expand(*[t] * 9) is None and f.kv_insert_rope(*[t] * 14) is None
    assert f.prefill() is None and f.kv_expand(*[None] * 9) is None and f.kv_insert_rope(*[None] * 14) is None
    with pytest.raises(TypeError):
        f.bind()
    with pytest.raises(ValueError):
        f.bind(0, 0, 0, 0, 0)


def _reload(monkeypatch):
    """The short way as a process finds it that loads the library now."""
    import mla_decode_attention_05_gb300 as mla
    monkeypatch.setattr(mla, "_fast", None)
    mla._load_fast(mla.lib())
    return mla._fast


def test_one_built_for_something_else_is_not_loaded(monkeypatch, tmp_path):
    """Another PyTorch, another interpreter, another header of the library."""
    import shutil
    import sysconfig

    from mla_decode_attention_05_gb300 import build
    build.build()
    import mla_decode_attention_05_gb300 as mla
    mla.lib()
    if mla._fast is None:
        pytest.skip("fastcall.so was not built here")
    assert _reload(monkeypatch) is not None
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0")
        assert _reload(m) is None
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-1-other.so")
        assert _reload(m) is None
    shutil.copytree(build.INCLUDE, tmp_path / "include")
    with open(tmp_path / "include" / "mla_decode.h", "a") as f:
        f.write("/* another argument somewhere */\n")
    with monkeypatch.context() as m:
        m.setattr(build, "INCLUDE", str(tmp_path / "include"))
        assert _reload(m) is None
    with monkeypatch.context() as m:
        m.setattr(build, "INCLUDE", str(tmp_path / "nowhere"))
        assert _reload(m) is None
    assert _reload(monkeypatch) is not None


@pytest.mark.parametrize("compiler", ["false", "/nowhere/to/be/found"])
def test_a_build_that_fails_leaves_none(monkeypatch, tmp_path, compiler):
    """What an earlier build left is gone where its sources have changed and
    the compiler fails or is missing."""
    from mla_decode_attention_05_gb300 import build
    (tmp_path / "fastcall.so").write_bytes(b"of an earlier build")
    (tmp_path / "fastcall-0123456789abcdef.so").write_bytes(b"of another PyTorch")
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path))
    monkeypatch.setenv("CXX", compiler)
    build._finish_fast(build._start_fast(False))
    assert list(tmp_path.iterdir()) == []


def test_two_builds_at_once(monkeypatch, tmp_path):
    """A file of an earlier build that another build removes first."""
    import os

    from mla_decode_attention_05_gb300 import build
    old = tmp_path / "fastcall.so"
    old.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path))
    monkeypatch.setenv("CXX", "false")
    remove = os.remove

    def late(path):
        remove(path)
        remove(path)
    monkeypatch.setattr(build.os, "remove", late)
    build._finish_fast(build._start_fast(False))
    assert not old.exists()
