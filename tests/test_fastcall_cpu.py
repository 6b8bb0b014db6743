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
