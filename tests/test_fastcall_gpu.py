"""The binding's short way (fastcall.so): the same results, refusals and given
buffers as the Python way, and the order of calls that follow one another
without a wait."""
import numpy as np
import pytest
import torch

from _ops import bf16, cu
from oracle import prefill as O

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


@pytest.fixture
def both(monkeypatch):
    """Runs f the short way and the Python way."""
    import mla_decode_attention_05_gb300 as mla
    mla.lib()
    assert mla._fast is not None, "fastcall.so was not built"
    fast = mla._fast

    def run(f):
        monkeypatch.setattr(mla, "_fast", fast)
        a = f()
        monkeypatch.setattr(mla, "_fast", None)
        b = f()
        monkeypatch.setattr(mla, "_fast", fast)
        return a, b
    return run


def _inputs(seed=1, n=70, H=3):
    rng = np.random.default_rng(seed)
    w_kv = bf16(rng, (H, 256, 512), 512 ** -0.5).cuda()
    return dict(qkv=bf16(rng, (n, 2112)).cuda(), q=bf16(rng, (n, H, 192)).cuda(), w=bf16(rng, (512,)).cuda(), w_kv=w_kv,
                slots=torch.randperm(192, generator=torch.Generator().manual_seed(seed))[:n].cuda(),
                pos=torch.arange(n, device="cuda") * 3, cs=torch.from_numpy(O.angle_table(3 * n)).cuda(),
                bt=torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda"), cu=cu([50, 20]), n=n, H=H)


def _taken(f):
    """Does the short way take this call?"""
    import mla_decode_attention_05_gb300 as mla
    seen = []

    class Spy:
        def __getattr__(self, name):
            real = getattr(fast, name)

            def call(*a):
                r = real(*a)
                seen.append(r is not None)
                return r
            return call
    fast, mla._fast = mla._fast, Spy()
    try:
        f()
    finally:
        mla._fast = fast
    return seen == [True]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_tensor"])
def test_same_results(both, fmt):
    import mla_decode_attention_05_gb300 as mla
    s = _inputs()
    n, H = s["n"], s["H"]
    width = {"bf16": 576, "fp8": 640, "fp8_tensor": 576}[fmt]
    kw = dict(kv_scales=torch.zeros((3, 64, 4), device="cuda") if fmt == "fp8" else None)

    def insert(q_out=True, in_place=False):
        cache = torch.zeros((3, 64, width), dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device="cuda")
        q = s["q"].clone()
        out = torch.zeros((n, H, 64), dtype=torch.bfloat16, device="cuda") if not in_place else None
        r = mla.kv_insert_rope(s["qkv"][:, 1536:2048], s["qkv"][:, 2048:], s["w"], s["slots"], cache, eps=1e-6,
                               positions=s["pos"], cos_sin=s["cs"], q_pe=q[..., 128:], q_out=out,
                               k_scale_inv=torch.full((1,), 0.5, device="cuda") if fmt == "fp8_tensor" else None,
                               fp8_per_tensor=fmt == "fp8_tensor", **kw)
        assert r[0] is cache and (r[1] is out if out is not None else r[1].data_ptr() == q[..., 128:].data_ptr())
        return cache, r[1].clone(), q
    for in_place in (False, True):
        a, b = both(lambda: insert(in_place=in_place))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert _taken(lambda: insert(in_place=in_place))
    cache = a[0]
    sc = kw["kv_scales"] if fmt == "fp8" else torch.full((1,), 2.0, device="cuda") if fmt == "fp8_tensor" else None
    w_uk, w_uv = s["w_kv"][:, :128], s["w_kv"][:, 128:]
    f = lambda **k: mla.kv_expand(cache, s["bt"], s["cu"], w_uk, w_uv, kv_scales=sc, **k)
    a, b = both(lambda: f(total=n))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and _taken(lambda: f(total=n))
    kv = torch.empty_like(a[0])
    a2, b2 = both(lambda: f(kv=kv))
    assert a2[0].data_ptr() == kv.data_ptr() and torch.equal(a2[0], a[0])
    args = (s["q"], kv[..., :128], a[1], kv[..., 128:], s["cu"], s["cu"])
    for causal in (True, False):
        f = lambda **k: mla.prefill(*args, softmax_scale=SCALE, causal=causal, **k)
        a, b = both(f)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and _taken(f)
    out, lse = torch.empty_like(a[0]), torch.empty_like(a[1])
    a2, _ = both(lambda: f(out=out, lse=lse, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")))
    assert a2[0].data_ptr() == out.data_ptr() and torch.equal(out, a[0]) and torch.equal(lse, a[1])
    f = lambda **k: mla.value_project(s["qkv"][:, :1536].unflatten(1, (3, 512)), w_uv, **k)
    a, b = both(f)
    assert torch.equal(a, b) and _taken(f)
    assert both(lambda: f(out=a))[0].data_ptr() == a.data_ptr()


def test_a_split_prefill_has_its_workspace(both):
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(4)
    q, kv, pe = bf16(rng, (20, 2, 192)).cuda(), bf16(rng, (3000, 2, 256)).cuda(), bf16(rng, (3000, 64)).cuda()
    f = lambda: mla.prefill(q, kv[..., :128], pe, kv[..., 128:], cu([20]), cu([3000]), softmax_scale=SCALE)
    a, b = both(f)
    assert mla.prefill_workspace_bytes(1, 2, 20, 3000) > 0 and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for way in (mla._fast, None):
        keep, mla._fast = mla._fast, way
        try:
            with pytest.raises(mla.MlaError, match="workspace"):
                mla.prefill(q, kv[..., :128], pe, kv[..., 128:], cu([20]), cu([3000]), softmax_scale=SCALE, workspace=small)
        finally:
            mla._fast = keep


def test_refusals_are_pythons():
    """Calls that the short way does not take reach the Python checks."""
    import mla_decode_attention_05_gb300 as mla
    s = _inputs(2)
    w_uk, w_uv = s["w_kv"][:, :128], s["w_kv"][:, 128:]
    attn = s["qkv"][:, :1536].unflatten(1, (3, 512))
    with pytest.raises(TypeError, match="attn must be torch.bfloat16"):
        mla.value_project(attn.float(), w_uv)
    with pytest.raises(ValueError, match="attn must be"):
        mla.value_project(attn[..., :256], w_uv)
    with pytest.raises(ValueError, match="out must be"):
        mla.value_project(attn, w_uv, out=torch.empty((2, 3, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        mla.value_project(attn, w_uv.cpu())
    kv = torch.zeros((70, 3, 256), dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros((70, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError, match="cu_seqlens_q"):
        mla.prefill(s["q"], kv[..., :128], pe, kv[..., 128:], s["cu"].long(), s["cu"], softmax_scale=SCALE)
    with pytest.raises(mla.MlaError, match="softmax_scale"):
        mla.prefill(s["q"], kv[..., :128], pe, kv[..., 128:], s["cu"], s["cu"], softmax_scale=-1.0)
    assert mla.prefill(s["q"], kv[..., :128], pe, kv[..., 128:], s["cu"], s["cu"], softmax_scale=1)[0].shape == (70, 3, 128)
    with pytest.raises(ValueError, match="cu_seqlens"):
        mla.kv_expand(torch.zeros((3, 64, 576), dtype=torch.bfloat16, device="cuda"), s["bt"], s["cu"][:2], w_uk, w_uv, total=70)
    cache = torch.zeros((3, 64, 576), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="slots"):
        mla.kv_insert_rope(s["qkv"][:, 1536:2048], s["qkv"][:, 2048:], s["w"], s["slots"][:5], cache, eps=1e-6,
                           positions=s["pos"], cos_sin=s["cs"])
    with pytest.raises(ValueError, match="overlap"):
        mla.kv_insert_rope(s["qkv"][:, 1536:2048], s["qkv"][:, 2048:], s["w"], s["slots"], cache, eps=1e-6,
                           positions=s["pos"], cos_sin=s["cs"], q_pe=s["q"][..., 128:],
                           q_out=torch.zeros((70, 3, 64), dtype=torch.bfloat16, device="cuda")[:1].expand(70, 3, 64))


def test_calls_that_follow_one_another():
    """Each kernel sets itself up while the one in front of it ends, and reads
    and writes only then: inputs overwritten right after a call, one output
    buffer for all, results read by the next operator."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(6)
    H, n = 8, 300
    w = bf16(rng, (H, 256, 512), 512 ** -0.5).cuda()
    xs = [bf16(rng, (n, H, 512)).cuda() for _ in range(6)]
    want = [mla.value_project(x, w[:, 128:]).clone() for x in xs]
    torch.cuda.synchronize()
    x, out, got = torch.empty_like(xs[0]), torch.empty_like(want[0]), []
    for _ in range(5):
        got.clear()
        for a in xs:
            x.copy_(a)
            mla.value_project(x, w[:, 128:], out=out)
            got.append(out.clone())
        assert all(torch.equal(g, v) for g, v in zip(got, want))
    # insert -> expand -> prefill -> the next prompt into the same cache and buffers
    lens = [130, 170]
    bt = torch.tensor([[3, 1, 0], [4, 2, 5]], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(m) for m in lens]).cuda()
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(lens)]).cuda()
    slots = bt[seq, pos // 64].long() * 64 + pos % 64
    cs, one = torch.from_numpy(O.angle_table(200)).cuda(), torch.ones(512, dtype=torch.bfloat16, device="cuda")
    prompts = [(bf16(rng, (n, 2112)).cuda(), bf16(rng, (n, H, 192), 1.5).cuda()) for _ in range(4)]
    cache = torch.zeros((6, 64, 576), dtype=torch.bfloat16, device="cuda")
    kv, pe = torch.empty((n, H, 256), dtype=torch.bfloat16, device="cuda"), torch.empty((n, 64), dtype=torch.bfloat16, device="cuda")
    o, l = torch.empty((n, H, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((H, n), device="cuda")
    rot = torch.empty((n, H, 192), dtype=torch.bfloat16, device="cuda")

    def one_prompt(qkv, q, wait):
        step = torch.cuda.synchronize if wait else (lambda: None)
        rot.copy_(q), step()
        mla.kv_insert_rope(qkv[:, 1536:2048], qkv[:, 2048:], one, slots, cache, eps=1e-6, positions=pos, cos_sin=cs,
                           q_pe=rot[..., 128:]), step()
        mla.kv_expand(cache, bt, cu(lens), w[:, :128], w[:, 128:], kv=kv, k_pe=pe), step()
        mla.prefill(rot, kv[..., :128], pe, kv[..., 128:], cu(lens), cu(lens), softmax_scale=SCALE, out=o, lse=l), step()
        return o.clone(), l.clone()
    want = [one_prompt(*p, True) for p in prompts]
    for _ in range(5):
        got = [one_prompt(*p, False) for p in prompts]
        assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v))


def test_other_threads_run_meanwhile(tmp_path):
    """The interpreter is free while a call allocates and launches: seen by a
    function in the library's place."""
    import ctypes
    import shutil
    import subprocess
    import sysconfig

    import mla_decode_attention_05_gb300 as mla
    L = mla.lib()
    cc = shutil.which("cc") or shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src, so = tmp_path / "held.c", tmp_path / "held.so"
    src.write_text("#include <Python.h>\nint calls, held;\n"
                   "int call(void) { calls++; held += PyGILState_Check(); return 0; }\n"
                   "size_t room(void) { call(); return 0; }\n")
    subprocess.check_call([cc, "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], str(src), "-o", str(so)])
    stub = ctypes.CDLL(str(so))
    at = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    s = _inputs(3)
    cache = torch.zeros((3, 64, 576), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((70, 3, 256), dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros((70, 64), dtype=torch.bfloat16, device="cuda")
    mla._fast.bind(at(stub.call), at(stub.call), at(stub.call), at(stub.room), at(stub.call))
    try:
        assert _taken(lambda: mla.kv_insert_rope(s["qkv"][:, 1536:2048], s["qkv"][:, 2048:], s["w"], s["slots"], cache,
                                                 eps=1e-6, positions=s["pos"], cos_sin=s["cs"]))
        assert _taken(lambda: mla.kv_expand(cache, s["bt"], s["cu"], s["w_kv"][:, :128], s["w_kv"][:, 128:], total=70))
        assert _taken(lambda: mla.prefill(s["q"], kv[..., :128], pe, kv[..., 128:], s["cu"], s["cu"], softmax_scale=SCALE))
        assert _taken(lambda: mla.value_project(s["qkv"][:, :1536].unflatten(1, (3, 512)), s["w_kv"][:, 128:]))
    finally:
        mla._fast.bind(*(at(f) for f in (L.mla_kv_insert_rope, L.mla_kv_expand, L.mla_prefill,
                                         L.mla_prefill_workspace_bytes, L.mla_value_project)))
    assert ctypes.c_int.in_dll(stub, "calls").value == 5 and ctypes.c_int.in_dll(stub, "held").value == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_tensor"])
@pytest.mark.parametrize("n,H", [(1, 5), (1, 1), (2, 1), (2, 5)])
def test_few_tokens_in_place(both, n, H, fmt):
    """A decode step's queries, rotated in place as views of their absorbed rows:
    taken for a single token and a single head too, with the Python way's bits."""
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(7)
    qkv, q0, w = bf16(rng, (n, 2112)).cuda(), bf16(rng, (n, H, 576)).cuda(), bf16(rng, (512,)).cuda()
    slots, pos = torch.arange(n, device="cuda") + 70, torch.arange(n, device="cuda") + 3
    cs = torch.from_numpy(O.angle_table(8)).cuda()

    def insert():
        width = 640 if fmt == "fp8" else 576
        cache = torch.zeros((2, 64, width), dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device="cuda")
        sc = torch.zeros((2, 64, 4), device="cuda") if fmt == "fp8" else None
        q = q0.clone()
        r = mla.kv_insert_rope(qkv[:, 1536:2048], qkv[:, 2048:], w, slots, cache, eps=1e-6, positions=pos, cos_sin=cs,
                               q_pe=q[..., 512:], kv_scales=sc, fp8_per_tensor=fmt == "fp8_tensor",
                               k_scale_inv=torch.full((1,), 0.5, device="cuda") if fmt == "fp8_tensor" else None)
        assert r[1].data_ptr() == q[..., 512:].data_ptr()
        return (cache, q) if sc is None else (cache, q, sc)
    a, b = both(insert)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and not torch.equal(a[1], q0)
    assert torch.equal(a[1][..., :512], q0[..., :512])
    assert _taken(insert)


def test_rows_that_overlap_are_left_to_the_python_way():
    import mla_decode_attention_05_gb300 as mla
    rng = np.random.default_rng(8)
    qkv, w = bf16(rng, (2, 2112)).cuda(), bf16(rng, (512,)).cuda()
    cache = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    z = torch.arange(2, device="cuda")
    cs = torch.from_numpy(O.angle_table(8)).cuda()
    flat = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    for n, H, strides in ((2, 3, (64, 64)), (2, 3, (128, 64)), (2, 3, (512, 32)), (1, 3, (0, 32)), (2, 1, (32, 0)), (2, 3, (64, 0))):
        out = flat.as_strided((n, H, 64), strides + (1,))
        with pytest.raises(ValueError, match="overlap"):
            mla.kv_insert_rope(qkv[:n, 1536:2048], qkv[:n, 2048:], w, z[:n], cache, eps=1e-6, positions=z[:n], cos_sin=cs,
                               q_pe=bf16(rng, (n, H, 64)).cuda(), q_out=out)
