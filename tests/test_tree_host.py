"""Refusals of the tree step's calls (pkv_slot_map, pkv_rope_append_axes,
pkv_decode_attn_tree, pkv_tree_commit): every argument is checked on the host
before any kernel is launched.  Runs without a GPU: the checks read only the
context's configuration, so a context made of it alone stands in for one, and
a call whose arguments pass ends at the missing device (PKV_ERR_CUDA)."""
import ctypes as C

import numpy as np
import pytest
import torch

from tests import _tree

BASE = 0x10000000


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_flight_b200 import build
    build.build()
    from paged_kv_flight_b200 import pkv as mod
    return mod


@pytest.fixture(autouse=True)
def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("made-up pointers: only where nothing can be launched")


def _ctx(pkv, fp8=False, d=128):
    """A context as far as the checks read it: its configuration, zeros behind."""
    blob = C.create_string_buffer(1 << 16)
    cfg = pkv.make_config(32, 8, d, 16, "fp8" if fp8 else "bf16", 1e4, 8, 64, 1000)
    C.memmove(blob, C.byref(cfg), C.sizeof(cfg))
    return blob


def _at(i, off=0):
    """Pointers far from one another, 16-byte aligned, never followed."""
    return BASE + (i << 28) + off


def _call(pkv, fn, good, order, **kw):
    a = dict(good, **kw)
    assert set(kw) <= set(good)
    return getattr(pkv.lib, fn)(*(a[k] for k in order))


SLOTS = ("ctx seq_lens new_lens parents batch block_tables stride held pages_out free cap count left n words cu slots "
         "positions mask stream").split()
ROPE = "ctx q k v n positions axes sections interleaved slots q_out k_pool v_pool k_scale v_scale stream".split()
TREE = "ctx q k_pool v_pool k_scale v_scale table stride lens cu mask words batch n out stream".split()
COMMIT = "ctx k_pool v_pool k_scale v_scale table stride lens path depth path_lens batch lens_out stream".split()


def _good(order, **numbers):
    g = {k: _at(i) for i, k in enumerate(order)}
    g.update(stream=None, **numbers)
    return g


def test_slot_map_refusals(pkv):
    good = _good(SLOTS, ctx=_ctx(pkv), batch=4, stride=64, cap=100, n=40, words=2)
    call = lambda **kw: _call(pkv, "pkv_slot_map", good, SLOTS, **kw)   # noqa: E731
    assert call() == pkv.PKV_ERR_CUDA                      # all checks passed
    assert call(batch=0, seq_lens=None) == pkv.PKV_OK
    bad = [dict(ctx=None), dict(batch=-1), dict(batch=9), dict(stride=0), dict(stride=65), dict(n=-1), dict(cap=-1),
           dict(words=0), dict(mask=None), dict(parents=None), dict(cu=_at(15, 2)), dict(mask=_at(18, 1))]
    bad += [{k: None} for k in "seq_lens new_lens block_tables held pages_out free count left cu slots positions".split()]
    # outputs over inputs and over one another; in place only where it is named
    bad += [dict(cu=good["seq_lens"]), dict(slots=good["parents"] + 4 * 39), dict(pages_out=good["held"] + 4),
            dict(left=good["held"]), dict(block_tables=good["free"]), dict(positions=good["slots"]),
            dict(mask=good["slots"]), dict(pages_out=good["count"]), dict(left=good["cu"] + 16)]
    for kw in bad:
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    assert call(pages_out=good["held"], left=good["count"]) == pkv.PKV_ERR_CUDA
    assert call(parents=None, mask=None, words=0) == pkv.PKV_ERR_CUDA       # a chain
    assert call(n=0, slots=None, positions=None) == pkv.PKV_ERR_CUDA
    assert call(n=1 << 29) == pkv.PKV_ERR_UNSUPPORTED
    assert call(cap=0, free=None) == pkv.PKV_ERR_CUDA


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_append_axes_refusals(pkv, fp8):
    sec = lambda *v: (C.c_int * len(v))(*v)   # noqa: E731
    good = _good(ROPE, ctx=_ctx(pkv, fp8), n=10, axes=3, sections=sec(16, 24, 24), interleaved=0)
    call = lambda **kw: _call(pkv, "pkv_rope_append_axes", good, ROPE, **kw)   # noqa: E731
    assert call() == pkv.PKV_ERR_CUDA
    assert call(q_out=good["q"]) == pkv.PKV_ERR_CUDA
    assert call(n=0, q=None) == pkv.PKV_OK
    bad = [dict(ctx=None), dict(n=-1), dict(axes=0), dict(axes=5), dict(sections=None),
           dict(sections=sec(16, 24, 23)), dict(sections=sec(90, -13, -13)), dict(sections=sec(64, 64, -64)),
           dict(sections=sec(10, 10, 44), interleaved=1), dict(axes=4, sections=sec(30, 20, 14, 0), interleaved=1),
           dict(q=_at(1, 8)), dict(k_pool=_at(11, 4)),
           dict(positions=_at(5, 2)), dict(q_out=good["q"] + 256), dict(q_out=good["k"]), dict(q_out=good["v"])]
    bad += [{k: None} for k in "q k v positions slots q_out k_pool v_pool".split()]
    bad += [dict(k_scale=None), dict(v_scale=None), dict(v_scale=_at(14, 4))] if fp8 else []
    for kw in bad:
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    assert call(sections=sec(24, 20, 20), interleaved=1) == pkv.PKV_ERR_CUDA
    assert call(axes=1, sections=sec(64)) == pkv.PKV_ERR_CUDA
    if not fp8:
        assert call(k_scale=None, v_scale=None) == pkv.PKV_ERR_CUDA


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_attn_tree_refusals(pkv, fp8):
    good = _good(TREE, ctx=_ctx(pkv, fp8), stride=64, words=2, batch=4, n=40)
    call = lambda **kw: _call(pkv, "pkv_decode_attn_tree", good, TREE, **kw)   # noqa: E731
    assert call() == pkv.PKV_ERR_CUDA
    assert call(batch=0, q=None) == pkv.PKV_OK and call(n=0, q=None) == pkv.PKV_OK
    assert call(n=1 << 29) == pkv.PKV_ERR_UNSUPPORTED
    bad = [dict(ctx=None), dict(batch=-1), dict(batch=9), dict(stride=0), dict(stride=65), dict(n=-1), dict(words=0),
           dict(q=_at(1, 8)), dict(out=_at(14, 8)), dict(cu=_at(9, 4)), dict(mask=_at(10, 2)), dict(out=good["q"]),
           dict(out=good["q"] + 16)]
    bad += [{k: None} for k in "q k_pool v_pool table lens cu mask out".split()]
    bad += [dict(k_scale=None), dict(v_scale=None)] if fp8 else []
    for kw in bad:
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_commit_refusals(pkv, fp8):
    good = _good(COMMIT, ctx=_ctx(pkv, fp8), stride=64, depth=5, batch=4)
    call = lambda **kw: _call(pkv, "pkv_tree_commit", good, COMMIT, **kw)   # noqa: E731
    assert call() == pkv.PKV_ERR_CUDA
    assert call(lens_out=good["lens"]) == pkv.PKV_ERR_CUDA
    assert call(depth=0, path=None) == pkv.PKV_ERR_CUDA
    assert call(batch=0, path=None) == pkv.PKV_OK
    bad = [dict(ctx=None), dict(batch=-1), dict(batch=9), dict(stride=0), dict(depth=-1), dict(lens_out=_at(12, 2)),
           dict(path=_at(8, 2)), dict(lens_out=good["lens"] + 4), dict(lens_out=good["path"] + 76),
           dict(lens_out=good["path_lens"]), dict(lens_out=good["table"])]
    bad += [{k: None} for k in "k_pool v_pool table lens path path_lens lens_out".split()]
    bad += [dict(k_scale=None), dict(v_scale=None)] if fp8 else []
    for kw in bad:
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw


def test_binding_checks_shapes(pkv):
    """The Python binding holds the tensors' shapes against one another (host
    tensors that report themselves as device tensors)."""
    class _OnDevice(torch.Tensor):
        @property
        def is_cuda(self):
            return True

    i = lambda *s: torch.zeros(*s, dtype=torch.int32).as_subclass(_OnDevice)   # noqa: E731
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16).as_subclass(_OnDevice)   # noqa: E731
    ctx = _ctx(pkv)
    with pytest.raises(ValueError, match="cu_q"):
        pkv.pkv_slot_map(ctx, i(4), i(4), i(4, 8), i(4), i(20), i(1), i(4), i(9), i(9), i(4), i(1))
    with pytest.raises(ValueError, match="tree_mask"):
        pkv.pkv_slot_map(ctx, i(4), i(4), i(4, 8), i(4), i(20), i(1), i(5), i(9), i(9), i(4), i(1), i(9), i(8, 1))
    with pytest.raises(ValueError, match="positions"):
        pkv.pkv_rope_append_axes(ctx, h(9, 32, 128), h(9, 8, 128), h(9, 8, 128), i(2, 9), [16, 24, 24], i(9),
                                 h(9, 32, 128), 0, 0, None, None)
    with pytest.raises(ValueError, match="tree_mask"):
        pkv.pkv_decode_attn_tree(ctx, h(9, 32, 128), 0, 0, None, None, i(2, 4), i(2), i(3), i(8, 1), h(9, 32, 128))
    with pytest.raises(ValueError, match="path_lens"):
        pkv.pkv_tree_commit(ctx, 0, 0, None, None, i(2, 4), i(2), i(2, 3), i(3), i(2))
    with pytest.raises(ValueError, match="k_new"):
        pkv.pkv_rope_append_axes(ctx, h(9, 32, 128), h(8, 8, 128), h(8, 8, 128), i(3, 9), [16, 24, 24], i(9),
                                 h(9, 32, 128), 0, 0, None, None)
    with pytest.raises(ValueError, match="device tensors"):
        pkv.pkv_tree_commit(ctx, 0, 0, None, None, i(2, 4), torch.zeros(2, dtype=torch.int32), i(2, 3), i(2), i(2))
    class _Elsewhere(_OnDevice):
        def get_device(self):
            return 3

    keep, pkv._cur_device = pkv._cur_device, lambda: 0
    try:
        with pytest.raises(ValueError, match="current device"):
            pkv.pkv_tree_commit(ctx, 0, 0, None, None, torch.zeros(2, 4, dtype=torch.int32).as_subclass(_Elsewhere), i(2),
                                i(2, 3), i(2), i(2))
    finally:
        pkv._cur_device = keep
    with pytest.raises(TypeError, match="path_lens"):
        pkv.pkv_tree_commit(ctx, 0, 0, None, None, i(2, 4), i(2), i(2, 3), i(2).long(), i(2))


def test_plain_forms_agree():
    """The plain forms of the tests against independent facts: ancestor sets
    by walking, a rotation's length, and a softmax over one key."""
    rng = np.random.default_rng(3)
    par = _tree.parents_of(rng, 40)
    seen = _tree.ancestors(par)
    for i in range(40):
        walk, x = set(), i
        while x != -1:
            walk.add(x)
            x = par[x]
        assert walk == set(np.flatnonzero(seen[i]))
    x = rng.standard_normal((5, 2, 64))
    y = _tree.rotate(x, rng.integers(0, 9000, (3, 5)), [12, 10, 10], True, 1e4)
    assert np.allclose((x ** 2).sum(-1), (y ** 2).sum(-1))
    k = rng.standard_normal((1, 1, 16, 64))
    o, _ = _tree.attention(x[:1], k, k, [0], [0, 1], np.zeros((1, 1), np.int32), np.ones((1, 1), np.int32), 16, 2)
    assert np.allclose(o[0, 1], k[0, 0, 0])


def test_marshal_module(pkv):
    """The binding's extension module: what it takes for a device tensor, and
    that a call's arguments arrive in order, None as NULL, whatever their sign."""
    m = pytest.importorskip("paged_kv_flight_b200._marshal")
    x = torch.zeros(3, dtype=torch.int32)
    assert m.pointer(x, 0, 3) is None and m.pointer(7, 0) is None and m.pointer(None, 2) is None     # not on a device
    with pytest.raises(TypeError):
        m.pointer(x)
    got = []
    kind = C.CFUNCTYPE(C.c_int, *[C.c_int64] * 20)
    back = kind(lambda *a: got.append(a) or 5)
    address = C.cast(back, C.c_void_p).value
    args = [1, None, -1, 2 ** 63, 2 ** 40 + 3] + list(range(5, 20))
    assert m.call(address, *args) == 5
    assert got[0] == tuple([1, 0, -1, -2 ** 63, 2 ** 40 + 3] + list(range(5, 20)))
    for bad in ((address, "x"), (address, 1.5), (), (address, *range(21))):
        with pytest.raises(TypeError):
            m.call(*bad)
    assert len(got) == 1


def test_binding_without_the_marshal_module():
    """The same refusals and calls where the extension module is not built."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import sys
sys.modules['paged_kv_flight_b200._marshal'] = None
import torch
from paged_kv_flight_b200 import pkv
from tests.test_tree_host import _ctx
class T(torch.Tensor):
    is_cuda = True
i = lambda *s: torch.zeros(*s, dtype=torch.int32).as_subclass(T)
h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16).as_subclass(T)
ctx = _ctx(pkv)
def status(f, *a, **k):
    try:
        return f(*a, check=False, stream=0, **k)
    except Exception as e:
        return type(e).__name__
want = pkv.PKV_ERR_CUDA, 'ValueError'
got = (status(pkv.pkv_slot_map, ctx, i(2), i(2), i(2, 4), i(2), i(9), i(1), i(3), i(5), i(5), i(2), i(1)),
       status(pkv.pkv_slot_map, ctx, i(2), i(3), i(2, 4), i(2), i(9), i(1), i(3), i(5), i(5), i(2), i(1)))
assert got == want, got
pool = 1 << 33
got = (status(pkv.pkv_rope_append_axes, ctx, h(2, 32, 128), h(2, 8, 128), h(2, 8, 128), i(1, 2), [64], i(2), h(2, 32, 128), pool, pool << 1, None, None),
       status(pkv.pkv_rope_append_axes, ctx, h(2, 32, 128), h(2, 8, 128), h(2, 8, 128), i(2, 2), [64], i(2), h(2, 32, 128), pool, pool << 1, None, None))
assert got == want, got
"""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


def test_binding_wants_every_tensor_on_the_current_device(pkv):
    """Not the first one alone: a length vector or a pool on another GPU is
    refused by name, before the library is called."""
    class _Here(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

    class _Elsewhere(_Here):
        def get_device(self):
            return 1

    i = lambda *s: torch.zeros(*s, dtype=torch.int32)   # noqa: E731
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)   # noqa: E731
    f = lambda *s: torch.zeros(*s)   # noqa: E731
    pools = dict(k_pool=h(9, 8, 16, 128), v_pool=h(9, 8, 16, 128), k_scale=f(9, 8), v_scale=f(9, 8))
    calls = {
        pkv.pkv_slot_map: dict(seq_lens=i(2), new_lens=i(2), block_tables=i(2, 4), pages_held=i(2), free_pages=i(9),
                               free_count=i(1), cu_q=i(3), slots=i(5), positions=i(5), pages_out=i(2), free_left=i(1),
                               parents=i(5), tree_mask=i(5, 1)),
        pkv.pkv_rope_append_axes: dict(q=h(2, 32, 128), k_new=h(2, 8, 128), v_new=h(2, 8, 128), positions=i(1, 2),
                                       sections=[64], slots=i(2), q_out=h(2, 32, 128), **pools),
        pkv.pkv_decode_attn_tree: dict(q=h(5, 32, 128), **pools, block_tables=i(2, 4), seq_lens=i(2), cu_q=i(3),
                                       tree_mask=i(5, 1), out=h(5, 32, 128)),
        pkv.pkv_tree_commit: dict(**pools, block_tables=i(2, 4), seq_lens=i(2), path=i(2, 3), path_lens=i(2),
                                  lens_out=i(2)),
    }
    keep, pkv._cur_device = pkv._cur_device, lambda: 0
    try:
        for call, args in calls.items():
            here = {k: v.as_subclass(_Here) if isinstance(v, torch.Tensor) else v for k, v in args.items()}
            assert call(None, **here, stream=0, check=False) == pkv.PKV_ERR_INVALID_ARG      # NULL context, all else taken
            for k, v in args.items():
                if isinstance(v, torch.Tensor):
                    with pytest.raises(ValueError, match=f"{k}: on cuda:1, the current device is cuda:0"):
                        call(None, **dict(here, **{k: v.as_subclass(_Elsewhere)}), stream=0)
    finally:
        pkv._cur_device = keep


def test_marshal_module_of_another_torch(pkv, tmp_path, monkeypatch):
    """A module built against other headers is not current, one that cannot be
    built again does not stay, and the binding uses none but its own torch's."""
    import os
    import subprocess
    import sys

    from paged_kv_flight_b200 import build
    stamp = build.marshal_stamp()
    assert torch.__version__ in stamp
    if os.path.exists(build.MARSHAL):
        assert build.marshal_current(stamp) and not build.marshal_current(stamp.replace("torch ", "torch 9"))
    old = tmp_path / "_marshal.so"
    old.write_bytes(b"\0torch 1.0, abi 1, cpython-30\0")
    monkeypatch.setattr(build, "MARSHAL", str(old))
    monkeypatch.setenv("CXX", "false")
    assert not build.marshal_current(stamp)
    build.build_marshal()
    assert not old.exists() and not list(tmp_path.iterdir())
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
from paged_kv_flight_b200 import build
build.marshal_stamp = lambda: 'torch 9'
from paged_kv_flight_b200 import pkv
assert pkv._pointer.__module__ == pkv._call.__module__ == pkv.__name__
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
