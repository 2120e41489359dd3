"""The operators around a step's attention without a GPU: refusals of the C entry points (host validation comes
before any CUDA call) and of the binding, workspace sizes, and the references the GPU tests compare with."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import ops_ref as R

P, I, L, F, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
FAKE = 0x10000   # an aligned stand-in device address; host validation never dereferences it


class Desc(ctypes.Structure):
    _fields_ = [("num_blocks", I), ("block_size", I), ("num_kv_heads", I), ("head_dim", I)]


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_slot_gb300.build import build_library
    return ctypes.CDLL(build_library())


def caller(fn, types, **defaults):
    """A call by argument name with everything else at a valid value."""
    fn.argtypes = [t for _, t, _ in types]
    def call(**kw):
        assert set(kw) <= {n for n, _, _ in types}
        return fn(*[kw.get(n, d) for n, _, d in types])
    return call


def test_rope_append_refusals(lib):
    head = [("q", P, FAKE), ("k", P, FAKE), ("v", P, FAKE)]
    tail = [("kc", P, FAKE), ("vc", P, FAKE), ("out", P, FAKE)]
    given = caller(lib.pkv_rope_append, head + [("pos", P, FAKE), ("f", P, FAKE), ("R", I, 64), ("inter", I, 0),
                   ("slots", P, FAKE), ("n", I, 0), ("N", I, 8)] + tail +
                   [("d", Desc, Desc(64, 16, 2, 64)), ("err", P, None), ("stream", P, None)])
    multi = caller(lib.pkv_rope_append_multi, head + [("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE), ("f", P, FAKE),
                   ("R", I, 64), ("inter", I, 0), ("B", I, 0), ("T", I, 1), ("N", I, 8)] + tail +
                   [("slots", P, FAKE), ("d", Desc, Desc(64, 16, 2, 64)), ("err", P, None), ("stream", P, None)])
    for call in (given, multi):
        assert call() == 0                                   # no tokens: nothing launched
        for name in ("q", "k", "v", "f", "kc", "vc", "out", "slots"):
            assert call(**{name: None}) == -1, name
        for name in ("q", "k", "v", "kc", "vc", "out"):
            assert call(**{name: FAKE + 8}) == -6, name
        assert call(f=FAKE + 4) == -6 and call(slots=FAKE + 4) == -6
        assert call(R=0) == -2 and call(R=80) == -2          # none, more than the head
        assert call(R=24) == -3                              # not a multiple of 16
        assert call(d=Desc(64, 16, 2, 96)) == -3             # head_dim
        assert call(d=Desc(64, 8, 2, 64)) == -3              # block size
        assert call(d=Desc(0, 16, 2, 64)) == -2
        assert call(N=0) == -2
    assert given(pos=None) == -1 and given(n=-1) == -2
    assert multi(bt=None) == -1 and multi(ctx=None) == -1
    assert multi(T=0) == -2 and multi(B=-1) == -2 and multi(nb=0) == -2
    assert multi(B=1 << 20, T=1 << 20) == -2                 # more tokens than 32 bits count
    scales = [("ks", P, FAKE), ("vs", P, FAKE), ("stride", I, 0)]
    fp8 = caller(lib.pkv_rope_append_fp8, head + [("pos", P, FAKE), ("f", P, FAKE), ("R", I, 64), ("inter", I, 0)] + scales +
                 [("slots", P, FAKE), ("n", I, 0), ("N", I, 8)] + tail +
                 [("d", Desc, Desc(64, 16, 2, 128)), ("err", P, None), ("stream", P, None)])
    assert fp8() == 0 and fp8(stride=2) == 0
    assert fp8(stride=1) == -2 and fp8(ks=None) == -1 and fp8(vs=None) == -1 and fp8(kc=FAKE + 4) == -6


def test_key_bounds_refusals(lib):
    f = caller(lib.pkv_key_bounds, [("kc", P, FAKE), ("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE), ("B", I, 0),
               ("new", I, 1), ("bounds", P, FAKE), ("d", Desc, Desc(64, 16, 2, 64)), ("err", P, None), ("s", P, None)])
    assert f() == 0 and f(B=3, new=0) == 0
    for name in ("kc", "bt", "ctx", "bounds"):
        assert f(**{name: None}) == -1, name
    assert f(new=-1) == -2 and f(B=-1) == -2 and f(B=70000) == -2 and f(nb=0) == -2 and f(nb=1 << 28) == -2
    assert f(kc=FAKE + 8) == -6 and f(bounds=FAKE + 8) == -6
    assert f(d=Desc(64, 16, 2, 60)) == -3 and f(d=Desc(64, 8, 2, 64)) == -3


def test_select_refusals_and_workspace(lib):
    lib.pkv_select_workspace_bytes.restype = Z
    lib.pkv_select_workspace_bytes.argtypes = [I, I, I]
    ws = lib.pkv_select_workspace_bytes
    up = lambda x: -(-x // 256) * 256
    u = 3 * 2 * 50                                            # sequences x heads x blocks
    assert ws(3, 2, 50) == up(up(up(u * 4) + u * 8) + u * 4) + 3 * 2 * 4 * 4
    assert ws(-1, 2, 50) == 0 and ws(0, 2, 50) == 0
    f = caller(lib.pkv_select_blocks, [("q", P, FAKE), ("bounds", P, FAKE), ("bt", P, FAKE), ("nb", I, 50), ("ctx", P, FAKE),
               ("B", I, 0), ("N", I, 8), ("first", I, 1), ("last", I, 1), ("M", I, 8), ("sel", P, FAKE),
               ("d", Desc, Desc(64, 16, 2, 64)), ("ws", P, FAKE), ("size", Z, ws(3, 2, 50)), ("err", P, None), ("s", P, None)])
    assert f() == 0
    for name in ("q", "bounds", "bt", "ctx", "sel"):
        assert f(**{name: None}) == -1, name
    assert f(ws=None) == -7 and f(B=3, size=ws(3, 2, 50) - 1) == -7
    assert f(first=5, last=4) == -2 and f(first=-1) == -2 and f(last=-1) == -2 and f(M=0, first=0, last=0) == -2
    assert f(q=FAKE + 8) == -6 and f(bounds=FAKE + 8) == -6 and f(ws=FAKE + 16) == -6
    assert f(N=6, d=Desc(64, 16, 4, 64)) == -2 and f(N=32) == -3 and f(d=Desc(64, 16, 2, 96)) == -3
    assert f(B=70000) == -2 and f(nb=0) == -2


def test_blocks_attention_refusals(lib):
    lib.pkv_splitk_workspace_bytes.restype = Z
    lib.pkv_splitk_workspace_bytes.argtypes = [I, I, I, I]
    need = lib.pkv_splitk_workspace_bytes(4, 8, 64, 4)
    args = [("bt", P, FAKE), ("nb", I, 50), ("ctx", P, FAKE), ("sel", P, FAKE), ("M", I, 8), ("B", I, 0), ("N", I, 8),
            ("scale", F, 0.1), ("out", P, FAKE), ("lse", P, None)]
    tail = [("pb", I, 0), ("parts", I, 0), ("ws", P, None), ("size", Z, 0), ("err", P, None), ("s", P, None)]
    f = caller(lib.pkv_decode_attn_blocks, [("q", P, FAKE), ("kc", P, FAKE), ("vc", P, FAKE)] + args +
               [("d", Desc, Desc(64, 16, 2, 64))] + tail)
    assert f() == 0 and f(pb=2, parts=4, ws=FAKE, size=need, B=0) == 0
    for name in ("q", "kc", "vc", "bt", "ctx", "sel", "out"):
        assert f(**{name: None}) == -1, name
    assert f(M=0) == -2 and f(pb=-1) == -2 and f(pb=2, parts=3, ws=FAKE, size=need) == -2
    assert f(pb=2, parts=4) == -7 and f(B=4, pb=2, parts=4, ws=FAKE, size=need - 1) == -7
    assert f(pb=2, parts=4, ws=FAKE + 16, size=need) == -6
    assert f(pb=1, parts=2049, ws=FAKE, size=1 << 40) == -3   # 4 heads x 2,049 weights: more than the merge holds
    assert f(pb=2 ** 31 - 1, parts=2, ws=FAKE, size=1 << 40) == -2   # more entries than 32 bits count
    assert f(kc=FAKE + 8) == -6 and f(out=FAKE + 2) == -6
    g = caller(lib.pkv_decode_attn_blocks_fp8, [("q", P, FAKE), ("kc", P, FAKE), ("vc", P, FAKE), ("ks", P, FAKE), ("vs", P, FAKE),
               ("stride", I, 0)] + args + [("d", Desc, Desc(64, 16, 2, 128))] + tail)
    assert g() == 0 and g(stride=2) == 0
    assert g(stride=3) == -2 and g(ks=None) == -1 and g(q=FAKE + 4) == -6 and g(d=Desc(64, 16, 2, 64)) == -3


def test_verify_refusals_and_workspace(lib):
    lib.pkv_verify_workspace_bytes.restype = Z
    lib.pkv_verify_workspace_bytes.argtypes = [I, I]
    ws = lib.pkv_verify_workspace_bytes
    assert ws(3, 1000) == 256 * -(-3 * 4 * 8 // 256) + 3 * 4
    assert ws(3, 1 << 19) == 0 and ws(-1, 10) == 0
    f = caller(lib.pkv_verify_draft, [("p", P, FAKE), ("ps", L, 1000), ("q", P, FAKE), ("qs", L, 1000), ("bf16", I, 0),
               ("tok", P, FAKE), ("lens", P, None), ("u", P, FAKE), ("r", P, FAKE), ("B", I, 0), ("T", I, 4), ("V", I, 1000),
               ("acc", P, FAKE), ("out", P, FAKE), ("ctx", P, None), ("ctx_out", P, None), ("ws", P, FAKE),
               ("size", Z, ws(3, 1000)), ("err", P, None), ("s", P, None)])
    assert f() == 0 and f(q=None, qs=0) == 0 and f(T=0, tok=None, u=None) == 0
    for name in ("p", "tok", "u", "r", "acc", "out"):
        assert f(**{name: None}) == -1, name
    assert f(ctx=FAKE) == -1 and f(ctx_out=FAKE) == -1 and f(ctx=FAKE, ctx_out=FAKE) == 0
    assert f(ps=999) == -2 and f(qs=999) == -2 and f(V=0) == -2 and f(T=-1) == -2 and f(T=1025) == -2 and f(B=70000) == -2
    assert f(V=1 << 19, ps=1 << 20, qs=1 << 20) == -3
    assert f(ws=None) == -7 and f(B=3, size=ws(3, 1000) - 1) == -7
    assert f(p=FAKE + 2) == -6 and f(p=FAKE + 2, bf16=1) == 0 and f(ws=FAKE + 8) == -6


def test_binding_refuses_host_tensors_types_and_shapes(monkeypatch):
    """The binding checks type, shape and place of every tensor before it takes an address (no GPU here: with the
    current device faked, host tensors are refused by name)."""
    from paged_kv_decode_slot_gb300 import binding as B
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    t = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype)
    q, k, kc = t(4, 8, 64), t(4, 2, 64), t(9, 16, 2, 64)
    rest = (t(4, dtype=torch.int32), t(32, dtype=torch.float64), t(4, dtype=torch.int64), kc, kc, q)
    with pytest.raises(ValueError, match="q before the rotation must be a CUDA tensor"):
        B.pkv_rope_append(q, k, k, *rest)
    with pytest.raises(TypeError):
        B.pkv_rope_append(None, k, k, *rest)
    with pytest.raises(ValueError, match="head_dim"):
        B.pkv_rope_append(t(4, 8, 128), k, k, *rest)
    with pytest.raises(ValueError):                          # 2 dims
        B.pkv_rope_append(t(4, 64), k, k, *rest)
    monkeypatch.setattr(B, "_arg", B._arg_py)                # (the compiled check does not take a stand-in for a GPU)
    with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
        B.pkv_key_bounds(kc, t(3, 4, dtype=torch.int32).pin_memory() if torch.cuda.is_available() else _Cuda(3, 4, dtype=torch.int32),
                         _Cuda(3, dtype=torch.int32), 1, t(9, 2, 2, 64))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        B.pkv_verify_draft(t(2, 3, 10, dtype=torch.float64), None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="vocab_size"):
        B.pkv_verify_draft(t(2, 3, 10), t(2, 2, 8), None, None, None, None, None, t(8, dtype=torch.uint8))


class _Cuda(torch.Tensor):
    """A host tensor that says it lives on the current device."""

    @staticmethod
    def __new__(cls, *shape, dtype):
        return torch.zeros(*shape, dtype=dtype).as_subclass(cls)

    def get_device(self):
        return 0


def test_binding_shapes_must_match(monkeypatch):
    from paged_kv_decode_slot_gb300 import binding as B
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_launch", lambda stream, dev: 0)
    monkeypatch.setattr(B, "_arg", B._arg_py)                # (the compiled check does not take a stand-in for a GPU)
    monkeypatch.setattr(B, "_maybe", B._maybe_py)
    c = lambda *shape, dtype=torch.bfloat16: _Cuda(*shape, dtype=dtype)
    i32 = torch.int32
    q, kc, bt, ctx = c(4, 8, 64), c(9, 16, 2, 64), c(4, 5, dtype=i32), c(4, dtype=i32)

    class Lib:
        def __getattr__(self, name):
            def called(*args):
                raise AssertionError(f"{name} was called")
            return called
    monkeypatch.setattr(B, "_lib", Lib())
    sel, ws, out = c(4, 2, 3, dtype=i32), c(512, dtype=torch.uint8), c(4, 8, 64)
    ok = dict(q=q, k_cache=kc, v_cache=kc, block_tables=bt, context_lens=ctx, selected=sel, scale=1.0, out=out)
    with pytest.raises(AssertionError, match="pkv_decode_attn_blocks"):
        B.pkv_decode_attn_blocks(**ok)
    for name, bad in (("v_cache", c(8, 16, 2, 64)), ("block_tables", c(3, 5, dtype=i32)), ("context_lens", c(5, dtype=i32)),
                      ("selected", c(4, 3, 3, dtype=i32)), ("out", c(4, 8, 128)), ("q", c(4, 8, 128))):
        with pytest.raises(ValueError):
            B.pkv_decode_attn_blocks(**{**ok, name: bad})
    for name, bad in (("selected", c(4, 2, 3, dtype=torch.int64)), ("k_cache", c(9, 16, 2, 64, dtype=torch.uint8)),
                      ("out", c(4, 8, 64, dtype=torch.float32))):
        with pytest.raises(TypeError):
            B.pkv_decode_attn_blocks(**{**ok, name: bad})
    with pytest.raises(ValueError):                          # scales of another pool
        B.pkv_decode_attn_blocks_fp8(q, c(9, 16, 2, 64, dtype=torch.uint8), c(9, 16, 2, 64, dtype=torch.uint8),
                                     c(8, 2, dtype=torch.float32), c(8, 2, dtype=torch.float32), bt, ctx, sel, 1.0, out)
    with pytest.raises(ValueError):                          # bounds of another head count
        B.pkv_select_blocks(q, c(9, 2, 3, 64), bt, ctx, sel, ws)
    with pytest.raises(ValueError, match="overlap"):
        base = torch.zeros(5, 8, 64, dtype=torch.bfloat16).as_subclass(_Cuda)
        B.pkv_rope_append(base[:4], c(4, 2, 64), c(4, 2, 64), ctx, c(32, dtype=torch.float64), c(4, dtype=torch.int64),
                          kc, kc, base[1:])


def test_compiled_argument_check_is_built_and_refuses_alike():
    from paged_kv_decode_slot_gb300 import binding as B
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    from paged_kv_decode_slot_gb300 import tensor_args
    x = torch.zeros(3, 4)
    for check in (tensor_args.arg, B._arg_py):
        for args, error in (((x, torch.float32, (3, 4), "x", 0), "x must be a CUDA tensor"), ((x, torch.int32, (3, 4), "x", 0), "torch.int32"),
                            ((x, torch.float32, (3,), "x", 0), "1 dims"), ((None, torch.float32, (3,), "x", 0), "torch.Tensor")):
            with pytest.raises((TypeError, ValueError), match=error):
                check(*args)
    assert tensor_args.maybe(None, torch.float32, (3,), "x", 0) is None
    with pytest.raises(TypeError):
        tensor_args.arg(x)


def test_compiled_calls_leave_what_is_not_plain_to_the_binding():
    """Host tensors, other types, missing arguments and sizes that do not fit: None, and nothing is called."""
    from paged_kv_decode_slot_gb300 import binding as B
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    from paged_kv_decode_slot_gb300 import tensor_args
    assert B._calls is tensor_args
    counts = dict(rope_append=13, rope_append_fp8=15, rope_append_multi=14, rope_append_multi_fp8=16, key_bounds=8, key_bounds_fp8=9,
                  select_blocks=12, decode_attn_blocks=15, decode_attn_blocks_fp8=17, verify_draft=15)
    t = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    for name, n in counts.items():
        f = getattr(tensor_args, name)
        for args in ((), (t,) * n, (None,) * n, (t,) * (n - 1) + (0,), (t,) * (n - 2) + (None, 0), (1,) * n, (1 << 80,) * n, ("x",) * (n + 1)):
            assert f(*args) is None, (name, len(args))
    with pytest.raises(TypeError):
        tensor_args.use_library(0)
    with pytest.raises(ImportError):
        tensor_args.use_library(ctypes.CDLL(None)._handle, B._launch)


@pytest.mark.filterwarnings("ignore")
def test_compiled_calls_and_tensors_without_memory():
    """Fake tensors that say they are on the GPU: no address, no exception past the interpreter."""
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    from paged_kv_decode_slot_gb300 import tensor_args
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        c = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")
        kc, tables, lens, bounds = c(9, 16, 2, 64), c(3, 4, dtype=torch.int32), c(3, dtype=torch.int32), c(9, 2, 2, 64)
        q, sel, ws, out = c(3, 8, 64), c(3, 2, 5, dtype=torch.int32), c(512, dtype=torch.uint8), c(3, 8, 64)
        p, tok, u = c(3, 3, 10), c(3, 2, dtype=torch.int32), c(3, 2, dtype=torch.float32)
        assert kc.is_cuda
        assert tensor_args.key_bounds(kc, tables, lens, 1, bounds, None, None, 0) is None
        assert tensor_args.select_blocks(q, bounds, tables, lens, sel, ws, 1, 1, None, 16, None, 0) is None
        assert tensor_args.decode_attn_blocks(q, kc, kc, tables, lens, sel, 1.0, out, None, 0, 0, None, None, None, 0) is None
        assert tensor_args.verify_draft(p, None, tok, u, u[:, 0].contiguous(), lens, c(3, 3, dtype=torch.int32), ws, None, None, None,
                                        None, None, None, 0) is None
        inv, new, slots = c(32, dtype=torch.float64), c(3, 1, 2, 64), c(3, 1, dtype=torch.int64)
        assert tensor_args.rope_append_multi(c(3, 1, 8, 64), new, new, tables, lens, inv, kc, kc, c(3, 1, 8, 64), slots, False, None,
                                             None, 0) is None


def test_plan_blocks_attention():
    from paged_kv_decode_slot_gb300.step import plan_blocks_attention as plan
    p = plan(64, 8, 128, 152)
    assert (p.mode, p.partition_blocks, p.max_partitions) == ("single", 0, 1)
    for args in ((1, 8, 128, 152), (20, 8, 250, 152), (4, 2, 33, 152), (200, 8, 1000, 152)):
        p = plan(*args)
        assert p.mode == "split" and p.partition_blocks * p.max_partitions >= args[2]
        assert p.partition_blocks * (p.max_partitions - 1) < args[2]


# ------------------------------------------------------------- the references against facts of their own
def test_reference_rotation():
    """A quarter turn maps (1, 0) to (0, 1); turns add up; lengths stay; far positions agree with the exact fraction."""
    x = np.array([[[1.0, 0.0] + [0.0] * 14]])
    y = R.rope(x, np.array([1]), np.array([math.pi / 2] + [0.0] * 7), True)
    assert np.allclose(y[0, 0, :2], [0, 1], atol=1e-15)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 32))
    f = 500000.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        y = R.rope(R.rope(x, np.array([3, 5, 9]), f, inter), np.array([7, -5, 100]), f, inter)
        assert np.allclose(y, R.rope(x, np.array([10, 0, 109]), f, inter), atol=1e-12)
        assert np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # inv_freq = pi's double: 2^31 - 1 half turns are off by what the double lacks of pi
    y = R.rope(np.array([[[1.0, 0.0] + [0.0] * 14]]), np.array([2 ** 31 - 1]), np.array([math.pi] + [0.0] * 7), True)
    assert abs(y[0, 0, 1] - (2 ** 31 - 1) * 1.2246467991473532e-16) < 1e-15 and abs(y[0, 0, 0] + 1) < 1e-13


def test_reference_selection_bounds_every_key():
    """No q . k of a block exceeds its score, and the first/last blocks are always there."""
    rng = np.random.default_rng(1)
    ctx = [160]
    tab, pool = R.tables(rng, ctx)
    keys, q = rng.standard_normal((pool, 16, 1, 16)), rng.standard_normal((1, 2, 16))
    b = R.key_bounds(keys, tab, ctx, 160, np.zeros((pool, 1, 2, 16)))
    score = np.array([max(np.where(x > 0, x * b[blk, 0, 1], x * b[blk, 0, 0]).sum() for x in q[0]) for blk in tab[0]])
    assert all((q[0] @ keys[blk, :, 0].T).max() <= s + 1e-12 for blk, s in zip(tab[0], score))
    sel = R.select(q, b, tab, ctx, 4, 1, 1)[0, 0]
    assert sel[0] == 0 and sel[-1] == 9 and list(sel) == sorted(sel)
    assert set(sel[1:3]) == set(1 + np.argsort(-score[1:9])[:2])


def test_reference_attention_and_verification():
    rng = np.random.default_rng(2)
    ctx = [40]
    tab, pool = R.tables(rng, ctx)
    k, v, q = rng.standard_normal((pool, 16, 1, 8)), rng.standard_normal((pool, 16, 1, 8)), rng.standard_normal((1, 1, 8))
    flat = lambda x: np.concatenate([x[tab[0, j], :min(16, 40 - 16 * j), 0] for j in range(3)])
    z = flat(k) @ q[0, 0]
    out, lse, _ = R.blocks_attention(q, k, v, tab, ctx, np.array([[[2, 0, 1]]]), 1.0)
    assert np.allclose(out[0, 0], np.exp(z) @ flat(v) / np.exp(z).sum()) and np.isclose(lse[0, 0], np.log(np.exp(z).sum()))
    p = np.array([[[0.5, 0.25, 0.25], [0.1, 0.2, 0.7]]])
    qd = np.array([[[0.25, 0.75, 0.0]]])
    tok = np.array([[1]])
    acc, out = R.verify(p, qd, tok, np.array([[0.3]]), np.array([0.31]))       # 0.3 * 0.75 < 0.25: stands, then from p_1
    assert acc[0] == 1 and list(out[0]) == [1, 2]
    acc, out = R.verify(p, qd, tok, np.array([[0.5]]), np.array([0.4]))        # refused: residual (0.25, 0, 0.25)
    assert acc[0] == 0 and list(out[0]) == [0, -1]
    acc, out = R.verify(p, qd, tok, np.array([[0.5]]), np.array([0.5]))        # the running sum must exceed: 0.25 does not
    assert list(out[0]) == [2, -1]
