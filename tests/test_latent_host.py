"""The latent cache and the operators on sequences' blocks without a GPU: refusals of the C entry points and of the binding,
workspace sizes."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import latent_ref as L
from test_ops_host import FAKE, Desc, caller

P, I, Q, F, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
GOOD = Desc(64, 16, 1, 576)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_slot_gb300.build import build_library
    lib = ctypes.CDLL(build_library())
    lib.pkv_latent_workspace_bytes.restype = lib.pkv_blocks_workspace_bytes.restype = Z
    return lib


def test_latent_append_refusals(lib):
    rows = [("kv", P, FAKE), ("qr", P, FAKE), ("ts", Q, 8 * 64), ("hs", Q, 64)]
    norm = [("f", P, FAKE), ("inter", I, 0), ("w", P, None), ("eps", F, 1e-6)]
    tail = [("N", I, 8), ("cache", P, FAKE), ("q", P, FAKE)]
    given = caller(lib.pkv_latent_append, rows + [("pos", P, FAKE)] + norm + [("slots", P, FAKE), ("n", I, 0)] + tail +
                   [("d", Desc, GOOD), ("err", P, None), ("stream", P, None)])
    multi = caller(lib.pkv_latent_append_multi, rows + [("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE)] + norm +
                   [("B", I, 0), ("T", I, 1)] + tail + [("slots", P, FAKE), ("d", Desc, GOOD), ("err", P, None), ("stream", P, None)])
    for call in (given, multi):
        assert call() == 0                                   # no tokens: nothing launched
        for name in ("kv", "qr", "f", "cache", "q", "slots"):
            assert call(**{name: None}) == -1, name
        for name in ("kv", "qr", "cache", "q", "w"):
            assert call(**{name: FAKE + 8}) == -6, name
        assert call(f=FAKE + 4) == -6 and call(slots=FAKE + 4) == -6
        assert call(ts=12) == -6 and call(hs=4) == -6 and call(ts=-8) == -2 and call(hs=-64) == -2
        assert call(eps=-1.0) == -2 and call(eps=float("nan")) == -2 and call(N=0) == -2
        assert call(d=Desc(64, 16, 1, 512)) == -3 and call(d=Desc(64, 16, 2, 576)) == -3 and call(d=Desc(64, 32, 1, 576)) == -3
        assert call(d=Desc(0, 16, 1, 576)) == -2
    assert given(pos=None) == -1 and given(n=-1) == -2 and given(n=2 ** 31 - 1) == -2
    assert multi(bt=None) == -1 and multi(ctx=None) == -1 and multi(T=0) == -2 and multi(B=-1) == -2 and multi(nb=0) == -2
    assert multi(nb=1 << 28) == -2 and multi(B=1 << 20, T=1 << 20) == -2


def test_latent_attention_refusals(lib):
    need = lib.pkv_latent_workspace_bytes(3, 2, 8)
    call = caller(lib.pkv_decode_attn_latent, [("q", P, FAKE), ("cache", P, FAKE), ("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE),
                  ("B", I, 0), ("T", I, 2), ("N", I, 8), ("scale", F, 1.0), ("out", P, FAKE), ("lse", P, None), ("d", Desc, GOOD),
                  ("ws", P, FAKE), ("bytes", Z, need), ("err", P, None), ("stream", P, None)])
    assert call() == 0
    for name in ("q", "cache", "bt", "ctx", "out"):
        assert call(**{name: None}) == -1, name
    for name in ("q", "cache", "out"):
        assert call(**{name: FAKE + 8}) == -6, name
    assert call(lse=FAKE + 2) == -6 and call(ws=FAKE + 16) == -6
    assert call(ws=None) == -7 and call(B=3, bytes=need - 1) == -7
    assert call(T=0) == -2 and call(T=65) == -3 and call(N=0) == -2 and call(B=-1) == -2 and call(nb=0) == -2 and call(nb=1 << 28) == -2
    assert call(B=1 << 20, N=1 << 12) == -2
    assert call(d=Desc(64, 16, 1, 512)) == -3 and call(d=Desc(64, 16, 4, 576)) == -3 and call(d=Desc(64, 8, 1, 576)) == -3


def test_workspace_sizes(lib):
    size = lib.pkv_latent_workspace_bytes
    assert size(0, 1, 1) > 0 and size(-1, 1, 1) == 0 and size(1, 65, 1) == 0 and size(1, 1, 0) == 0
    for T, N in ((1, 1), (1, 16), (2, 16), (1, 128), (4, 128), (3, 40)):
        a, b = size(1, T, N), size(1000, T, N)
        assert 0 < a <= b and a % 256 == 0 and b % 256 == 0       # one for a batch serves smaller ones
    assert size(1, 1, 16) < size(1, 1, 32) < size(1, 1, 128) == size(1, 1, 64)
    assert lib.pkv_blocks_workspace_bytes(1000) == 4000 and lib.pkv_blocks_workspace_bytes(0) == 0


def test_sequence_refusals(lib):
    fork = caller(lib.pkv_fork_sequences, [("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE), ("B", I, 0), ("par", P, FAKE), ("R", I, 0),
                  ("ref", P, FAKE), ("blocks", I, 9), ("bo", P, 2 * FAKE), ("co", P, 2 * FAKE), ("err", P, None), ("stream", P, None)])
    assert fork() == 0 and fork(bt=None, ctx=None, par=None, bo=None, co=None) == 0
    assert fork(ref=None) == -1
    for name in ("bt", "ctx"):
        assert fork(B=1, **{name: None}) == -1
    for name in ("par", "bo", "co"):
        assert fork(R=1, **{name: None}) == -1
    for name in ("bt", "ctx", "par", "ref", "bo", "co"):
        assert fork(**{name: 3 * FAKE + 2}) == -6, name
    assert fork(nb=0) == -2 and fork(nb=1 << 28) == -2 and fork(B=-1) == -2 and fork(R=-1) == -2 and fork(blocks=0) == -2
    assert fork(B=2 ** 31 - 1, R=2 ** 31 - 1) == -2
    # the new tables or lengths on the old ones
    assert fork(B=10, R=10, bo=FAKE) == -2 and fork(B=10, R=10, bo=FAKE + 9 * 16) == -2 and fork(B=10, R=10, co=FAKE + 36) == -2
    extend = caller(lib.pkv_extend_sequences, [("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE), ("new", P, FAKE), ("B", I, 0), ("ref", P, FAKE),
                    ("blocks", I, 9), ("copies", P, FAKE), ("ws", P, FAKE), ("bytes", Z, 36), ("err", P, None), ("stream", P, None)])
    assert extend() == 0
    for name in ("bt", "ctx", "new", "ref", "copies"):
        assert extend(**{name: None}) == -1 and extend(**{name: FAKE + 2}) == -6, name
    assert extend(ws=None) == -7 and extend(bytes=35) == -7 and extend(ws=FAKE + 2) == -6
    assert extend(nb=0) == -2 and extend(B=-1) == -2 and extend(blocks=0) == -2
    compact = caller(lib.pkv_compact_blocks, [("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE), ("B", I, -1), ("ref", P, FAKE), ("blocks", I, 9),
                     ("moves", P, FAKE), ("most", I, 4), ("n", P, FAKE), ("ws", P, FAKE), ("bytes", Z, 36), ("err", P, None),
                     ("stream", P, None)])
    assert compact() == -2 and compact(B=1, bt=None) == -1
    for name in ("ref", "moves", "n"):
        assert compact(**{name: None}) == -1, name
    assert compact(B=0, most=0) == -2 and compact(B=0, blocks=0) == -2 and compact(B=0, ws=None) == -7 and compact(B=0, bytes=8) == -7
    assert compact(B=0, moves=FAKE + 2) == -6 and compact(B=0, n=FAKE + 2) == -6
    one = (P * 2)(FAKE, FAKE)
    copy = caller(lib.pkv_copy_blocks_pools, [("pools", P, ctypes.cast(one, P)), ("n", I, 2), ("size", Q, 32), ("blocks", I, 9), ("pairs", P, FAKE),
                  ("k", I, 0), ("err", P, None), ("stream", P, None)])
    assert copy() == 0 and copy(pools=None) == -1 and copy(pairs=None) == -1
    assert copy(n=0) == -2 and copy(n=257) == -3 and copy(size=0) == -2 and copy(size=24) == -3 and copy(blocks=0) == -2 and copy(k=-1) == -2
    assert copy(pairs=FAKE + 2) == -6
    assert copy(pools=ctypes.cast((P * 2)(FAKE, None), P)) == -1 and copy(pools=ctypes.cast((P * 2)(FAKE, FAKE + 8), P)) == -6


def test_references():
    """Attention of one token is its row; rows by hand."""
    r = np.random.default_rng(0)
    cache, q = r.standard_normal((3, 16, 576)), r.standard_normal((1, 2, 1, 576))
    out, lse, *_ = L.attention(q, cache, np.array([[2]]), [1], 0.3)
    assert np.all(out[0, 0] == 0) and np.isneginf(lse[0, 0, 0])
    np.testing.assert_allclose(out[0, 1, 0], cache[2, 0, :512])
    t = np.array([[0, 1], [0, 1], [-1, -1]], dtype=np.int32)
    ctx, ref = np.array([20, 20, 0], dtype=np.int32), np.array([2, 2, 0, 0, 0], dtype=np.int32)
    tab, c, f, copies, refused = L.extend(t, ctx, [1, 1, 17], ref)
    assert not refused and tab.tolist() == [[0, 2], [0, 1], [3, 4]] and copies.tolist() == [[1, 2], [-1, -1], [-1, -1]]
    assert f.tolist() == [2, 1, 1, 1, 1] == L.counts(tab, c, 5).tolist()
    tab2, c2, f2 = L.fork(tab, c, [2, 2, -1], 5)
    assert f2.tolist() == [0, 0, 0, 2, 2]
    tab3, f3, moves, n = L.compact(tab2, c2, f2, 4)
    assert tab3[:2].tolist() == [[1, 0], [1, 0]] and moves[:n].tolist() == [[4, 0], [3, 1]] and f3.tolist() == [2, 2, 0, 0, 0]


def test_counts_near_2_to_the_31_are_refused(lib):
    """Loops over rows, blocks and pairs step past the end in 32 bits."""
    most = 2 ** 31 - 1 - 65536
    need = lib.pkv_blocks_workspace_bytes
    need.argtypes = [I]
    fork = caller(lib.pkv_fork_sequences, [("bt", P, None), ("nb", I, 1), ("ctx", P, None), ("B", I, 0), ("par", P, None), ("R", I, 0),
                  ("ref", P, FAKE), ("blocks", I, 9), ("bo", P, None), ("co", P, None), ("err", P, None), ("stream", P, None)])
    assert fork(blocks=most) == 0 and fork(blocks=most + 1) == -2
    args = dict(bt=FAKE, ctx=FAKE, par=FAKE, bo=1 << 60, co=1 << 61)
    assert fork(B=most + 1, **args) == -2 and fork(R=most + 1, **args) == -2 and fork(B=most, R=1, **args) == -2
    extend = caller(lib.pkv_extend_sequences, [("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE), ("new", P, FAKE), ("B", I, 0), ("ref", P, FAKE),
                    ("blocks", I, 9), ("copies", P, FAKE), ("ws", P, FAKE), ("bytes", Z, 1 << 40), ("err", P, None), ("stream", P, None)])
    assert extend(blocks=most) == 0 and extend(blocks=most + 1) == -2 and extend(B=most + 1) == -2
    compact = caller(lib.pkv_compact_blocks, [("bt", P, None), ("nb", I, 4), ("ctx", P, None), ("B", I, 0), ("ref", P, FAKE), ("blocks", I, 9),
                     ("moves", P, FAKE), ("most", I, 4), ("n", P, FAKE), ("ws", P, FAKE), ("bytes", Z, 1 << 40), ("err", P, None),
                     ("stream", P, None)])
    assert compact(blocks=most + 1) == -2 and compact(most=most + 1) == -2
    attend = caller(lib.pkv_decode_attn_latent, [("q", P, FAKE), ("cache", P, FAKE), ("bt", P, FAKE), ("nb", I, 4), ("ctx", P, FAKE),
                    ("B", I, 0), ("T", I, 2), ("N", I, 8), ("scale", F, 1.0), ("out", P, FAKE), ("lse", P, None), ("d", Desc, GOOD),
                    ("ws", P, FAKE), ("bytes", Z, 1 << 40), ("err", P, None), ("stream", P, None)])
    assert attend(nb=(2 ** 31 - 1 - 1024) // 16) == 0 and attend(nb=(2 ** 31 - 1 - 1024) // 16 + 1) == -2


def test_rows_wider_than_a_grid_are_refused(lib):
    most = 65535 * 512
    fork = caller(lib.pkv_fork_sequences, [("bt", P, None), ("nb", I, 1), ("ctx", P, None), ("B", I, 0), ("par", P, None), ("R", I, 0),
                  ("ref", P, FAKE), ("blocks", I, 9), ("bo", P, None), ("co", P, None), ("err", P, None), ("stream", P, None)])
    assert fork(nb=most) == 0 and fork(nb=most + 1) == -2
