"""Steps and the rows they take, without a GPU: refusals of the extension with the lengths for a step, a stack's inputs."""
from __future__ import annotations

from types import SimpleNamespace

from test_latent_host import I, P, Z, lib  # noqa: F401
from test_ops_host import FAKE, caller


def test_refusals_of_the_lengths_for_the_step(lib):  # noqa: F811
    extend = caller(lib.pkv_extend_sequences_step, [("bt", P, FAKE), ("nb", I, 4), ("ctx", P, 2 * FAKE), ("new", P, 3 * FAKE), ("B", I, 0),
                    ("ref", P, FAKE), ("blocks", I, 9), ("copies", P, FAKE), ("lens", P, 4 * FAKE), ("ws", P, FAKE), ("bytes", Z, 36),
                    ("err", P, None), ("stream", P, None)])
    assert extend() == 0 and extend(lens=None) == 0
    for name in ("bt", "ctx", "new", "ref", "copies"):
        assert extend(**{name: None}) == -1 and extend(**{name: 5 * FAKE + 2}) == -6, name
    assert extend(lens=4 * FAKE + 2) == -6
    # the lengths for the step on the lengths themselves, or on what the rows grow by
    assert extend(B=10, lens=2 * FAKE) == -2 and extend(B=10, lens=2 * FAKE + 36) == -2 and extend(B=10, lens=3 * FAKE - 36) == -2
    assert extend(ws=None) == -7 and extend(bytes=35) == -7 and extend(nb=0) == -2 and extend(B=-1) == -2 and extend(blocks=0) == -2


def test_a_stacks_inputs_are_its_layers():
    from paged_kv_decode_slot_gb300.step import DecodeStep, LatentDecodeStep, LayerStack, PrefixDecodeStep
    layer = lambda kind, **own: SimpleNamespace(fused=True, plan=None, input_names=lambda: kind.input_names(None), **own)
    names = LayerStack([layer(LatentDecodeStep), layer(LatentDecodeStep)]).input_names()
    assert names == ("block_tables", "context_lens", "kv_new.0", "q_rope.0", "q.0", "kv_new.1", "q_rope.1", "q.1")
    for kind in (DecodeStep, PrefixDecodeStep):
        names = LayerStack([layer(kind, k_new=0), layer(kind, k_new=0)]).input_names()
        assert names == ("block_tables", "context_lens", "q.0", "k_new.0", "v_new.0", "q.1", "k_new.1", "v_new.1")
