"""The calls of rotary positions, chunks and drawn tokens on a stream that is not the current
one: it is current while they look at their arguments and allocate."""
import inspect

import pytest
import torch

from test_streams import Stream, streams  # noqa: F401


@pytest.mark.parametrize("name,dims", [("rope_rows", 4), ("kv_append_rope_q8", 4), ("chunk_attention_q8", 4),
                                       ("verify_accept_tree_draw", 3)])
def test_the_given_stream_is_current_while_a_call_allocates(streams, monkeypatch, name, dims):  # noqa: F811
    from medusa_speculative_decoding_gb300 import api
    at = []

    class Looked(Exception):
        pass

    def look(*a, **k):
        at.append(streams[-1])
        raise Looked

    for f in ("_need", "_need_pool"):
        monkeypatch.setattr(api, f, look)
    f = getattr(api, name)
    n = [p for p in inspect.signature(f).parameters.values() if p.default is p.empty]
    with pytest.raises(Looked):
        f(*[torch.zeros([1] * dims) for _ in n], stream=Stream("side"))
    assert at == ["side"]
