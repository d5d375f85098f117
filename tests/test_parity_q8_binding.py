"""GPU tests of what the binding of the 8-bit paged cache refuses: a ValueError that names
the argument, with nothing launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def a():
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    return dict(k_pages=z(4, 2, 16, 64, d=torch.uint8), v_pages=z(4, 2, 16, 64, d=torch.uint8), k_scale=torch.ones(4, 2, device="cuda"),
                v_scale=torch.ones(4, 2, device="cuda"), page_table=z(2, 3), kv_len=z(2)), z


CALLS = {
    "tree_attention_q8": lambda z: dict(q=z(2, 1, 4, 64, d=torch.float32), k_tree=z(2, 1, 2, 64, d=torch.float32),
                                        v_tree=z(2, 1, 2, 64, d=torch.float32), mask=z(1, 1, d=torch.int64), scale=0.1),
    "kv_append_q8": lambda z: dict(k_rows=z(2, 1, 2, 64, d=torch.float32), v_rows=z(2, 1, 2, 64, d=torch.float32)),
    "kv_pages_fork": lambda z: {},
    "kv_pages_compact": lambda z: {},
}


@pytest.mark.parametrize("name", CALLS)
def test_missing_and_wrong_arguments(medusa, a, name):
    pool, z = a
    if name == "kv_pages_compact":
        del pool["kv_len"]
    args = {**pool, **CALLS[name](z)}
    f = getattr(medusa, name)
    for k in args:
        if k == "scale":
            continue
        wrongs = [None, args[k].cpu(), args[k].to(torch.float64)]
        if name != "kv_pages_compact" or k != "page_table":  # (a table of any batch may be compacted)
            wrongs.append(torch.cat([args[k]] * 2))
        for wrong in wrongs:
            with pytest.raises(ValueError):
                f(**{**args, k: wrong})
    torch.cuda.synchronize()
    f(**args)
    torch.cuda.synchronize()
