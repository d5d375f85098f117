"""More arguments that the 8-bit paged cache's entry points refuse: checked on the host,
with nothing enqueued.  No test here launches a kernel."""
import ctypes as C

import pytest

from test_q8_refusals import M, X, Y, append, attend  # noqa: F401  (M: fixture)

Z, V = C.c_void_p(12288), C.c_void_p(16384)


@pytest.mark.parametrize("args", [
    dict(last=Y, out=Y), dict(best=Y, hidden=X, h_next=Z, H=64, out=Y), dict(appended=X), dict(appended=Z, last=Z),
    dict(appended=Z, best=Z, hidden=X, h_next=V, H=64), dict(appended=Y), dict(out=Y, rows=Y), dict(appended=Z, rows=Z),
    dict(out=Y, table=Y), dict(appended=Z, table=Z)], ids=str)
def test_append_outputs_are_none_of_what_it_reads(M, args):  # noqa: F811
    """Every block reads lengths, rows and pages while one writes the new lengths."""
    assert append(M, **args) == -1


@pytest.mark.parametrize("R", [2 ** 31 - 1, 2 ** 31 - 65])
def test_append_of_too_many_rows(M, R):  # noqa: F811
    """The number of pages that R rows span is counted in 64 bits."""
    assert append(M, R=R) == -2


@pytest.mark.parametrize("scale", [2.36e38, 3.0e38, 3.4e38])
def test_attention_scales_that_overflow_in_log2_units(M, scale):  # noqa: F811
    """scale * log2 e has to be finite: infinite, it makes every zero score NaN."""
    assert attend(M, scale=scale, ws=X, ws_bytes=1 << 40) == -1
