"""A cache of no pages: planned as one that holds no tokens, whatever the table's width; its pointers and the table are not asked for."""
import pytest

from test_cache_host import FAKE, attend, lib, msg, problem, read, write  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("T", [1, 3, 40, 300])
def test_no_tiles_of_the_cache_are_planned(lib, T, dt, fmt):  # noqa: F811
    size = lib.msda_cache_attention_workspace_size
    for source in (0, T):
        full = dict(T=T, source=source, width=4000, longest=64000)
        assert size(dt, fmt, problem(**full)) > 0
        assert size(dt, fmt, problem(**full, pages=0)) == size(dt, fmt, problem(**full | dict(longest=0))) == 0


def test_sizes_count_what_there_is(lib):  # noqa: F811
    """Too many tiles for one call with pages, few without."""
    many = dict(B=1 << 12, T=1, source=1, N=8, M=8, width=1 << 20, longest=1 << 24)
    assert attend(lib, problem(**many)) == 2 and "too many" in msg(lib)
    assert attend(lib, problem(**many, pages=0), out=FAKE + 2) == 3 and "out" in msg(lib)


def test_other_arguments_are_still_asked_for(lib):  # noqa: F811
    """Each of these calls ends at the argument named, behind the cache's pointers, which are NULL."""
    none = dict.fromkeys(("cache_key", "cache_value", "key_scale", "value_scale", "table"))
    p = problem(pages=0)
    assert write(lib, p, start=None, **none) == 1 and "start" in msg(lib)
    assert read(lib, p, lengths=None, **none) == 1 and "lengths" in msg(lib)
    assert attend(lib, p, lse=None, **none) == 1 and "lse" in msg(lib)
    with_pages = problem()
    for call in (write, read, attend):
        assert call(lib, with_pages, **none) == 1 and "NULL" in msg(lib)
