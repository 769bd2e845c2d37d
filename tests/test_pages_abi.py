"""The page tables' header and its binding agree, and its C calls refuse what they cannot take (no GPU)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "dspark_pages.h")).read(), flags=re.S)


def test_binding_covers_the_header():
    from serial_draft_head_gb300 import pages
    text = header()
    names = set(re.findall(r"^int (dspark_pages_\w+)\(", text, flags=re.M))
    assert names == set(pages.EXPORTS)
    L = pages.load()
    assert all(hasattr(L, n) for n in names)
    assert int(re.search(r"#define DSPARK_PAGES_MAX_REQUESTS (\d+)", text).group(1)) == pages.PAGES_MAX_REQUESTS


def test_struct_matches_the_header():
    from serial_draft_head_gb300 import pages
    body = re.search(r"struct dspark_pages \{(.*?)\};", header(), flags=re.S).group(1)
    want = []
    for line in filter(None, (x.strip() for x in body.split(";"))):
        kind, name = re.match(r"(\w+)\s+(.*)", line).groups()
        size = 8 if name.startswith("*") or kind == "int64_t" else 4
        want.append((name.lstrip("*"), size))
    assert [(n, ctypes.sizeof(t)) for n, t in pages.dspark_pages._fields_] == want


def test_calls_refuse_without_touching_a_device():
    from serial_draft_head_gb300 import pages, walk
    L = pages.load()
    at = 1 << 20                                   # any address: nothing is launched
    good = dict(table=at, held=at, free=at, n_free=at, state=at, table_stride=8, n_pages=9, page_size=16, requests=4,
                max_pages=8)
    for bad in (dict(table=None), dict(held=None), dict(free=None), dict(n_free=None), dict(state=None),
                dict(table_stride=7), dict(n_pages=0), dict(page_size=0), dict(requests=0), dict(requests=1025),
                dict(max_pages=0), dict(n_pages=1 << 27), dict(max_pages=1 << 27, table_stride=1 << 27)):
        p = ctypes.addressof(pages.dspark_pages(**{**good, **bad}))
        keep = pages.dspark_pages(**{**good, **bad})
        p = ctypes.addressof(keep)
        assert L.dspark_pages_reset(p, None) == walk.EINVAL
        assert L.dspark_pages_trim(p, at, None) == walk.EINVAL
        assert L.dspark_pages_status(p, None) == walk.EINVAL
        assert L.dspark_pages_grow(p, at, at, 1, None, 0, 0, at, at, at, None) == walk.EINVAL
    keep = pages.dspark_pages(**good)
    p = ctypes.addressof(keep)
    for args in ((None, at, 1, None, 0, 0, at, at, at), (at, None, 1, None, 0, 0, at, at, at),
                 (at, at, -1, None, 0, 0, at, at, at), (at, at, 1, None, 0, 0, None, at, at),
                 (at, at, 1, None, 0, 0, at, None, at), (at, at, 1, None, 0, 0, at, at, None),
                 (at, at, 1, at, 0, 0, at, at, at), (at, at, 1, at, -1, 1, at, at, at)):
        assert L.dspark_pages_grow(p, *args, None) == walk.EINVAL
    assert L.dspark_pages_trim(p, None, None) == walk.EINVAL
    assert L.dspark_pages_reset(None, None) == walk.EINVAL


@pytest.mark.parametrize("kw", [dict(n_pages=0), dict(page_size=0), dict(requests=0), dict(requests=1025),
                                dict(max_pages=0), dict(n_pages=1 << 27), dict(max_pages=1 << 27)])
def test_pool_refuses_sizes(kw):
    from serial_draft_head_gb300 import Pages
    with pytest.raises(ValueError):
        Pages(**{**dict(n_pages=9, page_size=16, requests=4, max_pages=8), **kw}, device="cuda:0")
