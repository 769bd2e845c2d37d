"""The tree header, its binding and the mask helper agree (no GPU)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header():
    return open(os.path.join(ROOT, "include", "dspark_tree.h")).read()


def test_binding_covers_the_header():
    from serial_draft_head_gb300 import tree
    text = re.sub(r"/\*.*?\*/", "", header(), flags=re.S)
    names = set(re.findall(r"^int (dspark_tree_\w+)\(", text, flags=re.M))
    assert names == set(tree.EXPORTS)
    L = tree.load()
    for n in names:
        assert hasattr(L, n)
    defs = re.findall(r"^#define DSPARK_((?:TYPE|TREE)_\w+)\s+\(?(-?\d+)\)?", text, flags=re.M)
    assert len(defs) >= 6
    for name, value in defs:
        assert getattr(tree, name) == int(value)


@pytest.mark.parametrize("struct", ["dspark_tree_config", "dspark_tree_cache", "dspark_tree_batch"])
def test_structs_match_the_header(struct):
    from serial_draft_head_gb300 import tree
    text = re.sub(r"/\*.*?\*/", "", header(), flags=re.S)
    body = re.search(r"struct %s \{(.*?)\};" % struct, text, flags=re.S).group(1)
    want = []
    for line in body.split(";"):
        line = line.strip()
        if not line:
            continue
        kind, names = re.match(r"((?:const )?\w+)\s+(.*)", line, flags=re.S).groups()
        for n in names.split(","):
            n = n.strip()
            size = re.search(r"\[(\d)\]", n)
            ctype = ctypes.c_void_p if n.startswith("*") else \
                {"int": ctypes.c_int, "int64_t": ctypes.c_int64}[kind]
            want.append((re.sub(r"[\*\s]|\[\d\]", "", n),
                         ctypes.sizeof(ctype) * (int(size.group(1)) if size else 1)))
    got = [(n, ctypes.sizeof(t)) for n, t in getattr(tree, struct)._fields_]
    assert got == want


def test_create_refuses_without_touching_a_device():
    from serial_draft_head_gb300 import tree, walk
    L = tree.load()
    h = ctypes.c_void_p()
    good = dict(q_heads=4, kv_heads=2, head_dim=64, type=0, max_requests=1, max_nodes=8)
    for bad in (dict(q_heads=3), dict(kv_heads=0), dict(kv_heads=-2), dict(head_dim=0),
                dict(head_dim=68), dict(head_dim=256), dict(type=2), dict(max_requests=0),
                dict(max_requests=1025), dict(max_nodes=0), dict(max_nodes=257)):
        cfg = tree.dspark_tree_config(**{**good, **bad})
        assert L.dspark_tree_create(ctypes.byref(cfg), ctypes.byref(h)) == walk.EINVAL
        assert not h.value
    assert L.dspark_tree_create(None, ctypes.byref(h)) == walk.EINVAL
    assert L.dspark_tree_destroy(None) == walk.EINVAL
    assert L.dspark_tree_status(None, None) == walk.EINVAL
    assert "outside their bounds" in walk.dspark_walk_strerror(walk.EPAGES)


def test_ancestor_bits():
    from serial_draft_head_gb300 import tree
    first = torch.tensor([0, 4, 4, 74], dtype=torch.int32)
    parent = torch.tensor([-1, 0, 0, 1] + [-1] + list(range(69)), dtype=torch.int32)
    m = tree.ancestor_bits(parent, first)
    assert m.dtype == torch.int32 and tuple(m.shape) == (74, 3)
    assert m[:4, 0].tolist() == [1, 3, 5, 11] and (m[:4, 1:] == 0).all()
    for i in range(70):
        bits = [(int(m[4 + i, j // 32]) >> (j % 32)) & 1 for j in range(96)]
        assert bits == [1 if j <= i else 0 for j in range(96)]
    with pytest.raises(ValueError):
        tree.ancestor_bits(torch.tensor([0], dtype=torch.int32), first[:1].new_tensor([0, 1]))


def test_batch_is_packed_as_the_struct_lies():
    from serial_draft_head_gb300 import tree
    b = tree.dspark_tree_batch()
    mem = (ctypes.c_char * ctypes.sizeof(b)).from_buffer(b)
    tree._pack_batch(mem, 0, 11, 12, 13, -14, 15, 16, 17)
    assert (b.pages, b.start, b.first, b.pages_stride, b.max_pages, b.B, b.N) == \
        (11, 12, 13, -14, 15, 16, 17)
