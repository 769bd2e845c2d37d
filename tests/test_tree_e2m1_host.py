"""What the tree operators' C calls take and refuse of 4-bit caches and rotations, against a fake of
the CUDA runtime (no GPU)."""
import pytest

from test_tree_host import calls, create  # noqa: F401

AT = 1 << 20                                       # any address: nothing is launched


def made(D=128, **kw):
    """A 4-bit cache of two heads as its struct's bytes."""
    from serial_draft_head_gb300 import tree
    f = dict(k=AT, v=AT, k_scale=AT, v_scale=AT, n_pages=9, page_size=16, type=3, row=D // 2, scale=D // 16)
    f.update(kw)
    c = tree.dspark_tree_cache(**{n: f[n] for n in ("k", "v", "k_scale", "v_scale", "n_pages", "page_size", "type")})
    c.k_stride[:] = c.v_stride[:] = (32 * f["row"], 2 * f["row"], f["row"])
    c.k_scale_stride[:] = c.v_scale_stride[:] = (32 * f["scale"], 2 * f["scale"], f["scale"])
    return {"bytes": bytes(c).hex()}


def each(cache, D):
    """A call of each operator that takes a cache."""
    from serial_draft_head_gb300 import tree
    b = {"bytes": bytes(tree.dspark_tree_batch(pages=AT, start=AT, first=AT, pages_stride=4, max_pages=4, B=2, N=8)).hex()}
    st = {"bytes": bytes((tree.ctypes.c_int64 * 2)(8 * D, D)).hex()}
    r = {"bytes": bytes(tree.dspark_tree_rotation(turns=AT, eps=1e-6, rotary_dim=D // 2 // 16 * 16)).hex()}
    return [["dspark_tree_write", "handle", cache, b, AT, st, AT, st, None],
            ["dspark_tree_read", "handle", cache, b, AT, AT, None],
            ["dspark_tree_keep", "handle", cache, b, AT, 3, 3, AT, None],
            ["dspark_tree_attend", "handle", cache, b, AT, st, None, 0, 0, 0.125, 0.0, AT, AT, None],
            ["dspark_tree_place", "handle", cache, AT, r, AT, 8, AT, st, AT, st, AT, st, AT, None]]


@pytest.mark.parametrize("D,kw,rc", [
    (128, {}, 0), (64, {}, 0), (96, {}, 0), (32, {}, 0),
    (80, {}, -1), (48, {}, -1),                             # heads that are no multiple of 32
    (128, dict(k_scale=None), -1), (128, dict(v_scale=None), -1),
    (128, dict(k=AT + 8), -1), (128, dict(row=72), -1),     # rows off 16 bytes
    (128, dict(k_scale=AT + 4), -1), (128, dict(scale=12), -1),     # scales off 8, 4, 2 bytes
    (64, dict(v_scale=AT + 2), -1), (64, dict(scale=6), -1), (64, dict(scale=12), 0),
    (96, dict(k_scale=AT + 1), -1), (96, dict(scale=8), 0), (96, dict(scale=7), -1),
    (128, dict(type=4), -1), (128, dict(page_size=0), -1), (128, dict(n_pages=0), -1)])
def test_cache_of_4_bits(calls, D, kw, rc):  # noqa: F811
    what = each(made(D, **kw), D)
    done = calls([create(head_dim=D)] + what + [["dspark_tree_destroy", "handle"]])
    assert done[0][0] == 0
    for (name, *_), (got, log) in zip(what, done[1:-1]):
        assert (got == 0) == (rc == 0), name
        assert any("launch" in line for line in log) == (rc == 0), name


def test_rotations(calls):  # noqa: F811
    from serial_draft_head_gb300 import tree
    st = {"bytes": bytes((tree.ctypes.c_int64 * 2)(512, 64)).hex()}
    odd = {"bytes": bytes((tree.ctypes.c_int64 * 2)(512, 60)).hex()}

    def rotate(r=None, at=AT, N=8, q=AT, sq=st, k=AT, sk=st, oq=AT, ok=AT, **kw):
        f = {**dict(turns=AT, q_norm=AT, k_norm=AT, eps=1e-6, rotary_dim=64, interleaved=0), **kw}
        r = {"bytes": bytes(tree.dspark_tree_rotation(**f)).hex()}
        return ["dspark_tree_rotate", "handle", r, at, N, q, sq, k, sk, oq, ok, None]

    good = [rotate(), rotate(q_norm=None), rotate(rotary_dim=0, turns=None), rotate(rotary_dim=16), rotate(interleaved=1)]
    bad = [rotate(rotary_dim=80), rotate(rotary_dim=-16), rotate(rotary_dim=8), rotate(turns=None), rotate(eps=-1.0),
           rotate(eps=float("nan")), rotate(q_norm=AT + 4), rotate(k_norm=AT + 8), rotate(N=-1), rotate(at=None),
           rotate(q=None), rotate(k=None), rotate(q=AT + 2), rotate(sq=odd), rotate(sk=None), rotate(oq=None),
           rotate(ok=AT + 8)]
    done = calls([create()] + good + bad + [rotate(N=0), ["dspark_tree_destroy", "handle"]])
    assert [rc for rc, _ in done[1:1 + len(good)]] == [0] * len(good)
    assert all(any("launch" in line for line in log) for _, log in done[1:1 + len(good)])
    assert all(rc != 0 and not any("launch" in line for line in log) for rc, log in done[1 + len(good):-2])
    assert done[-2][0] == 0 and not any("launch" in line for line in done[-2][1])     # no rows: nothing to do
    # heads of a size that 16 does not divide are not rotated
    (rc, _), (rc2, _), _ = calls([create(head_dim=40), rotate(rotary_dim=16), ["dspark_tree_destroy", "handle"]])
    assert rc == 0 and rc2 != 0
    # a cache of more slots than an int32 holds has no slot numbers
    big = made(64, n_pages=1 << 28)
    r = {"bytes": bytes(tree.dspark_tree_rotation(turns=AT, eps=0.0, rotary_dim=64)).hex()}
    (rc, _), (rc2, _), _ = calls([create(), ["dspark_tree_place", "handle", big, AT, r, AT, 8, AT, st, AT, st, AT, st,
                                             AT, None], ["dspark_tree_destroy", "handle"]])
    assert rc == 0 and rc2 != 0


@pytest.mark.parametrize("struct", ["dspark_tree_rotation"])
def test_struct_matches_the_header(struct):
    import ctypes
    import os
    import re
    from serial_draft_head_gb300 import tree
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dspark_tree.h")
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    body = re.search(r"struct %s \{(.*?)\};" % struct, text, flags=re.S).group(1)
    want = [(re.sub(r".*\W", "", x.strip()), 8 if "*" in x else 4) for x in body.split(";") if x.strip()]
    assert [(n, ctypes.sizeof(t)) for n, t in getattr(tree, struct)._fields_] == want


def test_frequencies_become_turns():
    """The turns of a position, as fractions of 2^64, to the last bit: against sines of far positions."""
    import math
    from fractions import Fraction
    from serial_draft_head_gb300 import tree
    # pi by Machin's formula, in integers
    one = 10 ** 60

    def arctan_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    pi = Fraction(4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)
    assert abs(tree._TURN * 2 * pi - 1) < Fraction(1, 2 ** 150)
    for f in (1.0, 1e-4, 0.7943, -0.25, 123.5):
        turns = round((Fraction(f) * tree._TURN % 1) * 2 ** 64) % 2 ** 64
        assert tree._turns(f) == turns
        for pos in (1, 131071, 2 ** 31 - 1, -5):
            x = (pos * turns) % 2 ** 64 / 2 ** 64
            want = Fraction(f) * pos / (2 * pi) % 1
            d = abs(Fraction(x) - want)
            assert min(d, 1 - d) < 2.0 ** -31, (f, pos)
            assert math.isfinite(x)
