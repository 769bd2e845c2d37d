"""What a handle sets up when it is made, and what over a 4-bit cache when it is first used with one,
against a fake of the CUDA runtime (no GPU)."""
import json
import os
import subprocess
import sys

import pytest

from test_tree_e2m1_host import each, made
from test_tree_host import HERE, create, operators

# the fake, with the kernels that get attributes and the sizes of allocations in its log
FAKE = r"""
#define cudaFuncSetAttribute plain_set_attribute
#define cudaMalloc plain_malloc
#include "%s"
#undef cudaFuncSetAttribute
#undef cudaMalloc
int cudaFuncSetAttribute(const void *f, int attr, int value) {
  (void)attr, (void)value;
  return note("attribute %%p\n", f);
}
int cudaMalloc(void **p, size_t n) { return note("bytes %%zu\n", n), plain_malloc(p, n); }
"""


@pytest.fixture(scope="session")
def calls(tmp_path_factory):
    from serial_draft_head_gb300 import tree, walk
    tree.load()
    at = tmp_path_factory.mktemp("fake_setup")
    (at / "fake.c").write_text(FAKE % os.path.join(HERE, "fake_cudart.c"))
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(at / "fake.so"), str(at / "fake.c")], check=True)

    def run(what):
        res = subprocess.run([sys.executable, os.path.join(HERE, "fake_tree.py"), walk.library_path(), str(at / "fake.so")],
                             input=json.dumps(what), capture_output=True, text=True, timeout=120)
        assert res.returncode == 0, res.stderr
        return json.loads(res.stdout)

    return run


def kernels(log):
    return {line.split()[1] for line in log if line.startswith("attribute")}


def attend(D, B=2, N=8, cap=0.0):
    """An attend call over a 4-bit cache."""
    from serial_draft_head_gb300 import tree
    name, h, cache, _, *rest = each(made(D), D)[3]
    b = tree.dspark_tree_batch(pages=1 << 20, start=1 << 20, first=1 << 20, pages_stride=4, max_pages=4, B=B, N=N)
    rest[-4] = cap
    return [name, h, cache, {"bytes": bytes(b).hex()}] + rest


@pytest.mark.parametrize("D", [128, 64, 32])
@pytest.mark.parametrize("type", [0, 1])
def test_kernels_over_4_bits_are_set_up_when_they_are_used(calls, D, type):
    """Not in a handle's making: those that it sets up then are the ones of 16 bits and e4m3; each of the
    others before its first launch by the handle, once."""
    forms = [attend(D, N=2), attend(D, N=8), attend(D, N=16), attend(D, N=200), attend(D, N=2, cap=5.0)]
    first, *rest = calls([create(head_dim=D, type=type)] + forms + forms + [["dspark_tree_destroy", "handle"]])
    made_with = kernels(first[1])
    assert first[0] == 0 and made_with
    seen = set()
    for i, (rc, log) in enumerate(rest[:-1]):
        assert rc == 0 and any("launch" in line for line in log)
        now = kernels(log)
        assert not now & made_with and not now & seen
        assert bool(now) == (i < len(forms)), i
        seen |= now
    # a call over 16 bits sets nothing up
    plain = operators()[3]
    if type == 0 and D == 64:
        for rc, log in calls([create(head_dim=D), plain, plain, ["dspark_tree_destroy", "handle"]])[1:-1]:
            assert rc == 0 and not kernels(log) and any("launch" in line for line in log)


def test_heads_without_a_4_bit_cache_have_no_room_for_its_parts(calls):
    """Heads that 32 does not divide: their workspace goes by their own rows."""
    def size(D):
        (rc, log), _ = calls([create(head_dim=D, q_heads=2, kv_heads=2, max_nodes=8), ["dspark_tree_destroy", "handle"]])
        assert rc == 0
        return max(int(line.split()[1]) for line in log if line.startswith("bytes"))
    assert size(80) < size(96) == size(128) and size(40) < size(64)
