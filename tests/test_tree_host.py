"""What the tree operators' C calls ask of the CUDA runtime, against a fake of it (no GPU)."""
import json
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="session")
def calls(tmp_path_factory):
    """Runs a list of calls (see fake_tree.py); the results and each call's log."""
    from serial_draft_head_gb300 import tree, walk
    tree.load()
    fake = str(tmp_path_factory.mktemp("fake") / "fake_cudart.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", fake, os.path.join(HERE, "fake_cudart.c")],
                   check=True)

    def run(what):
        res = subprocess.run([sys.executable, os.path.join(HERE, "fake_tree.py"), walk.library_path(), fake],
                             input=json.dumps(what), capture_output=True, text=True, timeout=120)
        assert res.returncode == 0, res.stderr
        return json.loads(res.stdout)

    return run


def create(**kw):
    from serial_draft_head_gb300 import tree
    cfg = tree.dspark_tree_config(**{**dict(q_heads=8, kv_heads=2, head_dim=64, type=0, max_requests=4,
                                            max_nodes=64), **kw})
    return ["dspark_tree_create", {"bytes": bytes(cfg).hex()}, "out"]


def test_create_returns_with_its_memory_cleared(calls):
    """The status word and the counts that kernels on any stream go by are zero before the handle is
    there to be used: what clears them has been waited for, and waits for no work of others."""
    (rc, log), = calls([create()])
    assert rc == 0
    cleared = [i for i, line in enumerate(log) if line.startswith("memset")]
    assert cleared
    for i in cleared:
        stream = log[i].split()[2]
        assert any(line.startswith("synchronise stream %s " % stream) for line in log[i:])
        assert stream != "0" and not any(line.startswith("synchronise all") for line in log)


def operators(B=2, N=8):
    """One call of each operator on a handle of `create()`, over a 16-bit cache."""
    from serial_draft_head_gb300 import tree
    at = 1 << 20                                   # any address: nothing is launched
    cache = tree.dspark_tree_cache(k=at, v=at, n_pages=9, page_size=16, type=0)
    cache.k_stride[:] = cache.v_stride[:] = (16 * 128, 128, 64)
    batch = tree.dspark_tree_batch(pages=at, start=at, first=at, pages_stride=4, max_pages=4, B=B, N=N)
    strides = {"bytes": bytes((tree.ctypes.c_int64 * 2)(512, 64)).hex()}
    c, b = {"bytes": bytes(cache).hex()}, {"bytes": bytes(batch).hex()}
    return [["dspark_tree_write", "handle", c, b, at, strides, at, strides, None],
            ["dspark_tree_read", "handle", c, b, at, at, None],
            ["dspark_tree_keep", "handle", c, b, at, 3, 3, at, None],
            ["dspark_tree_attend", "handle", c, b, at, strides, None, 0, 0, 0.125, 0.0, at, at, None]]


def test_calls_work_on_the_handles_device(calls):
    """Whichever device is current: each call launches on the handle's and leaves the other current."""
    what = operators() + [["dspark_tree_status", "handle", None], ["dspark_tree_destroy", "handle"]]
    for now in (0, 1):
        done = calls([["device", 1], create(), ["device", now]] + what)[3:]
        for (name, *_), (rc, log) in zip(what, done):
            assert rc == 0, name
            work = [line for line in log if " on " in line]
            assert work and all(line.endswith(" on 1") for line in work), (name, log)
            devices = [line for line in log if line.startswith("device")]
            assert devices == ([] if now == 1 else ["device 1", "device 0"]), (name, log)


def test_grids_fit_the_device(calls):
    """Any number of requests and rows: a grid is at most 65,535 wide in its second direction."""
    def launch(what):  # noqa: E306
        (rc, _), (rc2, log), (rc3, _) = calls([create(kv_heads=kv, q_heads=kv), what, ["dspark_tree_destroy", "handle"]])
        assert (rc, rc2, rc3) == (0, 0, 0)
        return [tuple(int(x) for x in line.split()[2:5]) for line in log if line.startswith("launch grid")]
    for B, N in ((70001, 8), (2 ** 31 - 1, 1), (1, 2 ** 31 - 1)):
        for kv in (1, 8, 65535):
            for what in operators(B, N)[:3]:
                for x, y, z in launch(what):
                    assert 1 <= x < 2 ** 31 and 1 <= y <= 65535 and z == 1, (what[0], B, N, kv)
