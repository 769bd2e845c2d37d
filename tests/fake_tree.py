"""Calls of the library against tests/fake_cudart.c, in a process of its own: run as
`python fake_tree.py LIBRARY FAKE`, calls as JSON on stdin, results and the runtime calls that each
made as JSON on stdout.  A call is [name, argument, ...]; an argument is a number, {"bytes": hex} (the
address of such bytes), "handle", "out" (where create puts the handle), or null.  The name "device" sets
the current device."""
import ctypes
import json
import sys


def main():
    lib_path, fake_path = sys.argv[1:3]
    fake = ctypes.CDLL(fake_path, mode=ctypes.RTLD_GLOBAL)      # found before the runtime's own
    lib = ctypes.CDLL(lib_path)
    fake.fake_log.restype = ctypes.c_char_p
    handle, keep, results = ctypes.c_void_p(), [], []

    def value(a):
        if isinstance(a, dict):
            keep.append(ctypes.create_string_buffer(bytes.fromhex(a["bytes"])))
            return ctypes.c_void_p(ctypes.addressof(keep[-1]))
        if isinstance(a, float):
            return ctypes.c_float(a)
        if a == "handle":
            return handle
        if a == "out":
            return ctypes.byref(handle)
        return ctypes.c_void_p(a)

    for name, *args in json.load(sys.stdin):
        fake.fake_clear()
        if name == "device":
            rc = fake.cudaSetDevice(args[0])
        else:
            rc = getattr(lib, name)(*[value(a) for a in args])
        results.append([rc, fake.fake_log().decode().splitlines()])
    json.dump(results, sys.stdout)


main()
