"""Answers of the allocator's calls on shared pages where the pool or the host's memory is full."""
import subprocess
import sys

import numpy as np
import pytest


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_180_gb300 import build
    build.build()
    import paged_kv_cache_180_gb300 as p
    return p


@pytest.mark.parametrize("layers", [1, 2])
@pytest.mark.parametrize("tokens", [40, 33, 32, 16, 1])
def test_a_fork_without_room_is_answered_as_an_admission(pkv, layers, tokens):
    # every page is assigned: whether or not a partly filled last page would have to be copied, the answer is the credits'
    a = pkv.Allocator(3 * layers, layers, 16, 256, 3)
    assert a.admit(0, 40, 8)[0] == a.OK                    # 47 tokens: three pages a layer, all of the pool
    for layer in range(layers):
        for block in range(3):
            a.page(0, layer, block)
    assert a.state() == (0, 3 * layers)
    before = a.block_tables()
    for new, want in ((1, a.NO_CREDIT), (8, a.NO_CREDIT), (100, a.EXCEEDS_POOL)):
        assert a.admit(1, tokens, new)[0] == want
        rc, src, dst = a.fork(0, 1, tokens, new)
        assert rc == want and len(src) == len(dst) == 0, (tokens, new)
    assert np.array_equal(a.block_tables(), before) and a.state() == (0, 3 * layers)
    a.free_seq(0)
    assert a.admit(1, tokens, 1)[0] == a.OK                # the refused forks hold nothing


_COMPACT_WITHOUT_MEMORY = """
import ctypes, resource, sys
lib = ctypes.CDLL(sys.argv[1])
I, P = ctypes.c_int, ctypes.c_void_p
lib.pkv_alloc_create.argtypes = [I, I, I, I, I, P, ctypes.POINTER(P)]
lib.pkv_alloc_compact.argtypes = [P, P, P, I, ctypes.POINTER(ctypes.c_int32)]
lib.pkv_alloc_admit.argtypes = [P, I, I, I, P]
lib.pkv_alloc_page.argtypes = [P, I, I, I, P]
lib.pkv_alloc_page_refs.argtypes = [P, I]
pages, h, n = 1 << 24, P(), ctypes.c_int32(0)
assert lib.pkv_alloc_create(pages, 1, 16, 64, 2, None, ctypes.byref(h)) == 0
got = ctypes.c_int32(0)
assert lib.pkv_alloc_admit(h, 0, 40, 1, None) == 0
for b in range(3):
    assert lib.pkv_alloc_page(h, 0, 0, b, ctypes.byref(got)) == 0 and got.value == pages - 1 - b
src, dst = (I * 3)(), (I * 3)()
now = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (now + (8 << 20), now + (8 << 20)))
rc = lib.pkv_alloc_compact(h, src, dst, 3, ctypes.byref(n))
assert rc == 0 and n.value == 3, rc
assert sorted(zip(src, dst)) == [(pages - 3, 0), (pages - 2, 1), (pages - 1, 2)]
assert [lib.pkv_alloc_page_refs(h, p) for p in (0, 1, 2, 3, pages - 3, pages - 1)] == [1, 1, 1, 0, 0, 0]
print("ok")
"""


def test_compact_asks_for_no_memory(pkv):
    # a pool of 2^24 pages and 8 MiB of address space left: PKV_ERR_SHAPE stands for a capacity that is too small only
    r = subprocess.run([sys.executable, "-c", _COMPACT_WITHOUT_MEMORY, pkv.binding.LIB_PATH], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
