"""How the four warps of a decode CTA leave its chunk loop when a wait runs out (csrc/kvq3_stop.h), explored on the
CPU: every interleaving of four warps over a few chunks, each wait succeeding or running out on its own.  In no state
may warps wait at a barrier that another has left for good, and all leave at the same chunk (the drain and the merge
behind the loop count on that)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hadamard_rotated_bit_kvq3_gb300", "csrc")
WARPS, CHUNKS = 4, 3


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """(mark of a chunk, whether a mark stops at a chunk) of the kernel's own header, compiled for the host."""
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("stop")
    src, lib = str(at / "stop.cpp"), str(at / "stop.so")
    with open(src, "w") as f:
        f.write('#include "kvq3_stop.h"\n'
                'extern "C" unsigned mark_of(long long i) { return kvq3::stop_mark(i); }\n'
                'extern "C" int stops(unsigned m, long long i) { return kvq3::stops_at(m, i); }\n'
                'extern "C" unsigned none() { return kvq3::kNoStop; }\n')
    subprocess.run([cc, "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    dll = ctypes.CDLL(lib)
    dll.mark_of.argtypes, dll.mark_of.restype = [ctypes.c_longlong], ctypes.c_uint
    dll.stops.argtypes, dll.stops.restype = [ctypes.c_uint, ctypes.c_longlong], ctypes.c_int
    dll.none.restype = ctypes.c_uint
    return dll.none(), dll.mark_of, lambda m, i: bool(dll.stops(m, i))


def stuck_states(none, mark_of, stops):
    """End states of the exploration that are not `all done` or `all left at one chunk`.  A warp is (chunk, step):
    about to wait, at the barrier, about to read the mark, gone; (CHUNKS, wait) is past the last chunk."""
    WAIT, BARRIER, READ, GONE = range(4)
    start = (tuple((0, WAIT) for _ in range(WARPS)), none)
    seen, todo, bad = {start}, [start], []
    while todo:
        warps, mark = todo.pop()
        nexts = []
        if all(s == BARRIER for _, s in warps):
            nexts.append((tuple((c, READ) for c, _ in warps), mark))
        for w, (c, s) in enumerate(warps):
            def to(x, m=mark):
                nexts.append((tuple(sorted(warps[:w] + (x,) + warps[w + 1:])), m))   # warps are alike
            if s == WAIT and c < CHUNKS:
                to((c, BARRIER))                   # the copy arrived
                to((c, BARRIER), mark_of(c))       # its wait ran out
            elif s == READ:
                to((c, GONE) if stops(mark, c) else (c + 1, WAIT))
        if not nexts:
            done = all(x == (CHUNKS, WAIT) for x in warps)
            left = all(s == GONE for _, s in warps) and len({c for c, _ in warps}) == 1
            if not (done or left):
                bad.append(warps)
        for n in nexts:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return bad


def test_all_warps_leave_at_the_same_chunk(rule):
    assert stuck_states(*rule) == []


def test_a_mark_without_its_chunk_strands_warps():
    # the exploration finds what the rule is there for: a plain flag leaves warps at a barrier
    assert stuck_states(0, lambda i: 1, lambda m, i: m != 0)


def test_the_first_and_far_chunks(rule):
    none, mark_of, stops = rule
    for i in (0, 1, 2, 7, 1 << 20, (1 << 31) - 1, (1 << 32) - 3):
        assert mark_of(i) != none and stops(mark_of(i), i)
        assert not stops(none, i) and not stops(mark_of(i + 1), i) and not stops(mark_of(i), i + 1)


def test_the_decode_loop_takes_the_rule():
    src = open(os.path.join(CSRC, "kvq3_decode.cuh")).read()
    assert "*abort_s = stop_mark(i);" in src and "if (stops_at(*abort_s, i)) {" in src
    assert src.count("*abort_s") == 3 and src.count("*abort_s = kNoStop;") == 1
