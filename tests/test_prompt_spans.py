"""Slot ranges of prompt attention's key tiles (csrc/span.h), compiled for the host with
signed overflow trapping, against the same ranges in unbounded integers: rows whose
16-byte chunks number 2^31 and more, up to the longest row the kernels take."""
import ctypes
import subprocess

import pytest

from kv_cache_compression_calib_b200 import build

LONGEST = 0x7fffff00  # slots


@pytest.fixture(scope="module")
def span(tmp_path_factory):
    d = tmp_path_factory.mktemp("span")
    (d / "span.cc").write_text(
        '#include "span.h"\nextern "C" int span(int beg, int tiles, int bn, int seen, long long there, int *start) {\n'
        "    const tri::Span s = tri::unseen_span(beg, tiles, bn, seen, there);\n    *start = s.start;\n    return s.count;\n}\n")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-fsanitize=signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", build.CSRC, "-o", str(d / "span.so"), str(d / "span.cc")],
                   check=True)
    f = ctypes.CDLL(str(d / "span.so")).span
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_longlong, ctypes.POINTER(ctypes.c_int)]

    def call(*a):
        at = ctypes.c_int()
        return f(*a, ctypes.byref(at)), at.value

    return call


@pytest.mark.parametrize("d,bn", [(64, 128), (128, 128), (256, 64)])
@pytest.mark.parametrize("tokens", [1, 3, 256])
@pytest.mark.parametrize("paged", [True, False])
def test_spans_of_long_rows(span, d, bn, tokens, paged):
    chunks = d // 8  # of 16 bytes in a bf16 record
    for slots in (tokens, 1000, (1 << 31) // chunks - 1, (1 << 31) // chunks, (1 << 31) // chunks + 77, 1 << 30, LONGEST):
        tiles, seen = (slots + bn - 1) // bn, slots - tokens + 1
        there = (slots + bn - 1) // bn * bn if paged else slots + 1 + 10 ** 12
        for splits in (1, 2, 148):
            covered = []
            for s in range(splits):
                beg, end = tiles * s // splits, tiles * (s + 1) // splits
                count, start = span(beg, end - beg, bn, seen, there)
                want = range(max(beg * bn, seen), min(end * bn, there))
                assert count == len(want) and 0 <= count * chunks <= (256 + bn) * chunks
                if count:
                    assert start == want.start
                    covered.append((start, start + count))
            stop = min(tiles * bn, there)
            assert ((covered[0][0], covered[-1][1]) == (seen, stop)) if seen < stop else not covered
            assert all(a[1] == b[0] for a, b in zip(covered, covered[1:]))


def test_spans_of_nothing(span):
    assert span(5, 0, 128, 0x7fffffff, 4096)[0] == 0  # no key tile
    assert span(0, 3, 128, 384, 384)[0] == 0  # every row sees every slot
    assert span(2, 1, 128, -7, 200)[0] == 0 and span(0, 1, 128, -7, 200) == (128, 0)  # tokens without a slot
    assert span(3, 2, 64, 250, 260) == (10, 250)
