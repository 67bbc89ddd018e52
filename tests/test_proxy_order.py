"""Shared memory that a ranking of sequences has used is written by page copies next, which go by another proxy."""
import os
import re

import pytest

from paged_kv_cache_193_gb300 import build
from test_dependent_loads import _code


def _body(source, name):
    """The code of the function of that name, from its opening brace to the one that closes it."""
    at = source.index("{", re.search(r"\b%s\([^;{]*\)\s*\{" % name, source).start())
    depth = 0
    for i in range(at, len(source)):
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        if depth == 0:
            return source[at:i]
    raise AssertionError(name)


@pytest.mark.parametrize("name,function,words", [("pa_sparse_attend.cuh", "longest_row", ["len"]),
                                                 ("pa_rows.cu", "longest_unit", ["len", "order", "start"])])
def test_a_ranking_is_fenced_from_the_copies_behind_it(name, function, words):
    """A barrier orders the threads' loads and stores among themselves, not before what a copy writes to the same bytes:
    behind its last access every thread fences, and then meets the others."""
    body = _body(_code(os.path.join(build.CSRC, name)), function)
    fence = body.rindex("fence_proxy_async_smem()")
    barrier = body.rindex("__syncthreads()")
    assert max(m.start() for w in words for m in re.finditer(r"\b%s\[" % w, body)) < fence < barrier
