"""The windowed attention's work items (csrc/attn_plan.cuh), run on the host: a block's threads as threads.

Whatever the offsets, the list holds only items that were written, inside the batch, and no more
than it has room for; where the items are found from the offsets, no block has a second one."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from tests._util import ROOT

UNWRITTEN = -7777


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    tmp = tmp_path_factory.mktemp("plan")
    with open(os.path.join(ROOT, "transformer_esm_layer_gb300", "csrc", "attn_plan.cuh")) as f:
        text = re.sub(r"^#(include|pragma once).*$", "", f.read(), flags=re.M)
    (tmp / "attn_plan.inc").write_text(text)
    so = str(tmp / "plan.so")
    subprocess.run([gxx, "-std=c++20", "-O1", "-fwrapv", "-shared", "-fPIC", "-pthread", "-w",
                    f'-DATTN_PLAN_SOURCE="{tmp}/attn_plan.inc"', os.path.join(ROOT, "tests", "host_plan.cpp"), "-o", so],
                   check=True)
    return ctypes.CDLL(so)


def _offsets(cu):
    return np.asarray(cu, dtype=np.int32)


def _ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def _max_items(T, B):
    return (T + 127) // 128 + B


def _find(host, cu, T, heads, max_seqlen=65536):
    """The item count and every block's item where the kernel finds its items itself."""
    cu, B = _offsets(cu), len(cu) - 1
    grid = _max_items(T, B) * heads
    err = ctypes.c_uint(0)
    item = np.zeros(5, np.int32)
    out = []
    for it in range(grid):
        n = host.host_find_item(_ptr(cu), B, T, max_seqlen, 65536, heads, grid, it, _ptr(item), ctypes.byref(err))
        if it < n:
            out.append(tuple(int(v) for v in item))
    return grid, n, out, err.value


def _in_batch(row, rows, key, keys, T):
    return 0 <= row and 1 <= rows <= 128 and row + rows <= T and 0 <= key <= row and row + rows <= key + keys <= T


MALFORMED = [(1024, [0, 1024, 0, 1024]), (1024, [0, 1024, 0, 1024, 0, 1024, 0, 1024]), (400, [0, 300, 200, 400]),
             (400, [5, 400]), (400, [-3, 100, 400]), (400, [0, 500, 400]), (300, [0, -2 ** 31, 2 ** 31 - 1, 300])]


@pytest.mark.parametrize("T,cu", MALFORMED)
def test_items_from_malformed_offsets_stay_one_per_block(host, T, cu):
    grid, n, items, err = _find(host, cu, T, 4)
    assert err
    assert n <= grid
    for row, rows, key, keys, h in items:
        assert _in_batch(row, rows, key, keys, T) and 0 <= h < 4


@pytest.mark.parametrize("lengths", [[180], [0, 1, 127, 128, 129, 300, 2, 0, 515], [7] * 32])
@pytest.mark.parametrize("heads", [1, 4, 20])
def test_items_from_offsets_cover_the_batch_once(host, lengths, heads):
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T = int(cu[-1])
    _, n, items, err = _find(host, cu, T, heads)
    assert not err and n == len(items) == heads * sum(-(-L // 128) for L in lengths)
    seen = np.zeros((heads, T), int)
    for row, rows, key, keys, h in items:
        assert _in_batch(row, rows, key, keys, T)
        seen[h, row:row + rows] += 1
    assert np.all(seen == 1)


def _plan(host, cu, T, window=(20, 20, 3), backward=False, sort_above=0, max_seqlen=65536):
    """The listed items, and the room behind the list."""
    cu, B = _offsets(cu), len(cu) - 1
    room = _max_items(T, B)
    work = np.full((room + 64, 4), UNWRITTEN, np.int32)
    err = ctypes.c_uint(0)
    n = host.host_attn_plan(_ptr(cu), B, T, max_seqlen, 65536, room, *window, int(backward), sort_above,
                            _ptr(work[32:]), ctypes.byref(err))
    assert np.all(work[:32] == UNWRITTEN) and np.all(work[32 + room:] == UNWRITTEN)
    return work[32:32 + room], n, err.value


@pytest.mark.parametrize("T,cu", MALFORMED + [(2048, [0, 2048] * 4), (2048, [0, 2048] * 200)])
@pytest.mark.parametrize("sort_above", [0, 7, 15, 37, 10 ** 6])
@pytest.mark.parametrize("window,backward", [((20, 20, 3), False), ((-1, 0, 0), False), ((-1, 0, 0), True)])
def test_listed_items_of_malformed_offsets_were_written(host, T, cu, sort_above, window, backward):
    """Also where the batch has room for fewer items than are sorted, and its offsets hold more."""
    work, n, err = _plan(host, cu, T, window, backward, sort_above)
    assert err
    assert 0 <= n <= len(work)
    for row, rows, key, keys in work[:n]:
        assert _in_batch(row, rows, key, keys, T), (row, rows, key, keys)


@pytest.mark.parametrize("lengths", [[180], [0, 1, 127, 128, 129, 300, 2, 0, 515], [7] * 300, [0] * 256 + [2000, 5]])
@pytest.mark.parametrize("sort_above", [0, 3, 10 ** 6])
def test_listed_items_cover_the_batch_once(host, lengths, sort_above):
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T = int(cu[-1])
    work, n, err = _plan(host, cu, T, window=(200, 0, 1), sort_above=sort_above)
    assert not err and n == sum(-(-L // 128) for L in lengths)
    seen = np.zeros(T, int)
    for row, rows, key, keys in work[:n]:
        assert _in_batch(row, rows, key, keys, T)
        seen[row:row + rows] += 1
    assert np.all(seen == 1)
