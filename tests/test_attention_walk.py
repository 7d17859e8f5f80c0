"""The attention kernels' source, and the bf16 decode step's walk over its tiles, run on the host from it
(tests/csrc/attn_probe.cu)."""
import ctypes
import glob
import os

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
TILE, WARPS, PAIR_COST = 128, 8, 2
MARKER = 0x5eadbeef


@pytest.fixture(scope="module")
def probe():
    from gated_delta_rule_86_b200 import build
    build.build_probe()
    lib = ctypes.CDLL(os.path.join(HERE, "csrc", "libattn_probe.so"))
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.attn_probe_walk.argtypes = [vp, i32, i32, vp, i64, i32, i32, i32, i32, i64, i32, i32]
    lib.attn_probe_walk.restype = i64
    return lib


@pytest.mark.parametrize("lens,page_log2,vheads", [([333], 4, 4), ([1], 0, 1), ([128], 6, 2), ([129, 0, 500], 4, 3),
                                                   ([40, 257, 0, 0], 5, 1), ([700, 128, 3], 7, 2), ([5000], 0, 1)])
@pytest.mark.parametrize("gap", [0, 3])
def test_pages_are_looked_up_inside_the_table(probe, lens, page_log2, vheads, gap):
    """No entry behind a row or behind the last row is read: all of them hold a marker that never comes back."""
    size, n = 1 << page_log2, len(lens)
    width = max(-(-x // size) for x in lens)
    memory = torch.full((n + 2, width + gap), MARKER, dtype=torch.int32)
    for b, x in enumerate(lens):
        memory[b, : -(-x // size)] = 7
    seq = torch.tensor(lens, dtype=torch.int32)
    tiles = [-(-x // TILE) for x in lens]
    line = sum((t + PAIR_COST) * vheads for t in tiles if t)

    def hits(b, vh, count, warp):
        return probe.attn_probe_walk(seq.data_ptr(), n, vheads, memory.data_ptr(), width + gap, width, page_log2, b, vh, count,
                                     warp, MARKER)

    first = next(b for b, t in enumerate(tiles) if t)
    for warp in range(WARPS):
        for b, t in enumerate(tiles):   # a block with a pair of its own
            for vh in range(vheads):
                assert hits(b, vh, t, warp) == 0
        for count in range(1, line + 1):   # shares of every length from the line's begin on
            assert hits(first, 0, count, warp) == 0


def test_no_loads_that_promise_constant_data():
    """The kernels come up while their inputs' writers still run, so none of their loads may be a non-coherent one."""
    files = glob.glob(os.path.join(os.path.dirname(HERE), "gated_delta_rule_86_b200", "csrc", "attn_*.cuh"))
    assert len(files) >= 8
    for path in files:
        code = "\n".join(line.split("//")[0] for line in open(path).read().splitlines())
        assert "__ldg" not in code and "global.nc" not in code, path
