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
    lib.attn_probe_per_pair.argtypes = [i64, i64, i32, i32, i32]
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


# (pairs, tokens of a full row, head size, bf16, us with a block per pair, us with shares), measured on 148 SMs
MEASURED = [
    (1, 256, 128, 1, 5.03, 7.29), (1, 640, 128, 1, 7.96, 8.55), (1, 1024, 128, 1, 10.76, 9.62), (1, 1024, 64, 1, 9.39, 8.74),
    (4, 512, 128, 1, 6.92, 9.14), (4, 1024, 64, 1, 9.23, 8.70), (8, 2048, 128, 1, 18.29, 12.81), (64, 1024, 128, 1, 11.79, 13.82),
    (64, 1024, 64, 1, 9.84, 11.56), (128, 1024, 128, 1, 14.82, 19.63), (128, 1024, 64, 1, 10.58, 14.99), (144, 1024, 128, 1, 15.83, 20.47),
    (1, 128, 128, 0, 7.02, 9.00), (1, 512, 128, 0, 17.77, 11.41), (1, 1024, 128, 0, 31.93, 13.34), (1, 256, 64, 0, 8.63, 9.26),
    (1, 512, 64, 0, 14.13, 10.02), (1, 1024, 64, 0, 25.27, 11.07), (8, 1024, 128, 0, 32.15, 14.35), (32, 512, 128, 0, 18.32, 14.12),
    (32, 1024, 64, 0, 26.10, 14.52), (64, 256, 128, 0, 11.59, 13.72), (64, 512, 128, 0, 19.00, 17.91), (64, 1024, 64, 0, 28.19, 20.05),
    (128, 512, 128, 0, 20.13, 24.36), (128, 1024, 128, 0, 34.27, 38.40), (128, 1024, 64, 0, 35.82, 31.51), (144, 1024, 128, 0, 34.80, 39.21),
]


@pytest.mark.parametrize("pairs,tokens,d,bf16,alone,shared", MEASURED)
def test_decode_takes_the_faster_side(probe, pairs, tokens, d, bf16, alone, shared):
    assert probe.attn_probe_per_pair(pairs, tokens, d, bf16, 148) == (alone < shared)
