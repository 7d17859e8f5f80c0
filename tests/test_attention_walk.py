"""The attention kernels' source, and what runs of it on the host (tests/csrc/attn_probe.cu): the bf16 decode step's walk
over its tiles, and the rules by which variants are chosen, against the times measured on both sides."""
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
    lib.attn_probe_rows.argtypes = [i32] * 9 + [vp]
    lib.attn_probe_rows.restype = None
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


# fp32 prompts: head size, causal, batch, tokens, heads, heads of keys; us forward with blocks of 16 and of 64 rows; us of the
# gradient in one launch, in two with 16 rows, with 64 rows for queries and 16 for keys, with 64; measured on 148 SMs
ROWS = [
    (64, 1, 1, 256, 2, 2, 13.2, 22.5, 29.7, 45.1, None, 74.1),
    (64, 1, 1, 1024, 4, 4, 58.2, 79.8, 160.3, 202.9, None, 271.9),
    (64, 1, 1, 1024, 6, 6, 64.3, 79.7, 233.6, 222.3, None, 271.9),
    (64, 1, 1, 1024, 8, 8, 81.2, 80, 309, 285.9, 278.9, 272.7),
    (64, 1, 1, 8192, 1, 1, 438.4, 612.6, 2197.3, 1538.7, None, 2114.7),
    (64, 1, 8, 256, 4, 4, 28.7, 23.1, 108.1, 95.5, 86.2, 75.7),
    (64, 1, 32, 64, 4, 4, 12.8, 8.7, 51.6, 37.9, 32.2, 26),
    (64, 1, 4, 1024, 4, 4, 137.3, 125.3, 612.9, 479.9, None, 426.4),
    (64, 1, 1, 1024, 8, 2, 82.7, 80.4, 424.3, 476.8, 471.6, 722.8),
    (64, 1, 2, 1024, 16, 2, 245, 199.4, 1195.4, 1255, 1172.4, 1502.3),
    (64, 0, 1, 512, 8, 8, 34, 41.7, 166.3, 111.3, 124, 140.1),
    (64, 0, 1, 1024, 5, 5, 101.4, 80, 376.4, 386.2, 348.8, 271.5),
    (64, 0, 1, 1024, 8, 8, 120.5, 80.1, 588.9, 424, 357.1, 272),
    (64, 0, 1, 1024, 8, 2, 121.1, 80.1, 584.8, 537.1, 475.1, 721),
    (64, 0, 4, 512, 16, 2, 213.7, 142, 1138, 790.2, 713.2, 845.5),
    (64, 0, 1, 64, 64, 64, 7.7, 8.7, 29.6, 20.8, 23.2, 25.5),
    (128, 1, 1, 256, 2, 2, 21.6, 38.3, 36.3, 65.9, None, 130.5),
    (128, 1, 1, 1024, 5, 5, 127, 141.8, 268.4, 397.9, 414.6, 494.7),
    (128, 1, 1, 1024, 8, 8, 178.1, 141.8, 423.2, 557.6, 495.4, 494.9),
    (128, 1, 8, 256, 3, 3, 47.6, 38.7, 114.3, 146.9, None, 131.5),
    (128, 1, 8, 256, 4, 4, 57.6, 38.9, 146.5, 180.4, 146.7, 131.8),
    (128, 1, 32, 64, 4, 4, 25.5, 13.3, 67.9, 78.1, 56.2, 41.2),
    (128, 1, 1, 512, 16, 4, 99.8, 73.2, 260.1, 395.3, 349, 663.6),
    (128, 1, 2, 1024, 5, 5, 212.8, 142.7, 525.3, 668.3, None, 496),
    (128, 0, 1, 512, 8, 8, 79, 72.7, 226.9, 245.3, 233.7, 245.9),
    (128, 0, 2, 512, 6, 6, 117.4, 73.1, 322.2, 366.6, 293.6, 245.8),
    (128, 0, 1, 1024, 8, 8, 303.9, 141.8, 791.7, 950.4, 690.3, 481.8),
    (128, 0, 1, 1024, 8, 2, 304, 142.2, 787.5, 948.9, 688.7, 1265.1),
    (128, 0, 2, 1024, 16, 2, 1057.3, 560.4, 3109.1, 3564.4, 2755.2, 2953.7),
]


@pytest.mark.parametrize("d,causal,B,T,hq,hkv,f16,f64,one,two,mixed,g64", ROWS)
def test_fp32_blocks_take_the_faster_side(probe, d, causal, B, T, hq, hkv, f16, f64, one, two, mixed, g64):
    """Within a tenth of the fastest: a rule on sizes does not know where the last wave of blocks ends."""
    for packed in (0, 1):   # packed sequences of these lengths count as the dense batch
        rows = (ctypes.c_int32 * 4)()
        probe.attn_probe_rows(d, causal, B, T * (B if packed else 1), T * (B if packed else 1), hq, hkv, packed, 148, rows)
        fwd, alone, q, k = rows
        if packed and T < 512:
            continue   # whole tiles here; the rule takes the last tile of a packed sequence for half full
        assert (f16 if fwd == 16 else f64) <= 1.1 * min(f16, f64)
        took = one if alone else {(16, 16): two, (64, 16): mixed, (64, 64): g64}[q, k]
        assert took is None or took <= 1.1 * min(x for x in (one, two, mixed, g64) if x is not None)
