"""Parts of the prompt kernel on the GPU (tests/csrc/attn_probe.cu): its powers on the FMA units, and its failure path,
made to happen without a GPU fault.

Every wait of the kernel on a barrier of its block is bounded, but two softmax warps that share rows also meet at
barriers that are not.  The probe (tests/csrc/attn_probe.cu) runs the kernel with one softmax warp giving up, as if
its wait had run out, at each place where it can; the other warp of the pair may be past that wait.  The kernel must
return with the error recorded, and the next call must be right.
"""
import ctypes
import math
import os
import time

import pytest
import torch

import gated_delta_rule_86_b200 as kda

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(cuda_lib):
    lib = ctypes.CDLL(os.path.join(HERE, "csrc", "libattn_probe.so"))
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.attn_probe_give_up.argtypes = [i32, i32, vp, vp, vp, i32, i32, i32, i32, ctypes.c_float, vp]
    lib.attn_probe_give_up.restype = ctypes.c_int
    return lib


@pytest.mark.parametrize("hq,hkv", [(32, 8), (20, 20)])   # items of two heads, and of two row tiles
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("place", range(3))
def test_a_warp_that_gives_up_ends_the_kernel(probe, place, d, hq, hkv):
    T = 3000   # several items per block
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn((1, T, h, d), generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    want = kda.kda_attn_fwd(q, k, v)
    out = torch.empty_like(q)
    torch.cuda.synchronize()

    def run(quit):
        return probe.attn_probe_give_up(quit, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), 1, T, hq, hkv, d ** -0.5,
                                        out.data_ptr())

    for warp in range(16):
        t0 = time.perf_counter()
        assert run(16 * place + warp) == 4
        assert time.perf_counter() - t0 < 5
    assert run(-1) == 0
    assert torch.equal(out, want)


def test_powers_on_the_fma_units(probe):
    """2^x by the polynomial: its error as a function, 1.55e-7 (scanned in 64 bits), and the roundings of its six steps:
    the last one 2^-24, the one before it times |f| <= 1/2 of a factor of 0.7 and so on, less than 2^-24 together."""
    probe.attn_probe_powers.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32]
    n = 1 << 20
    x = torch.cat((torch.linspace(-1, 1, n, device="cuda"), torch.linspace(-125.9, 126.9, n, device="cuda"),
                   torch.arange(-126, 127, device="cuda").float().repeat(2)))
    y = torch.empty_like(x)
    assert probe.attn_probe_powers(x.data_ptr(), y.data_ptr(), x.numel()) == 0
    want = torch.exp2(x.double())
    assert ((y.double() - want).abs() / want).max().item() <= 1.55e-7 + 2 * 2.0 ** -24
    edge = torch.tensor([-126.0, -127.0, -1e30, -math.inf, math.nan, 0.0], device="cuda")
    y = torch.empty_like(edge)
    assert probe.attn_probe_powers(edge.data_ptr(), y.data_ptr(), edge.numel()) == 0
    assert ((y[:4].double() / 2.0 ** -126 - 1).abs() <= 2.0 ** -22).all()   # stays where it is below -126
    assert torch.isinf(y[4].bfloat16()) and abs(y[5].item() - 1) <= 2.0 ** -22
