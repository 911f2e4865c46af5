"""Which kernel an 8-bit integer product is given (no GPU: the query of the measurement
library launches nothing, and counts 256 compute units where there is none)."""

import ctypes
import os
import random

import pytest

import fp8_quantized_gemm_amd as bsq

CEILING = os.path.join(bsq._PKG, "libbsq_ceiling.so")
pytestmark = pytest.mark.skipif(not (os.path.exists(CEILING) and os.path.exists(bsq.LIB_PATH)), reason="libraries not built")

DIRECT16, DIRECT64, RING128, RING192, RING256, RING128X5, RING64, RING96 = range(8)
A, S, B, T, C = (0x1000000 * i for i in range(1, 6))         # aligned addresses, never dereferenced


@pytest.fixture(scope="module")
def choose():
    bsq.lib()
    L = ctypes.CDLL(CEILING)
    P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    L.bsq_int8_on.argtypes = [I, I, I, I64, I64, I64, P, P, P, P, P, P, I64, P]
    return lambda M, N, K, a=A, b=B: L.bsq_int8_on(-1, -1, 0, M, N, K, a, S, b, T, None, C, N, None)


def test_operands_off_16_bytes_take_the_direct_kernel(choose):
    for K in (1, 8, 15, 17, 4095, 4099, 8200):
        for M, N in ((1, 1), (1, 4096), (200, 300), (8192, 14336)):
            assert choose(M, N, K) in (DIRECT16, DIRECT64), (M, N, K)
    for a, b in ((A + 8, B), (A, B + 8), (A + 1, B + 1)):
        assert choose(4096, 4096, 4096, a, b) in (DIRECT16, DIRECT64)
    assert choose(4096, 4096, 4096) not in (DIRECT16, DIRECT64)
    assert choose(5, 7, 0) in (DIRECT16, DIRECT64)           # nothing to reduce


def test_every_choice_is_a_kernel_that_takes_the_operands(choose):
    rng = random.Random(0)
    seen = set()
    for _ in range(3000):
        M, N = (round(2 ** rng.uniform(0, 15)) for _ in "MN")
        K = round(2 ** rng.uniform(4, 16.9))
        K = K // 16 * 16 if rng.random() < 0.7 else K
        k = choose(M, N, K)
        assert 0 <= k < 8 and (K % 16 == 0 or k in (DIRECT16, DIRECT64)), (M, N, K, k)
        seen.add(k)
    assert seen == set(range(8)), seen                       # none that no call reaches


def test_ends_of_the_range(choose):
    assert choose(16384, 28672, 4096) == RING256             # many rounds of the largest tile
    assert choose(128, 2048, 2048) in (RING64, RING96)       # fewer tiles of 128 than compute units
