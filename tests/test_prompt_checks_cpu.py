"""Refusals of the prompt path's C entries that need numbers at the ends of their types (CPU only)."""
import ctypes

import pytest

import linear_attention_serving_chunkwise_gb300 as kda
from linear_attention_serving_chunkwise_gb300.build import build

BAD = kda.KDA_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return kda.load()


@pytest.mark.parametrize("dtype", [kda.KDA_BF16, kda.KDA_F32])
def test_chunk_attention_refuses_scales_whose_powers_of_two_overflow(lib, dtype):
    """Scores are kept in powers of two: scale / ln 2 has to be finite as well."""
    desc = lambda scale: kda.make_chunk_attention_desc(2, 40, 8, 2, 128, dtype, 10, 16, 5, scale, 16 * 2 * 128, 16 * 2 * 128)
    at = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(8)]
    for scale in (2.0 ** 126, -2.0 ** 126, 1e-45, 0.0):
        assert kda.chunk_attention_workspace_bytes(desc(scale)) > 0
        assert lib.kda_chunk_attention(ctypes.byref(desc(scale)), *at, 0, None) == kda.KDA_ERR_WORKSPACE
    for scale in (3e38, -3e38, 2.0 ** 127, float("inf"), float("nan")):
        assert kda.chunk_attention_workspace_bytes(desc(scale)) == 0
        assert lib.kda_chunk_attention(ctypes.byref(desc(scale)), *at, 1 << 40, None) == BAD
