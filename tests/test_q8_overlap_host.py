"""Outputs laid over inputs of the 8-bit cache's calls are refused on the host, except where a call can work in place."""
import ctypes

import pytest

from hybrid_head_sparse_decode_b200 import _native as N
from test_q8_host import FAKE, cache, lib, shape, tokens  # noqa: F401  (lib: the fixture)

Q = FAKE + (1 << 24)          # 2 x 8 x 128 bf16: 4096 bytes


@pytest.mark.parametrize("shift", [0, 16, -16, 4080, -4080])
def test_out_over_q(lib, shift):  # noqa: F811
    s, c = shape(), cache()
    sparse = (ctypes.c_uint8 * 8)()
    assert lib.lychee_decode_attn_q8(s, Q, c, FAKE, Q + shift, FAKE, 1 << 40, None, None) == N.ERR_INVALID_ARG
    assert lib.lychee_hybrid_decode_attn_q8(s, 8, 0, Q, c, FAKE, None, sparse, FAKE, Q + shift, FAKE + (1 << 28), FAKE, 1 << 40,
                                            None, None) == N.ERR_INVALID_ARG


@pytest.mark.parametrize("shift", [4, -4, 508, -508])
def test_sets_over_sets(lib, shift):  # noqa: F811
    sparse = (ctypes.c_uint8 * 8)()
    assert lib.lychee_hybrid_decode_attn_q8(shape(), 8, 0, Q, cache(), FAKE, None, sparse, Q + (1 << 24), Q + 8192,
                                            Q + (1 << 24) + shift, FAKE, 1 << 40, None, None) == N.ERR_INVALID_ARG


# one projection's output [T = 2, 8 + 2 + 2, 64] bf16: rows of 768 elements, 512 of them q's
@pytest.mark.parametrize("at,stride", [(0, 768), (16, 512), (-16, 512), (1024, 768), (1280, 768), (1536, 768), (-2032, 768),
                                       (2544, 768)])
def test_rotated_queries_over_rows(lib, at, stride):  # noqa: F811
    k = Q + 1024 if stride == 768 else Q + (1 << 20)
    t = tokens(q=Q, q_out=Q + at, q_stride=stride, k=k, v=k + 256, k_stride=768, v_stride=768, rot=64)
    assert lib.lychee_append_rope_q8(shape(d=64), cache(), t, FAKE, None, None) == N.ERR_INVALID_ARG
