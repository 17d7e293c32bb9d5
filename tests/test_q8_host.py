"""What the 8-bit paged cache's calls refuse on the host, before anything is launched (so it needs no
GPU), and the references of their GPU tests checked against themselves."""
import ctypes

import pytest
import torch

import q8_ref as R
from hybrid_head_sparse_decode_b200 import build, ops
from hybrid_head_sparse_decode_b200 import _native as N

FAKE = 0x10000   # never dereferenced: every call below ends on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.load()


def shape(**kw):
    f = dict(B=2, Hq=8, Hkv=2, d=128, page=64, num_pages=10, max_pages=4, dtype=N.BF16, code=N.E4M3)
    f.update(kw)
    return N.Q8Shape(*(f[n] for n, _ in N.Q8Shape._fields_))


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE)
    f.update(kw)
    return N.Q8CachePtrs(*(f[n] for n, _ in N.Q8CachePtrs._fields_))


BAD = [(dict(B=0), N.ERR_INVALID_ARG), (dict(Hkv=0), N.ERR_INVALID_ARG), (dict(page=0), N.ERR_INVALID_ARG),
       (dict(num_pages=0), N.ERR_INVALID_ARG), (dict(max_pages=0), N.ERR_INVALID_ARG), (dict(dtype=2), N.ERR_INVALID_ARG),
       (dict(code=2), N.ERR_INVALID_ARG), (dict(Hq=9), N.ERR_INVALID_ARG), (dict(Hq=6), N.ERR_UNSUPPORTED),
       (dict(Hq=32), N.ERR_UNSUPPORTED), (dict(Hq=256, Hkv=64), N.ERR_UNSUPPORTED), (dict(d=96), N.ERR_UNSUPPORTED),
       (dict(d=256), N.ERR_UNSUPPORTED), (dict(page=8), N.ERR_UNSUPPORTED), (dict(page=48), N.ERR_UNSUPPORTED),
       (dict(page=256), N.ERR_UNSUPPORTED), (dict(max_pages=(1 << 18) + 1), N.ERR_UNSUPPORTED),
       (dict(num_pages=1 << 24), N.ERR_UNSUPPORTED), (dict(B=1 << 22), N.ERR_UNSUPPORTED),
       (dict(B=1 << 17, max_pages=1 << 18), N.ERR_UNSUPPORTED)]


@pytest.mark.parametrize("change,status", BAD)
def test_bad_shapes(lib, change, status):
    s, c = shape(**change), cache()
    assert lib.lychee_q8_workspace_size(ctypes.byref(s), 0) == 0
    assert lib.lychee_decode_attn_q8(s, FAKE, c, FAKE, FAKE, FAKE, 1 << 40, None, None) == status
    roles = (ctypes.c_uint8 * 256)(*([1] * 256))
    assert lib.lychee_hybrid_decode_attn_q8(s, 8, 0, FAKE, c, FAKE, None, roles, None, FAKE, FAKE, FAKE, 1 << 40, None,
                                            None) == status
    assert lib.lychee_append_rope_q8(s, c, tokens(), FAKE, None, None) == status


def tokens(**kw):
    f = dict(k=FAKE, v=FAKE, q=None, q_out=None, k_stride=256, v_stride=256, q_stride=0, cos_sin=FAKE, cu_new=None, T=2,
             n_pos=100, rot=128, interleaved=0)
    f.update(kw)
    return N.Q8Tokens(*(f[n] for n, _ in N.Q8Tokens._fields_))


@pytest.mark.parametrize("change", [dict(k=None), dict(v=None), dict(q=FAKE), dict(q_out=FAKE), dict(T=-1), dict(T=3),
                                    dict(k=FAKE + 8), dict(v=FAKE + 2), dict(k_stride=255), dict(k_stride=260),
                                    dict(v_stride=128), dict(rot=4), dict(rot=130), dict(rot=136), dict(rot=0), dict(n_pos=0),
                                    dict(cos_sin=FAKE + 4), dict(q=FAKE, q_out=FAKE, q_stride=1000),
                                    dict(q=FAKE, q_out=FAKE + 8, q_stride=1024), dict(cu_new=FAKE + 2)])
def test_bad_tokens(lib, change):
    assert lib.lychee_append_rope_q8(shape(), cache(), tokens(**change), FAKE, None, None) == N.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(block_table=None),
                                    dict(k=FAKE + 1), dict(v=FAKE + 8), dict(k_scale=FAKE + 2), dict(block_table=FAKE + 1)])
def test_bad_caches(lib, change):
    s, c = shape(), cache(**change)
    assert lib.lychee_append_rope_q8(s, c, tokens(), FAKE, None, None) == N.ERR_INVALID_ARG
    assert lib.lychee_decode_attn_q8(s, FAKE, c, FAKE, FAKE, FAKE, 1 << 40, None, None) == N.ERR_INVALID_ARG


def test_attention_arguments(lib):
    s, c = shape(), cache()
    ok = [s, FAKE, c, FAKE, FAKE, FAKE, 1 << 40, None, None]
    for at, bad in ((1, None), (1, FAKE + 8), (3, None), (3, FAKE + 2), (4, None), (4, FAKE + 8), (7, FAKE + 1)):
        args = list(ok)
        args[at] = bad
        assert lib.lychee_decode_attn_q8(*args) == N.ERR_INVALID_ARG, at
    need = lib.lychee_q8_workspace_size(s, 0)
    for ws, n in ((None, 1 << 40), (FAKE + 128, 1 << 40), (FAKE, need - 1)):
        args = list(ok)
        args[5:7] = ws, n
        assert lib.lychee_decode_attn_q8(*args) == N.ERR_WORKSPACE


def test_hybrid_arguments(lib):
    s, c = shape(), cache()
    all_r, mixed, wrong = ((ctypes.c_uint8 * 8)(*r) for r in ([1] * 8, [1, 0] * 4, [1, 2] * 4))
    ok = [s, 8, 0, FAKE, c, FAKE, None, mixed, FAKE, FAKE, FAKE, FAKE, 1 << 40, None, None]
    for at, bad in ((1, 0), (1, 257), (1, -1), (2, -1), (2, 48), (2, 64), (2, 2048), (3, None), (5, None), (6, FAKE + 1),
                    (7, None), (7, wrong), (8, None), (8, FAKE + 2), (9, None), (9, FAKE + 8), (10, None), (10, FAKE + 1),
                    (13, FAKE + 2)):
        args = list(ok)
        args[at] = bad
        assert lib.lychee_hybrid_decode_attn_q8(*args) == N.ERR_INVALID_ARG, (at, bad)
    need = lib.lychee_q8_workspace_size(s, 8)
    assert need >= 2 * 8 * 256 * 4 and lib.lychee_q8_workspace_size(s, 257) == 0 and lib.lychee_q8_workspace_size(s, -1) == 0
    for ws, n in ((None, 1 << 40), (FAKE + 128, 1 << 40), (FAKE, need - 1)):
        args = list(ok)
        args[11:13] = ws, n
        assert lib.lychee_hybrid_decode_attn_q8(*args) == N.ERR_WORKSPACE
    # a block selection whose keys do not fit one CTA
    big = shape(page=128, max_pages=8193 + 8192, num_pages=20)
    assert lib.lychee_hybrid_decode_attn_q8(big, 64, 32, *ok[3:]) == N.ERR_UNSUPPORTED


def test_binding_refuses_what_the_library_cannot_take():
    k = torch.zeros(3, 2, 64)
    c = ops.Q8Cache(torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 16, 64, dtype=torch.int8),
                    torch.ones(4, 2), torch.ones(4, 2))
    tab, seq = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.append_rope_q8(k, k, c, tab, seq)
    with pytest.raises(TypeError):
        ops.append_rope_q8(k.half(), k.half(), c, tab, seq)
    with pytest.raises(ValueError):
        ops.append_rope_q8(k[0], k[0], c, tab, seq)
    with pytest.raises(ValueError, match="CUDA"):
        ops.decode_attn_q8(k, c, tab, seq)
    with pytest.raises(ValueError, match="CUDA"):
        ops.hybrid_decode_attn_q8(k, c, tab, seq, [1, 1], None, 2)
    with pytest.raises(TypeError):
        ops.alloc_q8_cache(4, 2, 16, 64, torch.float8_e5m2, "cpu")
    made = ops.alloc_q8_cache(4, 2, 16, 64, torch.int8, "cpu")
    assert made.k.shape == (4, 2, 16, 64) and made.v_scale.shape == (4, 2) and made.k.dtype == torch.int8
    with pytest.raises(N.LycheeError):
        ops.q8_workspace_size(1, 8, 2, 96, 16, 4, 2, torch.bfloat16, torch.int8)


def test_reference_scale_is_the_smallest_that_fits():
    for code, top in R.LARGEST.items():
        for amax in (top, top * 1.0001, top / 2, top / 2 * 1.0001, 1.0, 3e-5, 1e9):
            s = R.block_scale(torch.tensor([[amax, -amax / 3]]), code)
            assert amax / s <= top * (1 + 1e-6) and amax / (s / 2) > top
        assert R.block_scale(torch.zeros(1, 4), code) == 2.0 ** -60
        assert R.block_scale(torch.tensor([[float("inf"), float("nan"), 1.0]]), code) == R.block_scale(torch.ones(1, 1), code)


def test_reference_rotation_turns_by_the_angle():
    """Against complex products in fp64: a rotation keeps lengths and adds angles."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(3, 64, generator=g)
    a = torch.rand(16, generator=g, dtype=torch.float64) * 6
    cs = torch.cat([a.cos(), a.sin()]).float()
    for inter in (False, True):
        y = R.rotate(x, cs, inter).double()
        i1, i2 = (torch.arange(0, 32, 2), torch.arange(1, 32, 2)) if inter else (torch.arange(16), torch.arange(16, 32))
        z = torch.complex(x[:, i1].double(), x[:, i2].double()) * torch.polar(torch.ones_like(a), a)
        assert torch.allclose(y[:, i1], z.real, atol=1e-6) and torch.allclose(y[:, i2], z.imag, atol=1e-6)
        assert torch.equal(y[:, 32:], x[:, 32:].double())
