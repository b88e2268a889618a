"""The backward pass, the forward with statistics and the rotary positions
refuse bad arguments before touching a device (CPU)."""
import ctypes
import math

import pytest
import torch

import masked_grouped_query_b200 as mgq
from masked_grouped_query_b200 import _lib, build

P = ctypes.c_void_p
# Disjoint addresses, a megabyte apart.
A = [0x1000000 * (i + 1) for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _lse(lib, ptr=None, dims=(1, 4, 4, 4, 2, 64, 1, 0), cap=0.0):
    p = list(A[:5])
    for i, x in (ptr or {}).items():
        p[i] = x
    return lib.gqa_attn_fwd_lse(*[P(x) for x in p], *dims, cap, None)


def _bwd(lib, ptr=None, dims=(1, 4, 4, 4, 2, 64, 1, 0), cap=0.0, size=1 << 20):
    p = list(A[:11])
    p[6] = 0  # no gradient of lse
    for i, x in (ptr or {}).items():
        p[i] = x
    return lib.gqa_attn_bwd(*[P(x) for x in p], size, *dims, cap, None)


BAD_SIZES = [
    ((1, 4, 4, 3, 2, 64, 1, 0), 0.0, -4),
    ((1, 4, 4, 4, 2, 60, 1, 0), 0.0, -5),
    ((1, 4, 4, 4, 2, 264, 1, 0), 0.0, -5),
    ((-1, 4, 4, 4, 2, 64, 1, 0), 0.0, -3),
    ((1, -4, 4, 4, 2, 64, 1, 0), 0.0, -3),
    ((1, 4, 4, 0, 2, 64, 1, 0), 0.0, -3),
    ((1, 4, 4, 4, 2, 64, 1, 0), -1.0, -6),
    ((1, 4, 4, 4, 2, 64, 1, 0), math.nan, -6),
    ((1, 4, 4, 4, 2, 64, 1, 0), math.inf, -6),
    ((1, 1 << 20, 4, 1 << 12, 1, 256, 1, 0), 0.0, -10),
]


@pytest.mark.parametrize("dims,cap,code", BAD_SIZES)
def test_bad_sizes(lib, dims, cap, code):
    assert _lse(lib, dims=dims, cap=cap) == code
    assert _bwd(lib, dims=dims, cap=cap) == code
    if code != -6:
        assert lib.gqa_attn_bwd_scratch(*dims, None) == code


def test_backward_index_limits(lib):
    size = ctypes.c_size_t(0)
    for dims in ((1, 1, 0x7fffffff, 1, 1, 8, 0, 0), (1 << 16, 1, 1, 1 << 16, 1, 8, 0, 0),
                 (1 << 15, 1, 1 << 24, 1, 1, 8, 0, 0)):
        assert lib.gqa_attn_bwd_scratch(*dims, ctypes.byref(size)) == -10


def test_scratch_bytes(lib):
    # 1 KiB for every tile of 128 rows (runs are heads where a mask separates
    # long ones, whole groups otherwise) while no walk is cut.
    def tiles(*dims):
        size = ctypes.c_size_t(0)
        assert lib.gqa_attn_bwd_scratch(*dims, ctypes.byref(size)) == 0
        assert size.value % 1024 == 0
        return size.value // 1024

    assert tiles(1, 128, 128, 4, 1, 128, 1, 0) == 4          # 512 rows of one group
    assert tiles(32, 1, 4096, 32, 8, 128, 1, 0) == 256       # 4 rows each
    # 16 row tiles over 32 key tiles: 8 parts each, of 128 x 128 floats.
    assert tiles(2, 1, 4096, 32, 8, 128, 1, 0) == 16 + 16 * 8 * 64
    # One key tile under 40 row tiles: 10 parts of dK and of dV, 128 x 64 floats.
    assert tiles(1, 5120, 100, 1, 1, 64, 0, 0) == 40 + 2 * 10 * 32
    assert tiles(1, 300, 300, 4, 2, 64, 1, 0) == 4 * 3       # heads apart
    assert tiles(1, 300, 300, 4, 2, 64, 0, 0) == 2 * 5       # 600 rows of two heads
    assert tiles(1, 300, 300, 4, 2, 64, 0, 7) == 4 * 3
    assert tiles(0, 300, 300, 4, 2, 64, 1, 0) == 0


def test_bad_pointers(lib):
    for i in range(5):
        assert _lse(lib, {i: 0}) == -1
        assert _lse(lib, {i: A[i] + 8}) == -2
    assert _lse(lib, {4: A[0]}) == -11
    assert _lse(lib, {4: A[3] + 64}) == -11
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9, 10):
        assert _bwd(lib, {i: 0}) == -1
    for i in range(11):
        assert _bwd(lib, {i: A[i] + 8}) == -2
    assert _bwd(lib, {7: A[1]}) == -11        # dq over q
    assert _bwd(lib, {8: A[2] + 512}) == -11  # dk inside k
    assert _bwd(lib, {9: A[8]}) == -11        # dv over dk
    assert _bwd(lib, {10: A[5]}) == -11       # scratch over lse
    assert _bwd(lib, {6: A[7]}) == -11        # dlse inside dq
    assert _bwd(lib, size=1023) == -12
    assert "needs 2048" in _lib.load().gqa_attn_last_error_detail().decode()


def test_valid_calls_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    assert _lse(lib) == -7
    assert _bwd(lib) == -7
    assert _bwd(lib, {6: A[12]}) == -7
    assert _rot(lib) == -7
    assert _rot(lib, {2: A[0], 3: A[1]}) == -7                  # in place
    assert _rot(lib, {1: 0, 3: 0}, hkv=0) == -7                 # no keys
    # nothing to do: no device is asked for
    assert _lse(lib, {0: 0, 3: 0, 4: 0}, dims=(1, 0, 4, 4, 2, 64, 1, 0)) == 0
    assert _bwd(lib, {i: 0 for i in range(11)}, dims=(0, 4, 4, 4, 2, 64, 1, 0), size=0) == 0
    assert _rot(lib, {i: 0 for i in range(5)}, length=0) == 0


def _rot(lib, ptr=None, b=1, length=4, hq=4, hkv=2, d=64, sections=(8, 24), theta=10000.0, flags=0,
         axes=None):
    p = list(A[:5])
    for i, x in (ptr or {}).items():
        p[i] = x
    sec = (ctypes.c_int * max(1, len(sections)))(*sections)
    return lib.gqa_attn_rotary(*[P(x) for x in p], b, length, hq, hkv, d,
                               len(sections) if axes is None else axes, sec, theta, flags, None)


def test_rotary_refusals(lib):
    assert _rot(lib, flags=0x100) == -12
    assert _rot(lib, b=-1) == -3
    assert _rot(lib, hq=0, hkv=0) == -3
    assert _rot(lib, d=60) == -5
    assert _rot(lib, sections=()) == -12
    assert _rot(lib, sections=(1,) * 9) == -12
    assert _rot(lib, sections=(8, 0)) == -12
    assert _rot(lib, sections=(8, 25)) == -12           # 66 elements in a head of 64
    assert _rot(lib, sections=(0x7fffffff, 0x7fffffff)) == -12
    for theta in (0.0, -1.0, math.nan, math.inf):
        assert _rot(lib, theta=theta) == -12
    for i in range(5):
        assert _rot(lib, {i: 0}) == -1
        assert _rot(lib, {i: A[i] + 8}) == -2
    assert _rot(lib, {2: A[0] + 64}) == -11             # overlaps, not in place
    assert _rot(lib, {2: A[0]}, flags=0x8) == -11       # in place with another type
    assert _rot(lib, {2: A[0]}, flags=0x1) == -11       # in place with another layout
    assert _rot(lib, {2: A[1]}) == -11                  # q_out over k
    assert _rot(lib, {3: A[2]}) == -11                  # k_out over q_out
    assert _rot(lib, {3: A[4]}) == -11                  # k_out over the positions


def test_python_wrappers_refuse_host_tensors_and_wrong_types():
    q = torch.zeros(1, 4, 3, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 4, 3)
    with pytest.raises(ValueError, match="CUDA"):
        mgq.attention_lse(q, k, k)
    with pytest.raises(TypeError, match="bfloat16"):
        mgq.attention_lse(q.float(), k, k)
    with pytest.raises(ValueError, match="CUDA"):
        mgq.attention_backward(q, q, k, k, q, lse)
    with pytest.raises(TypeError):
        mgq.attention_backward(None, q.float(), k, k, q, lse)
    pos = torch.zeros(1, 1, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mgq.rotary(q, k, pos, sections=(32,))
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        mgq.rotary(q.half(), k, pos, sections=(32,))


@pytest.mark.gpu
def test_python_wrappers_refuse_mismatches():
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    q, k, o, lse = z(1, 4, 3, 64), z(1, 2, 5, 64), z(1, 4, 3, 64), z(1, 4, 3, dtype=torch.float32)
    good = dict(do=o, q=q, k=k, v=k, o=o, lse=lse)
    for name, bad, error in (("v", z(1, 2, 4, 64), ValueError), ("do", z(1, 4, 4, 64), ValueError),
                             ("o", o.float(), TypeError), ("lse", lse.double(), TypeError),
                             ("lse", z(1, 4, 4, dtype=torch.float32), ValueError),
                             ("q", z(1, 3, 4, 64).transpose(1, 2), ValueError),
                             ("k", z(2, 2, 5, 64), ValueError)):
        with pytest.raises(error):
            mgq.attention_backward(**{**good, name: bad})
    with pytest.raises(ValueError):
        mgq.attention_backward(**good, dk=q)
    with pytest.raises(_lib.GqaAttnError) as e:
        mgq.attention_backward(**good, dq=q)
    assert e.value.code == -11
    with pytest.raises(_lib.GqaAttnError) as e:
        mgq.attention_backward(**good, softcap=-1.0)
    assert e.value.code == -6
    with pytest.raises(ValueError):
        mgq.attention_lse(q, k, k, lse=z(1, 4, 2, dtype=torch.float32))
    pos = torch.zeros(2, 1, 3, dtype=torch.int32, device="cuda")
    kr = z(1, 2, 3, 64)
    for args, kw, error in (((q, k, pos), dict(sections=(16, 16)), ValueError),
                            ((q, kr.float(), pos), dict(sections=(16, 16)), TypeError),
                            ((q, kr, pos.float()), dict(sections=(16, 16)), TypeError),
                            ((q, kr, pos), dict(sections=(32,)), ValueError),
                            ((q, kr, pos), dict(sections=(16, 16), out=(q,)), TypeError),
                            ((q, kr, pos), dict(sections=(16, 16), out=(kr, q)), ValueError),
                            ((q, None, pos), dict(sections=(16, 16), out=(q, kr)), ValueError),
                            ((q, kr, pos), dict(sections=(16, 16), out_dtype=torch.half), TypeError),
                            ((q, kr, pos), dict(sections=(16, 17)), _lib.GqaAttnError)):
        with pytest.raises(error):
            mgq.rotary(*args, **kw)
