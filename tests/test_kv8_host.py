"""Host-side checks of the 8-bit paged cache: refusals that need no GPU, and the reference's
own form of it."""
import ctypes
import math

import pytest

import decode_qwen2_block_gb300 as blk
from decode_qwen2_block_gb300 import build as gpu_build

torch = pytest.importorskip("torch")
from kv8_reference import E5M2, quantise, scale_of, values  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    gpu_build.build()
    return blk.load()


def test_null_handles_are_refused(lib):
    w, b, p = blk.BlkWeights(), blk.BlkPagedBatch(), blk.BlkKv8Pool(16, 16, 16, 16)
    N = blk.BLK_ERR_NULL
    assert blk.blk_page_append_kv8(None, 16, 16, 64, 64, 16, 1, 16, 1, p, None) == N
    assert blk.blk_page_read_kv8(None, 16, 1, 16, 1, p, 16, 16, 64, 64, None) == N
    assert blk.blk_attn_paged_kv8(None, b, 16, 64, p, 16, 64, 16, 1 << 20, None) == N
    assert blk.blk_step_paged_kv8(None, w, b, 16, 16, 16, p, 16, 16, 1 << 20, None) == N
    assert blk.blk_step_paged_stack_kv8(None, (blk.BlkWeights * 1)(w), 1, b, (blk.BlkKv8Pool * 1)(p), 16,
                                        16, 16, 16, 16, 1 << 20, None) == N


def test_the_pool_structure_is_laid_out_as_in_c():
    assert ctypes.sizeof(blk.BlkKv8Pool) == 4 * 8 and blk.BlkKv8Pool.v_scale.offset == 24


def test_the_tensor_calls_refuse_what_is_not_theirs(lib):
    from decode_qwen2_block_gb300 import _native
    args = (None, 0, 4, 2, 64)
    i64, f16 = torch.zeros(3, dtype=torch.int64), torch.zeros((3, 2, 64), dtype=torch.float16)
    c = torch.zeros((5, 2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((5, 2, 16, 2), dtype=torch.uint8).view(torch.float8_e5m2)
    batch = blk.BlkPagedBatch()
    for call in (lambda: _native.page_append_kv8(args, f16, f16, i64, c, c, s, s, None),
                 lambda: _native.page_append_kv8(args, f16, f16, i64, f16, c, s, s, None),
                 lambda: _native.page_read_kv8(args, i64, c, c, s, s, f16, f16, None),
                 lambda: _native.attn_paged_kv8(args, batch, f16, c, c, s, s, f16, i64, None)):
        with pytest.raises(blk.BlkError) as e:          # (CPU tensors)
            call()
        assert e.value.status == blk.BLK_ERR_SHAPE
    for call in (lambda: _native.page_append_kv8(args, f16, f16, i64, c, c, s, None),
                 lambda: _native.page_read_kv8(args, i64, 1, 2, 3, 4, f16, f16, None),
                 lambda: _native.attn_paged_kv8(args, i64, f16, c, c, s, s, f16, i64, None),
                 lambda: _native.bind(1, 2, 3, 4)):
        with pytest.raises(TypeError):
            call()


def test_the_references_scales_are_torchs():
    byte = torch.arange(256, dtype=torch.uint8)
    a, b = scale_of(byte), byte.view(torch.float8_e5m2).double()
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


def test_the_reference_by_hand():
    """Blocks whose scale and codes are plain: a greatest magnitude of 127 2^k has the scale
    64 2^k and codes x / 2^k; the next larger number the next scale, 80 2^k."""
    x = torch.zeros((4, 32), dtype=torch.float16)
    x[0, :5] = torch.tensor([127.0, -126.0, 0.5, 1.5, -2.5])
    x[1, 0] = 127.125
    x[2, :2] = torch.tensor([2.0 ** -24, -2.0 ** -24])
    c, s = quantise(x)
    assert scale_of(s).flatten().tolist() == [64, 80, 2.0 ** -16, 0]
    assert (c.long() - 128)[0, :5].tolist() == [127, -126, 0, 2, -2]
    assert c[1, 0] - 128 == round(127.125 * 64 / 80) and (c[3] == 128).all()
    assert (c.long() - 128)[2, :2].tolist() == [0, 0]       # 2^-24 is a quarter of a step of 2^-22
    assert values(c, s)[0, :5].tolist() == [127, -126, 0, 2, -2]


def test_the_reference_holds_every_number_to_half_a_step():
    x = torch.arange(0x7c00, dtype=torch.int16).view(torch.float16)
    x = torch.cat((x, x.new_zeros(-x.numel() % 32))).view(-1, 32)
    c, s = quantise(x)
    v = values(c, s)
    step = scale_of(s) / 64
    assert torch.isfinite(v.half()).all() and torch.equal(v.half().double(), v)
    assert ((v - x.double()).abs() <= step / 2).all()
    a = x.double().amax(-1)
    assert (127 * step[:, 0] >= a).all()
    less = torch.tensor([0.0, *E5M2.tolist()], dtype=torch.float64)[(s.long() - 1).clamp(min=0).flatten()]
    assert ((127 * less / 64 < a) | (a == 0)).all()
    assert math.isclose(float(E5M2[-1]), 57344.0)
