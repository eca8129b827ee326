"""The compiled binding's checks on CUDA tensors: types, shapes, strides and devices come back as
Python errors, the library's refusals as CkError, and given outputs are the ones returned."""
import pytest
import torch

import int8_weight_quantized_gb300 as ck

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def i32(*shape):
    return t(*shape, dtype=torch.int32)


@pytest.mark.parametrize("call,error", [
    (lambda: ck.ck_attention(t(4, 2, 64), t(4, 1, 64, dtype=torch.float16), t(4, 1, 64), i32(2)), TypeError),
    (lambda: ck.ck_attention(t(4, 2, 64), t(4, 1, 64), t(5, 1, 64), i32(2)), ValueError),
    (lambda: ck.ck_attention(t(4, 2, 64), t(4, 1, 64), t(4, 1, 64), i32(2).long()), TypeError),
    (lambda: ck.ck_attention(t(4, 2, 64), t(4, 1, 64), t(4, 1, 64), i32(2), i32(3)), ValueError),
    (lambda: ck.ck_attention(t(64, 2, 4).transpose(0, 2), t(4, 1, 64), t(4, 1, 64), i32(2)), ValueError),
    (lambda: ck.ck_attention(t(4, 2, 64), t(4, 1, 64), t(4, 1, 64), i32(2), out=t(4, 2, 32)), ValueError),
    (lambda: ck.ck_attention(t(4, 2, 64), t(4, 1, 64), t(4, 1, 64), i32(2), scale="x"), TypeError),
    (lambda: ck.ck_attention(t(4, 2, 96), t(4, 1, 96), t(4, 1, 96), i32(2)), ck.CkError),
    (lambda: ck.ck_attention(t(4, 3, 64), t(4, 2, 64), t(4, 2, 64), i32(2)), ck.CkError),
    (lambda: ck.ck_paged_attention(t(2, 2, 64), ck.KVCache(t(3, 1, 8, 64), t(3, 1, 8, 32)), i32(2, 1), i32(2)), ValueError),
    (lambda: ck.ck_paged_attention(t(2, 2, 64), ck.KVCache(t(3, 1, 8, 128), t(3, 1, 8, 128)), i32(2, 1), i32(2)), ValueError),
    (lambda: ck.ck_paged_attention(t(2, 2, 64), ck.KVCache(*[t(3, 1, 8, 64, dtype=torch.int8)] * 2), i32(2, 1), i32(2)),
     ValueError),
    (lambda: ck.ck_paged_attention(t(2, 2, 64), ck.KVCache(*[t(3, 1, 8, 64, dtype=torch.float16)] * 2), i32(2, 1), i32(2)),
     ck.CkError),
    (lambda: ck.ck_paged_attention(t(2, 2, 64), ck.KVCache(t(3, 1, 8, 64), t(3, 1, 8, 64)), i32(3, 1), i32(2)), ValueError),
    (lambda: ck.ck_paged_attention(t(2, 2, 64), ck.KVCache(t(3, 1, 8, 64), t(3, 1, 8, 64)), i32(2, 100), i32(2),
                                   ws=t(16, dtype=torch.uint8)), ck.CkError),
    (lambda: ck.ck_qk_norm_rope(t(3, 256), None, None, 3, 0), ValueError),
    (lambda: ck.ck_qk_norm_rope(t(3, 250), None, None, 2, 1), ValueError),
    (lambda: ck.ck_qk_norm_rope(t(256, 3).t(), None, None, 2, 1), ValueError),
    (lambda: ck.ck_qk_norm_rope(t(3, 256), i32(2), t(9, 64, dtype=torch.float32), 2, 1), ValueError),
    (lambda: ck.ck_qk_norm_rope(t(3, 256), i32(3), t(9, 24, dtype=torch.float32), 2, 1), ck.CkError),
    (lambda: ck.ck_qk_norm_rope(t(3, 256), None, None, 2, 1, q_weight=t(32)), ValueError),
    (lambda: ck.ck_qk_norm_rope(t(3, 256), None, None, 2, 1, cache=ck.KVCache(t(3, 1, 8, 64), t(3, 1, 8, 64)),
                                slots=i32(3)), TypeError),
    (lambda: ck.ck_int4_linear(t(2, 256), i32(16, 31), t(16, 2)), ValueError),
    (lambda: ck.ck_int4_linear(t(2, 256), i32(16, 32), t(16, 3)), ValueError),
    (lambda: ck.ck_int4_linear(t(2, 256), i32(12, 32), t(12, 2)), ck.CkError),
    (lambda: ck.ck_int4_linear(t(2, 256), i32(16, 32), t(16, 2), bias=t(16, dtype=torch.float32)), TypeError),
    (lambda: ck.ck_int4_linear(t(2, 256), i32(16, 32), t(16, 2), out_dtype=torch.int32), ValueError),
    (lambda: ck.ck_int4_linear(t(2, 512)[:, ::2], i32(16, 32), t(16, 2)), ValueError),
])
def test_refusals(call, error):
    with pytest.raises(error):
        call()
    torch.cuda.synchronize()
    assert ck.ck_device_error() == 0


def test_given_outputs_are_returned():
    q, k, v, cu = t(4, 2, 64), t(4, 1, 64), t(4, 1, 64), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    out, lse = t(4, 2, 64), t(2, 4, dtype=torch.float32)
    a, b = ck.ck_attention(q, k, v, cu, out=out, lse=lse, return_lse=True)
    assert a is out and b is lse
    y = t(2, 16, dtype=torch.float32)
    assert ck.ck_int4_linear(t(2, 256), i32(16, 32), t(16, 2), y=y, out_dtype=torch.float32) is y
    qo, ko = t(3, 2, 64), t(3, 1, 64)
    r = ck.ck_qk_norm_rope(t(3, 256), None, None, 2, 1, q=qo, k=ko)
    assert r[0] is qo and r[1] is ko


def test_empty_batches():
    assert ck.ck_attention(t(0, 2, 64), t(0, 1, 64), t(0, 1, 64), i32(1)).shape == (0, 2, 64)
    cache = ck.KVCache(t(3, 1, 8, 64), t(3, 1, 8, 64))
    assert ck.ck_paged_attention(t(0, 2, 64), cache, i32(0, 1), i32(0)).shape == (0, 2, 64)
    q, k = ck.ck_qk_norm_rope(t(0, 256), None, None, 2, 1)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    assert ck.ck_int4_linear(t(0, 256), i32(16, 32), t(16, 2)).shape == (0, 16)


def test_the_stride_of_one_token_does_not_matter():
    """Views of one row of a wider tensor, whose row length need not be a multiple of anything."""
    x = torch.randn((3, 4 * 64 + 3), device="cuda").to(BF)
    q, k, v = x[:, :128].view(3, 2, 64)[:1], x[:, 128:192].view(3, 1, 64)[:1], x[:, 192:256].view(3, 1, 64)[:1]
    assert q.stride(0) == 259
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    assert torch.equal(ck.ck_attention(q, k, v, cu), v.expand(1, 2, 64))
    got = ck.ck_qk_norm_rope(x[:1, :256], None, None, 2, 1, norm=False)
    assert torch.equal(got[0], q) and torch.equal(got[1], k)
    cache = ck.KVCache(k.contiguous().view(1, 1, 1, 64), v.contiguous().view(1, 1, 1, 64))
    out = ck.ck_paged_attention(q, cache, i32(1, 1), i32(1) + 1)
    assert torch.equal(out, v.expand(1, 2, 64))
    with pytest.raises(ck.CkError):  # two tokens have one
        ck.ck_qk_norm_rope(x[:2, :256], None, None, 2, 1)


def test_an_output_that_does_not_fit_is_torchs_out_of_memory_error():
    """2^40 bytes of output for a view of one token repeated: refused by torch's allocator, under a
    limit that it keeps without asking the device."""
    torch.cuda.set_per_process_memory_fraction(0.5)
    try:
        q = t(1, 2, 64).expand(2 ** 32, 2, 64)
        with pytest.raises(torch.OutOfMemoryError):
            ck.ck_attention(q, t(1, 1, 64), t(1, 1, 64), i32(2))
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
