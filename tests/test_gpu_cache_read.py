"""Rows of the paged cache read back: 16-bit rows as they are, int8 rows as code * scale in fp32
rounded once (the same two operations in torch give the same bits)."""
import pytest
import torch

import int8_weight_quantized_gb300 as ck
from helpers import NAN16, assert_guards_intact, guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16 = torch.bfloat16, torch.float16


def make(lens, hkv, d, page, dtype, int8, seed, first=0, after=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    pool = torch.randperm(pages, generator=g, device=DEV)
    table = torch.zeros((len(lens), max([1] + need)), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pool[at:at + n].to(torch.int32)
        at += n
    shape = (pages, hkv, page, d)
    if int8:
        cache = ck.KVCache.empty(pages, page, hkv, d, dtype=torch.int8)
        for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            t.copy_(torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8))
            s.copy_(torch.randn(shape[:3], generator=g, device=DEV).mul_(3).exp2_() * 0.01)
    else:
        cache = ck.KVCache(*[torch.randn(shape, generator=g, device=DEV).to(dtype) for _ in range(2)])
    cu = torch.tensor([first] + [first + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device=DEV)
    return cache, table, cu, int(cu[-1]) + after


def expected(cache, table, lens, dtype):
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        rows = []
        for b, n in enumerate(lens):
            j = torch.arange(n, device=DEV)
            at, off = table[b].long()[j // cache.page_size], j % cache.page_size
            x = t[at, :, off]
            rows.append(x if s is None else (x.float() * s[at, :, off][..., None]).to(dtype))
        out.append(torch.cat(rows))
    return out


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("lens,hkv,d,page", [
    ([1], 1, 8, 1), ([300], 8, 128, 16), ([0, 5, 0, 17, 33], 2, 64, 16), ([700, 0, 129], 3, 96, 7), ([64], 1, 256, 64),
    ([9000, 1], 4, 72, 100), ([i % 5 for i in range(400)], 2, 64, 3), ([30000], 8, 128, 64),
])
def test_against_the_definition(lens, hkv, d, page, dtype, int8):
    cache, table, cu, total = make(lens, hkv, d, page, dtype, int8, seed=d)
    k, v = ck.ck_cache_read(cache, table, cu, total, dtype=dtype)
    want = expected(cache, table, lens, dtype)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("int8", [False, True])
def test_rows_that_no_sequence_has_stay(int8):
    lens = [40, 0, 21]
    cache, table, cu, total = make(lens, 2, 64, 16, BF, int8, seed=1, first=5, after=9)
    bufs = [guarded((total, 2, 64), BF, NAN16) for _ in range(2)]
    k, v = bufs[0][1], bufs[1][1]
    a, b = ck.ck_cache_read(cache, table, cu, total, k=k, v=v)
    assert a is k and b is v
    for got, want, (buf, _) in zip((k, v), expected(cache, table, lens, BF), bufs):
        assert torch.equal(got[5:66], want)
        assert (got[:5].view(torch.int16) == NAN16).all() and (got[66:].view(torch.int16) == NAN16).all()
        assert_guards_intact(buf, NAN16)


@pytest.mark.parametrize("int8", [False, True])
def test_pages_and_bounds_out_of_range(int8):
    cache, table, cu, total = make([40, 50, 30], 2, 64, 16, F16, int8, seed=2)
    want = expected(cache, table, [40, 50, 30], F16)
    for value in (-1, cache.num_pages, 2 ** 31 - 1):
        bad = table.clone()
        bad[1, 2] = value
        k, v = ck.ck_cache_read(cache, bad, cu, total, dtype=F16)
        assert ck.ck_device_error() == 128
        for got, w in zip((k, v), want):
            assert got[72:88].isnan().all()
            assert torch.equal(got[:72], w[:72]) and torch.equal(got[88:], w[88:])
    # more tokens than the table has pages for: those are NaN
    k, v = ck.ck_cache_read(cache, table[:, :2].contiguous(), cu, total, dtype=F16)
    assert ck.ck_device_error() == 128
    for got, w in zip((k, v), want):
        assert torch.equal(got[:32], w[:32]) and got[32:40].isnan().all() and got[72:90].isnan().all()
    for i, value in ((0, -3), (3, total + 1), (1, 95), (2, 7)):
        bad = cu.clone()
        bad[i] = value
        ck.ck_cache_read(cache, table, bad, total, dtype=F16)  # in range whatever the bounds say
        assert ck.ck_device_error() == 128


def test_scales_of_nan_and_infinity():
    cache, table, cu, total = make([20], 2, 64, 16, BF, True, seed=3)
    page = int(table[0, 1])
    cache.k_scale[page, 1, 2] = float("nan")
    cache.v_scale[page, 0, 3] = 1e37
    k, v = ck.ck_cache_read(cache, table, cu, total)
    assert k[18, 1].isnan().all() and not k[18, 0].isnan().any()
    want = expected(cache, table, [20], BF)
    assert torch.equal(v, want[1])


def test_offsets_beyond_32_bits():
    pages, page, hkv, d = 2 ** 15 + 8, 64, 8, 128
    cache = ck.KVCache(*[torch.empty((pages, hkv, page, d), dtype=BF, device=DEV) for _ in range(2)])
    at = torch.tensor([pages - 1, 2, 2 ** 15 + 1], device=DEV)
    for t in (cache.k, cache.v):
        t[at] = torch.randn((3, hkv, page, d), device=DEV).to(BF)
    cu = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
    table = at[None].to(torch.int32).contiguous()
    k, v = ck.ck_cache_read(cache, table, cu, 150)
    want = expected(cache, table, [150], BF)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_what_was_written_comes_back():
    """ck_qk_norm_rope's rows: 16-bit ones bit for bit, int8 ones within half a code of what went in (and
    the two roundings of code * scale)."""
    tokens, hq, hkv, d, page = 90, 4, 2, 64, 16
    qkv = torch.randn((tokens, (hq + 2 * hkv) * d), device=DEV).to(BF)
    table = torch.randperm(8, device=DEV).to(torch.int32)[None, :6].contiguous()
    j = torch.arange(tokens, device=DEV)
    slots = table[0].long()[j // page] * page + j % page
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    for kind in (BF, torch.int8):
        cache = ck.KVCache.empty(8, page, hkv, d, dtype=kind)
        _, k = ck.ck_qk_norm_rope(qkv, j.to(torch.int32), ck.rope_table(tokens, d), hq, hkv, cache=cache, slots=slots,
                                  return_k=True)
        v = qkv.view(tokens, -1, d)[:, hq + hkv:]
        for got, want in zip(ck.ck_cache_read(cache, table, cu, tokens), (k, v)):
            if kind == BF:
                assert torch.equal(got, want)
            else:  # half a code of max / 127, the scale's and the result's roundings, k's own to bf16
                top = want.float().abs().amax(-1, keepdim=True) * (1 + 2.0 ** -8)
                assert ((got.float() - want.float()).abs() <= top / 254 + top * 2.0 ** -7).all()


def test_streams_and_graphs():
    cache, table, cu, total = make([100, 30], 2, 64, 16, BF, True, seed=5)
    want = expected(cache, table, [100, 30], BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ck.ck_cache_read(cache, table, cu, total, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    k, v = torch.empty_like(got[0]), torch.empty_like(got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ck.ck_cache_read(cache, table, cu, total, k=k, v=v)
    cache.k.neg_()
    graph.replay()
    assert torch.equal(k, -want[0]) and torch.equal(v, want[1])


def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(dtype=torch.float32), TypeError), (lambda: dict(dtype=F16), ck.CkError), (lambda: dict(total=-1), ValueError),
    (lambda: dict(cu=t(2)), TypeError), (lambda: dict(cu=t(3, dtype=torch.int32)), ValueError), (lambda: dict(k=t(4, 1, 32)), ValueError),
    (lambda: dict(v=t(4, 1, 64, dtype=F16)), TypeError), (lambda: dict(table=t(1, 0, dtype=torch.int32)), ck.CkError),
])
def test_refusals(kw, error):
    cache = ck.KVCache(t(3, 1, 8, 64), t(3, 1, 8, 64))
    f = dict(table=t(1, 2, dtype=torch.int32), cu=t(2, dtype=torch.int32), total=4, dtype=None, k=None, v=None)
    f.update(kw())
    with pytest.raises(error):
        ck.ck_cache_read(cache, f["table"], f["cu"], f["total"], dtype=f["dtype"], k=f["k"], v=f["v"])
    torch.cuda.synchronize()
    assert ck.ck_device_error() == 0


def test_nothing_to_read():
    cache = ck.KVCache(t(3, 1, 8, 64), t(3, 1, 8, 64))
    k, v = ck.ck_cache_read(cache, t(0, 1, dtype=torch.int32), t(1, dtype=torch.int32), 0)
    assert k.shape == (0, 1, 64) and v.shape == (0, 1, 64)
