"""Norms of queries and keys with the position rotation and the way into the paged cache,
against the 64-bit definition.

Bound: the fp32 chain (a sum of at most 256 squares in a tree over 8-term sums, square root,
division, two products, two products and a sum of the rotation) is off by at most 32 units of
2^-24 of the terms' magnitude; then one rounding to 16 bits.  int8 rows: the scale by 40 such
units, a code by half a step of the scale on top."""
import pytest
import torch

import int8_weight_quantized_gb300 as ck
import transformer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(tokens, hq, hkv, d, rot, dtype, seed, page=16, extra=0, cache_dtype=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    width = (hq + 2 * hkv) * d
    qkv = torch.randn((tokens, width + extra), generator=g, device=DEV).mul_(1.5).to(dtype)[:, :width]
    qw = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dtype)
    kw = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dtype)
    table = ck.rope_table(4096, rot) if rot else None
    positions = torch.randint(0, 4096, (tokens,), generator=g, device=DEV, dtype=torch.int32)
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:tokens]
    cache = ck.KVCache.empty(pages, page, hkv, d, dtype=cache_dtype or dtype)
    return qkv, qw, kw, table, positions, slots, cache


def expected(qkv, hq, hkv, d, qw, kw, eps, norm, table, positions, interleaved):
    x = qkv.reshape(-1, hq + 2 * hkv, d)
    cos = sin = None
    if table is not None:
        cos, sin = table[positions.long()].chunk(2, 1)
    q = ref.norm_rope(x[:, :hq], qw, eps, norm, cos, sin, interleaved)
    k = ref.norm_rope(x[:, hq:hq + hkv], kw, eps, norm, cos, sin, interleaved)
    v = x[:, hq + hkv:].double()
    return q, k, v


def check16(got, want, dtype, what):
    y, mag = want
    fp32 = 32 * ref.U32 * mag
    ref.assert_within(got, y, (y.abs() + fp32) * ref.unit(dtype) + ref.least(dtype) + fp32, what)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,hq,hkv,d,rot,interleaved", [
    (1, 32, 8, 128, 128, False),
    (1, 1, 1, 64, 64, True),
    (37, 6, 2, 64, 32, False),
    (130, 7, 1, 96, 48, False),
    (19, 5, 5, 80, 80, True),
    (64, 16, 4, 128, 64, True),
    (33, 8, 2, 256, 256, False),
    (5, 3, 1, 8, 0, False),
    (21, 4, 4, 72, 16, False),
])
def test_rotated_rows_and_cache(tokens, hq, hkv, d, rot, interleaved, dtype):
    qkv, qw, kw, table, positions, slots, cache = make(tokens, hq, hkv, d, rot, dtype, 3, page=7, extra=8)
    before_k, before_v = cache.k.clone(), cache.v.clone()
    q, k = ck.ck_qk_norm_rope(qkv, positions, table, hq, hkv, qw, kw, eps=1e-5, interleaved=interleaved, cache=cache,
                              slots=slots, return_k=True)
    want_q, want_k, want_v = expected(qkv, hq, hkv, d, qw, kw, 1e-5, True, table, positions, interleaved)
    check16(q, want_q, dtype, "q")
    check16(k, want_k, dtype, "k")
    at, off = slots // 7, slots % 7
    assert torch.equal(cache.k[at, :, off], k)
    assert torch.equal(cache.v[at, :, off].double(), want_v)
    untouched = torch.ones(cache.k.shape[0] * 7, dtype=torch.bool, device=DEV)
    untouched[slots] = False
    rows = untouched.nonzero()[:, 0]
    assert torch.equal(cache.k[rows // 7, :, rows % 7], before_k[rows // 7, :, rows % 7])
    assert torch.equal(cache.v[rows // 7, :, rows % 7], before_v[rows // 7, :, rows % 7])
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("norm,weights", [(False, False), (True, False)])
def test_without_norm_or_weights(norm, weights):
    qkv, qw, kw, table, positions, _, _ = make(11, 4, 2, 64, 64, torch.bfloat16, 5)
    q, k = ck.ck_qk_norm_rope(qkv, positions, table, 4, 2, norm=norm)
    want_q, want_k, _ = expected(qkv, 4, 2, 64, None, None, 1e-6, norm, table, positions, False)
    check16(q, want_q, torch.bfloat16, "q")
    check16(k, want_k, torch.bfloat16, "k")


def test_neither_norm_nor_rotation_copies():
    qkv, *_ = make(9, 4, 2, 64, 0, torch.float16, 6)
    q, k = ck.ck_qk_norm_rope(qkv, None, None, 4, 2, norm=False)
    assert torch.equal(q, qkv.reshape(9, 8, 64)[:, :4]) and torch.equal(k, qkv.reshape(9, 8, 64)[:, 4:6])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (96, 5), (256, 16)])
def test_int8_cache_rows(d, page, dtype):
    tokens, hq, hkv = 43, 4, 2
    qkv, qw, kw, table, positions, slots, cache = make(tokens, hq, hkv, d, d if d % 16 == 0 else 0, dtype, 7, page=page,
                                                       cache_dtype=torch.int8)
    qkv[3, :] = 0  # zero rows: scale 0, codes 0
    q, k = ck.ck_qk_norm_rope(qkv, positions, table, hq, hkv, qw, kw, cache=cache, slots=slots)
    assert k is None
    _, (want_k, mag), want_v = expected(qkv, hq, hkv, d, qw, kw, 1e-6, True, table, positions, False)
    at, off = slots // page, slots % page
    for name, want, m in (("k", want_k, mag), ("v", want_v, want_v.abs())):
        codes = getattr(cache, name)[at, :, off]
        scale = getattr(cache, name + "_scale")[at, :, off]
        top = want.abs().amax(-1)
        ref.assert_within(scale, top / 127, 40 * ref.U32 * m.amax(-1) / 127, name + " scale")
        step = scale.double()[..., None]
        ref.assert_within(codes.double() * step, want, 0.5 * step + 40 * ref.U32 * m.amax(-1, keepdim=True), name)
        assert int(codes.abs().max()) <= 127
        assert not codes[3].any() and not scale[3].any()
    # values are quantized from the 16-bit input itself: bit-exact by the row quantizer's rule
    # (on the CPU: torch's CUDA division by a plain number multiplies by its reciprocal)
    x = want_v.float().cpu()
    s = x.abs().amax(-1) / 127
    c = torch.where(s[..., None] > 0, (x / s[..., None].clamp_min(1e-38)).round().clamp(-127, 127), torch.zeros_like(x))
    assert torch.equal(cache.v_scale[at, :, off].cpu(), s)
    assert torch.equal(cache.v[at, :, off].cpu(), c.to(torch.int8))


def test_negative_slots_stay_out_of_the_cache():
    qkv, qw, kw, table, positions, slots, cache = make(20, 4, 2, 64, 64, torch.bfloat16, 8)
    slots[::3] = -1
    ck.ck_qk_norm_rope(qkv, positions, table, 4, 2, qw, kw, cache=cache, slots=slots)
    kept = slots[slots >= 0]
    assert int((cache.k.abs().sum((1, 3)) > 0).sum()) == kept.numel()
    assert ck.ck_device_error() == 0


def test_out_of_range_indices_are_reported_and_skipped():
    """The kernel's own bounds checks: nothing outside is read or written."""
    assert ck.ck_device_error() == 0
    qkv, qw, kw, table, positions, slots, cache = make(20, 4, 2, 64, 64, torch.bfloat16, 9)
    positions[4] = 4096
    positions[5] = -1
    slots[6] = cache.num_pages * cache.page_size
    q, k = ck.ck_qk_norm_rope(qkv, positions, table, 4, 2, qw, kw, cache=cache, slots=slots, return_k=True)
    assert q[4:6].isnan().all() and k[4:6].isnan().all()
    ok = [i for i in range(20) if i not in (4, 5)]
    assert not q[ok].isnan().any()
    assert ck.ck_device_error(clear=True) == 128
    assert ck.ck_device_error() == 0


def test_on_another_stream_and_in_a_graph():
    qkv, qw, kw, table, positions, slots, cache = make(50, 8, 2, 128, 128, torch.bfloat16, 10)
    q0, k0 = ck.ck_qk_norm_rope(qkv, positions, table, 8, 2, qw, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q1, k1 = ck.ck_qk_norm_rope(qkv, positions, table, 8, 2, qw, kw, stream=side)
    side.synchronize()
    assert torch.equal(q0, q1) and torch.equal(k0, k1)
    q2, k2 = torch.empty_like(q0), torch.empty_like(k0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.ck_qk_norm_rope(qkv, positions, table, 8, 2, qw, kw, q=q2, k=k2)
    qkv.mul_(-0.5)
    g.replay()
    q3, k3 = ck.ck_qk_norm_rope(qkv, positions, table, 8, 2, qw, kw)
    torch.cuda.synchronize()
    assert torch.equal(q2, q3) and torch.equal(k2, k3) and not torch.equal(q2, q0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_int8_rows_that_codes_cannot_hold_have_nan_scales(d, dtype):
    """A position out of range, a NaN or an infinity leaves no plausible row in an int8 cache: the
    row's scale is NaN, and what reads it is NaN; every other row is as it was."""
    assert ck.ck_device_error() == 0
    tokens, hq, hkv, page = 24, 4, 2, 8
    qkv, qw, kw, table, positions, _, clean = make(tokens, hq, hkv, d, d, dtype, 11, page=page, cache_dtype=torch.int8)
    slots = torch.arange(tokens, device=DEV)
    ck.ck_qk_norm_rope(qkv, positions, table, hq, hkv, qw, kw, cache=clean, slots=slots)
    qkv, positions = qkv.clone(), positions.clone()
    x = qkv.view(tokens, hq + 2 * hkv, d)
    k_bad, v_bad = torch.zeros((2, tokens, hkv), dtype=torch.bool, device=DEV)
    for token, position in ((4, 4096), (5, -1)):
        positions[token] = position
        k_bad[token] = True
    for token, head, at, fill in ((6, 0, 0, float("nan")), (7, 1, d - 1, float("inf")), (8, 0, 5, -float("inf"))):
        x[token, hq + head, at] = fill
        k_bad[token, head] = True
    for token, head, at, fill in ((9, 1, d // 2, float("nan")), (10, 0, 3, float("inf")), (6, 1, 1, -float("inf"))):
        x[token, hq + hkv + head, at] = fill
        v_bad[token, head] = True
    cache = ck.KVCache.empty(clean.num_pages, page, hkv, d, dtype=torch.int8)
    ck.ck_qk_norm_rope(qkv, positions, table, hq, hkv, qw, kw, cache=cache, slots=slots)
    assert ck.ck_device_error(clear=True) == 128
    at, off = slots // page, slots % page
    for name, bad in (("k", k_bad), ("v", v_bad)):
        scale, want = [getattr(c, name + "_scale")[at, :, off] for c in (cache, clean)]
        assert scale[bad].isnan().all(), name
        assert torch.equal(scale[~bad], want[~bad])
        codes, want = [getattr(c, name)[at, :, off] for c in (cache, clean)]
        assert torch.equal(codes[~bad], want[~bad])
    if d > 128:
        return
    # one sequence to a page: tokens 0..7, 8..15, 16..23; all but the last hold such rows
    q = torch.randn((3, hq, d), device=DEV).to(dtype)
    blocks = torch.arange(3, dtype=torch.int32, device=DEV)[:, None]
    lens = torch.full((3,), page, dtype=torch.int32, device=DEV)
    out = ck.ck_paged_attention(q, cache, blocks, lens).view(3, hkv, hq // hkv, d)
    reads = (k_bad | v_bad).view(3, page, hkv).any(1)
    assert reads[:2].all() and not reads[2].any()
    assert out[reads].isnan().all()
    assert torch.equal(out[2], ck.ck_paged_attention(q, clean, blocks, lens).view(3, hkv, hq // hkv, d)[2])


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_int8_rows_without_norm_or_rotation(fill):
    qkv, *_, slots, cache = make(9, 2, 1, 64, 0, torch.bfloat16, 12, cache_dtype=torch.int8)
    qkv = qkv.clone()
    qkv.view(9, 4, 64)[3, 2, 63] = qkv.view(9, 4, 64)[5, 3, 0] = fill
    ck.ck_qk_norm_rope(qkv, None, None, 2, 1, norm=False, cache=cache, slots=slots)
    at, off = slots // 16, slots % 16
    assert cache.k_scale[at, 0, off].isnan().nonzero().flatten().tolist() == [3]
    assert cache.v_scale[at, 0, off].isnan().nonzero().flatten().tolist() == [5]
