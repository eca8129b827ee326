"""Attention of one new token over the paged cache, against the 64-bit definition (the bound's
terms are derived in transformer_ref.attend; one rounding of the output on top)."""
import pytest
import torch

import int8_weight_quantized_gb300 as ck
import transformer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(lens, hq, hkv, d, page, dtype, int8, seed, poison=True, q_std=1.5):
    """A shuffled pool; every row that no sequence owns is NaN (16-bit) or has a NaN scale."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    pool = torch.randperm(pages, generator=g, device=DEV)
    width = max(1, max(need)) + 1
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=DEV)
    shape = (pages, hkv, page, d)
    if int8:
        cache = ck.KVCache.empty(pages, page, hkv, d, dtype=torch.int8)
        for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            t.copy_(torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8))
            s.copy_(torch.rand(shape[:3], generator=g, device=DEV) * 0.02 + 0.004)
    else:
        cache = ck.KVCache(*[torch.randn(shape, generator=g, device=DEV).to(dtype) for _ in range(2)])
    owned = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    at = 0
    for b, n in enumerate(lens):
        mine = pool[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine.to(torch.int32)
        rows = torch.arange(n, device=DEV)
        if n:
            owned[mine[rows // page], rows % page] = True
    if poison:
        for t in ((cache.k_scale, cache.v_scale) if int8 else (cache.k, cache.v)):
            hidden = ~owned[:, None, :].expand(pages, hkv, page)
            t[hidden] = float("nan")
    q = (torch.randn((len(lens), hq, d), generator=g, device=DEV) * q_std).to(dtype)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def rows_of(cache, table, b, n, page, h):
    j = torch.arange(n, device=DEV)
    at, off = table[b].long()[j // page], j % page
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = t[at, h, off].double()
        out.append(x if s is None else x * s[at, h, off].double()[:, None])
    return out


def check(q, cache, table, lens, out, lse, window=0, sinks=0, scale=None):
    dtype, d = q.dtype, q.shape[2]
    hkv, page = cache.k.shape[1], cache.page_size
    g = q.shape[1] // hkv
    int8 = cache.k.dtype == torch.int8
    # weights meet 16-bit values in their own type; int8 codes in fp16
    p_type = torch.float16 if int8 else dtype
    scale = d ** -0.5 if scale is None else scale
    for b, n in enumerate(lens.tolist()):
        for h in range(hkv):
            k, v = rows_of(cache, table, b, n, page, h)
            j = torch.arange(n, device=DEV)
            seen = torch.ones(n, dtype=torch.bool, device=DEV) if not window else (j >= n - window) | (j < sinks)
            rows = slice(h * g, (h + 1) * g)
            want, want_lse, tol, lse_tol = ref.attend(q[b, rows], k, v, scale, seen[None].expand(g, n),
                                                      ref.unit(p_type), ref.least(p_type))
            if n:
                tol = tol + (want.abs() + tol) * ref.unit(dtype) + ref.least(dtype)
            ref.assert_within(out[b, rows], want, tol, "sequence %d head %d" % (b, h))
            if lse is not None:
                if n == 0:
                    assert (lse[b, rows] == -float("inf")).all()
                else:
                    ref.assert_within(lse[b, rows], want_lse, lse_tol, "lse %d" % b)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,hq,hkv,d,page", [
    ([1], 8, 2, 128, 16),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], 4, 1, 64, 16),
    ([274], 32, 8, 128, 16),
    ([700, 0, 3, 1025, 129], 12, 2, 128, 7),
    ([90, 511], 3, 3, 64, 1),
    ([257], 40, 2, 128, 100),
    ([5000, 4999], 16, 1, 128, 64),
])
def test_against_the_definition(lens, hq, hkv, d, page, dtype, int8):
    q, cache, table, n = make(lens, hq, hkv, d, page, dtype, int8, seed=len(lens) + d)
    out, lse = ck.ck_paged_attention(q, cache, table, n, return_lse=True)
    check(q, cache, table, n, out, lse)
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (100, 0), (130, 5), (4096, 4), (33, 1000)])
def test_window_and_first_tokens(window, sinks, int8):
    lens = [0, 1, 4, 100, 133, 135, 136, 999]
    q, cache, table, n = make(lens, 8, 2, 64, 16, torch.bfloat16, int8, seed=window + sinks)
    # what the window hides is poisoned too
    for b, length in enumerate(lens):
        j = torch.arange(length, device=DEV)
        hidden = j[(j < length - window) & (j >= sinks)]
        at, off = table[b].long()[hidden // 16], hidden % 16
        for t in ((cache.k_scale, cache.v_scale) if int8 else (cache.k, cache.v)):
            t[at, :, off] = float("inf")
    out, lse = ck.ck_paged_attention(q, cache, table, n, window=window, sinks=sinks, return_lse=True)
    for t in (cache.k_scale, cache.v_scale) if int8 else (cache.k, cache.v):
        t.nan_to_num_(0.0, 0.0, 0.0)
    check(q, cache, table, n, out, lse, window, sinks)


@pytest.mark.parametrize("int8", [False, True])
def test_many_sequences_and_a_long_one(int8):
    lens = [(37 * i * i + 11) % 300 for i in range(150)] + [20011]
    q, cache, table, n = make(lens, 8, 2, 128, 32, torch.bfloat16, int8, seed=77)
    out, lse = ck.ck_paged_attention(q, cache, table, n, return_lse=True)
    check(q, cache, table, n, out, lse)
    again = ck.ck_paged_attention(q, cache, table, n)
    assert torch.equal(out, again)  # the same split and order of sums every time


def test_sharp_scores_and_strides():
    lens = [300, 41]
    q, cache, table, n = make(lens, 8, 2, 128, 16, torch.float16, False, seed=5, q_std=12.0)
    wide = torch.zeros((2, 8 * 128 + 64), dtype=torch.float16, device=DEV)
    wide[:, :1024] = q.reshape(2, -1)
    view = wide[:, :1024].view(2, 8, 128)
    out, lse = ck.ck_paged_attention(view, cache, table, n, return_lse=True, scale=0.3)
    check(q, cache, table, n, out, lse, scale=0.3)


@pytest.mark.parametrize("gain", [1e-30, 1e-6, 1e6, 1e30])
def test_int8_queries_and_scales_of_any_size(gain):
    """int8 codes meet bf16 queries and fp32 scales over their whole range."""
    q, cache, table, n = make([123, 4], 4, 2, 64, 16, torch.bfloat16, True, seed=6)
    q = (q.float() * gain).to(torch.bfloat16)
    cache.k_scale.mul_(1.0 / gain)
    cache.v_scale.mul_(gain)
    out, lse = ck.ck_paged_attention(q, cache, table, n, return_lse=True)
    check(q, cache, table, n, out, lse)


def test_zero_scale_rows():
    q, cache, table, n = make([70], 4, 2, 64, 16, torch.bfloat16, True, seed=8)
    cache.v_scale[table[0].long()[:4]] = 0.0
    out = ck.ck_paged_attention(q, cache, table, n)
    check(q, cache, table, n, out, None)
    cache.v_scale.zero_()
    assert not ck.ck_paged_attention(q, cache, table, n).any()


def test_out_of_range_indices_are_reported():
    """A length beyond the table and a page beyond the pool: bounds-checked, NaN, reported."""
    assert ck.ck_device_error() == 0
    q, cache, table, n = make([50, 50, 50, 50], 4, 2, 64, 16, torch.bfloat16, False, seed=9)
    good = ck.ck_paged_attention(q, cache, table, n)
    n[1] = table.shape[1] * 16 + 1
    table[2, 1] = cache.num_pages
    out = ck.ck_paged_attention(q, cache, table, n)
    assert out[1].isnan().all() and out[2].isnan().all()
    assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    assert ck.ck_device_error(clear=True) == 128
    n[1] = -1
    assert ck.ck_paged_attention(q, cache, table, n)[1].isnan().all()
    assert ck.ck_device_error(clear=True) == 128


def test_streams_share_nothing_and_graphs_replay():
    q, cache, table, n = make([900, 20, 3000], 8, 2, 128, 16, torch.bfloat16, False, seed=10)
    want = ck.ck_paged_attention(q, cache, table, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [[ck.ck_paged_attention(q, cache, table, n, stream=s) for _ in range(5)] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for per in outs for o in per)
    out = torch.empty_like(want)
    ws = torch.full((ck.load_library().ck_paged_attention_workspace_size(3, 8, 2, 128, table.shape[1] * 16),), 255, dtype=torch.uint8,
                    device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.ck_paged_attention(q, cache, table, n, out=out, ws=ws)
    n[0], n[2] = 10, 2999
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ck.ck_paged_attention(q, cache, table, n))


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float16, 64)])
@pytest.mark.parametrize("scale", [1e-36, 1e-38, 1e-40, 1e-44])
@pytest.mark.parametrize("lens", [[70], [3, 33, 900]])
def test_tiny_value_scales_beside_zero_ones(scale, dtype, d, lens):
    """Scales down to subnormal ones, as rows of tiny values leave them, with zero rows among them."""
    q, cache, table, n = make(lens, 4, 2, d, 16, dtype, True, seed=31, poison=False)
    cache.v_scale.fill_(scale)
    cache.v_scale.view(-1)[::3] = 0.0
    out, lse = ck.ck_paged_attention(q, cache, table, n, return_lse=True)
    check(q, cache, table, n, out, lse)
    cache.k_scale.mul_(scale)
    out, lse = ck.ck_paged_attention(q, cache, table, n, return_lse=True)
    check(q, cache, table, n, out, lse)


@pytest.mark.parametrize("hq", [4, 20])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ratio", [1e-2, 1e-4, 1e-6, 1e-8, 1e-12])
@pytest.mark.parametrize("lens,at", [([1], [0]), ([100], [0]), ([100], [99]), ([40, 300], [17, 140]), ([2500], [1300])])
def test_value_scales_that_differ_within_a_sequence(lens, at, ratio, d, hq):
    """Nearly all the weight on a key whose value row is small beside the others.

    The kernel rounds the product of weight and value scale to fp16 once, relative to at most the
    largest such product P = max_j w_j s_j: unit(fp16) of each, or least(fp16) of P where it is
    subnormal, so that codes of at most 127 bring m * least * 127 P.  The rest as in
    transformer_ref.attend; the scale's base-2 logarithm brings 2^-22 of itself."""
    hkv, page = 2, 16
    q, cache, table, n = make(lens, hq, hkv, d, page, torch.bfloat16, True, seed=int(1 / ratio) % 1000, poison=False)
    g = hq // hkv
    # scores: some 40 for the chosen key, within 3 of zero for the others
    q = (torch.ones_like(q).float() * torch.linspace(0.9, 1.1, d, device=DEV)).to(torch.bfloat16)
    cache.k_scale.fill_(0.01)
    cache.k.copy_(torch.where(torch.arange(d, device=DEV) % 2 == 0, cache.k, -cache.k.roll(1, -1)))
    for b, j in enumerate(at):
        page_at = int(table[b, j // page])
        cache.k[page_at, :, j % page] = 127
        cache.k_scale[page_at, :, j % page] = 40.0 / (127 * d ** 0.5)
        cache.v_scale[page_at, :, j % page] *= ratio
    out, lse = ck.ck_paged_attention(q, cache, table, n, return_lse=True)
    fp16, u = torch.float16, ref.U32
    for b, length in enumerate(lens):
        for h in range(hkv):
            rows = slice(h * g, (h + 1) * g)
            k, v = rows_of(cache, table, b, length, page, h)
            j = torch.arange(length, device=DEV)
            s = cache.v_scale[table[b].long()[j // page], h, j % page].double()
            seen = torch.ones((g, length), dtype=torch.bool, device=DEV)
            want, want_lse, _, lse_tol = ref.attend(q[b, rows], k, v, d ** -0.5, seen, 0.0, 0.0)
            score = q[b, rows].double() @ k.t() * d ** -0.5
            w = torch.exp(score - score.amax(-1, keepdim=True))
            total = w.sum(-1, keepdim=True)
            dots = (q[b, rows].double().abs() @ k.abs().t() * d ** -0.5).amax(-1, keepdim=True)
            span = (score.amax(-1, keepdim=True) - score).amax(-1, keepdim=True)
            logs = s.log2().abs().amax()
            eps = (d + 8) * u * dots + 2.0 ** -21 + 4 * u * span + 2.0 ** -22 * logs + ref.unit(fp16)
            tol = (2 * eps + (length + 8) * u) * (w @ v.abs()) / total
            tol = tol + length * ref.least(fp16) * 127 * (w * s).amax(-1, keepdim=True) / total
            tol = tol + (want.abs() + tol) * ref.unit(torch.bfloat16) + ref.least(torch.bfloat16)
            ref.assert_within(out[b, rows], want, tol, "sequence %d head %d" % (b, h))
            ref.assert_within(lse[b, rows], want_lse, lse_tol, "lse")


def test_a_large_value_row_that_nobody_weighs():
    """One key of weight e^-60 with a value scale 1e12 times the others' costs these nothing."""
    q, cache, table, n = make([200, 1500], 8, 2, 64, 16, torch.float16, True, seed=33, poison=False)
    q = torch.ones_like(q)
    cache.k_scale.fill_(0.005)
    want = ck.ck_paged_attention(q, cache, table, n)
    for b, j in ((0, 60), (1, 700)):
        page_at = int(table[b, j // 16])
        cache.k[page_at, :, j % 16] = -127
        cache.k_scale[page_at, :, j % 16] = 60.0 / (127 * 8.0)
        cache.v_scale[page_at, :, j % 16] = 0.0
        clean = ck.ck_paged_attention(q, cache, table, n)
        cache.v_scale[page_at, :, j % 16] = 1e12
        out = ck.ck_paged_attention(q, cache, table, n)
        assert out.isfinite().all()
        # both round each product of weight and scale once, to a unit of 2^-11 (twice, independently),
        # and the outputs once; the large row itself brings 1e12 * 127 * e^-60 = 1e-12
        assert (out.float() - clean.float()).abs().max() <= 4 * 2.0 ** -11 * 127 * 0.024


def test_launches_are_counted():
    """The count of kernels goes by what a call enqueues: a split call joins in a second launch."""
    for length, launches in ((100, 1), (512, 1), (513, 2), (3000, 2)):
        q, cache, table, n = make([length], 4, 2, 64, 1, torch.bfloat16, False, seed=41)
        table = table[:, :length].contiguous()
        ck.ck_profile_begin(with_events=False)
        ck.ck_paged_attention(q, cache, table, n)
        assert ck.ck_profile_end()["attention"][1] == launches
        ck.ck_profile_begin(with_events=False)
        ck.ck_paged_attention(q, cache, table, n, window=100, sinks=4)
        assert ck.ck_profile_end()["attention"][1] == 1


def test_windows_up_to_the_largest_integer():
    q, cache, table, n = make([3000, 41], 4, 2, 64, 16, torch.bfloat16, False, seed=42)
    want = ck.ck_paged_attention(q, cache, table, n)
    most = 2 ** 63 - 1
    for window, sinks in ((most, 0), (most, 4), (most, most), (most - 3, 4), (5, most)):
        ck.ck_profile_begin(with_events=False)
        out = ck.ck_paged_attention(q, cache, table, n, window=window, sinks=sinks)
        assert ck.ck_profile_end()["attention"][1] == 2  # split, as without a window
        assert torch.equal(out, want)
