"""Attention over whole prompts against the 64-bit definition (the bound's terms are derived in
transformer_ref.attend; one rounding of the output on top)."""
import pytest
import torch

import int8_weight_quantized_gb300 as ck
import transformer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(q_lens, k_lens, hq, hkv, d, dtype, seed, q_std=1.5):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    tq, tk = sum(q_lens), sum(k_lens)
    q = (torch.randn((tq, hq, d), generator=g, device=DEV) * q_std).to(dtype)
    k, v = [torch.randn((tk, hkv, d), generator=g, device=DEV).to(dtype) for _ in range(2)]
    cu = [torch.tensor([0] + list(x), device=DEV).cumsum(0).to(torch.int32) for x in (q_lens, k_lens)]
    return q, k, v, cu[0], cu[1]


def seen_by(n, m, causal, window, sinks):
    i = torch.arange(n, device=DEV)[:, None] + (m - n)
    j = torch.arange(m, device=DEV)[None]
    if not causal:
        return torch.ones((n, m), dtype=torch.bool, device=DEV)
    seen = j <= i
    if window:
        seen &= (i - j < window) | (j < sinks)
    return seen


def check(q, k, v, cu_q, cu_k, out, lse, causal=True, window=0, sinks=0, scale=None, heads=None):
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    cq, ck_ = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cq) - 1):
        qs, ks = slice(cq[b], cq[b + 1]), slice(ck_[b], ck_[b + 1])
        n, m = cq[b + 1] - cq[b], ck_[b + 1] - ck_[b]
        if n == 0:
            continue
        seen = seen_by(n, m, causal, window, sinks)
        for h in heads or range(hq):
            want, want_lse, tol, lse_tol = ref.attend(q[qs, h], k[ks, h // (hq // hkv)], v[ks, h // (hq // hkv)], scale,
                                                      seen, ref.unit(q.dtype), ref.least(q.dtype))
            tol = tol + (want.abs() + tol) * ref.unit(q.dtype) + ref.least(q.dtype)
            ref.assert_within(out[qs, h], want, tol, "sequence %d head %d" % (b, h))
            if lse is not None:
                none = ~seen.any(-1)
                assert (lse[h, qs][none] == -float("inf")).all()
                ref.assert_within(lse[h, qs][~none], want_lse[~none], lse_tol[~none], "lse %d %d" % (b, h))


MIXED = [1, 2, 127, 128, 129, 255, 256, 257, 0, 300]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_batches(d, dtype, causal):
    q, k, v, cq, cku = make(MIXED, MIXED, 4, 2, d, dtype, seed=d)
    out, lse = ck.ck_attention(q, k, v, cq, causal=causal, return_lse=True)
    check(q, k, v, cq, cku, out, lse, causal)
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d", [(6, 2, 64), (8, 1, 128), (3, 3, 128), (16, 1, 64)])
def test_more_keys_than_queries_and_fewer(hq, hkv, d, causal):
    """Chunks of a prompt against all keys so far; queries before the first key see nothing."""
    q_lens, k_lens = [1, 5, 130, 64, 200, 33, 7], [500, 5, 700, 0, 90, 300, 1]
    q, k, v, cq, cku = make(q_lens, k_lens, hq, hkv, d, torch.bfloat16, seed=hq)
    out, lse = ck.ck_attention(q, k, v, cq, cku, causal=causal, return_lse=True)
    check(q, k, v, cq, cku, out, lse, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 4), (100, 0), (128, 1), (129, 130), (300, 5), (2000, 4)])
def test_window_and_first_tokens(window, sinks, d):
    lens = [1, 700, 129, 385]
    q, k, v, cq, cku = make(lens, lens, 2, 1, d, torch.bfloat16, seed=window + sinks)
    out, lse = ck.ck_attention(q, k, v, cq, window=window, sinks=sinks, return_lse=True)
    check(q, k, v, cq, cku, out, lse, True, window, sinks)


def test_window_with_more_keys_than_queries():
    q, k, v, cq, cku = make([150, 40], [900, 41], 4, 2, 128, torch.float16, seed=3)
    out, lse = ck.ck_attention(q, k, v, cq, cku, window=70, sinks=4, return_lse=True)
    check(q, k, v, cq, cku, out, lse, True, 70, 4)


def test_long_prompt():
    q, k, v, cq, cku = make([3001], [3001], 4, 2, 128, torch.bfloat16, seed=4)
    out, lse = ck.ck_attention(q, k, v, cq, return_lse=True)
    check(q, k, v, cq, cku, out, lse)
    again = ck.ck_attention(q, k, v, cq)
    assert torch.equal(out, again)


def test_views_of_a_fused_projection():
    hq, hkv, d, t = 6, 2, 128, 333
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device=DEV).to(torch.bfloat16)
    x = qkv.view(t, hq + 2 * hkv, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    cu = torch.tensor([0, 100, 333], dtype=torch.int32, device=DEV)
    out = ck.ck_attention(q, k, v, cu)
    assert torch.equal(out, ck.ck_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu))
    check(q, k, v, cu, cu, out, None)


def test_sharp_scores_and_rising_maxima():
    """Scores that grow along the keys: the running maximum rises at every tile."""
    n, d = 1000, 64
    q, k, v, cq, cku = make([n], [n], 2, 1, d, torch.bfloat16, seed=6, q_std=1.0)
    k = (k.float() * 0.1 + torch.linspace(0, 6, n, device=DEV)[:, None, None]).to(torch.bfloat16)
    q = q.abs()
    out, lse = ck.ck_attention(q, k, v, cq, causal=False, return_lse=True, scale=0.5)
    check(q, k, v, cq, cku, out, lse, causal=False, scale=0.5)
    k2 = k.flip(0).contiguous()
    out, lse = ck.ck_attention(q, k2, v, cq, causal=False, return_lse=True, scale=0.5)
    check(q, k2, v, cq, cku, out, lse, causal=False, scale=0.5)


def test_negative_and_zero_scale():
    q, k, v, cq, cku = make([200], [200], 2, 1, 64, torch.float16, seed=11)
    for scale in (-0.125, 0.0):
        out, lse = ck.ck_attention(q, k, v, cq, scale=scale, return_lse=True)
        check(q, k, v, cq, cku, out, lse, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,row,window,sinks", [
    ([300], 299, 0, 0), ([300], 130, 0, 0), ([300], 10, 50, 4), ([40, 300, 5], 339, 0, 0), ([700], 2, 64, 1),
])
def test_what_a_query_does_not_see_has_no_part(lens, row, window, sinks, fill, d):
    """A key and value row of NaN or infinities changes the rows that see it, and no other."""
    q, k, v, cq, cku = make(lens, lens, 2, 1, d, torch.bfloat16, seed=row)
    clean, clean_lse = ck.ck_attention(q, k, v, cq, window=window, sinks=sinks, return_lse=True)
    k, v = k.clone(), v.clone()
    k[row], v[row] = fill, fill
    out, lse = ck.ck_attention(q, k, v, cq, window=window, sinks=sinks, return_lse=True)
    sees = torch.zeros(sum(lens), dtype=torch.bool, device=DEV)
    lo = 0
    for n in lens:
        if lo <= row < lo + n:
            sees[lo:lo + n] = seen_by(n, n, True, window, sinks)[:, row - lo]
        lo += n
    hidden = ~sees
    assert not out[hidden].isnan().any()
    # rows that do not see it agree with the clean run to the rounding of their weights
    ref.assert_within(out[hidden], clean[hidden], 4 * ref.unit(torch.bfloat16) * (clean[hidden].abs().double() + 1), "rows")
    ref.assert_within(lse[:, hidden], clean_lse[:, hidden], torch.full_like(lse[:, hidden], 1e-4), "lse")


def test_value_rows_of_nan_alone():
    """NaN in the value rows only: their scores are ordinary, their weights are not zero."""
    q, k, v, cq, cku = make([257], [257], 2, 1, 128, torch.float16, seed=9)
    v = v.clone()
    v[200, 0, 5] = float("nan")
    v[140, 0, 7] = float("inf")
    out = ck.ck_attention(q, k, v, cq)
    clean = v.clone()
    clean[200, 0, 5] = clean[140, 0, 7] = 0
    assert out[200:, :, 5].isnan().all() and not out[:200, :, 5].isnan().any()
    assert (out[140:, :, 7] == float("inf")).all() and out[:140, :, 7].isfinite().all()
    keep = [c for c in range(128) if c not in (5, 7)]
    check(q[:, :, :], k, clean, cq, cku, torch.where(torch.isfinite(out), out, ck.ck_attention(q, k, clean, cq)), None)
    assert out[:, :, keep].isfinite().all()


def test_bounds_out_of_range_are_reported():
    """Sequence bounds beyond the tensors: checked in the kernel, NaN for their rows, reported."""
    assert ck.ck_device_error() == 0
    q, k, v, cq, cku = make([64, 64], [64, 64], 2, 1, 64, torch.bfloat16, seed=12)
    bad = cku.clone()
    bad[2] = 129
    out = ck.ck_attention(q, k, v, cq, bad)
    assert out[64:].isnan().all()
    assert torch.equal(out[:64], ck.ck_attention(q, k, v, cq)[:64])
    assert ck.ck_device_error(clear=True) == 128


def test_other_streams_and_graphs():
    q, k, v, cq, cku = make([500, 77], [500, 77], 4, 2, 128, torch.bfloat16, seed=13)
    want = ck.ck_attention(q, k, v, cq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [ck.ck_attention(q, k, v, cq, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.ck_attention(q, k, v, cq, out=out)
    q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ck.ck_attention(q, k, v, cq))


@pytest.mark.parametrize("hq,hkv", [(3, 1), (4, 1), (10, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 3)])
def test_many_more_tiles_than_multiprocessors(hq, hkv, d, window, sinks):
    """Blocks go from item to item, with odd and even numbers of heads to a key head; empty and
    one-token sequences stand between long ones."""
    lens = [1500, 0, 1, 2049, 128, 0, 1281, 3, 256, 257] * 2
    q, k, v, cq, cku = make(lens, lens, hq, hkv, d, torch.bfloat16, seed=hq + d)
    out, lse = ck.ck_attention(q, k, v, cq, window=window, sinks=sinks, return_lse=True)
    check(q, k, v, cq, cku, out, lse, True, window, sinks, heads=(0, hq - 1))
    # the other heads: as the same head computed alone
    for h in range(1, hq - 1):
        kv = h // (hq // hkv)
        one = ck.ck_attention(q[:, h:h + 1], k[:, kv:kv + 1], v[:, kv:kv + 1], cq, window=window, sinks=sinks)
        ref.assert_within(out[:, h:h + 1], one, 4 * ref.unit(torch.bfloat16) * (one.abs().double() + 1), "head")
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("hq", [3, 4])
def test_hidden_infinities_with_shared_heads(hq):
    """What the last tests ask, with more heads to a key head: each head's rows stand alone."""
    q, k, v, cq, cku = make([300, 140], [300, 140], hq, 1, 64, torch.bfloat16, seed=hq)
    want = ck.ck_attention(q, k, v, cq)
    v = v.clone()
    v[220] = float("inf")
    v[300 + 100] = float("nan")
    out = ck.ck_attention(q, k, v, cq)
    hidden = torch.ones(440, dtype=torch.bool, device=DEV)
    hidden[220:300] = hidden[400:440] = False
    ref.assert_within(out[hidden], want[hidden], 4 * ref.unit(torch.bfloat16) * (want[hidden].abs().double() + 1), "rows")
    assert not out[~hidden].isfinite().any()


@pytest.mark.parametrize("hq", [2, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [1, 31, 32, 33, 128, 160])
def test_numbers_of_first_tokens(sinks, d, hq):
    """A few first tokens are a narrow key tile, more of them whole tiles."""
    lens = [700, 33, 520]
    q, k, v, cq, cku = make(lens, lens, hq, 1, d, torch.float16, seed=sinks)
    out, lse = ck.ck_attention(q, k, v, cq, window=90, sinks=sinks, return_lse=True)
    check(q, k, v, cq, cku, out, lse, True, 90, sinks)


@pytest.mark.parametrize("row", [0, 3, 4, 31, 32, 127])
def test_first_tokens_beside_hidden_rows(row):
    """NaN in a row of the first key tile: only the queries that see it change."""
    q, k, v, cq, cku = make([600], [600], 2, 1, 64, torch.bfloat16, seed=row)
    clean = ck.ck_attention(q, k, v, cq, window=100, sinks=4)
    k, v = k.clone(), v.clone()
    k[row] = v[row] = float("nan")
    out = ck.ck_attention(q, k, v, cq, window=100, sinks=4)
    sees = seen_by(600, 600, True, 100, 4)[:, row]
    assert out[sees].isnan().all()
    ref.assert_within(out[~sees], clean[~sees], 4 * ref.unit(torch.bfloat16) * (clean[~sees].abs().double() + 1), "rows")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [3, 127, 128, 200, 383, 450])
def test_one_key_far_above_the_others(at, d, dtype):
    """A maximum hundreds above all before it, in any part of any tile: sums start anew there."""
    q, k, v, cq, cku = make([512], [512], 2, 1, d, dtype, seed=at)
    k = k.clone()
    k[at] = (30.0 * q[at // 2, 0].float().sign()).to(dtype)
    for causal in (True, False):
        out, lse = ck.ck_attention(q, k, v, cq, causal=causal, return_lse=True, scale=1.0)
        check(q, k, v, cq, cku, out, lse, causal, scale=1.0)


@pytest.mark.parametrize("hq", [3, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_hidden_infinities_among_many_sequences(hq, d):
    """Infinities and NaN in some sequences' value rows, with more tiles than multiprocessors."""
    lens = [300, 140] * 24
    q, k, v, cq, cku = make(lens, lens, hq, 1, d, torch.bfloat16, seed=hq)
    want = ck.ck_attention(q, k, v, cq)
    v = v.clone()
    starts = cq.tolist()
    sees = torch.zeros(sum(lens), dtype=torch.bool, device=DEV)
    for s, row, fill in ((0, 220, float("inf")), (7, 100, float("nan")), (30, 0, -float("inf")), (46, 299, float("nan"))):
        v[starts[s] + row] = fill
        sees[starts[s] + row:starts[s + 1]] = True
    out = ck.ck_attention(q, k, v, cq)
    ref.assert_within(out[~sees], want[~sees], 4 * ref.unit(torch.bfloat16) * (want[~sees].abs().double() + 1), "rows")
    assert not out[sees].isfinite().any()


def prefilled(q):
    return torch.full_like(q, 7.0), torch.full((q.shape[1], q.shape[0]), 7.0, device=DEV)


@pytest.mark.parametrize("hq", [3, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bounds", [[0, 64, 700, 1000], [0, 64, 700, 641], [0, 64, 700, 2 ** 31 - 1], [-5, 64, 700, 640],
                                    [-2 ** 31, 64, 700, 640], [0, 64, 5000, 640]])
def test_query_bounds_out_of_range_give_nan(bounds, d, hq):
    """Rows of the tensor that a sequence with bounds outside it names are NaN, with lse; the other
    sequences' rows are right, and the word is set."""
    assert ck.ck_device_error() == 0
    total = 640
    q, k, v, _, _ = make([total], [total], hq, 1, d, torch.bfloat16, seed=21)
    cku = torch.tensor([0, 64, 264, 640], dtype=torch.int32, device=DEV)
    cu = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    out, lse = prefilled(q)
    ck.ck_attention(q, k, v, cu, cku, out=out, lse=lse, return_lse=True)
    assert ck.ck_device_error(clear=True) == 128
    bad = torch.zeros(total, dtype=torch.bool, device=DEV)
    for lo, hi in zip(bounds, bounds[1:]):
        if lo < 0 or hi > total:
            bad[max(lo, 0):max(min(hi, total), 0)] = True
        elif lo <= hi:
            b = bounds.index(lo)
            ks = slice(cku[b].item(), cku[b + 1].item())
            one = [torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (hi - lo, ks.stop - ks.start)]
            want = ck.ck_attention(q[lo:hi], k[ks], v[ks], *one)
            ref.assert_within(out[lo:hi], want, 4 * ref.unit(torch.bfloat16) * (want.abs().double() + 1), "rows")
    assert out[bad].isnan().all() and lse[:, bad].isnan().all()
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("hq", [3, 4])
@pytest.mark.parametrize("which", ["q", "k", "both"])
def test_bounds_that_descend_are_reported(which, hq):
    """A sequence whose bounds descend has no rows of its own; the word says so even where no other
    row depends on it.  (Rows that two sequences claim get either's.)"""
    assert ck.ck_device_error() == 0
    q, k, v, cu, _ = make([1280], [1280], hq, 1, 64, torch.bfloat16, seed=22)
    up = torch.tensor([0, 900, 900, 1280], dtype=torch.int32, device=DEV)
    down = torch.tensor([0, 1000, 50, 1280], dtype=torch.int32, device=DEV)
    out, lse = prefilled(q)
    ck.ck_attention(q, k, v, up if which == "k" else down, up if which == "q" else down, out=out, lse=lse, return_lse=True)
    assert ck.ck_device_error(clear=True) == 128
    if which == "both":  # rows that one sequence alone claims
        want = ck.ck_attention(q[:1000], k[:1000], v[:1000], torch.tensor([0, 1000], dtype=torch.int32, device=DEV))
        ref.assert_within(out[:50], want[:50], 4 * ref.unit(torch.bfloat16) * (want[:50].abs().double() + 1), "first")
        want = ck.ck_attention(q[50:], k[50:], v[50:], torch.tensor([0, 1230], dtype=torch.int32, device=DEV))
        ref.assert_within(out[1000:], want[950:], 4 * ref.unit(torch.bfloat16) * (want[950:].abs().double() + 1), "last")
    if which == "q":
        assert not (out == 7.0).all(-1).any()


def milliseconds(fn):
    fn()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    fn()
    ev[1].record()
    torch.cuda.synchronize()
    return ev[0].elapsed_time(ev[1])


@pytest.mark.parametrize("n,hq,hkv,d,window,causal", [(2048, 4, 1, 128, 0, True), (4096, 4, 1, 128, 0, True), (4096, 3, 1, 64, 0, True),
                                                      (2048, 2, 2, 128, 300, True), (2000, 2, 1, 64, 0, False)])
def test_a_channel_of_infinities(n, hq, hkv, d, window, causal):
    """One value channel that has overflowed in every token: the other channels are right, and the
    call does not take the time of a computation row by row."""
    q, k, v, cq, cku = make([n, 50], [n, 50], hq, hkv, d, torch.float16, seed=n + d)
    clean = v.clone()
    clean[..., 3] = 0.0
    v = v.clone()
    v[..., 3] = float("inf")
    sinks = 4 if window else 0
    call = lambda x: ck.ck_attention(q, k, x, cq, causal=causal, window=window, sinks=sinks, return_lse=True)  # noqa: E731
    out, lse = call(v)
    assert (out[..., 3] == float("inf")).all()
    out[..., 3] = 0.0
    check(q, k, clean, cq, cku, out, lse, causal, window, sinks)
    took, plain = milliseconds(lambda: call(v)), milliseconds(lambda: call(clean))
    print("channel of infinities: %d tokens, heads %d of %d: %.3f ms, %.3f without" % (n, hq, d, took, plain))
    assert took < 10.0
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_a_hidden_row_at_the_end_of_a_long_prompt(d):
    n = 6000
    q, k, v, cq, cku = make([n], [n], 2, 1, d, torch.bfloat16, seed=41)
    clean, clean_lse = ck.ck_attention(q, k, v, cq, return_lse=True)
    v = v.clone()
    v[n - 1] = float("nan")
    out, lse = ck.ck_attention(q, k, v, cq, return_lse=True)
    assert out[n - 1].isnan().all()
    assert torch.equal(lse, clean_lse)
    ref.assert_within(out[:n - 1], clean[:n - 1], 4 * ref.unit(torch.bfloat16) * (clean[:n - 1].abs().double() + 1), "rows")
    assert ck.ck_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3), (70, 40)])
def test_every_kind_of_value_among_visible_and_hidden_rows(window, sinks, d):
    """Infinities of both signs and NaN scattered over values: each output is what its visible keys
    make it, finite ones to the usual bound."""
    n = 400
    q, k, v, cq, cku = make([n], [n], 2, 1, d, torch.bfloat16, seed=window + d)
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    clean = v.clone()
    v = v.clone()
    for fill, often in ((float("inf"), 0.002), (-float("inf"), 0.002), (float("nan"), 0.001)):
        at = torch.rand(v.shape, generator=g, device=DEV) < often
        v[at], clean[at] = fill, 0.0
    out, lse = ck.ck_attention(q, k, v, cq, window=window, sinks=sinks, return_lse=True)
    seen = seen_by(n, n, True, window, sinks).double()
    plus, minus, nan = [(seen @ x[:, 0].double()) > 0 for x in (v == float("inf"), v == -float("inf"), v.isnan())]
    for h in range(2):
        o = out[:, h]
        assert torch.equal(o.isnan(), nan | (plus & minus))
        assert torch.equal(o == float("inf"), plus & ~minus & ~nan)
        assert torch.equal(o == -float("inf"), minus & ~plus & ~nan)
    some = (plus | minus | nan)[:, None].expand_as(out)
    clean_out = ck.ck_attention(q, k, clean, cq, window=window, sinks=sinks)
    check(q, k, clean, cq, cku, torch.where(some, clean_out, out), lse, True, window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 40])
def test_rows_whose_scores_are_all_minus_infinity(window, d):
    """A softmax over scores of minus infinity alone is 0 / 0, as over the cache; a row that sees a
    finite score beside them, and one that sees no key, are not that."""
    n = 300
    q, k, v, _, _ = make([n + 20], [n], 2, 1, d, torch.bfloat16, seed=51)
    q[..., 0] = q[..., 0].abs() + 0.5
    k = k.clone()
    k[:200] = 0.0
    k[:200, :, 0] = -float("inf")
    cu_q, cu_k = [torch.tensor([0, x], dtype=torch.int32, device=DEV) for x in (n + 20, n)]
    out, lse = ck.ck_attention(q, k, v, cu_q, cu_k, window=window, return_lse=True)
    assert (out[:20] == 0).all() and (lse[:, :20] == -float("inf")).all()
    assert out[20:220].isnan().all() and (lse[:, 20:220] == -float("inf")).all()
    assert out[220:].isfinite().all()
    cache = ck.KVCache(*[x[:, 0].view(n // 10, 1, 10, d).contiguous() for x in (k, v)])
    table = torch.arange(n // 10, dtype=torch.int32, device=DEV)[None]
    for length in (1, 100, 200, 300):
        one, one_lse = ck.ck_paged_attention(q[length + 19:length + 20], cache, table,
                                             torch.tensor([length], dtype=torch.int32, device=DEV), window=window,
                                             return_lse=True)
        assert torch.equal(one.isnan(), out[length + 19:length + 20].isnan())
        assert torch.equal(one_lse[0].isinf(), lse[:, length + 19].isinf())
