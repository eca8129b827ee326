"""The operators around the linear layers reject bad arguments before any device work, through
the C ABI (with pointers that are never dereferenced) and through the binding."""
import ctypes
import struct

import pytest
import torch

import int8_weight_quantized_gb300 as ck

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    from int8_weight_quantized_gb300 import build
    build.build()
    return ck.load_library()


def cache(**kw):
    f = dict(k=4096, v=4096, k_scale=4096, v_scale=4096, num_pages=4, page_size=16, kv_heads=2, head_dim=64, dtype=0)
    f.update(kw)
    return struct.pack("@PPPPqqqqi", *[f[n] for n in ("k", "v", "k_scale", "v_scale", "num_pages", "page_size", "kv_heads",
                                                    "head_dim", "dtype")])


def norm_rope(lib, **kw):
    f = dict(qkv=P, stride=512, tokens=3, hq=4, hkv=2, d=64, dtype=0, norm=1, qw=None, kw=None, eps=1e-6, rot=64,
             inter=0, pos=P, table=P, max_pos=10, q=P, k=None, cache=cache(), slots=P)
    f.update(kw)
    c = f["cache"]
    return lib.ck_qk_norm_rope(f["qkv"], f["stride"], f["tokens"], f["hq"], f["hkv"], f["d"], f["dtype"], f["norm"],
                               f["qw"], f["kw"], f["eps"], f["rot"], f["inter"], f["pos"], f["table"], f["max_pos"],
                               f["q"], f["k"], c, f["slots"], None)


@pytest.mark.parametrize("kw,what", [
    (dict(dtype=2), "dtype"), (dict(hq=3), "multiple of kv_heads"), (dict(hkv=0), "multiple of kv_heads"),
    (dict(d=60), "head_dim"), (dict(d=264), "head_dim"), (dict(rot=24), "rot_dim"), (dict(rot=128), "rot_dim"),
    (dict(norm=2), "norm"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(stride=504), "qkv_stride"),
    (dict(stride=516), "qkv_stride"), (dict(tokens=-1), "tokens"), (dict(tokens=2 ** 31), "tokens"),
    (dict(max_pos=0), "max_pos"), (dict(qkv=None), "qkv must not be NULL"), (dict(qkv=ODD), "qkv must be 16-byte"),
    (dict(q=None), "q_out"), (dict(pos=None), "positions"), (dict(pos=ODD), "positions must be aligned"),
    (dict(table=None), "cos_sin"), (dict(qw=ODD), "q_weight"), (dict(k=ODD), "k_out"), (dict(slots=None), "slots"),
    (dict(cache=cache(head_dim=128)), "cache holds"), (dict(cache=cache(dtype=1)), "cache dtype"),
    (dict(cache=cache(k=0)), "c->k must not be NULL"), (dict(cache=cache(dtype=2, v_scale=0)), "v_scale"),
    (dict(cache=cache(page_size=0)), "page_size"),
])
def test_norm_rope_refusals(lib, kw, what):
    assert norm_rope(lib, **kw) == ck.CK_ERR_INVALID_ARG
    assert what in ck.ck_last_error()


def paged(lib, **kw):
    f = dict(q=P, stride=256, cache=cache(), table=P, blocks=50, lens=P, batch=3, hq=4, dtype=0, scale=0.1, window=0,
             sinks=0, out=P, lse=None, ws=P, nbytes=1 << 40)
    f.update(kw)
    c = f["cache"]
    return lib.ck_paged_attention(f["q"], f["stride"], c, f["table"],
                                  f["blocks"], f["lens"], f["batch"], f["hq"], f["dtype"], f["scale"], f["window"],
                                  f["sinks"], f["out"], f["lse"], f["ws"], f["nbytes"], None)


@pytest.mark.parametrize("kw,what", [
    (dict(dtype=3), "dtype"), (dict(cache=None), "cache"), (dict(hq=5), "multiple of kv_heads"),
    (dict(cache=cache(head_dim=96)), "head_dim"), (dict(window=-1), "window"), (dict(sinks=-2), "sinks"),
    (dict(stride=248), "q_stride"), (dict(scale=float("inf")), "scale"), (dict(batch=-1), "batch"),
    (dict(blocks=0), "max_blocks"), (dict(blocks=2 ** 40), "max_blocks"), (dict(q=None), "q must"),
    (dict(table=None), "block_table"), (dict(lens=None), "seq_lens"), (dict(out=ODD), "out must be 16-byte"),
    (dict(lse=ODD), "lse"), (dict(ws=None), "workspace"), (dict(nbytes=0), "workspace too small"),
    (dict(cache=cache(dtype=1)), "cache dtype"),
])
def test_paged_attention_refusals(lib, kw, what):
    assert paged(lib, **kw) == ck.CK_ERR_INVALID_ARG
    assert what in ck.ck_last_error()


def prompt(lib, **kw):
    f = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, cq=P, ck=P, batch=2, tq=9, tk=9, hq=4, hkv=2, d=64, dtype=0,
             scale=0.1, causal=1, window=0, sinks=0, out=P, lse=None)
    f.update(kw)
    return lib.ck_attention(f["q"], f["qs"], f["k"], f["ks"], f["v"], f["vs"], f["cq"], f["ck"], f["batch"], f["tq"],
                            f["tk"], f["hq"], f["hkv"], f["d"], f["dtype"], f["scale"], f["causal"], f["window"],
                            f["sinks"], f["out"], f["lse"], None)


@pytest.mark.parametrize("kw,what", [
    (dict(dtype=2), "dtype"), (dict(hq=3), "multiple of kv_heads"), (dict(d=80), "head_dim"),
    (dict(window=-1), "window"), (dict(causal=2), "causal"), (dict(causal=0, window=5), "causal = 1"),
    (dict(qs=128), "q_stride"), (dict(ks=129), "k_stride"), (dict(vs=0), "v_stride"), (dict(scale=float("nan")), "scale"),
    (dict(batch=-1), "batch"), (dict(tq=2 ** 31), "total_q"), (dict(tk=-1), "total_k"), (dict(q=None), "q must"),
    (dict(k=None), "k must"), (dict(v=ODD), "v must"), (dict(cq=None), "cu_q"), (dict(ck=ODD), "cu_k"),
    (dict(out=None), "out"),
])
def test_attention_refusals(lib, kw, what):
    assert prompt(lib, **kw) == ck.CK_ERR_INVALID_ARG
    assert what in ck.ck_last_error()


def int4(lib, **kw):
    f = dict(x=P, w=P, s=P, bias=None, res=None, y=P, M=2, N=16, K=256, group=128, dtype=0, out=0)
    f.update(kw)
    return lib.ck_int4_linear(f["x"], f["w"], f["s"], f["bias"], f["res"], f["y"], f["M"], f["N"], f["K"], f["group"],
                              f["dtype"], f["out"], None)


@pytest.mark.parametrize("kw,what", [
    (dict(dtype=2), "dtype"), (dict(out=4), "out_dtype"), (dict(N=12), "multiple of 8"), (dict(K=192), "multiple of 128"),
    (dict(group=48), "group"), (dict(K=384, group=256), "multiple of group"), (dict(M=-1), "M must"),
    (dict(N=2 ** 30, K=2 ** 20), "2^39"), (dict(x=None), "x must"), (dict(w=ODD), "w4"), (dict(s=None), "w_scale"),
    (dict(y=ODD), "y must"), (dict(bias=ODD), "bias"), (dict(res=ODD), "residual"),
])
def test_int4_refusals(lib, kw, what):
    assert int4(lib, **kw) == ck.CK_ERR_INVALID_ARG
    assert what in ck.ck_last_error()


def test_int4_weight_refusals(lib):
    assert lib.ck_int4_prepare_weight(P, 16, 256, 100, P, P, None) == ck.CK_ERR_INVALID_ARG
    assert "group" in ck.ck_last_error()
    assert lib.ck_int4_prepare_weight(None, 16, 256, 128, P, P, None) == ck.CK_ERR_INVALID_ARG
    assert lib.ck_int4_pack(P, 12, 256, P, None) == ck.CK_ERR_INVALID_ARG


def test_nothing_to_do_is_ok(lib):
    assert norm_rope(lib, tokens=0, qkv=None, q=None) == ck.CK_OK
    assert paged(lib, batch=0, q=None) == ck.CK_OK
    assert prompt(lib, batch=0, q=None) == ck.CK_OK
    assert prompt(lib, tq=0, q=None) == ck.CK_OK
    assert int4(lib, M=0, x=None, y=None) == ck.CK_OK


def test_no_device_is_reported_not_faked(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for st in (norm_rope(lib), paged(lib), prompt(lib), int4(lib)):
        assert st in (ck.CK_ERR_CUDA, ck.CK_ERR_UNSUPPORTED_DEVICE)


def test_workspace_sizes(lib):
    assert lib.ck_paged_attention_workspace_size(-1, 8, 2, 64, 4096) == 0
    assert lib.ck_paged_attention_workspace_size(1, 8, 2, 64, 100) == 0  # short tables need none
    assert 0 < lib.ck_paged_attention_workspace_size(1 << 20, 8, 2, 128, 1 << 20) < 1 << 28


def test_binding_checks(lib):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ck.ck_qk_norm_rope(x.float(), None, None, 2, 1)
    with pytest.raises(ValueError):
        ck.ck_qk_norm_rope(x, None, None, 2, 1)  # not a CUDA tensor
    with pytest.raises(TypeError):
        ck.KVCache(torch.zeros((2, 1, 4, 64)), torch.zeros((2, 1, 4, 64)))
    with pytest.raises(ValueError):
        ck.KVCache(torch.zeros((2, 4, 64), dtype=torch.int8), torch.zeros((2, 4, 64), dtype=torch.int8))
    cache = ck.KVCache(*[torch.zeros((2, 1, 4, 64), dtype=torch.int8)] * 2)
    with pytest.raises(ValueError):  # not CUDA tensors
        ck.ck_paged_attention(x.view(4, 4, 64), cache, None, None)
    with pytest.raises(TypeError):
        ck.ck_int4_linear(x.float(), None, None)
    with pytest.raises(TypeError):
        ck.ck_attention(x.view(4, 4, 64).float(), x.view(4, 4, 64), x.view(4, 4, 64), None)


def test_rope_table():
    t = ck.rope_table(5, 4, base=100.0, device="cpu")
    assert t.shape == (5, 4) and t.dtype == torch.float32
    want = torch.tensor([3.0, 0.3], dtype=torch.float64)
    assert torch.allclose(t[3].double(), torch.cat([want.cos(), want.sin()]), atol=1e-7)
