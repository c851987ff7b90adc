"""The serving ops' refusals, on the host (no GPU): sizes, NULL pointers, page sizes, strides and
workspaces are checked before any CUDA call (placeholder addresses are never dereferenced on
these paths), and the binding refuses host tensors, wrong shapes and wrong types."""
import ctypes

import pytest
import torch

from zeroth_order_fine_b200 import zo


@pytest.fixture(scope="module")
def L():
    from zeroth_order_fine_b200 import build
    build.build()
    return zo.lib()


P = ctypes.c_void_p(0x10000)
Q = ctypes.c_void_p(0x20000)


def tables(L, **kw):
    a = dict(old=P, new=P, R=4, page=16, table=P, blocks=8, ring=P, pages=64, state=P, out=Q, cu=P,
             slots=P, toks=32)
    a.update(kw)
    return L.zo_op_block_tables(a["old"], a["new"], a["R"], a["page"], a["table"], a["blocks"],
                                a["ring"], a["pages"], a["state"], a["out"], a["cu"], a["slots"],
                                a["toks"], None)


@pytest.mark.parametrize("kw", [dict(R=-1), dict(page=0), dict(page=4), dict(page=24), dict(page=512),
                                dict(page=-16), dict(blocks=0), dict(pages=0), dict(toks=-1),
                                dict(old=None), dict(new=None), dict(table=None), dict(ring=None),
                                dict(state=None), dict(out=None), dict(cu=None), dict(slots=None),
                                dict(out=P), dict(pages=1 << 27), dict(pages=0x7fffffff)])
def test_block_tables_refuses(L, kw):
    assert tables(L, **kw) == zo.ZO_ERR_ARG


def write(L, **kw):
    a = dict(qkv=P, ld=3 * 128, slots=P, T=4, cache=P, n=64, H=1, kv=1, hd=128, dt=1)
    a.update(kw)
    return L.zo_op_kv_write(a["qkv"], a["ld"], a["slots"], a["T"], a["cache"], a["n"], a["H"], a["kv"],
                            a["hd"], a["dt"], None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(n=0), dict(H=-1), dict(kv=0), dict(hd=0), dict(dt=2),
                                dict(ld=3 * 128 - 1), dict(qkv=None), dict(slots=None),
                                dict(cache=None)])
def test_kv_write_refuses(L, kw):
    assert write(L, **kw) == zo.ZO_ERR_ARG


def test_kv_write_of_no_rows_is_a_no_op(L):
    assert write(L, T=0, qkv=None, slots=None, cache=None) == zo.ZO_OK


def attn(L, **kw):
    a = dict(q=P, ldq=512, cache=P, slots=1024, table=P, blocks=8, page=16, cu=P, lens=P, R=2, T=4,
             new=2, H=4, kv=2, hd=128, dt=1, out=P, ldo=512, ws=P, wsb=1 << 40, impl=0)
    a.update(kw)
    return L.zo_op_attention_paged(a["q"], a["ldq"], a["cache"], a["slots"], a["table"], a["blocks"],
                                   a["page"], a["cu"], a["lens"], a["R"], a["T"], a["new"], a["H"],
                                   a["kv"], a["hd"], a["dt"], a["out"], a["ldo"], a["ws"], a["wsb"],
                                   a["impl"], None)


@pytest.mark.parametrize("kw", [dict(R=-1), dict(T=-1), dict(new=-1), dict(blocks=0), dict(page=12),
                                dict(page=4), dict(page=512), dict(H=0), dict(kv=0), dict(H=5),
                                dict(hd=0), dict(dt=3), dict(impl=3), dict(impl=-1), dict(ldq=511),
                                dict(ldo=511), dict(slots=0), dict(slots=1000), dict(slots=1 << 31),
                                dict(q=None), dict(cache=None), dict(table=None), dict(cu=None),
                                dict(lens=None), dict(out=None), dict(ws=None),
                                dict(ws=ctypes.c_void_p(0x10008)), dict(wsb=0)])
def test_attention_paged_refuses(L, kw):
    assert attn(L, **kw) == zo.ZO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(hd=96, ldq=4 * 96, ldo=4 * 96),
                                dict(impl=2, dt=0),                      # tensor cores need bf16
                                dict(impl=2, hd=32),
                                dict(impl=2, ldq=513), dict(impl=2, ldo=513),
                                dict(impl=2, q=ctypes.c_void_p(0x10002)),
                                dict(impl=2, cache=ctypes.c_void_p(0x10008)),
                                dict(impl=2, out=ctypes.c_void_p(0x10004)),
                                dict(impl=2, H=258, kv=2, ldq=258 * 128, ldo=258 * 128)])
def test_attention_paged_unsupported(L, kw):
    assert attn(L, **kw) == zo.ZO_ERR_UNSUPPORTED


def test_attention_paged_without_rows_is_a_no_op(L):
    assert attn(L, R=0, q=None, cache=None) == zo.ZO_OK
    assert attn(L, T=0, q=None, cache=None) == zo.ZO_OK


def adapt(L, **kw):
    a = dict(x=P, W=P, bias=None, A=P, B=P, ids=P, sc=P, n=4, r=16, y=P, M=8, N=256, K=128, dt=1, act=0,
             acc=0, ws=P, wsb=1 << 40, impl=0)
    a.update(kw)
    return L.zo_op_linear_adapters(a["x"], a["W"], a["bias"], a["A"], a["B"], a["ids"], a["sc"],
                                   a["n"], a["r"], a["y"], a["M"], a["N"], a["K"], a["dt"], a["act"],
                                   a["acc"], a["ws"], a["wsb"], a["impl"], None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(N=0), dict(K=0), dict(n=0), dict(r=0), dict(r=257),
                                dict(n=8193, r=8), dict(dt=2), dict(act=2), dict(act=1, acc=1),
                                dict(impl=3), dict(x=None), dict(W=None), dict(A=None), dict(B=None),
                                dict(ids=None), dict(sc=None), dict(y=None), dict(ws=None), dict(wsb=0),
                                dict(ws=ctypes.c_void_p(0x10010))])
def test_linear_adapters_refuses(L, kw):
    assert adapt(L, **kw) == zo.ZO_ERR_ARG


@pytest.mark.parametrize("kw", [dict(impl=2, dt=0), dict(impl=2, K=124), dict(impl=2, N=252),
                                dict(impl=2, n=1, r=12), dict(impl=2, x=ctypes.c_void_p(0x10004)),
                                dict(impl=2, y=ctypes.c_void_p(0x10004))])
def test_linear_adapters_unsupported(L, kw):
    assert adapt(L, **kw) == zo.ZO_ERR_UNSUPPORTED


def test_linear_adapters_of_no_rows_is_a_no_op(L):
    assert adapt(L, M=0, x=None, y=None, ws=None) == zo.ZO_OK


def test_workspace_sizes(L):
    assert zo.zo_op_attention_paged_workspace(1, 1, 32, 8, 128) > 0
    for M in (1, 128, 129, 4096):
        # the rows' shrink at least, whatever form they take
        assert zo.zo_op_linear_adapters_workspace(M, 256, 128, 4, 16) >= M * 16 * 4
        assert zo.zo_op_linear_adapters_workspace(M, 256, 128, 4, 16, torch.float32) >= M * 16 * 4
    assert zo.zo_op_linear_adapters_workspace(-1, 256, 128, 4, 16) == 0


def test_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    b = torch.zeros(8, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        zo.zo_op_block_tables(i, i, torch.zeros(4, 8, dtype=torch.int32), i, i, i, 16, max_tokens=8)
    with pytest.raises(ValueError, match="CUDA"):
        zo.zo_op_kv_write(torch.zeros(4, 384, dtype=torch.bfloat16), i, b, 1, 1, 128)
    with pytest.raises(ValueError, match="CUDA"):
        zo.zo_op_attention_paged(b, b, torch.zeros(4, 8, dtype=torch.int32), 16, i, i, 1, 2, 1, 128)
    with pytest.raises(ValueError, match="CUDA"):
        zo.zo_op_linear_adapters(b, b, b, torch.zeros(8, 8, dtype=torch.bfloat16), i,
                                 torch.ones(2))
    with pytest.raises(ValueError, match="accumulate"):
        zo.zo_op_linear_adapters(b, b, b, b, i, torch.ones(2), accumulate=True)
    with pytest.raises(ValueError, match="rank"):
        zo.zo_op_linear_adapters(b, b, b, b, i, torch.ones(3))
