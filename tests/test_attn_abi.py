"""Refusals of the attention-side calls, on the host, before any GPU is touched (CPU)."""
import ctypes

import pytest
import torch

from bit_gemv_sherry_b200 import sherry as S

A16 = 0x100000     # never dereferenced: the checks fail first
WS = 0x200000


def rope(**kw):
    a = S.RopeArgs(q=A16, k=A16, q_out=A16, k_out=A16, q_stride=512, k_stride=128, q_out_stride=512,
                   k_out_stride=128, positions=A16, inv_freq=A16, T=3, Hq=8, Hk=2, D=64, R=64, eps=1e-5)
    for n, v in kw.items():
        setattr(a, n, v)
    return S.lib().sherry_qk_norm_rope(ctypes.addressof(a), None)


@pytest.mark.parametrize("status,kw", [
    (1, dict(q=None)), (1, dict(k_out=None)), (1, dict(positions=None)), (1, dict(inv_freq=None)),
    (2, dict(T=0)), (2, dict(Hq=-1)), (2, dict(Hq=0, Hk=0)), (2, dict(D=60)), (2, dict(D=264)), (2, dict(D=0)),
    (2, dict(R=72)), (2, dict(R=12)), (2, dict(R=-8)), (2, dict(q_stride=508)), (2, dict(k_out_stride=64)),
    (3, dict(q=A16 + 8)), (3, dict(k_out=A16 + 4)), (3, dict(q_weight=A16 + 4)), (3, dict(q_stride=514)),
    (3, dict(positions=A16 + 2)), (3, dict(in_type=1, q_stride=516)), (3, dict(out_type=1, k_out_stride=132)),
    (4, dict(in_type=2)), (4, dict(out_type=-1)), (4, dict(T=1 << 31)),
])
def test_rope_refusals(status, kw):
    assert rope(**kw) == status


def test_rope_null_args():
    assert S.lib().sherry_qk_norm_rope(None, None) == 1


def kv4(**kw):
    a = S.Kv4Args(cache=A16, pages=10, H=2, D=64, page_table=A16, width=4, table_stride=4, ctx_lens=A16,
                  cu_q=None, B=3, T=3)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


BAD_CACHE = [
    (1, dict(cache=None)), (1, dict(page_table=None)), (1, dict(ctx_lens=None)),
    (2, dict(pages=0)), (2, dict(H=0)), (2, dict(width=0)), (2, dict(table_stride=3)), (2, dict(B=0)),
    (2, dict(T=0)), (2, dict(T=4)),
    (3, dict(cache=A16 + 8)), (3, dict(page_table=A16 + 2)), (3, dict(cu_q=A16 + 1)),
    (4, dict(D=96)), (4, dict(pages=1 << 31)), (4, dict(width=1 << 26, table_stride=1 << 26)),
    (4, dict(B=65536, T=65536)), (4, dict(T=1 << 31, cu_q=A16)),
]


@pytest.mark.parametrize("status,kw", BAD_CACHE)
def test_cache_refusals(status, kw):
    a = kv4(**kw)
    L = S.lib()
    assert L.sherry_kv4_write(ctypes.addressof(a), A16, A16, 0, 128, 128, None) == status
    assert L.sherry_kv4_read(ctypes.addressof(a), A16, A16, 1, 128, 128, None) == status
    assert L.sherry_attn_kv4(ctypes.addressof(a), A16, 512, A16, 512, 8, 0, 1.0, WS, 1 << 30, None) == status


@pytest.mark.parametrize("status,args", [
    (1, (None, A16, 0, 128, 128)), (1, (A16, None, 0, 128, 128)), (4, (A16, A16, 2, 128, 128)),
    (2, (A16, A16, 0, 124, 128)), (2, (A16, A16, 0, 128, 64)), (3, (A16 + 8, A16, 0, 128, 128)),
    (3, (A16, A16, 0, 130, 128)), (3, (A16, A16, 1, 128, 132)),
])
def test_write_and_read_refusals(status, args):
    a = kv4()
    assert S.lib().sherry_kv4_write(ctypes.addressof(a), *args, None) == status
    assert S.lib().sherry_kv4_read(ctypes.addressof(a), *args, None) == status


@pytest.mark.parametrize("status,args", [
    (1, (None, 512, A16, 512, 8, 0, 1.0, WS, 1 << 30)), (1, (A16, 512, None, 512, 8, 0, 1.0, WS, 1 << 30)),
    (2, (A16, 512, A16, 512, 7, 0, 1.0, WS, 1 << 30)), (2, (A16, 512, A16, 512, 0, 0, 1.0, WS, 1 << 30)),
    (2, (A16, 512, A16, 512, 8, -1, 1.0, WS, 1 << 30)), (2, (A16, 504, A16, 512, 8, 0, 1.0, WS, 1 << 30)),
    (3, (A16 + 2, 512, A16, 512, 8, 0, 1.0, WS, 1 << 30)), (3, (A16, 516, A16, 512, 8, 0, 1.0, WS, 1 << 30)),
    (3, (A16, 512, A16, 512, 8, 0, 1.0, WS + 16, 1 << 30)), (7, (A16, 512, A16, 512, 8, 0, 1.0, None, 1 << 30)),
    (7, (A16, 512, A16, 512, 8, 0, 1.0, WS, 8)),
])
def test_attn_refusals(status, args):
    a = kv4()
    assert S.lib().sherry_attn_kv4(ctypes.addressof(a), *args, None) == status


def test_null_cache_argument():
    L = S.lib()
    assert L.sherry_kv4_write(None, A16, A16, 0, 128, 128, None) == 1
    assert L.sherry_attn_kv4(None, A16, 512, A16, 512, 8, 0, 1.0, WS, 1 << 30, None) == 1


def test_cache_sizes_and_status_text():
    L = S.lib()
    assert L.sherry_kv4_bytes(3, 2, 64) == 3 * 2 * 2 * 64 * 36
    assert L.sherry_kv4_bytes(3, 2, 128) == 3 * 2 * 2 * 64 * 68
    for bad in ((0, 2, 64), (3, 0, 64), (3, 2, 80), (1 << 31, 1, 64)):
        assert L.sherry_kv4_bytes(*bad) == 0
    assert b"page" in L.sherry_status_string(8)
    assert S.attn_kv4_workspace_bytes(0, 8, 64) == 0 and S.attn_kv4_workspace_bytes(1, 8, 64) > 0


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 2, 64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        S.qk_norm_rope(q, q, i, torch.zeros(32))
    with pytest.raises(TypeError):
        S.qk_norm_rope(None, None, i, torch.zeros(32))
    cache = torch.zeros(1, 2, 2, 64 * 36, dtype=torch.uint8)
    with pytest.raises(TypeError):
        S.kv4_write(cache, q, q, i.view(1, 1), i)
    with pytest.raises(TypeError):
        S.attn_kv4(q.bfloat16(), cache, i.view(1, 1), i)
    with pytest.raises(ValueError):
        S.kv4_cache(1, 2, 96, "cpu")


@pytest.mark.parametrize("ws", [torch.zeros(64, dtype=torch.uint8), torch.zeros(64), None, 4096])
def test_binding_refuses_scratch_of_another_device_or_type(ws):
    """What attn_kv4 asks of the caller's scratch before a kernel gets its address."""
    with pytest.raises(TypeError):
        S._bytes(ws, "ws", 0)
