"""Host-side checks of the paged KV4 cache's entry points: what they refuse, before anything is launched, and
what the workspace query answers (no call here reaches a kernel)."""
import ctypes as C
import threading

import pytest
import torch

import w2a4_gemm_b200 as q
from w2a4_gemm_b200 import build

BAD, UNSUPPORTED, OK = q.QIFT_ERR_INVALID_ARG, q.QIFT_ERR_UNSUPPORTED, q.QIFT_OK
A = 0x100000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return q.lib()


def _append(L, **kw):
    a = dict(q=A, q_stride=6144, k=A << 8, k_stride=6144, v=A << 9, v_stride=6144, tokens=4, q_heads=32, kv_heads=8,
             head_dim=128, rope=A, rope_len=64, rope_dim=128, inter=0, positions=A, slots=A, block=128, q_out=A << 10,
             kc=A, ks=A, vc=A, vs=A, pages=8, size=16, stream=None)
    a.update(kw)
    return L.qift_append_kv(*a.values())


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(q_heads=-1), dict(kv_heads=0), dict(head_dim=0), dict(pages=-1), dict(size=0),
    dict(q=None), dict(q_out=None), dict(q_heads=0), dict(k=None), dict(v=None), dict(slots=None),
    dict(positions=None), dict(kc=None), dict(vs=None),
    dict(q_stride=6140), dict(q_stride=4088), dict(k_stride=1016), dict(v_stride=0), dict(k_stride=2 ** 62),
    dict(k=A + 8), dict(q_out=(A << 10) + 2), dict(kc=A + 8), dict(rope=A + 4), dict(slots=A + 4), dict(ks=A + 4),
    dict(block=3), dict(block=256), dict(block=-2), dict(rope_dim=144), dict(rope_dim=0), dict(rope_dim=17),
    dict(inter=2), dict(rope_len=-1),
    dict(q_out=A), dict(q_out=A + 45056 - 16), dict(q_out=(A << 8) - 16), dict(q_out=A << 9),  # overlaps
])
def test_append_refuses(L, kw):
    assert _append(L, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(head_dim=96), dict(head_dim=512), dict(size=8), dict(size=48), dict(size=8192),
                                dict(rope_dim=24), dict(tokens=2 ** 31), dict(pages=2 ** 60)])
def test_append_unsupported(L, kw):
    assert _append(L, **kw) == UNSUPPORTED


def test_append_of_no_tokens_is_a_no_op(L):
    assert _append(L, tokens=0) == OK


def _gather(L, **kw):
    a = dict(kc=A, ks=A, vc=A, vs=A, pages=8, size=16, kv_heads=8, head_dim=128, slots=A, tokens=4, block=128, k=A, v=A,
             stream=None)
    a.update(kw)
    return L.qift_gather_kv(*a.values())


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(block=5), dict(block=256), dict(slots=None), dict(k=None),
                                dict(v=A + 2), dict(kc=None), dict(pages=-1), dict(kv_heads=0), dict(slots=A + 4)])
def test_gather_refuses(L, kw):
    assert _gather(L, **kw) == BAD


def test_gather_unsupported_and_empty(L):
    assert _gather(L, head_dim=32) == UNSUPPORTED
    assert _gather(L, size=24) == UNSUPPORTED
    assert _gather(L, tokens=0) == OK


def _attention(L, **kw):
    a = dict(q=A, q_stride=4096, tokens=6, q_heads=32, kv_heads=8, head_dim=128, cu_q=A, batch=3, max_q=4, kc=A, ks=A,
             vc=A, vs=A, pages=64, size=16, table=A, max_pages=20, kv_lens=A, max_kv=0, prefix=None, prefix_len=0,
             window=0, sinks=0, scale=0.1, block=128, out=A, dt=1, lse=None, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return L.qift_paged_attention(*a.values())


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(batch=-1), dict(max_q=-1), dict(q_heads=0), dict(q_heads=33), dict(kv_heads=0),
    dict(max_pages=-1), dict(max_kv=-1), dict(prefix_len=-1), dict(window=-1), dict(sinks=-1), dict(dt=2),
    dict(q=None), dict(out=None), dict(kv_lens=None), dict(table=None), dict(prefix_len=5), dict(kc=None), dict(ks=None),
    dict(cu_q=None), dict(q=A + 8), dict(out=A + 8), dict(kc=A + 4), dict(vs=A + 4), dict(table=A + 1), dict(lse=A + 2),
    dict(q_stride=4092), dict(q_stride=4088), dict(block=6), dict(block=256), dict(scale=float("nan")),
    dict(scale=float("inf")),
    dict(prefix=A, prefix_len=50, ws=None), dict(prefix=A, prefix_len=50, ws_bytes=16),
    dict(prefix=A, prefix_len=50, ws=A + 8),
])
def test_attention_refuses(L, kw):
    assert _attention(L, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(head_dim=80), dict(size=4), dict(max_pages=2 ** 30), dict(tokens=2 ** 40)])
def test_attention_unsupported(L, kw):
    assert _attention(L, **kw) == UNSUPPORTED


@pytest.mark.parametrize("out,dt", [(0, 1), (6 * 8192 - 16, 1), (-6 * 8192 + 16, 1), (-6 * 16384 + 16, 0)])
def test_attention_refuses_a_result_over_its_queries(L, out, dt):
    assert _attention(L, out=A + out, dt=dt, tokens=6) == BAD
    assert _attention(L, q=A << 8, out=A, ws=None, prefix=A, prefix_len=5) == BAD  # apart: only the workspace is missing


@pytest.mark.parametrize("kw", [  # rows whose number passes 32 bits, or 64
    dict(q_heads=65536, kv_heads=1, max_q=2 ** 31 - 1, batch=1, q_stride=65536 * 128),
    dict(q_heads=65536, kv_heads=1, max_q=65536, batch=2 ** 31 - 1, q_stride=65536 * 128),
    dict(q_heads=65536, kv_heads=1, max_q=2 ** 20, batch=2 ** 20, q_stride=65536 * 128),
    dict(tokens=2 ** 27, prefix=A, prefix_len=64), dict(q_heads=65536, kv_heads=1, tokens=2 ** 16, prefix=A, prefix_len=64)])
def test_attention_refuses_more_rows_than_it_can_number(L, kw):
    assert _attention(L, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(tokens=0), dict(batch=0, tokens=0), dict(max_q=0, tokens=0)])
def test_attention_of_nothing_is_a_no_op(L, kw):
    assert _attention(L, **kw) == OK


def test_workspace_query(L):
    size = q.qift_paged_attention_workspace
    assert size(0, 32, 8, 128, 0, 1, 16, 10) == 0
    assert size(1, 32, 8, 128, 1, 1, 16, 4) == 0                       # one split: no partial results
    one = size(1, 32, 8, 128, 1, 1, 16, 8192)
    assert one > 0 and one % 4 == 0
    assert size(1, 32, 8, 128, 1, 1, 16, 8192, max_kv=64) == 0         # the host knows that the sequence is short
    assert size(4, 32, 8, 128, 4, 1, 16, 4, prefix_len=7) > 0          # prefix and own keys are joined
    with pytest.raises(ValueError):
        size(1, 30, 8, 128, 1, 1, 16, 4)
    with pytest.raises(ValueError):
        size(1, 32, 8, 100, 1, 1, 16, 4)


def test_binding_refuses_cpu_tensors():
    c = [torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 16)] * 2
    x = torch.zeros(1, 1, 64, dtype=torch.float16)
    s = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        q.qift_append_kv(x, x, s, 64, *c)
    with pytest.raises(ValueError):
        q.qift_gather_kv(*c, s, 64)
    with pytest.raises(ValueError):
        q.qift_paged_attention(x, None, 1, *c, torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))


@pytest.mark.parametrize("name", ["max_q", "max_kv", "prefix_len", "window", "sinks", "page_size", "q_heads"])
def test_sizes_past_32_bits_are_refused_not_cut(name):
    a = dict(tokens=1, q_heads=32, kv_heads=8, head_dim=128, batch=1, max_q=1, page_size=16, max_pages=4, max_kv=0,
             prefix_len=0, window=0, sinks=0)
    assert q.qift_paged_attention_workspace(**a) >= 0
    for more in (2 ** 32, 2 ** 31):
        with pytest.raises(ValueError, match=name):
            q.qift_paged_attention_workspace(**{**a, name: a[name] + more})


@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 3), dict(sinks=2 ** 32), dict(block=2 ** 32), dict(max_kv=2 ** 33 + 1),
                                dict(prefix_len=2 ** 32), dict(max_q=2 ** 32 + 1), dict(window=-2 ** 32)])
def test_binding_refuses_sizes_past_32_bits(kw):
    c = [torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 16)] * 2
    x = torch.zeros(1, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="32 bits"):
        q.qift_paged_attention(x, None, **{"max_q": 1, **kw}, k_cache=c[0], k_scales=c[1], v_cache=c[2], v_scales=c[3],
                               page_table=torch.zeros(1, 1, dtype=torch.int32), kv_lens=torch.ones(1, dtype=torch.int32))
    if "block" in kw:
        with pytest.raises(ValueError, match="32 bits"):
            q.qift_append_kv(x, x, torch.zeros(1, dtype=torch.int64), kw["block"], *c)
        with pytest.raises(ValueError, match="32 bits"):
            q.qift_gather_kv(*c, torch.zeros(1, dtype=torch.int64), kw["block"])


def test_a_pin_of_one_thread_leaves_another_threads_answers(L):
    size, sizes = q.qift_paged_attention_workspace, (1, 32, 8, 128, 1, 1, 16, 512)
    want, got = size(*sizes), []
    def pinned():
        q.qift_debug_set_attention_path("wide")
        got.append(size(*sizes))
    t = threading.Thread(target=pinned)
    t.start()
    t.join()
    assert got[0] != want and size(*sizes) == want


def test_attention_path_pin(L):
    size = q.qift_paged_attention_workspace
    assert L.qift_debug_set_attention_path(7) == BAD
    q.qift_debug_set_attention_path("wide")
    try:
        assert size(1, 32, 8, 128, 1, 1, 16, 8192) > 0
        with pytest.raises(ValueError):
            size(1, 8, 2, 256, 1, 1, 16, 8192)                         # not for this head_dim
    finally:
        q.qift_debug_set_attention_path("auto")
    assert size(1, 8, 2, 256, 1, 1, 16, 8192) > 0
