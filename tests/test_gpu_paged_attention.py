"""The paged KV4 cache on the GPU: rows appended and read back against the CPU oracle and the stated order of
operations, bit for bit; attention against the formula in 64 bits.

Tolerance of attention in the cache's domain, for a row with weights w_j = softmax(u)_j and values v_j, d by d, with
A = sum_j w_j |v_j|:
  * each weight times its value's scale is rounded to binary16: half a step, 2^-11 of it at most, so 2^-11 A; weights
    under 2^-18 of the largest are subnormal and off by up to 2^-29 of the largest each, which for the lengths here
    (under 2^15 keys) is 2^-14 of A's largest;
  * a score's error e_u moves the weights by at most 2 e_u relative: the product adds D + D/2 * 72-fold values in
    groups of 16, each addition off by at most 2^-22 of partial sums that stay under 80 sum|q|, so
    e_u <= (D/16 + 1) 2^-22 80 sum|q| max_j s_j scale; the 2^u, scalings and sums add under 2^-17 relative;
  * a binary16 result is off by 2^-11 of the value (2^-25 where it is subnormal).
"""
import math

import numpy as np
import pytest
import torch

import oracle
import w2a4_gemm_b200 as qg
from w2a4_gemm_b200 import build

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    qg.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def empty_cache(pages, heads, size, d):
    """A pool that nothing was written to: scales NaN, so that a row read by mistake shows."""
    c = [torch.full((pages, heads, size, d // 2), 0x77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.full((pages, heads, size), NAN, device="cuda") for _ in range(2)]
    return [c[0], s[0], c[1], s[1]]


def rope_table(n, dim):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def rope_np(x, tab, positions, dim, interleaved):
    """The stated order of operations in numpy float32 (each rounded)."""
    x = x.astype(np.float32).copy()
    c, s = tab[positions][:, None, :dim // 2], tab[positions][:, None, dim // 2:]
    ia = np.arange(0, dim, 2) if interleaved else np.arange(dim // 2)
    ib = ia + 1 if interleaved else ia + dim // 2
    a, b = x[..., ia], x[..., ib]
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def hadamard_np(x, block):
    if not block:
        return x
    y, h = x.astype(np.float32), 1
    shape = y.shape
    while h < block:
        y = y.reshape(-1, 2, h)
        y = np.stack([y[:, 0] + y[:, 1], y[:, 0] - y[:, 1]], axis=1)
        h *= 2
    return y.reshape(shape) * np.float32(1.0 / math.sqrt(block))


def quantise_np(x16):
    x = x16.astype(np.float32)
    m = np.abs(x).max(-1)
    inv = np.where(m > 0, np.float32(7) / np.where(m > 0, m, 1), 0).astype(np.float32)
    q = np.clip(np.rint(x * inv[..., None]), -7, 7).astype(np.int8)
    return q, (m / np.float32(7)).astype(np.float32)


def unpack(p):
    p = p.view(torch.int8)
    return torch.stack([(p << 4) >> 4, p >> 4], -1).flatten(-2)


# --------------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("d,block", [(64, 64), (64, 0), (128, 128), (128, 2), (128, 16), (128, 32), (256, 256), (256, 64)])
def test_append_without_rope_is_quantize_kv(d, block):
    T, H, size = 37, 3, 16
    x = torch.randn(2, T, H, d, device="cuda", generator=gen(d + block)).half()
    x[0, 3] = 0
    cache = empty_cache(5, H, size, d)
    slots = torch.randperm(5 * size, device="cuda", generator=gen(1))[:T].contiguous()
    assert qg.qift_append_kv(x[0], x[1], slots, block, *cache) is None
    for i in range(2):
        packed, s = oracle.quantize_kv(x[i].reshape(T * H, d).cpu().numpy(), block)
        at = (slots // size, slice(None), slots % size)
        assert np.array_equal(cache[2 * i][at].reshape(T * H, d // 2).cpu().numpy(), packed)
        assert np.array_equal(cache[2 * i + 1][at].flatten().cpu().numpy().view(np.uint32), s.view(np.uint32))


@pytest.mark.parametrize("d,rope_dim,interleaved,block,hq,hk,size", [
    (128, 128, False, 128, 4, 2, 16), (128, 128, True, 128, 5, 1, 32), (64, 32, False, 64, 1, 1, 16),
    (64, 48, True, 32, 3, 3, 64), (256, 256, False, 256, 2, 1, 128), (256, 64, True, 0, 1, 2, 16),
    (128, 16, False, 64, 8, 8, 4096), (64, 64, False, 64, 7, 1, 16)])
def test_append_with_rope_bit_for_bit(d, rope_dim, interleaved, block, hq, hk, size):
    T, far = 29, 5000
    g = gen(d + rope_dim)
    qkv = torch.randn(T, hq + 2 * hk + 1, d, device="cuda", generator=g).half()  # heads behind them belong to no one
    qkv[:, :, 1] *= 30
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:hq + 2 * hk]
    pages = T // size + 4
    cache = empty_cache(pages, hk, size, d)
    slots = torch.randperm(pages * size, device="cuda", generator=g)[:T].contiguous()
    slots[4], slots[9], slots[20] = -1, pages * size, -(2 ** 40)
    positions = torch.randint(0, far, (T,), device="cuda", generator=g)
    positions[0], positions[1], positions[2], positions[3] = 0, far - 1, far, -1
    tab = rope_table(far, rope_dim)
    q_out = torch.full((T, hq, d), 5.0, device="cuda").half()
    got = qg.qift_append_kv(k, v, slots, block, *cache, q=q, positions=positions, rope=tab.cuda(),
                            interleaved=interleaved, q_out=q_out)
    assert got is q_out
    on = np.ones(T, bool)
    on[2:4] = False
    pos = np.clip(positions.cpu().numpy(), 0, far - 1)
    def turned(x, rope):
        x = x.cpu().numpy().astype(np.float32)
        return hadamard_np(rope_np(x, tab.numpy(), pos, rope_dim, interleaved) if rope else x, block).astype(np.float16)
    want = turned(q, True)
    want[~on] = 5.0
    assert np.array_equal(q_out.cpu().numpy().view(np.uint16), want.view(np.uint16))
    on[[4, 9, 20]] = False
    kept = torch.from_numpy(on).cuda()
    at = (slots[kept] // size, slice(None), slots[kept] % size)
    for i, (x, rope) in enumerate(((k, True), (v, False))):
        codes, s = quantise_np(turned(x, rope)[on])
        assert np.array_equal(unpack(cache[2 * i][at]).cpu().numpy(), codes)
        assert np.array_equal(cache[2 * i + 1][at].cpu().numpy().view(np.uint32), s.view(np.uint32))
        rest = torch.ones(pages, size, dtype=torch.bool, device="cuda")
        rest[slots[kept] // size, slots[kept] % size] = False
        assert torch.isnan(cache[2 * i + 1].movedim(1, 2)[rest]).all()  # no other slot was touched
        assert (cache[2 * i].movedim(1, 2)[rest] == 0x77).all()


@pytest.mark.parametrize("d,block", [(64, 64), (128, 128), (128, 0), (256, 32)])
def test_gather_bit_for_bit(d, block):
    H, size, pages = 3, 32, 7
    g = gen(d)
    cache = [torch.randint(0, 256, (pages, H, size, d // 2), device="cuda", generator=g).to(torch.uint8),
             torch.rand(pages, H, size, device="cuda", generator=g)] * 2
    cache[2] = cache[2].flip(0).contiguous()
    slots = torch.randint(0, pages * size, (41,), device="cuda", generator=g)
    slots[5], slots[6] = -1, pages * size
    got = qg.qift_gather_kv(*cache, slots, block)
    for i in range(2):
        at = (slots.clamp(0, pages * size - 1) // size, slice(None), slots.clamp(0, pages * size - 1) % size)
        want = oracle.dequantize_kv(cache[2 * i][at].reshape(-1, d // 2).cpu().numpy(),
                                    cache[2 * i + 1][at].flatten().cpu().numpy(), block).reshape(41, H, d)
        want[5:7] = 0
        assert np.array_equal(got[i].cpu().numpy(), want)


def test_append_then_gather_of_no_tokens():
    cache = empty_cache(1, 2, 16, 64)
    x = torch.empty(0, 2, 64, device="cuda").half()
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    q = qg.qift_append_kv(x, x, s, 64, *cache, q=x, positions=s, rope=rope_table(4, 64).cuda())
    k, v = qg.qift_gather_kv(*cache, s, 64)
    assert q.shape == k.shape == v.shape == (0, 2, 64)


# ------------------------------------------------------------------------------------------ attention
def make(q_lens, kv_lens, hq, hk, d, size, prefix=0, seed=0, gain=1.0):
    """A ragged batch over a pool whose unused rows hold NaN scales.  kv_lens count the prefix."""
    g = gen(seed)
    own = [max(n - prefix, 0) for n in kv_lens]
    n_own, n_pre = [-(-n // size) for n in own], -(-prefix // size)
    pages = sum(n_own) + n_pre + 2
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(own), max(n_own + [1])), -7, dtype=torch.int32, device="cuda")
    at = n_pre
    cache = empty_cache(pages, hk, size, d)
    def fill(page, count):
        for i in range(2):
            x = torch.randn(hk, count, d, device="cuda", generator=g) * (gain if i else 1.0)
            s = x.abs().amax(-1) / 7
            c = torch.round(x / s[..., None]).to(torch.int8)
            cache[2 * i][page, :, :count] = ((c[..., 0::2] & 15) | (c[..., 1::2] << 4)).view(torch.uint8)
            cache[2 * i + 1][page, :, :count] = s
    for j in range(n_pre):
        fill(int(order[j]), min(size, prefix - j * size))
    for b, n in enumerate(own):
        for j in range(n_own[b]):
            table[b, j] = order[at]
            fill(int(order[at]), min(size, n - j * size))
            at += 1
    T = sum(q_lens)
    return dict(q=torch.randn(T, hq, d, device="cuda", generator=g).half(),
                cu_q=torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32, device="cuda"),
                max_q=max(q_lens + [1]), cache=cache, table=table,
                kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device="cuda"),
                prefix_table=order[:n_pre].contiguous() if prefix else None, prefix=prefix)


def reference(m, window=0, sinks=0, scale=None, prefix=None):
    """The formula in 64 bits: (out in the cache's domain, lse, A, sum|q| max s scale) per row."""
    kc, ks, vc, vs = m["cache"]
    pages, hk, size, half = kc.shape
    d = 2 * half
    q = m["q"].double()
    T, hq, _ = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, A = torch.zeros(2, T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    reach = torch.zeros(T, hq, dtype=torch.float64, device="cuda")
    cu, lens, P = m["cu_q"].tolist(), m["kv_lens"].tolist(), m["prefix"]
    for b, n in enumerate(lens):
        nq = cu[b + 1] - cu[b]
        if not nq:
            continue
        def rows(c, s, h):
            pre = m["prefix_table"][:-(-P // size)].long() if P else []
            parts = []
            if P:
                parts.append((unpack(c[pre, h]).double() * s[pre, h].double()[..., None]).reshape(-1, d)[:min(P, n)])
            if n > P:
                t = m["table"][b, :-(-(n - P) // size)].long()
                x = torch.zeros(len(t), size, d, dtype=torch.float64, device="cuda")
                good = (t >= 0) & (t < pages)
                x[good] = unpack(c[t[good], h]).double() * s[t[good], h].double()[..., None]
                x[~good] = NAN
                parts.append(x.reshape(-1, d)[:n - P])
            return torch.cat(parts) if parts else torch.zeros(0, d, dtype=torch.float64, device="cuda")
        i = torch.arange(nq, device="cuda")[:, None] + n - nq
        j = torch.arange(n, device="cuda")[None, :]
        see = (j <= i) & ((j > i - window) | (j < sinks) if window else torch.ones_like(j <= i))
        for h in range(hk):
            k, v = rows(kc, ks, h), rows(vc, vs, h)
            lost = torch.isnan(k).any(-1)  # pages that are not there
            vis = see & ~lost[None]
            k, v = torch.nan_to_num(k), torch.nan_to_num(v)
            for x in range(h * hq // hk, (h + 1) * hq // hk):
                u = (q[cu[b]:cu[b + 1], x] @ k.T * scale).masked_fill(~vis, -math.inf)
                l = torch.logsumexp(u, -1) if n else torch.full((nq,), -math.inf, dtype=torch.float64, device="cuda")
                w = torch.where(vis, torch.exp(u - torch.where(l.isinf(), 0, l)[:, None]), 0)
                out[cu[b]:cu[b + 1], x], A[cu[b]:cu[b + 1], x] = w @ v, w @ v.abs()
                lse[cu[b]:cu[b + 1], x] = l
                s_max = torch.nan_to_num(k.abs().amax() / 7) if n else 0
                reach[cu[b]:cu[b + 1], x] = q[cu[b]:cu[b + 1], x].abs().sum(-1) * s_max * scale
    return out, lse, A, reach


def score_error(reach, d):
    return reach * (d / 16 + 1) * 2.0 ** -22 * 80


def bound(A, reach, ref, half):
    t = A * (2.0 ** -11 + 2 * score_error(reach, A.shape[-1])[..., None] + 2.0 ** -17) + A.amax(-1, keepdim=True) * 2.0 ** -14
    return t + (2.0 ** -11 * ref.abs() + 2.0 ** -25 if half else 2.0 ** -22 * ref.abs() + 1e-38)


def paths(m):
    return ("stream", "wide") if m["q"].shape[-1] <= 128 else ("stream",)


@pytest.fixture(autouse=True)
def _automatic():
    yield
    qg.qift_debug_set_attention_path("auto")


def call(m, **kw):
    return qg.qift_paged_attention(m["q"], m["cu_q"], m["max_q"], *m["cache"], m["table"], m["kv_lens"],
                                   prefix_table=m["prefix_table"], prefix_len=m["prefix"], **kw)


def check(m, window=0, sinks=0, scale=None, dtypes=(torch.float32, torch.float16), **kw):
    """Both kernels on the same call."""
    ref, lse, A, reach = reference(m, window, sinks, scale)
    cu = m["cu_q"].tolist()
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        for dt in dtypes:
            out = torch.full(m["q"].shape, 77.0, device="cuda", dtype=dt)
            l = torch.full(m["q"].shape[:2], 77.0, device="cuda")
            call(m, window=window, sinks=sinks, scale=scale, out=out, out_dtype=dt, lse=l, **kw)
            inside = slice(cu[0], cu[-1])
            err = (out.double() - ref).abs()[inside]
            tol = bound(A, reach, ref, dt == torch.float16)[inside]
            assert not torch.isnan(err).any(), path
            assert (err <= tol).all(), (path, float((err / tol).max()), (err / tol).flatten(1).amax(1).tolist()[:40])
            assert (out[:cu[0]] == 77).all() and (out[cu[-1]:] == 77).all()
            none = lse[inside].isinf()
            assert torch.equal(l[inside].isinf() & (l[inside] < 0), none)
            assert (out[inside][none] == 0).all()
            e_u = score_error(reach, ref.shape[-1])
            assert ((l.double() - lse)[inside][~none].abs() <= (e_u + 2.0 ** -16 + lse.abs() * 2.0 ** -20)[inside][~none]).all()
    qg.qift_debug_set_attention_path("auto")
    return out


LAYOUTS = [(4, 1, 128, 16), (8, 8, 128, 32), (7, 1, 64, 64), (16, 1, 64, 16), (6, 3, 256, 16), (24, 1, 128, 128), (16, 1, 256, 32)]


@pytest.mark.parametrize("hq,hk,d,size", LAYOUTS)
def test_decode_ragged(hq, hk, d, size):
    lens = [1, 0, 2, 15, 16, 17, 31, 32, 33, 64, 127, 128, 129, 500, 700]
    check(make([1] * len(lens), lens, hq, hk, d, size, seed=d + hq))


@pytest.mark.parametrize("hq,hk,d,size", LAYOUTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (37, 0), (64, 4), (100, 70), (2000, 3)])
def test_decode_window(hq, hk, d, size, window, sinks):
    lens = [1, 3, 36, 37, 38, 41, 64, 65, 101, 170, 333, 900]
    check(make([1] * len(lens), lens, hq, hk, d, size, seed=window), window, sinks, dtypes=(torch.float32,))


@pytest.mark.parametrize("hq,hk,d,size", LAYOUTS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
def test_several_tokens_and_rows_that_see_nothing(hq, hk, d, size, window, sinks):
    # more tokens than keys: the first of them stand before the sequence's start and see nothing
    m = make([3, 0, 5, 1, 2, 8, 4], [100, 40, 3, 0, 260, 8, 133], hq, hk, d, size, seed=3)
    check(m, window, sinks)


@pytest.mark.parametrize("hq,hk,d,size", LAYOUTS[:5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
def test_prompts(hq, hk, d, size, window, sinks):
    check(make([130, 65, 1, 257], [130, 200, 77, 700], hq, hk, d, size, seed=5), window, sinks)


@pytest.mark.parametrize("hq,hk,d,size", LAYOUTS)
@pytest.mark.parametrize("prefix,window,sinks", [(1, 0, 0), (64, 0, 0), (301, 0, 0), (301, 40, 5), (1000, 400, 0), (77, 200, 90)])
def test_shared_prefix(hq, hk, d, size, prefix, window, sinks):
    own = [1, 5, 16, 40, 129, 2, 33]
    m = make([1, 1, 2, 3, 1, 0, 1], [prefix + n for n in own], hq, hk, d, size, prefix=prefix, seed=prefix)
    check(m, window, sinks, dtypes=(torch.float32,))


def test_sequences_that_end_inside_the_prefix():
    m = make([1, 2, 1, 1, 4], [10, 64, 200, 0, 2], 8, 2, 128, 16, prefix=150, seed=9)
    check(m)
    check(m, 20, 3)


@pytest.mark.parametrize("hq,hk,d,prefix,window", [(8, 2, 128, 0, 0), (8, 2, 64, 0, 50), (4, 1, 128, 300, 0), (16, 1, 64, 0, 0),
                                                    (24, 1, 64, 0, 0), (2, 1, 256, 70, 0), (2, 2, 64, 300, 90)])
@pytest.mark.parametrize("far", [400, 3000])
def test_long_sequences_among_short_ones(hq, hk, d, prefix, window, far):
    # each sequence's row tiles are found through the offsets, and its length chooses its kernel
    q_lens = [0, 1] + [1] * 20 + [500] + [1, 2, 0, 3] * 4 + [90, 0, 1] + [1] * 30
    kv_lens = [n + prefix + (37 * i * i) % far for i, n in enumerate(q_lens)]
    kv_lens[5], kv_lens[7] = 0, 1
    m = make(q_lens, kv_lens, hq, hk, d, 32, prefix, seed=hq + d)
    check(m, window, 3 if window else 0, dtypes=(torch.float16,))
    ref, lse, A, reach = reference(m, window, 3 if window else 0)
    T, behind = sum(q_lens), 150
    q = torch.cat([torch.full((3, hq, d), NAN, device="cuda").half(), m["q"], torch.full((behind, hq, d), NAN, device="cuda").half()])
    out = torch.full(q.shape, 77.0, device="cuda")
    l = torch.full(q.shape[:2], 77.0, device="cuda")
    call(dict(m, q=q, cu_q=m["cu_q"] + 3), window=window, sinks=3 if window else 0, out=out, out_dtype=torch.float32, lse=l)
    assert ((out[3:3 + T].double() - ref).abs() <= bound(A, reach, ref, False)).all()
    none = lse.isinf()
    assert torch.equal(l[3:3 + T] == -math.inf, none) and (out[3:3 + T][none] == 0).all()
    for x in (out, l):
        assert (x[:3] == 77).all() and (x[3 + T:] == 77).all()


def test_an_empty_sequence_among_long_ones_sees_nothing():
    # the prefix's rows are those of the whole batch: one that sees nothing lies between rows that see all
    m = make([1] * 9 + [3], [400 + b for b in range(4)] + [0] + [500 + b for b in range(4)] + [2], 4, 2, 128, 16,
             prefix=300, seed=19)
    check(m)


def test_prefix_for_many_rows_equals_its_keys_in_every_table():
    # The same keys, once as a prefix and once as pages that all tables begin with: the same sums in another order.
    hq, hk, d, size, prefix = 32, 8, 128, 16, 640
    m = make([1] * 40, [prefix + 3 * b for b in range(40)], hq, hk, d, size, prefix=prefix, seed=2)
    a = check(m, dtypes=(torch.float32,))
    whole = dict(m, table=torch.cat([m["prefix_table"][None].expand(40, -1), m["table"]], 1).contiguous(),
                 prefix_table=None, prefix=0)
    b = check(whole, dtypes=(torch.float32,))
    assert (a - b).abs().max() < 2e-3 * b.abs().max()


def test_long_sequence_is_split():
    m = make([1, 1], [20011, 5], 8, 2, 128, 64, seed=1)
    check(m)
    check(m, max_kv=64)  # a bound that is wrong changes how the work is split, not what it is


@pytest.mark.parametrize("path,d", [("stream", 64), ("stream", 128), ("stream", 256), ("wide", 64), ("wide", 128)])
def test_result_rotated_back(path, d):
    m = make([1, 7, 40], [90, 30, 333], 8, 2, d, 16, seed=4)
    qg.qift_debug_set_attention_path(path)
    x = call(m, out_dtype=torch.float32)
    for block in (2, 16, 32, 64, d):
        y = call(m, out_dtype=torch.float32, block=block)
        want = torch.from_numpy(hadamard_np(x.cpu().numpy(), block)).double()
        # the same sums before the rotation; its log2(block) stages and the last product round once each
        rms = x.double().pow(2).mean(-1, keepdim=True).sqrt().cpu() * math.sqrt(block)
        assert ((y.double().cpu() - want).abs() <= 2.0 ** -20 * rms + 1e-9).all()


@pytest.mark.parametrize("gain", [1e-6, 1e3])
def test_small_and_large_values(gain):
    m = make([1, 3], [300, 90], 8, 2, 128, 16, seed=6, gain=gain)
    check(m, dtypes=(torch.float32,))


def test_values_of_very_different_size_and_zero_rows():
    m = make([1, 2], [200, 64], 4, 1, 128, 16, seed=8)
    vs = m["cache"][3]
    vs[:, :, 0::3] = 0.0                                   # tokens whose values are all zero
    vs[:, :, 1::3] *= 1e-5
    m["cache"][1][0, :, 3] = 0.0                           # a key that is all zero
    check(m, dtypes=(torch.float32,))
    vs.zero_()
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        assert (call(m) == 0).all()


def test_peaked_scores():
    m = make([2, 1], [500, 90], 8, 2, 128, 16, seed=10)
    m["q"] *= 40
    check(m)


@pytest.mark.parametrize("prefix", [0, 200])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 1], [5000, 300, 0]), ([9, 40], [2100, 1300])])
def test_a_query_with_nan_or_infinity_is_not_hidden_and_spoils_no_other(q_lens, kv_lens, prefix):
    m = make(q_lens, kv_lens, 8, 2, 64, 32, prefix, seed=12)
    clean = dict(m, q=m["q"].clone())
    m["q"][0, 1, 7], m["q"][1, 6, 63] = NAN, math.inf
    ref, lse, A, reach = reference(clean)
    good = torch.ones(m["q"].shape[:2], dtype=torch.bool, device="cuda")
    good[0, 1] = good[1, 6] = False
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        l = torch.empty(m["q"].shape[:2], device="cuda")
        out = call(m, out_dtype=torch.float32, lse=l)
        assert ((out.double() - ref).abs() <= bound(A, reach, ref, False))[good].all(), path
        assert torch.isnan(out[~good]).all() and torch.isnan(l[~good]).all(), path
        assert not torch.isnan(l[good]).any()


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_key_with_no_number_spoils_only_rows_that_see_it(d, window):
    # rows of one block on both sides of it; scales of keys, of values and of both
    m = make([40], [200], 4, 1, d, 16, seed=d)
    ref, _, A, reach = reference(m, window)
    positions = torch.arange(160, 200, device="cuda")
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        for bad, ks, vs in ((178, math.inf, 1.0), (178, 1.0, math.inf), (193, NAN, NAN), (166, math.inf, NAN)):
            cache = [c.clone() for c in m["cache"]]
            cache[1][m["table"][0, bad // 16], 0, bad % 16] = ks
            cache[3][m["table"][0, bad // 16], 0, bad % 16] = vs
            out = call(dict(m, cache=cache), window=window, out_dtype=torch.float32)
            see = (positions >= bad) & ((positions < bad + window) if window else True)
            err = (out.double() - ref).abs()
            assert (err <= bound(A, reach, ref, False))[~see].all(), (path, bad, ks, vs)


def test_rows_outside_every_sequence_are_left():
    m = make([1, 2, 1], [40, 50, 60], 4, 2, 64, 16, seed=11)
    m["q"] = torch.cat([m["q"], m["q"].flip(0)])           # four rows of padding behind
    check(m)
    m["cu_q"] += 2                                          # ... and two in front
    check(m)


@pytest.mark.parametrize("q_lens", [[1] * 20, [3, 0, 70, 5]])
def test_padding_before_and_behind_with_a_prefix(q_lens):
    m = make(q_lens, [400 + n for n in q_lens], 4, 1, 64, 32, prefix=390, seed=13)
    T, ahead, behind = sum(q_lens), 7, 90
    pad = lambda n: torch.full((n, 4, 64), NAN, device="cuda").half()
    ref, _, A, reach = reference(m)
    padded = dict(m, q=torch.cat([pad(ahead), m["q"], pad(behind)]), cu_q=m["cu_q"] + ahead)
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        out, l = torch.full((T + ahead + behind, 4, 64), 77.0, device="cuda"), torch.full((T + ahead + behind, 4), 77.0, device="cuda")
        call(padded, out=out, lse=l, out_dtype=torch.float32)
        assert ((out[ahead:ahead + T].double() - ref).abs() <= bound(A, reach, ref, False)).all(), path
        for x in (out, l):
            assert (x[:ahead] == 77).all() and (x[ahead + T:] == 77).all()


def test_pages_that_are_not_there():
    m = make([1, 1, 1], [100, 80, 40], 4, 2, 128, 16, seed=12)
    m["table"][0, 2], m["table"][1, 0], m["table"][2, 0] = -1, 2 ** 31 - 1, m["cache"][0].shape[0]
    check(m)
    short = dict(m, table=m["table"][:, :3].contiguous())   # keys beyond the table are not there either
    a = call(short, out_dtype=torch.float32)
    assert torch.isfinite(a).all()


def test_contradicting_offsets_stay_inside():
    m = make([2, 2], [40, 50], 4, 2, 64, 16, seed=13)
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        for cu in ([0, 3, 2], [-5, 2, 4], [0, 2, 400], [4, 4, 4]):
            out = torch.full((4, 4, 64), 7.0, device="cuda").half()
            call(dict(m, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda")), out=out)
        call(dict(m, kv_lens=torch.tensor([-3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()


def test_uniform_batch_without_offsets():
    m = make([3] * 5, [9, 70, 33, 3, 128], 8, 4, 128, 16, seed=14)
    a, b = call(m), call(dict(m, cu_q=None))
    assert torch.equal(a, b)


def test_strided_queries():
    m = make([1, 4], [77, 200], 8, 2, 128, 16, seed=15)
    wide = torch.randn(5, 13, 128, device="cuda").half()
    wide[:, 2:10] = m["q"]
    assert torch.equal(call(m), call(dict(m, q=wide[:, 2:10])))


@pytest.mark.parametrize("path", ["stream", "wide"])
def test_a_pool_past_32_bits(path):
    qg.qift_debug_set_attention_path(path)
    d, hk, size = 128, 8, 64
    pages = 2 ** 31 // (hk * size * d // 2) + 70            # over 2^31 bytes of codes
    m = make([1], [150], 8, hk, d, size, seed=16)
    small = m["cache"]
    big = [torch.zeros(pages, *t.shape[1:], dtype=t.dtype, device="cuda") for t in small]
    shift = pages - small[0].shape[0]
    for b, s in zip(big, small):
        b[shift:] = s
    want = call(m)
    got = call(dict(m, cache=big, table=m["table"] + shift))
    assert torch.equal(want, got)
    slots = (torch.arange(3, device="cuda") + pages * size - 3)
    x = torch.randn(3, hk, d, device="cuda").half()
    qg.qift_append_kv(x, x, slots, 128, *big)
    k, v = qg.qift_gather_kv(*big, slots, 128)
    err = (k.float() - x.float()).abs()
    assert torch.equal(k, v) and err.max() < 0.5 * x.float().norm(dim=-1).max() / 7


@pytest.mark.parametrize("path", ["stream", "wide"])
def test_other_stream_and_captured_graphs(path):
    qg.qift_debug_set_attention_path(path)
    m = make([1, 1], [9000, 4000], 8, 2, 128, 16, seed=17)
    want = call(m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(m, stream=s)
    s.synchronize()
    assert torch.equal(want, got)
    m2 = dict(m, q=m["q"].flip(0).contiguous())
    want2 = call(m2)
    graphs, outs = [], []
    for x in (m, m2):                                       # each captures a workspace of its own
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call(x))
        graphs.append(gr)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)
    m["kv_lens"][0] = 1234                                  # lengths are read on the device, at replay
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], call(m))


def test_same_call_twice_gives_the_same_bits():
    m = make([1] * 6 + [90], [3000, 40, 777, 5000, 1, 60, 4000], 32, 8, 128, 16, prefix=0, seed=18)
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        assert torch.equal(call(m), call(m))


def test_refusals_leave_the_result_alone():
    m = make([1], [40], 4, 2, 128, 16)
    out = torch.full((1, 4, 128), 3.0, device="cuda").half()
    for bad in (dict(q=m["q"].float()), dict(q=m["q"][:, :, :64]), dict(q=m["q"].transpose(0, 1)), dict(kv_lens=m["kv_lens"].long()),
                dict(table=m["table"][0]), dict(cu_q=m["cu_q"][:1]), dict(prefix=16), dict(max_q=-1)):
        with pytest.raises((ValueError, qg.QiftError)):
            call(dict(m, **bad), out=out)
    with pytest.raises(ValueError):
        call(m, out=out[:, :2])
    with pytest.raises(ValueError):
        call(m, out=out, out_dtype=torch.float32)
    with pytest.raises(qg.QiftError):
        call(m, out=out, block=3)
    torch.cuda.synchronize()
    assert (out == 3).all()


# ----------------------------------------------------------------------------------- as it would be used
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_a_layer_prompt_then_single_tokens(window, sinks):
    """Projections by the W2A4 linear, rows appended, attention, and the output projection fed in the rotated
    domain: a prompt and then tokens one by one give the same rows as the whole text at once."""
    hq, hk, d, n_in, size = 8, 2, 128, 512, 16
    T, block = 70, 128
    g = gen(21)
    w = torch.randn((hq + 2 * hk) * d, n_in, device="cuda", generator=g) * 0.02
    wo = torch.randn(n_in, hq * d, device="cuda", generator=g) * 0.02
    c, s, _ = qg.qift_quantize_weights(qg.qift_rotate(w, block), "qift")
    co, so, _ = qg.qift_quantize_weights(qg.qift_rotate(wo, block), "qift")
    rope = rope_table(128, d).cuda()
    x = torch.randn(T, n_in, device="cuda", generator=g).half()
    table = torch.randperm(8, device="cuda", generator=g).to(torch.int32)[None, :5].contiguous()

    def layer(cache, x, first):
        n = x.shape[0]
        qx, sx = qg.qift_quantize_acts(x, block)
        qkv = qg.qift_linear(qx, sx, c, s, "qift").view(n, hq + 2 * hk, d)
        at = torch.arange(first, first + n, device="cuda")
        slots = table[0].long()[at // size] * size + at % size
        q = qg.qift_append_kv(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, block, *cache, q=qkv[:, :hq], positions=at,
                              rope=rope)
        o = qg.qift_paged_attention(q, None, n, *cache, table, torch.tensor([first + n], device="cuda", dtype=torch.int32),
                                    window=window, sinks=sinks)
        qo, sa = qg.qift_quantize_acts(o.view(n, hq * d), 0)
        return o, qg.qift_linear(qo, sa, co, so, "qift")

    one, two = empty_cache(8, hk, size, d), empty_cache(8, hk, size, d)
    o_all, y_all = layer(one, x, 0)
    parts = [layer(two, x[:40], 0)] + [layer(two, x[i:i + 1], i) for i in range(40, T)]
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))    # the same rows in the cache
    o_parts = torch.cat([p[0] for p in parts]).float()
    # each side is off by at most the bound above; values are at most 7 * max scale
    assert (o_all.float() - o_parts).abs().max() <= 2 * (2.0 ** -11 + 2.0 ** -12 + 2e-3) * 7 * one[3][~one[3].isnan()].max()
    assert torch.isfinite(y_all).all() and y_all.shape == (T, n_in)


def test_wait_that_runs_out_is_reported_and_the_context_survives():
    m = make([200], [300], 8, 2, 128, 16, seed=20)
    qg.qift_debug_set_attention_path("wide")
    want = call(m)
    assert qg.qift_device_error() == (qg.QIFT_OK, 0)
    qg.qift_debug_set_wait_limit(20_000_000)               # about 10 ms a wait
    qg.qift_debug_stall_next_attention()
    call(m)
    status, word = qg.qift_device_error()
    qg.qift_debug_set_wait_limit(0)
    assert status == qg.QIFT_ERR_TIMEOUT and word != 0
    assert qg.qift_device_error() == (qg.QIFT_OK, 0)
    assert torch.equal(call(m), want)
    assert qg.qift_device_error() == (qg.QIFT_OK, 0)


def test_the_kernel_for_many_rows_takes_head_dims_up_to_128():
    m = make([40], [50], 2, 1, 256, 16, seed=22)
    qg.qift_debug_set_attention_path("wide")
    with pytest.raises(qg.QiftError) as e:
        call(m)
    assert e.value.status == qg.QIFT_ERR_UNSUPPORTED


def test_the_choice_of_kernel_is_by_cost():
    """A long prompt runs on the tensor memory kernel: its bits are those of the pinned call, and not those of the other."""
    m = make([3000], [3000], 32, 8, 128, 16, seed=23)
    auto = call(m)
    got = {}
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        got[path] = call(m)
    assert torch.equal(auto, got["wide"]) and not torch.equal(auto, got["stream"])
    one = dict(make([1] * 3, [500, 60, 7], 32, 8, 128, 16, seed=24))
    qg.qift_debug_set_attention_path("auto")
    auto = call(one)
    qg.qift_debug_set_attention_path("stream")
    assert torch.equal(auto, call(one))


# ------------------------------------------------------------------------------- as a server would call them
def test_a_captured_step_follows_lengths_slots_and_positions():
    """One graph of append and attention, replayed for step after step of a batch whose members differ in length
    and in the number of new tokens, on a stream of its own while another graph of the same kind runs beside it."""
    hq, hk, d, size, B, T = 8, 2, 128, 16, 4, 60
    tab = rope_table(4096, d).cuda()
    def batch(seed):
        g = gen(seed)
        s = dict(qkv=torch.randn(T, hq + 2 * hk, d, device="cuda", generator=g).half(), cache=empty_cache(B * 12, hk, size, d),
                 table=torch.randperm(B * 12, device="cuda", generator=g).to(torch.int32).view(B, 12),
                 cu=torch.zeros(B + 1, dtype=torch.int32, device="cuda"), lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
                 slots=torch.full((T,), -1, device="cuda"), positions=torch.zeros(T, dtype=torch.int64, device="cuda"))
        return s
    def step(s, cache):
        q = qg.qift_append_kv(s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:], s["slots"], d, *cache, q=s["qkv"][:, :hq],
                              positions=s["positions"], rope=tab)
        return qg.qift_paged_attention(q, s["cu"], 40, *cache, s["table"], s["lens"], block=d)
    def advance(s, counts, at):
        table = s["table"].cpu()
        slots, positions = [], []
        for b, n in enumerate(counts):
            for i in range(n):
                p = at[b] + i
                slots.append(int(table[b, p // size]) * size + p % size)
                positions.append(p)
            at[b] += n
        pad = T - len(slots)
        s["slots"].copy_(torch.tensor(slots + [-1] * pad))
        s["positions"].copy_(torch.tensor(positions + [0] * pad))
        s["cu"].copy_(torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32))
        s["lens"].copy_(torch.tensor(at, dtype=torch.int32))
        return len(slots)
    batches, streams, graphs, outs = [batch(1), batch(2)], [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for s, stream in zip(batches, streams):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(s, s["cache"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(step(s, s["cache"]))
        graphs.append(graph)
    eager = [[c.clone() for c in s["cache"]] for s in batches]
    at = [[0] * B, [0] * B]
    for counts in ([40, 1, 3, 0], [1, 1, 1, 1], [1, 0, 40, 1], [2, 30, 1, 1], [1, 1, 1, 1]):
        used = [advance(s, c, a) for s, c, a in zip(batches, (counts, counts[::-1]), at)]
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for s, cache, out, n in zip(batches, eager, outs, used):
            want = step(s, cache)
            assert torch.equal(out[:n], want[:n]) and not torch.isnan(out[:n]).any()
            for x, y in zip(s["cache"], cache):
                assert torch.equal(torch.nan_to_num(x.float(), 5e4), torch.nan_to_num(y.float(), 5e4))


def test_tokens_whose_elements_pass_32_bits():
    T, hq, hk, d, last = 600_000, 32, 8, 128, 50  # 3.7e9 elements in, 2.5e9 out
    g = gen(4)
    qkv = torch.zeros(T, hq + 2 * hk, d, dtype=torch.float16, device="cuda")
    qkv[-last:] = torch.randn(last, hq + 2 * hk, d, device="cuda", generator=g).half()
    slots = torch.full((T,), -1, device="cuda")
    slots[-last:] = torch.arange(last, device="cuda") * 16
    big, small = empty_cache(last, hk, 16, d), empty_cache(last, hk, 16, d)
    q = qg.qift_append_kv(qkv[:, hq:hq + hk], qkv[:, hq + hk:], slots, d, *big, q=qkv[:, :hq])
    tail = qkv[-last:].clone()
    del qkv
    few = qg.qift_append_kv(tail[:, hq:hq + hk], tail[:, hq + hk:], slots[-last:].clone(), d, *small, q=tail[:, :hq])
    assert torch.equal(q[-last:], few)
    for x, y in zip(big, small):
        assert torch.equal(torch.nan_to_num(x.float(), 5e4), torch.nan_to_num(y.float(), 5e4))
    # every token a sequence of one key, so that its result is that key's value; the last ones have one each
    table = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    table[-last:, 0] = torch.arange(last, dtype=torch.int32, device="cuda")
    lens = torch.ones(T, dtype=torch.int32, device="cuda")
    lse = torch.empty(T, hq, device="cuda")
    out = qg.qift_paged_attention(q, None, 1, *big, table, lens, lse=lse)
    _, v = qg.qift_gather_kv(*big, slots[-last:].clone(), 0)
    want = v.repeat_interleave(hq // hk, 1).float()
    assert ((out[-last:].float() - want).abs() <= want.abs() * (2.0 ** -11 * 3 + 2.0 ** -17)).all()  # the weight, and either result's rounding
    assert (out[0].float() - want[0]).abs().amax() <= want[0].abs().amax() * 2.0 ** -9
    k, _ = qg.qift_gather_kv(*big, slots[-last:].clone(), 0)
    u = (q[-last:].double() * k.repeat_interleave(hq // hk, 1).double()).sum(-1) / math.sqrt(d)
    # k read back is rounded to binary16: half a step, 2^-11, of each of its values
    reach = (q[-last:].double() * k.repeat_interleave(hq // hk, 1).double()).abs().sum(-1) / math.sqrt(d)
    s_max = small[1].nan_to_num(0.0).amax()
    e_u = score_error(q[-last:].double().abs().sum(-1) * s_max / math.sqrt(d), d)
    assert ((lse[-last:].double() - u).abs() <= reach * 2.0 ** -11 + e_u + 2.0 ** -16 + u.abs() * 2.0 ** -20).all()


# ------------------------------------------------------------------------------------------ numbers at their ends
@pytest.mark.parametrize("prefix", [0, 16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_an_infinite_query_gives_no_number_whatever_the_codes_signs(d, prefix):
    """Every key a row sees may answer an infinity with -infinity (or with infinity, or by a code of 0 with NaN): no
    softmax is defined, and the row must not be taken for one that sees nothing."""
    hq, hk, size, n = 4, 2, 16, 9
    m = make([n], [prefix + n], hq, hk, d, size, prefix, seed=30 + d)
    ref, lse, A, reach = reference(m)
    for sign in (7, -7, 0):
        for at in (0, 1, 2, 5, 8, d // 2, d - 2, d - 1):
            cache = [c.clone() for c in m["cache"]]
            if at % 2:
                cache[0][..., at // 2] = (cache[0][..., at // 2] & 0x0F) | ((sign & 15) << 4)
            else:
                cache[0][..., at // 2] = (cache[0][..., at // 2] & 0xF0) | (sign & 15)
            x = dict(m, cache=cache, q=m["q"].clone())
            ref, lse, A, reach = reference(x)
            bad = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
            bad[0, 1] = bad[0, 2] = bad[n - 1, 3] = True   # position prefix sees one key of its own
            x["q"][0, 1, at], x["q"][0, 2, at], x["q"][n - 1, 3, at] = math.inf, -math.inf, math.inf
            for path in paths(m):
                qg.qift_debug_set_attention_path(path)
                l = torch.empty(n, hq, device="cuda")
                out = call(x, out_dtype=torch.float32, lse=l)
                assert torch.isnan(out[bad]).all() and torch.isnan(l[bad]).all(), (path, sign, at, l[bad].tolist())
                assert ((out.double() - ref).abs() <= bound(A, reach, ref, False))[~bad].all(), (path, sign, at)
                assert torch.isfinite(l[~bad]).all()


def test_an_infinite_query_that_sees_nothing_is_empty():
    m = make([5], [3], 4, 2, 64, 16, seed=31)               # the first two rows stand before the sequence
    m["q"][0, 1, 4], m["q"][1, 2, 7] = math.inf, NAN
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        l = torch.zeros(5, 4, device="cuda")
        out = call(m, out_dtype=torch.float32, lse=l)
        assert (out[:2] == 0).all() and (l[:2] == -math.inf).all() and torch.isfinite(out[2:]).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("behind", [None, 0.0, 300.0])
@pytest.mark.parametrize("n", [190, 3000])
def test_keys_with_zero_values_far_above_the_others(n, behind, d):
    """Keys whose value rows are all zero (a scale of 0) meet no product that could overflow, but their weights are
    in the sum: scores up to 2^140 above those before, one sequence for each, with a last key further above or not.

    A weight is held to 2^-29 of the largest weight times its value's scale, a scale below 2^-28 counting as 2^-28:
    7 codes times n such errors of weights up to 1 are added to the bound."""
    B, hq = 75, 4
    m = make([1] * B, [n] * B, hq, 1, d, 16, seed=n + d)
    kc, ks, vc, vs = m["cache"]
    kc.zero_()
    kc[..., 0] = 7                                          # a key is (7, 0, 0, ...) s, a query (1, 0, 0, ...)
    m["q"].zero_()
    m["q"][..., 0] = 1
    for b in range(B):
        at = torch.arange(n, device="cuda")
        page, row = m["table"][b].long()[at // 16], at % 16
        log2 = torch.zeros(n, device="cuda")
        log2[n // 2:] = 103 + 0.5 * b
        if behind is not None:
            log2[-1] = behind
        ks[page, 0, row] = log2 * math.log(2) * math.sqrt(d) / 7
        zero = (log2 > 1) & (log2 < 299)
        vs[page[zero], 0, row[zero]] = 0.0
        vc[page[zero], 0, row[zero]] = 0
    ref, lse, A, reach = reference(m)
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        l = torch.empty(B, hq, device="cuda")
        out = call(m, out_dtype=torch.float32, lse=l)
        e_u = score_error(reach, d) + 2.0 ** -16 + lse.abs() * 2.0 ** -20
        assert ((l.double() - lse).abs() <= e_u).all(), (path, (l - lse).abs().amax(1).tolist())
        assert ((out.double() - ref).abs() <= bound(A, reach, ref, False) + 7 * n * 2.0 ** -57).all(), path


@pytest.mark.parametrize("shape", [(0, 64), (8, 0), (0, 0)])
def test_an_empty_rope_table_is_refused_and_not_taken_for_none(shape):
    cache = empty_cache(1, 1, 16, 64)
    x = torch.randn(2, 1, 64, device="cuda", generator=gen(1)).half()
    at = torch.arange(2, device="cuda")
    q_out = torch.full((2, 1, 64), 5.0, device="cuda").half()
    with pytest.raises(ValueError, match="rope"):
        qg.qift_append_kv(x, x, at, 64, *cache, q=x, positions=at, rope=torch.empty(shape, device="cuda"), q_out=q_out)
    torch.cuda.synchronize()
    assert (q_out == 5).all() and torch.isnan(cache[1]).all() and torch.isnan(cache[3]).all()


def guarded(shape, dtype, fill=77):
    """A tensor inside a larger one, and what tells whether anything around it was written."""
    n = math.prod(shape)
    whole = torch.full((n + 2 * 4096,), fill, dtype=dtype, device="cuda")
    return whole[4096:4096 + n].view(shape), lambda: bool((whole[:4096] == fill).all() and (whole[4096 + n:] == fill).all())


@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (16, 1, 128), (3, 3, 256)])
def test_contradicting_offsets_write_nowhere_else(hq, hk, d, prefix):
    """Offsets, lengths and tables that contradict the call's sizes: nothing around the result, its log-sum-exp and the
    workspace is written, and under bounds checks no index leaves its array."""
    q_lens, size = [1, 2, 0, 30, 1, 1, 5, 1], 16
    m = make(q_lens, [prefix + 40 + 90 * (i % 4) for i in range(8)], hq, hk, d, size, prefix, seed=33)
    T, far = sum(q_lens), 2 ** 31 - 1
    starts = [m["cu_q"].tolist(), [0, 3, 2, 1, 9, 9, 4, 40, 2], [-5, 2, 4, -far, 0, 7, 11, 12, 400], [far] * 9, [-far] * 9,
              [0] * 8 + [T], [0] * 8 + [far], [T] + [0] * 8, [T - 1] * 9, list(range(T, T - 9, -1)), [0, T, 0, T, 0, T, 0, T, 0]]
    lens = [m["kv_lens"].tolist(), [far, -far, -3, 0, 2 ** 30, far, 1, -1]]
    tables = [m["table"], torch.full_like(m["table"], far), torch.full_like(m["table"], -far)]
    for path in paths(m):
        qg.qift_debug_set_attention_path(path)
        for max_q in (1, 7, 30):
            for max_kv in (0, 1):
                bytes_ = qg.qift_paged_attention_workspace(T, hq, hk, d, 8, max_q, size, m["table"].shape[1], max_kv, prefix)
                for cu in starts:
                    for n in lens:
                        for table in tables:
                            out, out_ok = guarded((T, hq, d), torch.float16)
                            l, l_ok = guarded((T, hq), torch.float32)
                            ws, ws_ok = guarded((bytes_,), torch.uint8)
                            call(dict(m, cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q=max_q, table=table,
                                      kv_lens=torch.tensor(n, dtype=torch.int32, device="cuda")),
                                 out=out, lse=l, workspace=ws, max_kv=max_kv, block=d)
                            assert out_ok() and l_ok() and ws_ok(), (path, max_q, max_kv, cu, n)


@pytest.mark.parametrize("d,rope_dim,interleaved", [(64, 64, False), (128, 48, True), (256, 128, False)])
def test_append_and_gather_write_nowhere_else(d, rope_dim, interleaved):
    T, hq, hk, size, pages, far = 21, 5, 3, 16, 3, 50
    g = gen(34)
    x = torch.randn(T, hq + 2 * hk, d, device="cuda", generator=g).half()
    edge = [-1, -2 ** 63, 2 ** 63 - 1, pages * size, pages * size - 1, 0, 2 ** 31, -2 ** 31, 2 ** 32]
    slots = torch.tensor(edge + list(range(1, T - len(edge) + 1)), device="cuda")
    positions = torch.tensor(list(range(12)) + [far - 1, far, -1, 2 ** 62, -2 ** 63, 2 ** 63 - 1, 2 ** 32, 0, 0], device="cuda")
    made = [guarded((pages, hk, size, d // 2), torch.uint8), guarded((pages, hk, size), torch.float32),
            guarded((pages, hk, size, d // 2), torch.uint8), guarded((pages, hk, size), torch.float32),
            guarded((T, hq, d), torch.float16)]
    cache = [t for t, _ in made[:4]]
    qg.qift_append_kv(x[:, hq:hq + hk], x[:, hq + hk:], slots, d, *cache, q=x[:, :hq], positions=positions,
                      rope=rope_table(far, rope_dim).cuda(), interleaved=interleaved, q_out=made[4][0])
    assert all(ok() for _, ok in made)
    kept = ((slots >= 0) & (slots < pages * size) & (positions >= 0) & (positions < far)).tolist()
    written = {int(s) for s, k in zip(slots.tolist(), kept) if k}
    for s in cache[1::2]:
        now = (s.movedim(1, 2).reshape(pages * size, hk) != 77).all(1)
        assert {i for i, w in enumerate(now.tolist()) if w} == written
    k, v = qg.qift_gather_kv(*cache, slots, d)
    outside = (slots < 0) | (slots >= pages * size)
    assert (k[outside] == 0).all() and (v[outside] == 0).all()


def test_no_tokens_need_no_rope_table():
    cache = empty_cache(1, 1, 16, 64)
    x, at = torch.empty(0, 1, 64, device="cuda").half(), torch.empty(0, dtype=torch.int64, device="cuda")
    assert qg.qift_append_kv(x, x, at, 64, *cache, q=x, positions=at, rope=torch.empty(0, 64, device="cuda")).shape == x.shape


@pytest.mark.parametrize("path", ["stream", "wide"])
@pytest.mark.parametrize("d,hk,hq", [(128, 8, 32), (64, 2, 16)])
def test_steps_that_follow_at_once_see_one_anothers_rows(path, d, hk, hq):
    """Sixty steps of append and attention one behind the other, with one buffer of queries and one workspace: each
    kernel may start while the one before it runs, and reads what that one writes (a scale's neighbours in a line too)."""
    B, steps, size = 4, 60, 16
    g = gen(41)
    per = steps // size + 3
    qkv = torch.randn(steps, B, hq + 2 * hk, d, device="cuda", generator=g).half()
    table = torch.randperm(B * per, device="cuda", generator=g).to(torch.int32).view(B, per)
    at = torch.arange(steps, device="cuda")[:, None] + torch.tensor([0, 5, 15, 16], device="cuda")
    slots = (table.long()[torch.arange(B, device="cuda")[None], at // size] * size + at % size).contiguous()
    lens = (at + 1).to(torch.int32)
    rope = rope_table(200, d).cuda()
    q = torch.empty(B, hq, d, device="cuda").half()
    qg.qift_debug_set_attention_path(path)
    workspace = torch.empty(qg.qift_paged_attention_workspace(B, hq, hk, d, B, 1, size, per, prefix_len=0), device="cuda",
                            dtype=torch.uint8)
    first = [torch.randint(0, 256, (B * per, hk, size, d // 2), device="cuda", generator=g).to(torch.uint8),
             torch.rand(B * per, hk, size, device="cuda", generator=g)]
    first += [x.flip(0).contiguous() for x in first]

    def step(t, cache, out):
        qg.qift_append_kv(qkv[t][:, hq:hq + hk], qkv[t][:, hq + hk:], slots[t], d, *cache, q=qkv[t][:, :hq], positions=at[t],
                          rope=rope, q_out=q)
        qg.qift_paged_attention(q, None, 1, *cache, table, lens[t], block=d, out=out[t], workspace=workspace)

    want, got = torch.empty(2, steps, B, hq, d, device="cuda").half()
    alone, chained = [c.clone() for c in first], [c.clone() for c in first]
    for t in range(steps):
        step(t, alone, want)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for t in range(steps):
            step(t, chained, got)
    for _ in range(10):
        for a, b in zip(chained, first):
            a.copy_(b)
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(alone, chained))
