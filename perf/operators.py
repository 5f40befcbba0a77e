"""Workloads of the paged KV4 cache: appending keys and values with the position rotation, attention over the
cache with a window and first tokens that stay visible, and attention for a batch that shares a prefix.

A case is one call as a serving program makes it.  ``run`` computes it in plain torch where ``own`` is false and
through the library's entry points where it is true; ``exact`` is the definition in 64 bits.

Layouts (those of ``qift_append_kv`` and ``qift_paged_attention``):
  cache    uint8 [pages, kv_heads, page_size, head_dim / 2], two's-complement nibbles, the lower index low
  scales   float32 [pages, kv_heads, page_size]
  slot     page * page_size + offset in the page; -1 marks a row that is padding
  rope     float32 [positions, rope_dim]: the cosines of a position, then its sines
"""
import math
import random

import torch

own = False

APPEND, ATTENTION = "append", "attention"


# ------------------------------------------------------------------------------------------------- cases
def _append(name, tokens, padded, q_heads, kv_heads, head_dim, page_size, rope_dim, interleaved, block, far):
    return dict(name=name, kind=APPEND, tokens=tokens, padded=padded, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, page_size=page_size, rope_dim=rope_dim, interleaved=interleaved, block=block,
                far=far)


def _attention(name, batch, q_min, q_max, own_min, own_max, prefix, q_heads, kv_heads, head_dim, page_size, window,
               sinks, block):
    return dict(name=name, kind=ATTENTION, batch=batch, q_min=q_min, q_max=q_max, own_min=own_min, own_max=own_max,
                prefix=prefix, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size,
                window=window, sinks=sinks, block=block)


def listed():
    return [
        # One generated token of one user: 8B-shaped heads (32 query, 8 key/value, 128 wide).  Latency only.
        _append("append 1 token", 1, 0, 32, 8, 128, 16, 128, False, 128, 131072),
        # A decode batch padded for a captured graph; narrow heads, half of each rotated, in adjacent pairs.
        _append("append 61 padded d64", 61, 7, 16, 4, 64, 32, 32, True, 64, 8192),
        # A long prompt with 7B-shaped heads (32 query, 32 key/value).
        _append("append 8192 prompt", 8192, 0, 32, 32, 128, 16, 128, False, 128, 8192),
        # One user's next token early in a chat: latency only.
        _attention("decode 1x200", 1, 1, 1, 200, 200, 0, 32, 8, 128, 16, 0, 0, 128),
        # A batch of 16 users, 7B-shaped heads (each query head with its own keys).
        _attention("decode 16x4096 mha", 16, 1, 1, 300, 4096, 0, 32, 32, 128, 16, 0, 0, 128),
        # A full serving batch with long contexts: the cache is read at the memory's rate or not at all.
        _attention("decode 64x16384", 64, 1, 1, 8000, 16384, 0, 32, 8, 128, 16, 0, 0, 0),
        # One very long document: few rows, so the work has to be split over its length.
        _attention("decode 1x131071", 1, 1, 1, 131071, 131071, 0, 32, 8, 128, 64, 0, 0, 128),
        # Streaming generation: a window and four first tokens that stay visible; contexts far beyond the window.
        _attention("decode window 33x40000", 33, 1, 1, 3000, 40000, 0, 64, 8, 64, 32, 4096, 4, 64),
        # Prompts in chunks, with what came before in the cache, windowed.
        _attention("chunks window 3x2500", 3, 1100, 2500, 2600, 6000, 0, 32, 8, 128, 16, 1024, 4, 128),
        # A whole prompt of 8192 tokens, causal.
        _attention("prompt 8192", 1, 8192, 8192, 8192, 8192, 0, 32, 8, 128, 16, 0, 0, 128),
        # A few users behind one system prompt.
        _attention("prefix 2001 by 16", 16, 1, 1, 20, 300, 2001, 32, 8, 128, 16, 0, 0, 128),
        # Many short answers drawn from one long document.
        _attention("prefix 32768 by 128", 128, 1, 1, 10, 1000, 32768, 32, 8, 128, 16, 0, 0, 128),
    ]


HEADS = [(32, 8, 128), (32, 32, 128), (64, 8, 64), (16, 4, 64), (28, 4, 128), (40, 8, 128), (16, 1, 128), (8, 2, 256),
         (12, 12, 64)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    q_heads, kv_heads, head_dim = rng.choice(HEADS)
    page_size = rng.choice([16, 32, 64, 128])
    block = rng.choice([0, head_dim, head_dim])
    kind = rng.choice(["append", "decode", "decode", "prompt", "prefix"])
    if kind == "append":
        tokens = min(_log(rng, 1, 8192), 8192 * 96 * 128 // ((q_heads + 2 * kv_heads) * head_dim))
        c = _append("", tokens, rng.randint(0, min(9, tokens - 1)), q_heads, kv_heads, head_dim, page_size,
                    rng.choice([0, head_dim // 2, head_dim, head_dim]), rng.random() < 0.4, block,
                    _log(rng, max(64, tokens), 131072))
        del c["name"]
        return c
    window, sinks = (0, 0) if rng.random() < 0.5 else (_log(rng, 100, 8000), rng.choice([0, 1, 4, 100]))
    prefix = 0
    if kind == "prompt":
        batch, q_max = _log(rng, 1, 8), _log(rng, 17, 8192)
        q_min = rng.randint(1, q_max)
        own_max = q_max + (0 if rng.random() < 0.4 else _log(rng, 1, 8192))
        own_min = rng.randint(q_max, own_max)
    else:
        batch = _log(rng, 1, 64) if kind == "decode" else _log(rng, 2, 128)
        q_min, q_max = (1, 1) if rng.random() < 0.7 else (1, rng.randint(2, 8))
        own_max = q_max + (_log(rng, 1, 131072) if kind == "decode" else _log(rng, 1, 1000))
        own_min = rng.randint(q_max, own_max)
        if kind == "prefix":
            prefix = _log(rng, 100, 32768)
    # No drawn case costs more than the largest listed one: neither in products (half of the square is masked
    # there) nor in keys and values.
    products, values = 8192 * 8192 * 32 * 128 // 2, 64 * 12000 * 8 * 128
    while batch > 1 and (batch * q_max * (own_max + prefix) * q_heads * head_dim > products
                         or batch * own_max * kv_heads * head_dim > values):
        batch -= 1
    while q_max * (own_max + prefix) * q_heads * head_dim > products:
        q_max, own_max = q_max * 3 // 4, own_max * 3 // 4
        q_min, own_min = min(q_min, q_max), min(max(own_min * 3 // 4, q_max), own_max)
    c = _attention("", batch, q_min, q_max, own_min, own_max, prefix, q_heads, kv_heads, head_dim, page_size, window,
                   sinks, block)
    del c["name"]
    return c


def _spread(count, lo, hi, phase):
    """`count` whole numbers spread evenly over [lo, hi], both ends among them, in no order of size."""
    got = [lo + int(((i * 0.6180339887498949 + phase) % 1.0) * (hi - lo + 1)) for i in range(count)]
    got[-1] = lo
    got[0] = hi
    return got


def _lengths(case):
    """(tokens asked, keys of its own) of each sequence."""
    return (_spread(case["batch"], case["q_min"], case["q_max"], 0.5),
            _spread(case["batch"], case["own_min"], case["own_max"], 0.0))


# ------------------------------------------------------------------------------------------------ inputs
def _quantise(x):
    """Random rows as the cache holds them: nibbles and scales of the rows' INT4 values."""
    scale = x.abs().amax(-1) / 7.0
    q = torch.round(x / scale.unsqueeze(-1)).clamp_(-7, 7).to(torch.int8)
    return ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8).contiguous(), scale


def _rope_table(positions, dim, device):
    if not dim:
        return None
    inverse = 500000.0 ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * inverse
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = random.Random(seed)
    hq, hk, d, ps = case["q_heads"], case["kv_heads"], case["head_dim"], case["page_size"]
    s = dict(case)
    if case["kind"] == APPEND:
        t = case["tokens"]
        pages = -(-t // ps) + 9
        # Queries, keys and values are slices of one projection's output, as a model has them.
        qkv = torch.randn(t, hq + 2 * hk, d, device=device, generator=g)
        qkv[:, :, 3] *= 12.0  # a channel that stands out, as keys have them before the rotation
        s["q"], s["k"], s["v"] = qkv.half().split([hq, hk, hk], dim=1)
        slots = torch.randperm(pages * ps, device=device, generator=g)[:t].contiguous()
        slots[torch.randperm(t, device=device, generator=g)[:case["padded"]]] = -1
        s["slots"] = slots
        first = r.randint(0, max(0, case["far"] - t))
        s["positions"] = torch.arange(first, first + t, device=device)
        s["rope"] = _rope_table(case["far"], case["rope_dim"], device)
        for n in ("k", "v"):
            s[n + "_cache"] = torch.zeros(pages, hk, ps, d // 2, device=device, dtype=torch.uint8)
            s[n + "_scales"] = torch.zeros(pages, hk, ps, device=device)
        return s
    q_lens, own_lens = _lengths(case)
    shared = -(-case["prefix"] // ps)
    own_pages = [-(-n // ps) for n in own_lens]
    pages = shared + sum(own_pages) + 3
    for n in ("k", "v"):
        s[n + "_cache"], s[n + "_scales"] = _quantise(torch.randn(pages, hk, ps, d, device=device, generator=g))
    order = torch.randperm(pages, device=device, generator=g).to(torch.int32)
    s["prefix_table"] = order[:shared].contiguous() if shared else None
    table = torch.zeros(case["batch"], max(own_pages), device=device, dtype=torch.int32)
    at = torch.arange(max(own_pages), device=device)[None, :] < torch.tensor(own_pages, device=device)[:, None]
    table[at] = order[shared:shared + sum(own_pages)]
    s["page_table"] = table
    s["kv_lens"] = torch.tensor([n + case["prefix"] for n in own_lens], device=device, dtype=torch.int32)
    s["cu_q"] = torch.tensor([0] + q_lens, device=device).cumsum(0).to(torch.int32)
    s["q"] = torch.randn(sum(q_lens), hq, d, device=device, generator=g).half()
    s["own_longest"] = max(own_lens)
    return s


# ------------------------------------------------------------------------------------------- plain forms
def _unpack(p):
    """Nibbles to the whole numbers that they are, as float32."""
    p = p.view(torch.int8)
    return torch.stack([(p << 4) >> 4, p >> 4], dim=-1).flatten(-2).float()


def _hadamard(x, block):
    """Rows times the Walsh-Hadamard matrix of `block` over its root: sums and differences at distance 1, 2, 4 and
    so on, the order that `qift_rotate` is defined by."""
    if not block:
        return x
    h, shape = 1, x.shape
    while h < block:
        x = x.reshape(-1, 2, h)
        x = torch.stack([x[:, 0] + x[:, 1], x[:, 0] - x[:, 1]], dim=1)
        h *= 2
    return x.reshape(shape) * torch.tensor(1.0 / math.sqrt(block), dtype=torch.float32, device=x.device)


def _rotate(x, s):
    """Position rotation of [tokens, heads, d] rows, in float32."""
    if s["rope"] is None:
        return x
    half = s["rope_dim"] // 2
    c, n = s["rope"][s["positions"]][:, None].split([half, half], dim=-1)
    rest = x[..., s["rope_dim"]:]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if s["interleaved"] else (x[..., :half], x[..., half:2 * half])
    y = (a * c - b * n, b * c + a * n)
    y = torch.stack(y, dim=-1).flatten(-2) if s["interleaved"] else torch.cat(y, dim=-1)
    return torch.cat([y, rest], dim=-1)


def _plain_append(s):
    seven = torch.full((), 7.0, device=s["k"].device)  # a tensor: division by a number multiplies by its inverse
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    page, at = slots // s["page_size"], slots % s["page_size"]
    out = {"q": _hadamard(_rotate(s["q"].float(), s), s["block"]).half()}
    for n in ("k", "v"):
        x = s[n].float()
        x = _hadamard(_rotate(x, s) if n == "k" else x, s["block"]).half().float()
        m = x.abs().amax(-1)
        inverse = torch.where(m > 0, seven / m, torch.zeros_like(m))
        q = torch.round(x * inverse.unsqueeze(-1)).clamp(-7, 7).to(torch.int8)
        s[n + "_cache"][page, :, at] = ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.uint8)[kept]
        s[n + "_scales"][page, :, at] = (m / seven)[kept]
        # What the cache now holds for these rows, as the values that it stands for.
        y = torch.zeros_like(x)
        y[kept] = _unpack(s[n + "_cache"][page, :, at]) * s[n + "_scales"][page, :, at].unsqueeze(-1)
        out[n] = y.half()
    return out


def _rows(s, name, table, count):
    """[.., count, d] values of the first `count` tokens of a table of pages, kv heads before tokens."""
    table = table.long()
    x = _unpack(s[name + "_cache"][table]) * s[name + "_scales"][table].unsqueeze(-1)
    x = x.movedim(-3, -4)  # [.., kv, pages, page_size, d]
    return x.flatten(-3, -2)[..., :count, :]


def _plain_attention(s):
    b, hq, hk, d, p = s["batch"], s["q_heads"], s["kv_heads"], s["head_dim"], s["prefix"]
    device, group = s["q"].device, hq // hk
    q_max = s["q_max"]
    first, last = s["cu_q"][:-1].long(), s["cu_q"][1:].long()
    i = torch.arange(q_max, device=device)
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)  # [b, q_max]; rows past a sequence's end are not kept
    # [b, kv, group * q_max, d]
    q = s["q"].float()[row].reshape(b, q_max, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * q_max, d)
    scores = q @ _rows(s, "k", s["page_table"], s["own_longest"]).transpose(-1, -2)
    if p:  # the prefix's keys meet the rows of the whole batch
        every = q.transpose(0, 1).reshape(hk, b * group * q_max, d)
        shared = every @ _rows(s, "k", s["prefix_table"], p).transpose(-1, -2)
        scores = torch.cat([shared.reshape(hk, b, group * q_max, p).transpose(0, 1), scores], dim=-1)
    scores *= 1.0 / math.sqrt(d)
    where = (s["kv_lens"].long() - (last - first))[:, None, None] + i[:, None]  # [b, q_max, 1] position of a row
    j = torch.arange(scores.shape[-1], device=device)
    seen = j <= where
    if s["window"]:
        seen &= (j > where - s["window"]) | (j < s["sinks"])
    seen = seen[:, None, None].expand(b, hk, group, q_max, j.numel()).reshape(scores.shape)
    scores.masked_fill_(~seen, -math.inf)
    del seen
    scores -= scores.amax(-1, keepdim=True)
    weights = scores.exp_()
    weights /= weights.sum(-1, keepdim=True)
    out = weights[..., p:] @ _rows(s, "v", s["page_table"], s["own_longest"])
    if p:
        every = weights[..., :p].transpose(0, 1).reshape(hk, b * group * q_max, p)
        out += (every @ _rows(s, "v", s["prefix_table"], p)).reshape(hk, b, group * q_max, d).transpose(0, 1)
    out = out.reshape(b, hk, group, q_max, d).permute(0, 3, 1, 2, 4).reshape(b, q_max, hq, d)
    return _hadamard(out[i[None, :] < (last - first)[:, None]], s["block"]).half()


def run(state):
    if own:
        import w2a4_gemm_b200 as qg
        cache = (state["k_cache"], state["k_scales"], state["v_cache"], state["v_scales"])
        if state["kind"] == APPEND:
            q = qg.qift_append_kv(state["k"], state["v"], state["slots"], state["block"], *cache, q=state["q"],
                                  positions=state["positions"], rope=state["rope"],
                                  interleaved=state["interleaved"])
            k, v = qg.qift_gather_kv(*cache, state["slots"], 0)
            return {"q": q, "k": k, "v": v}
        return qg.qift_paged_attention(state["q"], state["cu_q"], state["q_max"], *cache, state["page_table"],
                                       state["kv_lens"], window=state["window"], sinks=state["sinks"],
                                       prefix_table=state["prefix_table"], prefix_len=state["prefix"],
                                       block=state["block"])
    return _plain_append(state) if state["kind"] == APPEND else _plain_attention(state)


# -------------------------------------------------------------------------------------------------- work
def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["kind"] == APPEND:
        t = case["tokens"]
        read = t * (hq + 2 * hk) * d * 2 + t * 16 + t * case["rope_dim"] * 4
        written = t * hq * d * 2 + (t - case["padded"]) * hk * (d + 8) + 2 * t * hk * d * 2
        # a rotation is 6 operations for a pair, the Walsh-Hadamard transform one for a value and stage
        stages = max(1, case["block"]).bit_length() - 1
        flops = t * (hq + hk) * case["rope_dim"] * 3 + t * (hq + 2 * hk) * d * (stages + 1) + t * 2 * hk * d * 3
        return {"bytes": read + written, "flops": flops}
    q_lens, own_lens = _lengths(case)
    w, sinks, p = case["window"], case["sinks"], case["prefix"]
    pairs = keys = 0
    lowest = p  # the shared keys from here on are inside some row's window
    for nq, n in zip(q_lens, own_lens):
        total = n + p
        low = max(0, total - nq - w + 1) if w else 0  # the first key of the first row's window
        keys += total - max(low, p) + (max(0, min(sinks, low) - p) if w else 0)
        lowest = min(lowest, low)
        if w:
            pairs += sum(min(x + 1, w) + min(sinks, max(0, x + 1 - w)) for x in range(total - nq, total))
        else:
            pairs += nq * total - nq * (nq - 1) // 2
    keys += p - lowest + (min(sinks, lowest) if w else 0)
    tokens = sum(q_lens)
    return {"bytes": keys * hk * (d + 8) + 2 * tokens * hq * d * 2 + 4 * (keys // case["page_size"] + 2 * case["batch"]),
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------------------------------------- exact
def _matrix(n, device):
    """The Walsh-Hadamard matrix of n over its root: the sign is the parity of the bits that row and column share."""
    if not n:
        return None
    i = torch.arange(n, device=device)
    shared, parity = i[:, None] & i[None, :], torch.zeros(n, n, device=device, dtype=torch.long)
    for bit in range(n.bit_length()):
        parity ^= (shared >> bit) & 1
    return (1.0 - 2.0 * parity.double()) / math.sqrt(n)


def _turned(x, matrix):
    return x if matrix is None else (x.unflatten(-1, (-1, matrix.shape[0])) @ matrix).flatten(-2)


def _whole(packed):
    """Nibbles as whole numbers, in 64 bits."""
    n = packed.long()
    n = torch.stack([n % 16, n // 16], dim=-1).flatten(-2)
    return torch.where(n > 7, n - 16, n).double()


def _exact_append(s):
    matrix, device = _matrix(s["block"], s["k"].device), s["k"].device
    turn = torch.eye(s["head_dim"], device=device, dtype=torch.float64).repeat(s["tokens"], 1, 1)
    half = s["rope_dim"] // 2
    for i in range(half):  # each token's rotation, as a matrix
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        row = s["rope"][s["positions"]].double()
        turn[:, a, a] = turn[:, b, b] = row[:, i]
        turn[:, b, a], turn[:, a, b] = row[:, half + i], -row[:, half + i]
    out = {"q": _turned(torch.einsum("thd,ted->the", s["q"].double(), turn), matrix)}
    for n in ("k", "v"):
        x = s[n].double()
        x = _turned(torch.einsum("thd,ted->the", x, turn) if n == "k" else x, matrix)
        x = x.half().double()  # the quantiser's input is defined as a binary16 value
        top = x.abs().amax(-1, keepdim=True)
        y = torch.round(x * 7.0 / top.clamp(min=1e-30)) * (top / 7.0)
        y[s["slots"] < 0] = 0.0
        out[n] = y
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == APPEND:
        return _exact_append(s)
    hq, hk, d, ps, p = (case[n] for n in ("q_heads", "kv_heads", "head_dim", "page_size", "prefix"))
    matrix, device = _matrix(case["block"], s["q"].device), s["q"].device
    out = torch.zeros(s["q"].shape, device=device, dtype=torch.float64)
    shared = [] if not p else s["prefix_table"].tolist()
    at = 0
    for nq, n, table in zip(*_lengths(case), s["page_table"].tolist()):
        total = n + p
        where = torch.arange(total - nq, total, device=device)[:, None]
        j = torch.arange(total, device=device)[None, :]
        hidden = j > where
        if case["window"]:
            hidden |= (j <= where - case["window"]) & (j >= case["sinks"])
        ids = [torch.tensor(t, device=device) for t in (shared, table[:-(-n // ps)])]
        for h in range(hk):
            kv = []
            for name in ("k", "v"):
                parts = [(_whole(s[name + "_cache"][t, h]) * s[name + "_scales"][t, h].double().unsqueeze(-1)).flatten(0, 1)[:c]
                         for t, c in zip(ids, (p, n)) if c]
                kv.append(torch.cat(parts))
            for x in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = s["q"][at:at + nq, x].double() @ kv[0].T / math.sqrt(d)
                score.masked_fill_(hidden, -math.inf)
                out[at:at + nq, x] = _turned(torch.softmax(score, dim=-1) @ kv[1], matrix)
        at += nq
    return out
