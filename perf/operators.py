"""The attention operators of libar.so as measured cases: one rank's heads between
the q/k/v projection and the output projection whose partial sums the
all-reduce adds up.

Three operators, called one after another in a decode step:

norm_rope, norm_rope_grad
    norms of queries and keys for each head with the rotation in the same pass,
    and its gradient;
cache
    a token's keys and values quantised into a paged cache of 4 bits, and read
    back;
attend
    attention over that cache.

The cache is made of tiles of 32 tokens of one head, 34 D bytes each: K codes
(16 D), V codes (16 D), K scales (D), V scales (D).  Codes are E2M1 (values 0,
0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two in a byte, the even channel in the low
half; 32 channels of a token share the scale 2**(byte - 127), and 255 stands
for a group that held an infinity or a NaN.  Places within a tile, for token t,
channel c, group g = c // 32, W = D // 16 and G = D // 32:
    K code byte    t * D/2 + c/2
    V code byte    ((t/8 * 16 + c/W) * 8 + t%8) * W/2 + c%W/2
    K scale byte   (g * 16 + t/8 * 4 + t%4) * 2 + t%8/4
    V scale byte   (t/8 * G + g) * 8 + t%8
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of eight sequences, one rank of eight: 8 query heads, 1 key head
        {"name": "norm_rope_step", "op": "norm_rope", "tokens": 8, "heads": 8, "kv_heads": 1, "dim": 128,
         "rotated": 128, "interleaved": False, "table": 32768},
        # 680 tokens of a whole layer of 40 heads, small heads of which half the channels turn, in pairs side by side
        {"name": "norm_rope_partial", "op": "norm_rope", "tokens": 680, "heads": 40, "kv_heads": 8, "dim": 64,
         "rotated": 32, "interleaved": True, "table": 8192},
        # a long prompt through a whole layer of 7168 = 56 x 128
        {"name": "norm_rope_prompt", "op": "norm_rope", "tokens": 8192, "heads": 56, "kv_heads": 8, "dim": 128,
         "rotated": 128, "interleaved": False, "table": 32768},
        # a training step on 440 tokens of one rank's 5 of 40 heads
        {"name": "norm_rope_grad_share", "op": "norm_rope_grad", "tokens": 440, "heads": 5, "kv_heads": 1, "dim": 128,
         "rotated": 128, "interleaved": False, "table": 8192},
        # a training step on 4096 tokens of a whole layer of 8192 = 64 x 128
        {"name": "norm_rope_grad_layer", "op": "norm_rope_grad", "tokens": 4096, "heads": 64, "kv_heads": 8, "dim": 128,
         "rotated": 128, "interleaved": False, "table": 32768},
        # one new token for each of 440 sequences, one rank's key head
        {"name": "cache_step", "op": "cache", "tokens": 440, "kv_heads": 1, "dim": 128, "page": 64, "order": "scattered"},
        # a long prompt into the cache, all eight key heads
        {"name": "cache_prompt", "op": "cache", "tokens": 16384, "kv_heads": 8, "dim": 128, "page": 64, "order": "pages"},
        # the smallest decode call: four short sequences, one of the slots unused, one rank's heads
        {"name": "attend_step_short", "op": "attend", "batch": 4, "q_max": 1, "kv_min": 77, "kv_max": 413, "empty": 1,
         "heads": 8, "kv_heads": 1, "dim": 128, "page": 64, "window": 0},
        # one sequence of 200003 tokens on one rank: long and narrow
        {"name": "attend_step_long", "op": "attend", "batch": 1, "q_max": 1, "kv_min": 200003, "kv_max": 200003, "empty": 0,
         "heads": 8, "kv_heads": 1, "dim": 128, "page": 256, "window": 0},
        # a serving batch of ragged lengths over a whole layer
        {"name": "attend_step_batch", "op": "attend", "batch": 128, "q_max": 1, "kv_min": 2048, "kv_max": 8192, "empty": 0,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # drafted tokens being checked: up to five queries a sequence, 7 heads to a key head, small heads, a window
        {"name": "attend_draft", "op": "attend", "batch": 32, "q_max": 5, "kv_min": 501, "kv_max": 9001, "empty": 2,
         "heads": 28, "kv_heads": 4, "dim": 64, "page": 32, "window": 4096},
        # two prompts, each in chunks of 2048 tokens over what the cache holds already
        {"name": "attend_prompt", "op": "attend", "batch": 2, "q_max": 2048, "kv_min": 5999, "kv_max": 8192, "empty": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "cache", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 1, 2, 4, 8])
    if op in ("norm_rope", "norm_rope_grad"):
        heads = kv_heads * rng.randint(1, 8)
        rotated = rng.choice([dim, dim, dim // 2])
        most = (8192 * 64 * 128 if op == "norm_rope" else 4096 * 72 * 128) // ((heads + kv_heads) * dim)
        return {"op": op, "tokens": _log(rng, 1, min(8192, most)), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rotated": rotated, "interleaved": rng.random() < 0.3, "table": rng.choice([8192, 32768])}
    page = rng.choice([32, 64, 128, 256])
    if op == "cache":
        return {"op": op, "tokens": _log(rng, 1, 16384 * 8 * 128 // max(kv_heads * dim, 8 * 128)), "kv_heads": kv_heads,
                "dim": dim, "page": page, "order": rng.choice(["scattered", "pages"])}
    heads = kv_heads * rng.randint(1, 12)
    if rng.random() < 0.7:  # steps: the tokens in all are bounded by what the largest listed step holds
        batch = _log(rng, 1, 160)
        kv_max = _log(rng, 1, max(1, min(200003, 128 * 4096 * 8 * 128 // (batch * kv_heads * dim))))
        q_max = rng.choice([1, 1, 2, 5])
        while batch * q_max * heads * kv_max > 128 * 64 * 8192 and (q_max > 1 or kv_max > 1):
            q_max, kv_max = max(1, q_max // 2), max(1, kv_max // 2)
    else:  # chunks of prompts
        batch = rng.randint(1, 3)
        q_max = _log(rng, 6, 2048)
        kv_max = _log(rng, q_max, 8192)
        while batch * q_max * heads * kv_max * dim > 2 * 2048 * 32 * 8192 * 128:
            q_max, kv_max = max(1, q_max // 2), max(1, kv_max // 2)
    return {"op": op, "batch": batch, "q_max": q_max, "kv_min": rng.choice([0, 1, kv_max // 2, kv_max]), "kv_max": kv_max,
            "empty": rng.choice([0, 0, 1]) if batch > 1 else 0, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "window": rng.choice([0, 0, max(1, kv_max // 3)])}


def _lengths(case):
    """Queries and cached tokens (the queries' own among them) of each sequence: by the case alone."""
    rng = random.Random("%(batch)d %(q_max)d %(kv_min)d %(kv_max)d" % case)
    q, kv = [], []
    for b in range(case["batch"]):
        n = case["kv_max"] if b == 0 else rng.randint(case["kv_min"], case["kv_max"])
        m = case["q_max"] if b == 0 or case["q_max"] > 5 else rng.randint(1, case["q_max"])
        if b >= case["batch"] - case["empty"]:
            n, m = 0, 1  # a slot of the batch without a sequence
        q.append(m)
        kv.append(n)
    return q, kv


def _seen(n, i, q, window):
    """How many tokens query i of q sees in a sequence of n."""
    last = n - q + i
    first = max(0, last - window + 1) if window else 0
    return max(0, last + 1 - first)


def work(case):
    d = case["dim"]
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * d
        side = case["tokens"] * (8 + 4 * case["rotated"]) + 4 * d
        if case["op"] == "norm_rope":
            return {"bytes": 4 * n + side, "flops": 8 * n}
        return {"bytes": 6 * n + side + 8 * d, "flops": 16 * n}
    if case["op"] == "cache":
        n = 2 * case["tokens"] * case["kv_heads"] * d
        return {"bytes": 4 * n + 2 * n * 17 // 32 + 16 * case["tokens"], "flops": 8 * n}
    qs, kvs = _lengths(case)
    pairs = sum(_seen(n, i, q, case["window"]) for q, n in zip(qs, kvs) for i in range(q))
    tokens = sum(min(n, case["window"] + q - 1) if case["window"] else n for q, n in zip(qs, kvs))
    rows = sum(qs) * case["heads"]
    return {"bytes": tokens * case["kv_heads"] * d * 17 // 16 + rows * (4 * d + 4), "flops": 4 * d * case["heads"] * pairs}


# ------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _keys(g, *shape):
    """bf16 rows whose channels differ in size, as keys and values do."""
    size = torch.exp(0.5 * _normal(g, shape[-1]))
    return (_normal(g, *shape) * size).to(torch.bfloat16)


def _make_cache(k, v, dim, page):
    """The cache's bytes for keys and values (pages * page_size, heads, dim) by slot."""
    slots, heads = k.shape[0], k.shape[1]

    def quantise(x):
        x = x.reshape(slots, heads, dim // 32, 32)
        bits = x.view(torch.int16).to(torch.int32) & 0x7FFF
        byte = (((bits.amax(-1) + 0x20) >> 7) - 2).clamp(2, 252)
        mag = torch.ldexp(x.float().abs(), 127 - byte.unsqueeze(-1)).reshape(slots, heads, dim)
        del bits
        code = torch.zeros(mag.shape, dtype=torch.uint8, device=mag.device)
        # borders between neighbours; a value on a border goes to the even code
        for n, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
            code += (mag >= border) if n % 2 else (mag > border)
        code += 8 * (x.reshape(slots, heads, dim) < 0).to(torch.uint8)
        code = code[..., 0::2] | (code[..., 1::2] << 4)
        return code.reshape(-1, page // 32, 32, heads, dim // 2), byte.to(torch.uint8).reshape(-1, page // 32, 32, heads, dim // 32)

    def place(x, shape, order):  # (pages, tiles, 32, heads, n) -> (pages, heads, tiles, bytes)
        x = x.permute(0, 3, 1, 2, 4)
        lead = x.shape[:3]
        x = x.reshape(*lead, *shape).permute(0, 1, 2, *[3 + i for i in order])
        return x.reshape(*lead, -1)

    kc, ks = quantise(k)
    vc, vs = quantise(v)
    G = dim // 32
    return torch.cat([place(kc, (32, dim // 2), (0, 1)), place(vc, (4, 8, 16, dim // 32), (0, 2, 1, 3)),
                      place(ks, (4, 2, 4, G), (3, 0, 2, 1)), place(vs, (4, 8, G), (0, 2, 1))], -1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "kept": {}}
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        t, hq, r = case["tokens"], case["heads"], case["rotated"]
        qkv = _keys(g, t, hq + 2 * hk, d)  # the projection's output; the values in it are not touched
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"] = (1 + 0.2 * _normal(g, d)).to(torch.bfloat16)
        s["k_weight"] = (1 + 0.2 * _normal(g, d)).to(torch.bfloat16)
        turn = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
        angle = torch.arange(case["table"], dtype=torch.float64, device=DEV)[:, None] * turn
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.randint(0, case["table"], (t,), generator=g, device=DEV)
        s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(t, hk, d, dtype=torch.bfloat16, device=DEV)
        if case["op"] == "norm_rope_grad":
            s["q_grad"] = _normal(g, t, hq, d).to(torch.bfloat16)
            s["k_grad"] = _normal(g, t, hk, d).to(torch.bfloat16)
            s["dq_weight"] = torch.empty(d, dtype=torch.float32, device=DEV)
            s["dk_weight"] = torch.empty(d, dtype=torch.float32, device=DEV)
    elif case["op"] == "cache":
        t, page = case["tokens"], case["page"]
        pages = 2 * -(-t // page) + 1
        s["k"], s["v"] = _keys(g, t, hk, d), _keys(g, t, hk, d)
        if case["order"] == "scattered":  # each token to a page of its own sequence
            slots = torch.randperm(pages * page, generator=g, device=DEV)[:t]
        else:  # a sequence over whole pages in any order, begun inside one
            at = torch.arange(t, device=DEV) + seed % page
            slots = torch.randperm(pages, generator=g, device=DEV)[at // page] * page + at % page
        s["slots"] = slots
        s["cache"] = torch.zeros(pages, hk, page // 32, 34 * d, dtype=torch.uint8, device=DEV)
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    else:
        page, hq = case["page"], case["heads"]
        qs, kvs = _lengths(case)
        per = max(1, -(-max(kvs) // page))
        used = [-(-n // page) for n in kvs]
        pages = sum(used) + 2
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(len(kvs), per, dtype=torch.int32, device=DEV)
        at = torch.arange(per, device=DEV) < torch.tensor(used, device=DEV)[:, None]
        table[at] = order[:sum(used)]
        s["page_table"] = table
        s["cache"] = _make_cache(_keys(g, pages * page, hk, d), _keys(g, pages * page, hk, d), d, page)
        s["q"] = (2 * _normal(g, sum(qs), hq, d)).to(torch.bfloat16)
        start = [0]
        for m in qs:
            start.append(start[-1] + m)
        s["q_start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        s["kv_len"] = torch.tensor(kvs, dtype=torch.int32, device=DEV)
        s["q_max"], s["kv_max"] = max(qs), max(kvs)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(sum(qs), hq, dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------------- plain forms

def _pairs(x, r, interleaved):
    if interleaved:
        return x[..., 0:r:2], x[..., 1:r:2]
    return x[..., :r // 2], x[..., r // 2:r]


def _join(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _norm_rope(x, w, cs, r, interleaved):
    x = x.float()
    z = x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * w.float()
    a, b = _pairs(z, r, interleaved)
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    return _join(a * c - b * s, b * c + a * s, z[..., r:], interleaved).to(torch.bfloat16)


def _norm_rope_grad(gy, x, w, cs, r, interleaved):
    gy, x, w = gy.float(), x.float(), w.float()
    a, b = _pairs(gy, r, interleaved)
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    g = _join(a * c + b * s, b * c - a * s, gy[..., r:], interleaved)
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * inv
    dw = (g * n).sum((0, 1), dtype=torch.float64).float()
    h = g * w
    return (inv * (h - n * (h * n).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _quantise(x):
    """x (tokens, heads, D) as codes and scale bytes."""
    t, h, d = x.shape
    y = x.float().reshape(t, h, d // 32, 32)
    most = y.abs().amax(-1)
    _, e = torch.frexp(most)  # most = m 2**e, 0.5 <= m < 1
    byte = (e + 126 + (torch.ldexp(most, 3 - e) >= 7).int() - 2).clamp(2, 252)
    byte = torch.where(torch.isfinite(y).all(-1), torch.where(most > 0, byte, 2), 255)
    mag = torch.ldexp(y.abs(), (127 - byte).unsqueeze(-1)).clamp(max=6.0)
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    mag = torch.round(mag / step) * step  # round() takes a half to the even multiple
    code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, torch.where(mag < 6, 6.0, 7.0)))
    code = torch.nan_to_num(code).to(torch.uint8) + 8 * torch.signbit(y).to(torch.uint8)
    return code.reshape(t, h, d), byte.to(torch.uint8)


def _values(code, byte):
    """What codes (..., D) and scale bytes (..., D/32) stand for."""
    mag = (code & 7).float()
    mag = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    mag = torch.where(code >= 8, -mag, mag)
    scale = torch.ldexp(torch.ones((), device=byte.device), byte.int() - 127)
    scale = torch.where(byte == 255, math.nan, scale)
    return (mag.reshape(*byte.shape, 32) * scale.unsqueeze(-1)).reshape(code.shape)


def _unpack(tiles, d):
    """The codes and scales of keys and values in tiles (..., 34 D), each (..., 32, D or D/32)."""
    lead, n, G = tiles.shape[:-1], tiles.dim() - 1, d // 32

    def part(lo, hi, shape, order, last):
        x = tiles[..., lo:hi].reshape(*lead, *shape)
        return x.permute(*range(n), *[n + i for i in order]).reshape(*lead, 32, last)

    def codes(x):
        return torch.stack([x & 15, x >> 4], -1).flatten(-2)

    return (codes(part(0, 16 * d, (32, d // 2), (0, 1), d // 2)), part(32 * d, 33 * d, (G, 4, 4, 2), (1, 3, 2, 0), G),
            codes(part(16 * d, 32 * d, (4, 16, 8, d // 32), (0, 2, 1, 3), d // 2)), part(33 * d, 34 * d, (4, G, 8), (0, 2, 1), G))


def _cache(k, v, slots, dims):
    """Writes tokens into a cache of codes and scales by slot, and reads them back."""
    out = []
    for x in (k, v):
        code, byte = _quantise(x)
        codes = torch.zeros(dims, x.shape[1], x.shape[2], dtype=torch.uint8, device=x.device)
        scales = torch.zeros(dims, x.shape[1], x.shape[2] // 32, dtype=torch.uint8, device=x.device)
        codes[slots] = code
        scales[slots] = byte
        out.append(_values(codes[slots], scales[slots]).to(torch.bfloat16))
    return out


def _attend(s, case):
    d, hk, page, window = case["dim"], case["kv_heads"], case["page"], case["window"]
    group, b, q_max = case["heads"] // hk, case["batch"], s["q_max"]
    tiles = s["cache"][s["page_table"].long()].transpose(1, 2)  # batch, heads, pages, tiles, bytes
    kc, ks, vc, vs = _unpack(tiles, d)
    flat = lambda x: x.reshape(b, hk, -1, x.shape[-1])  # noqa: E731
    k, v = _values(flat(kc), flat(ks)), _values(flat(vc), flat(vs))
    n = k.shape[2]
    start, kv = s["q_start"].long(), s["kv_len"].long()
    qlen = start[1:] - start[:-1]
    i = torch.arange(q_max, device=k.device)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].reshape(b, q_max, hk, group, d).permute(0, 2, 1, 3, 4).reshape(b, hk, q_max * group, d)
    last = (kv - qlen)[:, None] + i
    j = torch.arange(n, device=k.device)
    seen = (j <= last[..., None]) & (j < kv[:, None, None])
    if window:
        seen &= j > last[..., None] - window
    v = torch.where(seen.any(1)[:, None, :, None], v, 0.0)
    p = torch.matmul(q, k.transpose(2, 3).contiguous()) * d ** -0.5
    p = torch.where(seen[:, None, :, None, :], p.reshape(b, hk, q_max, group, n), -math.inf)
    top = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    o = torch.matmul(p.reshape(b, hk, q_max * group, n), v).reshape(b, hk, q_max, group, d)
    o = torch.where(total == 0, 0.0, o / total)
    token = torch.arange(s["q"].shape[0], device=k.device)
    seq = torch.bucketize(token, start[1:], right=True)
    at = token - start[seq]
    o = o.permute(0, 2, 1, 3, 4)[seq, at].reshape(-1, hk * group, d)
    return o.to(torch.bfloat16), lse.permute(0, 2, 1, 3)[seq, at].reshape(-1, hk * group)


def _workspace(s, size):
    """Scratch memory that a program keeps beside its buffers: zeroed once."""
    if "workspace" not in s["kept"]:
        s["kept"]["workspace"] = torch.zeros(max(16, size()), dtype=torch.uint8, device=DEV)
    return s["kept"]["workspace"]


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from allreduce_reduction_way_amd import ar
        if op == "norm_rope":
            ar.ar_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"], s["q_out"],
                               s["k_out"], eps=EPS, interleaved=case["interleaved"])
            return s["q_out"], s["k_out"]
        if op == "norm_rope_grad":
            ws = _workspace(s, lambda: ar.ar_qk_norm_rope_bwd_workspace(case["tokens"], case["heads"], case["kv_heads"], case["dim"]))
            ar.ar_qk_norm_rope_bwd(s["q_grad"], s["k_grad"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                   s["positions"], s["q_out"], s["k_out"], s["dq_weight"], s["dk_weight"], ws, eps=EPS,
                                   interleaved=case["interleaved"])
            return s["q_out"], s["k_out"], s["dq_weight"], s["dk_weight"]
        if op == "cache":
            ar.ar_kv4_write(s["k"], s["v"], s["slots"], s["cache"], case["page"])
            ar.ar_kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"], case["page"])
            return s["k_out"], s["v_out"]
        ws = _workspace(s, lambda: ar.ar_kv4_attention_workspace(case["batch"], s["q"].shape[0], s["q_max"], s["kv_max"],
                                                                 case["heads"], case["kv_heads"], case["dim"]))
        ar.ar_kv4_attention(s["q"], s["cache"], s["page_table"], s["q_start"], s["kv_len"], s["out"], s["lse"], ws,
                            page_size=case["page"], kv_heads=case["kv_heads"], max_q=s["q_max"], max_kv=s["kv_max"],
                            window=case["window"])
        return s["out"], s["lse"]
    if op == "norm_rope":
        cs = s["cos_sin"][s["positions"]]
        return [_norm_rope(s[x], s[x + "_weight"], cs, case["rotated"], case["interleaved"]) for x in ("q", "k")]
    if op == "norm_rope_grad":
        cs = s["cos_sin"][s["positions"]]
        dq, dqw = _norm_rope_grad(s["q_grad"], s["q"], s["q_weight"], cs, case["rotated"], case["interleaved"])
        dk, dkw = _norm_rope_grad(s["k_grad"], s["k"], s["k_weight"], cs, case["rotated"], case["interleaved"])
        return dq, dk, dqw, dkw
    if op == "cache":
        return _cache(s["k"], s["v"], s["slots"], s["cache"].shape[0] * case["page"])
    return _attend(s, case)


# ------------------------------------------------------------------------- the definitions in 64 bits

def _exact_norm_rope(case, s, which):
    x, w = s[which].double(), s[which + "_weight"].double()
    r, half = case["rotated"], case["rotated"] // 2
    c = torch.arange(case["dim"], device=DEV)
    i = torch.arange(half, device=DEV)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    table = s["cos_sin"].double()[s["positions"]]
    cos = torch.ones(x.shape[0], 1, case["dim"], dtype=torch.float64, device=DEV)
    sin = torch.zeros_like(cos)
    cos[:, 0, first], cos[:, 0, second] = table[:, :half], table[:, :half]
    sin[:, 0, first], sin[:, 0, second] = -table[:, half:], table[:, half:]
    mate = c.clone()
    mate[first], mate[second] = second, first
    unit = x / (x.square().sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
    if case["op"] == "norm_rope":
        z = unit * w
        return z * cos + z[..., mate] * sin
    gy = s[which + "_grad"].double()
    g = gy * cos + (gy * sin)[..., mate]
    size = (x.square().sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
    along = (g * w * unit).sum(-1, keepdim=True) / case["dim"]
    return (g * w - unit * along) / size, (g * unit).flatten(0, 1).sum(0)


_LADDER = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_cache(x):
    """The nearest value that the group's scale allows; between two, the one of the even code."""
    y = x.double().reshape(*x.shape[:-1], -1, 32)
    most = y.abs().amax(-1, keepdim=True)
    scale = torch.full_like(most, 2.0 ** -125)
    for e in range(-124, 126):  # the least power of two that leaves the largest below 7
        scale = torch.where(most >= 7 * 2.0 ** (e - 1), 2.0 ** e, scale)
    best = torch.zeros_like(y)
    off = (y.abs() - best).abs()
    for n, v in enumerate(_LADDER[1:], 1):
        far = (y.abs() - v * scale).abs()
        take = far <= off if n % 2 == 0 else far < off
        best, off = torch.where(take, v * scale, best), torch.where(take, far, off)
    best = torch.where(torch.isfinite(y).all(-1, keepdim=True), torch.copysign(best, y), math.nan)
    return best.reshape(x.shape)


def _exact_attend(case, s):
    d, hk, page = case["dim"], case["kv_heads"], case["page"]
    group, W, G = case["heads"] // hk, d // 16, d // 32
    ladder = torch.tensor(_LADDER + tuple(-v for v in _LADDER), dtype=torch.float64, device=DEV)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    c = torch.arange(d, device=DEV)
    qs, kvs = _lengths(case)
    at = 0
    for b, (m, n) in enumerate(zip(qs, kvs)):
        j = torch.arange(n, device=DEV)
        tile = s["cache"][s["page_table"][b].long()[j // page], :, j % page // 32]  # n, heads, bytes
        t = (j % 32)[:, None]

        def values(code_at, scale_at):
            code = tile.gather(2, code_at[:, None, :].expand(-1, hk, -1)).int()
            code = torch.where(c % 2 == 1, code >> 4, code & 15)
            byte = tile.gather(2, scale_at[:, None, :].expand(-1, hk, -1)).double()
            return ladder[code] * 2.0 ** (byte - 127)

        if n:
            k = values(t * (d // 2) + c // 2, 32 * d + (c // 32 * 16 + t // 8 * 4 + t % 4) * 2 + t % 8 // 4)
            v = values(16 * d + ((t // 8 * 16 + c // W) * 8 + t % 8) * (W // 2) + c % W // 2, 33 * d + (t // 8 * G + c // 32) * 8 + t % 8)
            pos = n - m + torch.arange(m, device=DEV)
            seen = j <= pos[:, None]
            if case["window"]:
                seen &= j > pos[:, None] - case["window"]
            for h in range(case["heads"]):
                x = s["q"][at:at + m, h].double() @ k[:, h // group].T / math.sqrt(d)
                x = x.masked_fill(~seen, -math.inf)
                total = torch.logsumexp(x, 1)
                lse[at:at + m, h] = total
                out[at:at + m, h] = torch.exp(x - torch.where(torch.isinf(total), 0.0, total)[:, None]) @ v[:, h // group]
        at += m
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return [_exact_norm_rope(case, s, x) for x in ("q", "k")]
    if case["op"] == "norm_rope_grad":
        (dq, dqw), (dk, dkw) = _exact_norm_rope(case, s, "q"), _exact_norm_rope(case, s, "k")
        return dq, dk, dqw, dkw
    if case["op"] == "cache":
        return [_exact_cache(s[x]) for x in ("k", "v")]
    return _exact_attend(case, s)
