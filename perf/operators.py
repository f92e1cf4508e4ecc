"""Measured cases of the softmax-attention layer's serving operators: rotary positions, the append
to a paged 8-bit key / value cache, and the attention that reads this cache.

A hybrid stack interleaves the delta-rule layers with softmax-attention layers; these operators
are that layer's counterpart of the prologue, the state update and the decode step.

``own`` False: plain torch operations in 32 bits (64 for the angles); True: the package's calls.
"""

import math
import statistics

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 60       # exponents of the power-of-two scales that an append writes
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------- cases

def _rope(name, tokens, heads, kv_heads, head_dim, rot_dim, layout, scaling, inverse, max_pos, dtype):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                rot_dim=rot_dim, layout=layout, scaling=scaling, inverse=inverse, max_pos=max_pos, dtype=dtype)


def _append(name, seqs, new, ragged, max_len, kv_heads, head_dim, page, dtype):
    return dict(name=name, op="append", seqs=seqs, new=new, ragged=ragged, max_len=max_len,
                kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype)


def _attend(name, seqs, new, max_len, spread, heads, kv_heads, head_dim, page, dtype):
    return dict(name=name, op="attend", seqs=seqs, new=new, max_len=max_len, spread=spread, heads=heads,
                kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype)


def listed():
    return [
        # the new tokens of 256 decoding sequences, a quarter of the head rotated, far positions
        _rope("rope_decode_256", 256, 16, 2, 128, 32, "half", "yarn", False, 262144, "bf16"),
        # a prefill of 4 x 8192 tokens, the whole head rotated in adjacent pairs
        _rope("rope_prefill_4x8k", 32768, 32, 8, 128, 128, "interleaved", "none", False, 8192, "bf16"),
        # the gradient through the rotation for a packed batch of odd length, in fp32
        _rope("rope_gradient_packed", 76091, 8, 1, 64, 64, "half", "linear", True, 32768, "fp32"),
        # one new token for each of 256 decoding sequences
        _append("append_decode_256", 256, 1, False, 500, 2, 128, 64, "bf16"),
        # a prefill of 4 x 8192 tokens written to the cache
        _append("append_prefill_4x8k", 4, 8192, False, 8192, 8, 128, 64, "bf16"),
        # 32 packed prompts of ragged lengths behind earlier tokens, small pages
        _append("append_packed_32", 32, 2048, True, 3000, 4, 64, 16, "fp32"),
        # one sequence early in its decode: latency alone
        _attend("attend_one_short", 1, 1, 333, 0.0, 16, 2, 128, 64, "bf16"),
        # 256 decoding sequences with the lengths of a serving batch
        _attend("attend_decode_256", 256, 1, 16384, 1.0, 16, 2, 128, 64, "bf16"),
        # one sequence at the longest context
        _attend("attend_long_256k", 1, 1, 262144, 0.0, 32, 4, 128, 64, "bf16"),
        # verification of four speculative tokens, small pages, wide groups
        _attend("attend_verify_4", 64, 4, 12345, 0.7, 32, 4, 128, 16, "bf16"),
        # every query head with a cache head of its own, in fp32
        _attend("attend_heads_fp32", 16, 1, 4099, 0.5, 8, 8, 64, 32, "fp32"),
        # a chunk of a long prompt attending to what the cache holds
        _attend("attend_chunk_512", 4, 512, 8192, 0.3, 32, 4, 128, 64, "bf16"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    head_dim = rng.choice([64, 128, 128])
    if op == "rope":
        heads, kv_heads = rng.choice([(16, 2), (32, 8), (8, 1), (8, 8), (12, 4)])
        rot_dim = rng.choice([head_dim // 4, head_dim // 2, head_dim, head_dim - 6])
        most = 32768 * 40 * 128 * 2 // ((heads + kv_heads) * head_dim * SIZE[dtype])
        c = _rope("", _log(rng, 1, min(most, 100000)), heads, kv_heads, head_dim, rot_dim,
                  rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "ntk", "yarn"]),
                  rng.random() < 0.4, _log(rng, 1000, 1000000), dtype)
    elif op == "append":
        page = rng.choice([16, 32, 64, 128])
        kv_heads = rng.choice([1, 2, 4, 8])
        if rng.random() < 0.5:
            c = _append("", _log(rng, 1, 400), rng.choice([1, 1, 2, 3, 5, 16]), False, rng.randint(40, 900),
                        kv_heads, head_dim, page, dtype)
        else:
            new = _log(rng, 20, 4000)
            seqs = _log(rng, 1, max(2, 16000 // new))
            c = _append("", seqs, new, rng.random() < 0.7, new + rng.randint(0, 300), kv_heads, head_dim, page, dtype)
    else:
        heads, kv_heads = rng.choice([(16, 2), (32, 4), (8, 8), (8, 1), (24, 8), (20, 1)])
        page = rng.choice([16, 32, 64, 128])
        new = rng.choice([1, 1, 1, 2, 4, 7, 16, 100])
        max_len = _log(rng, 1, 100000)
        most = max(1, min(256, 1000000 // (max_len * kv_heads), 4000000 // (max_len * new)))
        c = _attend("", _log(rng, 1, most), new, max_len, rng.choice([0.0, 0.5, 1.0]), heads, kv_heads, head_dim,
                    page, dtype)
    del c["name"]
    return c


# ---------------------------------------------------------------- sizes that go by the case alone

def _spread_lengths(n, longest, sigma):
    """n lengths up to `longest`, log-normal quantiles (all `longest` for sigma 0)."""
    if sigma == 0.0 or n == 1:
        return [longest] * n
    nd = statistics.NormalDist()
    top = nd.inv_cdf((n - 0.5) / n)
    return [max(1, int(longest * math.exp(sigma * (nd.inv_cdf((i + 0.5) / n) - top)))) for i in range(n)]


def _lengths(c):
    """(tokens in the cache with the new ones, new tokens) of each sequence, before the shuffle."""
    n = c["seqs"]
    if c["op"] == "attend":
        return [(x, c["new"]) for x in _spread_lengths(n, c["max_len"], c["spread"])]
    if not c["ragged"]:
        total = [c["new"] + (7 * i + 3) % (c["max_len"] - c["new"] + 1) for i in range(n)] if c["max_len"] > c["new"] \
            else [c["new"]] * n
        return [(x, c["new"]) for x in total]
    new = _spread_lengths(n, c["new"], 0.8)
    return [(x + (11 * i) % (c["max_len"] - c["new"] + 1), x) for i, x in enumerate(new)]


def work(case):
    c, d = case, case["head_dim"]
    e = SIZE[c["dtype"]]
    if c["op"] == "rope":
        values = c["tokens"] * (c["heads"] + c["kv_heads"]) * d
        rotated = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rot_dim"]
        return {"bytes": 2 * values * e + 4 * c["tokens"] + 4 * c["rot_dim"], "flops": 3 * rotated}
    pairs = _lengths(c)
    hk = c["kv_heads"]
    if c["op"] == "append":
        new = sum(x for _, x in pairs)
        pages = sum((total - 1) // c["page"] - (total - x) // c["page"] + 1 for total, x in pairs)
        return {"bytes": 2 * new * hk * d * (e + 1) + pages * (2 * hk * 4 + 4) + 4 * c["seqs"],
                "flops": 4 * new * hk * d}
    cached = sum(x for x, _ in pairs)
    pages = sum(-(-x // c["page"]) for x, _ in pairs)
    rows = c["seqs"] * c["new"] * c["heads"]
    seen = sum(max(0, x - c["new"] + 1 + t) for x, _ in pairs for t in range(c["new"]))
    return {"bytes": 2 * cached * hk * d + pages * (2 * hk * 4 + 4) + 4 * c["seqs"] + 2 * rows * d * e + 4 * rows,
            "flops": 4 * seen * c["heads"] * d}


# ---------------------------------------------------------------- inputs

def _frequencies(c):
    """Radians per token of each pair in 64 bits, and the factor on cos and sin."""
    rot, base, context, factor = c["rot_dim"], 10000.0, 8192.0, 8.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    if c["scaling"] == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        f = f / factor
    if c["scaling"] != "yarn":
        return f, 1.0
    edge = lambda turns: rot * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), rot - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _codes(g, shape):
    """What earlier appends left: values of unit variance at the scale that a page takes."""
    x = torch.empty(shape, dtype=E4M3, device=DEV)
    flat, step = x.view(-1), 1 << 28
    for at in range(0, flat.numel(), step):
        n = min(step, flat.numel() - at)
        flat[at:at + n] = (torch.randn(n, generator=g, device=DEV) * 64).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    return x


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(DTYPES[c["dtype"]])  # noqa: E731
    d, hk = c["head_dim"], c["kv_heads"]
    if c["op"] == "rope":
        f, amplitude = _frequencies(c)
        return dict(c, q=rand(c["tokens"], c["heads"], d), k=rand(c["tokens"], hk, d), frequencies=f.to(DEV),
                    amplitude=amplitude, positions=torch.randint(0, c["max_pos"], (c["tokens"],), generator=g,
                                                                 device=DEV, dtype=torch.int32))
    pairs = _lengths(c)
    order = torch.randperm(len(pairs), generator=torch.Generator().manual_seed(seed)).tolist()
    lens = [pairs[i][0] for i in order]
    new = [pairs[i][1] for i in order]
    need = [-(-x // c["page"]) for x in lens]
    widest, pool = max(need), sum(need)
    # a sequence's pages lie anywhere in the pool; entries behind its last page name page 0
    slots = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    start = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
    column = torch.arange(widest, device=DEV)
    valid = column[None, :] < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(valid, slots[(start[:, None] + column[None, :]).clamp(max=pool - 1)], 0).to(torch.int32).contiguous()
    scale = lambda: torch.exp2(torch.randint(-8, -5, (pool, hk), generator=g, device=DEV).float())  # noqa: E731
    s = dict(c, k_cache=_codes(g, (pool, hk, c["page"], d)), v_cache=_codes(g, (pool, hk, c["page"], d)),
             k_scale=scale(), v_scale=scale(), table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if c["op"] == "append":
        total = sum(new)
        s["k"], s["v"] = rand(total, hk, d), rand(total, hk, d)
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV) \
            if c["ragged"] else None
    else:
        s["q"] = rand(c["seqs"], c["new"], c["heads"], d)
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, cos, sin, s):
    """x [T, H, d]: the first rot_dim channels rotated by the tokens' angles."""
    rot = s["rot_dim"]
    x = x.to(cos.dtype)
    cos, sin = cos[:, None, :], sin[:, None, :]
    if s["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["frequencies"][None, :]
    cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    if s["inverse"]:   # the transposed rotation: the gradient of the inputs from that of the outputs
        sin = -sin
    return tuple(_rotate(x, cos, sin, s).to(x.dtype) for x in (s["q"], s["k"]))


def _append_places(s):
    """For each new token its sequence and its position in the cache."""
    n = s["seqs"]
    if s["cu"] is None:
        count = torch.full((n,), s["new"], device=DEV, dtype=torch.int64)
        first = torch.arange(n, device=DEV) * s["new"]
    else:
        count, first = (s["cu"][1:] - s["cu"][:-1]).long(), s["cu"][:-1].long()
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), count, output_size=s["k"].shape[0])
    old = s["lens"].long() - count
    return seq, torch.arange(s["k"].shape[0], device=DEV) - first[seq] + old[seq], old


def _power_scale(amax):
    """The smallest power of two s with amax <= 448 s, its exponent held to [-60, 60]."""
    mantissa, exponent = torch.frexp(amax)
    e = exponent - 9 + (mantissa > 0.875).int()
    e = torch.where(amax > 0, e.clamp(MIN_EXP, MAX_EXP), MIN_EXP)
    return torch.exp2(e.float())


def _plain_append(s):
    seq, pos, old = _append_places(s)
    page = s["table"].long()[seq, pos // s["page"]]
    at = pos % s["page"]
    begin = pos - at                                         # the page's first position in its sequence
    kept = torch.zeros(s["k_cache"].shape[0], dtype=torch.int64, device=DEV)
    kept[page] = (old[seq] - begin).clamp(min=0)             # earlier tokens in the page
    touched = torch.zeros_like(kept, dtype=torch.bool)
    touched[page] = True
    token = torch.arange(s["page"], device=DEV)
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float()
        high = torch.zeros_like(scale)
        high.scatter_reduce_(0, page[:, None].expand(-1, high.shape[1]), x.abs().amax(-1), "amax")
        needed = _power_scale(high)
        now = torch.where((kept > 0)[:, None], torch.maximum(scale, needed), needed)
        now = torch.where(touched[:, None], now, scale)
        ratio = scale / now
        again = ((kept > 0)[:, None] & (now != scale)).nonzero()[:, 0].unique()   # pages whose scale has grown
        grown = cache[again].float()
        old_codes = (token[None, :] < kept[again][:, None])[:, None, :, None] & \
            (now != scale)[again][:, :, None, None]
        cache[again] = torch.where(old_codes, grown * ratio[again][:, :, None, None], grown).to(E4M3)
        cache[page, :, at] = (x / now[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        scale.copy_(now)
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _read_cache(cache, scale, table, dtype):
    """[N, Hkv, L, d]: the values that the codes of the table's pages stand for."""
    x = cache[table].to(dtype) * scale[table].to(dtype)[..., None, None]      # [N, pages, Hkv, P, d]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _softmax_over_cache(q, k, v, lens, dtype):
    """q [N, T, Hq, d], k and v [N, Hkv, L, d]: (o [N, T, Hq, d], lse [N, T, Hq])."""
    n, t, hq, d = q.shape
    hk = k.shape[1]
    rows = q.to(dtype).view(n, t, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)
    score = rows @ k.transpose(-1, -2) / math.sqrt(d)
    last = lens.long()[:, None] - t + torch.arange(t, device=q.device)[None, :]          # [N, T]
    last = last.repeat_interleave(hq // hk, dim=1)                                       # [N, T G]
    hidden = torch.arange(k.shape[2], device=q.device)[None, None, :] > last[:, :, None]
    score = score.masked_fill(hidden[:, None], -math.inf)
    high = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(high == -math.inf, 0, high))
    total = weight.sum(-1, keepdim=True)
    o = (weight @ v) / torch.where(total == 0, 1, total)
    lse = (high + total.log()).squeeze(-1)
    back = lambda x: x.view(n, hk, t, hq // hk, -1).permute(0, 2, 1, 3, 4).reshape(n, t, hq, -1)  # noqa: E731
    return back(o), back(lse).squeeze(-1)


def _plain_attend(s):
    table = s["table"].long()
    k = _read_cache(s["k_cache"], s["k_scale"], table, torch.float32)
    v = _read_cache(s["v_cache"], s["v_scale"], table, torch.float32)
    o, lse = _softmax_over_cache(s["q"], k, v, s["lens"], torch.float32)
    return o.to(s["q"].dtype), lse


def run(state):
    s = state
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    import gated_delta_rule_70_b200 as kda
    if s["op"] == "rope":
        return kda.rope(s["q"], s["k"], s["positions"], s["frequencies"], amplitude=s["amplitude"],
                        layout=s["layout"], inverse=s["inverse"])
    if s["op"] == "append":
        kda.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                         s["lens"], cu_seqlens=s["cu"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    return kda.cache_attend(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                            want_lse=True)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rope(s):
    # a pair (a, b) is the complex number a + i b, and the rotation its product with r e^{+-i angle}
    angle = s["positions"].double()[:, None] * s["frequencies"]
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), -angle if s["inverse"] else angle)[:, None]
    half, out = s["rot_dim"] // 2, []
    for x in (s["q"].double(), s["k"].double()):
        pairs = x[..., :2 * half].unflatten(-1, (2, half)).movedim(-2, -1) if s["layout"] == "half" \
            else x[..., :2 * half].unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y = x.clone()
        y[..., :2 * half] = z.movedim(-1, -2).flatten(-2) if s["layout"] == "half" else z.flatten(-2)
        out.append(y)
    return tuple(out)


def _exact_attend(s):
    n, t, hq, d = s["q"].shape
    hk = s["kv_heads"]
    o = torch.zeros(n, t, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((n, t, hq), -math.inf, dtype=torch.float64, device=DEV)
    for i, length in enumerate(s["lens"].tolist()):
        pages = s["table"][i, :-(-length // s["page"])].long()
        k = (s["k_cache"][pages].double() * s["k_scale"][pages].double()[:, :, None, None]).transpose(0, 1)
        v = (s["v_cache"][pages].double() * s["v_scale"][pages].double()[:, :, None, None]).transpose(0, 1)
        k, v = k.reshape(hk, -1, d)[:, :length], v.reshape(hk, -1, d)[:, :length]
        q = s["q"][i].double().view(t, hk, hq // hk, d)
        score = torch.einsum("tgjd,gld->tgjl", q, k) * d ** -0.5
        ahead = torch.arange(length, device=DEV)[None, :] - torch.arange(t, device=DEV)[:, None] > length - t
        score = score.masked_fill(ahead[:, None, None, :], -math.inf)
        lse[i] = torch.logsumexp(score, -1).view(t, hq)
        weight = torch.nan_to_num(torch.exp(score - lse[i].view(t, hk, hq // hk, 1)), nan=0.0)
        o[i] = torch.einsum("tgjl,gld->tgjd", weight, v).reshape(t, hq, d)
    return o, lse


def _exact_append(s):
    # page by page: the codes are the values over the page's scale, before their rounding to 8 bits
    out = []
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        code, sc = cache.double(), scale.double()
        first = 0
        for i, length in enumerate(s["lens"].tolist()):
            count = s["new"] if s["cu"] is None else int(s["cu"][i + 1] - s["cu"][i])
            rows = x[first:first + count].double().transpose(0, 1)                   # [Hkv, new, d]
            first += count
            old, pages = length - count, s["table"][i].tolist()
            for p in range(old // s["page"], -(-length // s["page"])):
                begin, end = max(old, p * s["page"]), min(length, (p + 1) * s["page"])
                part, kept, at = rows[:, begin - old:end - old], begin - p * s["page"], pages[p]
                high = part.abs().amax((1, 2))
                now = torch.exp2(torch.ceil(torch.log2(high / E4M3_MAX)).clamp(MIN_EXP, MAX_EXP))
                if kept:
                    now = torch.maximum(now, sc[at])
                    code[at, :, :kept] *= (sc[at] / now)[:, None, None]
                code[at, :, kept:kept + end - begin] = (part / now[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX)
                sc[at] = now
        out.append((code, sc))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[s["op"]](s)
