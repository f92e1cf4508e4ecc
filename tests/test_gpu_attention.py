"""Rotary positions, the 8-bit cache append and the cache attention on the GPU, against the plain
64-bit implementations of tests/attention_ref.py.

Tolerances (derived from the number formats, u = eps / 2 of a type: bf16 2^-8, fp16 2^-11, fp32 2^-24)

rope     The angle is formed modulo a turn with an error below 2^-33 turns, the signed fraction is
         rounded to fp32 (|x| <= 1 half-turn: 2^-25 pi < 2^-23.3 radians), sincospi is within 2^-23,
         three products / sums and the amplitude round by u each: (|a| + |b|) amplitude 2^-21 covers
         their sum, and the output's rounding adds u |y|.  Positions here stay below 2^20, which
         leaves the frequency's own 2^-53 far below.
append   Codes and scales are equal: a power-of-two scale makes x / s exact, and the rounding is one.
attend   A score sums d products in fp32: error <= 2 (d + 4) 2^-24 S, S = scale sum |q_i k_i| (twice: a
         tensor-core sum may truncate); the exponential, the sums over the row and the joins of split
         parts stay below 2^-18; a weight rounds to fp16 (bf16 calls: 2^-11) or to two fp16 parts (fp32
         calls: 2^-22).  All of these are relative errors of weights, so the output moves by at most
         twice their sum (numerator and denominator) times sum w |v| / sum w; then u |o|.  Weights below
         fp16's normal range (2^-14 of the largest) lose 2^-25 of the largest each, which for the up to
         600 tokens and the scales used here is below 2^-15 sum w max|v| -- the term 2^-14 * max |v|.
"""

import math

import numpy as np
import pytest
import torch

import gated_delta_rule_70_b200 as pkg
from gated_delta_rule_70_b200 import attention as A
from gated_delta_rule_70_b200 import kda
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
WEIGHT = {"bf16": 2.0 ** -11, "fp32": 2.0 ** -22}


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(2025)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


# ---------------------------------------------------------------- rope

def rope_check(x, y, pos, freq, amp, layout, inverse, dtype):
    want, size = ref.rope(f64(x).reshape(-1, *x.shape[-2:]), pos.cpu().numpy(), freq.cpu().numpy(), amp, layout, inverse)
    got = f64(y).reshape(want.shape)
    bound = abs(amp) * size * 2.0 ** -21 + U[dtype] * np.abs(want) * (size > 0) + 1e-38
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) - bound)
    rot = 2 * len(freq)
    assert np.array_equal(got[..., rot:], f64(x).reshape(want.shape)[..., rot:])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens, hq, hk, d, rot", [
    (1, 1, 0, 8, 2), (3, 2, 1, 64, 64), (9, 16, 2, 128, 32), (17, 3, 3, 128, 128), (33, 5, 2, 64, 58),
    (64, 4, 1, 256, 256), (7, 2, 2, 40, 24), (300, 8, 8, 64, 16), (5, 130, 7, 16, 6),
])
def test_rope(dtype, layout, tokens, hq, hk, d, rot):
    g = torch.Generator().manual_seed(tokens * 1000 + rot)
    q = torch.randn((tokens, hq, d), generator=g).to(DT[dtype]).cuda()
    k = torch.randn((tokens, hk, d), generator=g).to(DT[dtype]).cuda() if hk else None
    pos = torch.randint(-5, 1 << 20, (tokens,), generator=g, dtype=torch.int32)
    pos[0] = 0
    pos = pos.cuda()
    freq, amp = pkg.rope_frequencies(rot, 10000.0, device="cuda")
    for inverse, amp in ((False, amp), (True, 1.25)):
        yq, yk = pkg.rope(q, k, pos, freq, amplitude=amp, layout=layout, inverse=inverse)
        rope_check(q, yq, pos, freq, amp, layout, inverse, dtype)
        if hk:
            rope_check(k, yk, pos, freq, amp, layout, inverse, dtype)


@pytest.mark.parametrize("layout, rot", [("half", 32), ("half", 58), ("interleaved", 58), ("interleaved", 64)])
def test_rope_in_place_strided_and_neighbours(layout, rot):
    """q and k as parts of one projection: rotated in place, the v part and the gaps untouched."""
    fused = torch.randn((2, 7, 8, 64), device="cuda").bfloat16()
    before = fused.clone()
    q, k = fused[:, :, :4], fused[:, :, 4:6]
    pos = torch.arange(14, dtype=torch.int32, device="cuda") * 1001
    freq, _ = pkg.rope_frequencies(rot, device="cuda")
    want = pkg.rope(q, k, pos, freq, layout=layout)
    out = pkg.rope(q, k, pos, freq, layout=layout, out=(q, k))
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(fused[:, :, 6:], before[:, :, 6:])
    rope_check(before[:, :, :4], want[0], pos, freq, 1.0, layout, False, "bf16")


def test_rope_nan_and_inf_stay_in_their_pair():
    x = torch.ones((2, 1, 64), device="cuda")
    x[0, 0, 3], x[1, 0, 60] = math.nan, math.inf
    pos = torch.tensor([5, 7], dtype=torch.int32, device="cuda")
    for layout, rot, near in (("half", 32, {3, 19}), ("interleaved", 30, {2, 3}), ("interleaved", 58, {2, 3})):
        freq, _ = pkg.rope_frequencies(rot, device="cuda")
        y, _ = pkg.rope(x, None, pos, freq, layout=layout)
        bad = (~torch.isfinite(y)).nonzero().tolist()
        assert {c for t, _, c in bad if t == 0} == near and [c for t, _, c in bad if t == 1] == [60]


def test_rope_far_positions():
    """Positions at the end of int32: the angle keeps 2^31 * 2^-53 turns, 2^-19.3 radians."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 262143], dtype=torch.int32, device="cuda")
    x = torch.randn((4, 1, 64), device="cuda")
    freq, _ = pkg.rope_frequencies(64, device="cuda")
    y, _ = pkg.rope(x, None, pos, freq)
    # the angle itself in extended precision: position * frequency exactly as a fraction
    from fractions import Fraction
    pi2 = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")
    h = 32
    for t in range(4):
        for i in range(h):
            a = float((Fraction(int(pos[t])) * Fraction(float(freq[i]))) % pi2)
            c, s = math.cos(a), math.sin(a)
            u, v = float(x[t, 0, i]), float(x[t, 0, i + h])
            tol = (abs(u) + abs(v)) * (2.0 ** -21 + 2.0 ** -19)
            assert abs(float(y[t, 0, i]) - (u * c - v * s)) <= tol
            assert abs(float(y[t, 0, i + h]) - (v * c + u * s)) <= tol


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_inverse_is_the_gradient(layout):
    """<g, R x> differences: the inverse call on g is the gradient of <g, rope(x)>, which is linear in x."""
    x = torch.randn((6, 3, 64), device="cuda")
    g = torch.randn((6, 3, 64), device="cuda")
    pos = torch.randint(0, 300000, (6,), dtype=torch.int32, device="cuda")
    freq, amp = pkg.rope_frequencies(48, scaling="yarn", factor=4.0, original_context=4096, device="cuda")
    kw = dict(amplitude=amp, layout=layout)
    gx, _ = pkg.rope(g, None, pos, freq, inverse=True, **kw)
    for at in ((0, 0, 0), (2, 1, 23), (3, 2, 24), (5, 0, 47), (1, 1, 63)):
        e = torch.zeros_like(x)
        e[at] = 1.0
        hi, _ = pkg.rope(x + e, None, pos, freq, **kw)
        lo, _ = pkg.rope(x - e, None, pos, freq, **kw)
        diff = float(((hi.double() - lo.double()) / 2 * g.double()).sum())
        # two channels of each call enter, of size <= 2 amp max|x| and rounded to 2^-21 of it, times |g| < 5
        assert abs(diff - float(gx[at])) <= 2 * 2 * amp * 6 * 2.0 ** -21 * 5


# ---------------------------------------------------------------- caches

def make_cache(lens, hk, d, p, seed, spare=3, columns=None, scales=(-8, -5)):
    """A pool with `spare` unused pages, its pages handed out in random order; codes random and
    NaN-free, scales powers of two."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(int(x), 0) // p) for x in lens]
    pool = sum(need) + spare
    columns = max(max(need), 1) if columns is None else columns
    order = torch.randperm(pool, generator=g).tolist()
    table = torch.full((len(lens), columns), -7, dtype=torch.int32)   # behind the last page: never read
    for n, c in enumerate(need):
        for j in range(min(c, columns)):
            table[n, j] = order.pop()
    def pages():
        x = (torch.randn((pool, hk, p, d), generator=g) * 64).clamp(-448, 448)
        return x.to(torch.float8_e4m3fn).cuda()
    def scale():
        return torch.exp2(torch.randint(scales[0], scales[1] + 1, (pool, hk), generator=g).float()).cuda()
    return [pages(), pages(), scale(), scale(), table.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda()]


def host(c):
    return [codes(c[0]), codes(c[1]), c[2].cpu().numpy(), c[3].cpu().numpy(), c[4].cpu().numpy(), c[5].cpu().numpy()]


def append_check(k, v, c, counts, **kw):
    h = host(c)
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    pkg.cache_append(k, v, *c, status=status, **kw)
    for x, cache, scale, i in ((k, c[0], c[2], 0), (v, c[1], c[3], 1)):
        rows = f64(x).reshape(-1, *x.shape[-2:])
        want, s = ref.append(rows, h[i], h[2 + i], h[4], h[5], counts)
        assert np.array_equal(f64(scale), s)
        assert np.array_equal(codes(cache), want)
    return int(status)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("p, d, hk, new, lens", [
    (16, 64, 1, 1, [1]), (16, 64, 2, 1, [16, 17, 33, 1, 0, 5]), (64, 128, 2, 1, [64, 65, 1, 500]),
    (32, 128, 3, 5, [5, 7, 36, 64, 3, 0]), (128, 64, 2, 16, [16, 140, 128, 9]),
    (16, 128, 1, 100, [100, 215, 50]), (64, 128, 1, 333, [333, 400]), (128, 128, 2, 130, [131, 257]),
])
def test_append_dense(dtype, p, d, hk, new, lens):
    c = make_cache(lens, hk, d, p, seed=p + new)
    g = torch.Generator().manual_seed(new)
    shape = (len(lens), new, hk, d)
    size = torch.exp2(torch.randint(-3, 4, shape[:3], generator=g).float())[..., None]   # pages grow their scale
    k, v = ((torch.randn(shape, generator=g) * size).to(DT[dtype]).cuda() for _ in range(2))
    assert append_check(k, v, c, [new] * len(lens)) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [2, 3, 8, 9, 16, 17, 32, 33, 64, 65, 128])
def test_append_each_size_of_a_page_share(dtype, d, new):
    """From two new tokens of a page to all of it: every number of warps and of values a thread holds."""
    lens = [new, new + 1, 128, 128 + new // 2, 300]
    c = make_cache(lens, 1, d, 128, seed=new)
    g = torch.Generator().manual_seed(d + new)
    k, v = (torch.randn((5, new, 1, d), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    assert append_check(k, v, c, [new] * 5) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("p, d, counts, old", [
    (16, 64, [3, 0, 40, 1, 17], [0, 5, 13, 15, 16]), (64, 128, [1, 1, 1], [63, 64, 0]),
    (32, 64, [0, 0, 5, 0], [1, 2, 3, 4]), (16, 128, [200], [7]), (128, 64, [1] * 40, list(range(100, 140))),
])
def test_append_packed(dtype, p, d, counts, old):
    lens = [a + b for a, b in zip(counts, old)]
    c = make_cache(lens, 2, d, p, seed=len(counts))
    total = sum(counts)
    fused = torch.randn((total, 7, d), device="cuda").to(DT[dtype])      # k and v as parts of one projection
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    assert append_check(fused[:, 3:5], fused[:, 5:], c, counts, cu_seqlens=cu) == 0


def test_append_special_values():
    """Zeros, subnormals, the largest values, infinities and NaN; scales that somebody else wrote."""
    d, p = 64, 16
    rows = torch.zeros((10, 1, 1, d))
    rows[1, 0, 0, 5] = 1e-40                      # below every scale: codes 0
    rows[2] = 3e38                                # beyond 448 * 2^60
    rows[3, 0, 0, 0] = math.inf
    rows[4, 0, 0, 0], rows[4, 0, 0, 1] = math.nan, 3.0
    rows[5] = math.nan
    rows[6, 0, 0, :4] = torch.tensor([448.0, -448.0, 1.0, -0.0])
    rows[7, 0, 0, :2] = torch.tensor([448.0 * (1 + 2.0 ** -7), 1.0])
    rows[8, 0, 0, :3] = torch.tensor([0.5, -17.3, 2.0 ** -9])
    rows[9, 0, 0, 0] = 1000.0
    for dtype in ("bf16", "fp32"):
        lens = [1, 1, 1, 1, 1, 1, 1, 1, 5, 9]
        c = make_cache(lens, 1, d, p, seed=3)
        c[2][:] = 0.013                           # not a power of two
        c[3][:] = 2.0 ** -20
        x = rows.to(DT[dtype]).cuda()
        assert append_check(x, x.clone(), c, [1] * 10) == 0


def test_append_bad_pages_and_lengths():
    """Reported, left out, and nothing else written."""
    for bad, bit in ((-1, A.KDA_STATUS_BAD_PAGE), (10 ** 6, A.KDA_STATUS_BAD_PAGE), (None, A.KDA_STATUS_BAD_LENGTH)):
        lens = [40, 40, 40]
        c = make_cache(lens, 2, 64, 16, seed=11)
        k = torch.randn((3, 30, 2, 64), device="cuda").bfloat16()
        if bad is None:
            c[5][:] = torch.tensor([60, 40, -3], dtype=torch.int32, device="cuda")   # 48 places a sequence
        else:
            c[4][1, 1] = bad
        assert append_check(k, k.clone(), c, [30, 30, 30]) == bit
        with pytest.raises(kda.KdaError) as e:
            pkg.cache_append(k, k, *c, check=True)
        assert e.value.status == kda.KDA_ERR_INVALID_ARGUMENT


def test_append_bad_cu_seqlens():
    for cu in ([1, 5, 9], [0, 12, 9], [0, 5, 8], [-4, 5, 9], [0, 50, 9], [0, -3, 9]):
        c = make_cache([40, 40], 1, 64, 16, seed=1)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        x = torch.randn((9, 1, 64), device="cuda")
        pkg.cache_append(x, x, *c, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), status=word)
        assert int(word) & kda.KDA_STATUS_BAD_CU_SEQLENS


# ---------------------------------------------------------------- attention

def attend_check(q, c, dtype, scale=None, values=None, **kw):
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    o, lse = pkg.cache_attend(q, *c, scale=scale, want_lse=True, status=status, **kw)
    h = host(c)
    h[3] = np.clip(h[3], 2.0 ** -60, 2.0 ** 60)
    want, wl, mean_v, size = ref.attend(f64(q), *h[:4], h[4], h[5], scale)
    d = q.shape[-1]
    rel = 2 * (d + 4) * 2.0 ** -24 * size + 2.0 ** -18
    top = np.abs(want).max() if values is None else values
    bound = (2 * (rel + WEIGHT[dtype]))[..., None] * mean_v + U[dtype] * np.abs(want) + 1e-37
    if dtype == "bf16":
        bound = bound + 2.0 ** -14 * np.where(mean_v > 0, top, 0.0)
    got, gl = f64(o), f64(lse)
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), empty) and np.all(got[empty] == 0)
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)
    gl, wl = np.where(empty, 0, gl), np.where(empty, 0, wl)
    assert np.all(np.abs(gl - wl) <= rel + 2.0 ** -22 * np.abs(wl))
    return int(status)


SHAPES = [
    # p, d, heads, kv heads, new tokens, lengths
    (16, 64, 1, 1, 1, [1]),
    (64, 128, 8, 1, 1, [1, 2, 7, 8, 9, 15, 16, 17]),
    (64, 128, 16, 2, 1, [63, 64, 65, 127, 128, 129, 0, 600]),
    (16, 128, 16, 2, 2, [1, 2, 3, 31, 33, 0, 300]),
    (32, 64, 12, 4, 3, [5, 2, 64, 511]),
    (128, 128, 8, 8, 1, [130, 1, 512, 513]),
    (128, 64, 4, 4, 5, [5, 3, 127, 129]),
    (64, 128, 20, 1, 1, [77, 200]),
    (32, 128, 32, 4, 4, [100, 4, 33, 550]),
    (64, 64, 24, 2, 7, [7, 64, 200]),
    (16, 128, 6, 2, 37, [40, 36, 90]),
    (64, 128, 8, 1, 16, [16, 100, 8]),
    (64, 128, 5, 5, 70, [70, 130]),
    (32, 64, 40, 1, 20, [20, 66]),
    (64, 128, 16, 1, 2, [128, 64, 63, 0, 1, 500]),
    (16, 64, 17, 1, 9, [300, 9, 4, 129]),
    (128, 128, 6, 3, 200, [200, 450]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("p, d, hq, hk, new, lens", SHAPES)
def test_attend(dtype, p, d, hq, hk, new, lens):
    c = make_cache(lens, hk, d, p, seed=p + hq + new)
    q = torch.randn((len(lens), new, hq, d), generator=torch.Generator().manual_seed(hq)).to(DT[dtype]).cuda()
    assert attend_check(q, c, dtype) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_strided_queries_and_scale(dtype):
    lens = [70, 3, 129]
    c = make_cache(lens, 2, 128, 64, seed=5)
    fused = torch.randn((3, 2, 10, 128), device="cuda").to(DT[dtype])
    assert attend_check(fused[:, :, 2:8], c, dtype, scale=0.31) == 0
    assert attend_check(fused[:, :, :4], c, dtype, scale=-0.05) == 0
    assert attend_check(fused[:, :, 4:6], c, dtype, scale=0.0) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_sharp_rows(dtype):
    """Scores of several hundred: one token takes the whole row, wherever it lies."""
    lens = [300, 299, 65]
    c = make_cache(lens, 1, 128, 16, seed=9)
    kv = ref.e4m3_decode(codes(c[0])) * c[2].cpu().numpy()[..., None, None]
    q = torch.zeros((3, 1, 4, 128))
    for n, places in enumerate(([0, 299, 150, 63], [0, 298, 17, 64], [0, 64, 63, 1])):
        for h, j in enumerate(places):
            q[n, 0, h] = torch.from_numpy(kv[int(c[4][n, j // 16]), 0, j % 16]) * 20
    assert attend_check(q.to(DT[dtype]).cuda(), c, dtype) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_wide_scales_and_queries(dtype):
    """Page scales over a wide range, keys and values alike; queries of every size."""
    lens = [200, 130]
    c = make_cache(lens, 2, 64, 32, seed=21, scales=(-24, 8))
    c[2] *= 2.0 ** -6
    q = (torch.randn((2, 3, 4, 64)) * torch.tensor([1e-30, 1e-3, 1.0, 8.0])[None, None, :, None])
    values = float((ref.e4m3_decode(codes(c[1])) * c[3].cpu().numpy()[..., None, None]).__abs__().max())
    assert attend_check(q.to(DT[dtype]).cuda(), c, dtype, values=values) == 0


def test_attend_scales_out_of_range():
    """Zero, tiny and huge value scales: taken as 2^-60 and 2^60; key scales of any size, zero too."""
    c = make_cache([64, 64, 64, 64], 1, 64, 16, seed=2)
    c[3][c[4][0].long()] = 0.0
    c[3][c[4][1].long()] = 1e-30
    c[3][c[4][2].long()] = 1e30
    c[2][c[4][3].long()] = 0.0
    q = torch.randn((4, 1, 2, 64), device="cuda")
    assert attend_check(q, c, "fp32") == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("p", [16, 64, 128])
@pytest.mark.parametrize("group", [2, 4, 9])
def test_attend_ignores_nan_where_masked(dtype, p, group):
    """NaN codes behind the last token, in other pages and in tokens that later rows alone see, and NaN
    scales of pages that nobody reads."""
    new, lens, hq = 4, [70, 5, 130, 3], 2 * group
    c = make_cache(lens, 2, 128, p, seed=31)
    q = torch.randn((4, new, hq, 128), device="cuda").to(DT[dtype])
    clean = pkg.cache_attend(q, *c, want_lse=True)
    nan = torch.full((), 0x7f, dtype=torch.uint8, device="cuda")
    for cache in (c[0].view(torch.uint8), c[1].view(torch.uint8)):
        used = torch.zeros(cache.shape[0], dtype=torch.bool, device="cuda")
        for n, length in enumerate(lens):
            pages = c[4][n, :-(-length // p)].long()
            used[pages] = True
            if length % p:
                cache[pages[-1], :, length % p:] = nan
        cache[~used] = nan
        c[2][~used] = math.nan
        c[3][~used] = math.nan
    o, lse = pkg.cache_attend(q, *c, want_lse=True)
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])
    # the last token of sequences 0 and 2 becomes NaN in one value channel: the last row alone sees it
    for n, length in ((0, 70), (2, 130)):
        page, at = int(c[4][n, (length - 1) // p]), (length - 1) % p
        c[1].view(torch.uint8)[page, 1, at, 77] = nan
    o, lse = pkg.cache_attend(q, *c, want_lse=True)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, -1, group:, 77] = hit[2, -1, group:, 77] = True
    assert torch.equal(torch.isnan(o), hit) and torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse, clean[1])
    # a key of the second-to-last token: the last two rows of its head see it, whole
    page, at = int(c[4][0, 68 // p]), 68 % p
    c[0].view(torch.uint8)[page, 0, at, 3] = nan
    o, _ = pkg.cache_attend(q, *c, want_lse=True)
    assert torch.isnan(o[0, 2:, :group]).all() and not torch.isnan(o[0, :2]).any() and not torch.isnan(o[1]).any()


def test_attend_bad_pages_and_lengths():
    lens = [100, 40, 64]
    c = make_cache(lens, 2, 64, 16, seed=8)
    q = torch.randn((3, 2, 4, 64), device="cuda")
    c[4][0, 2], c[4][1, :], c[4][2, 0] = -1, 10 ** 6, -2 ** 31
    assert attend_check(q, c, "fp32") == A.KDA_STATUS_BAD_PAGE
    with pytest.raises(kda.KdaError) as e:
        pkg.cache_attend(q, *c, check=True)
    assert e.value.status == kda.KDA_ERR_INVALID_ARGUMENT
    c = make_cache([100, 40, 64], 2, 64, 16, seed=8)
    c[4][1:, 3:] = 0
    c[4][1:, :] = c[4][0, 0]                      # all of the row is read where the length is too large
    c[5][:] = torch.tensor([100, 10 ** 9, -5], dtype=torch.int32, device="cuda")
    assert attend_check(q, c, "fp32") == A.KDA_STATUS_BAD_LENGTH


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_many_sequences(dtype):
    """More sequences than blocks, empty ones among them; pages shared by sequences (a common prefix)."""
    g = torch.Generator().manual_seed(4)
    lens = [int(x) for x in torch.randint(0, 40, (700,), generator=g)]
    c = make_cache(lens, 1, 64, 16, seed=12)
    c[4][:, 0] = c[4][0, 0].clamp(min=0)
    q = torch.randn((700, 1, 2, 64), generator=g).to(DT[dtype]).cuda()
    assert attend_check(q, c, dtype) == 0


@pytest.mark.parametrize("dtype, new", [("bf16", 1), ("fp32", 1), ("bf16", 5), ("fp32", 5)])
@pytest.mark.parametrize("every", [1000, 37, 5])
def test_attend_short_among_long(dtype, new, every):
    """Sequences whose few tokens cost less than their own start beside ones that are split: shares that end
    before a sequence's first token, or hold nothing at all."""
    g = torch.Generator().manual_seed(every)
    lens = [int(x) for x in torch.randint(0, 6, (220,), generator=g)]
    lens[::every] = [600 - 7 * i for i in range(len(lens[::every]))]
    c = make_cache(lens, 2, 128, 32, seed=every)
    q = torch.randn((220, new, 8, 128), generator=g).to(DT[dtype]).cuda()
    assert attend_check(q, c, dtype) == 0


@pytest.mark.parametrize("dtype, new", [("bf16", 1), ("fp32", 1), ("bf16", 9)])
@pytest.mark.parametrize("n", [257, 2049])
def test_attend_more_sequences_than_are_summed_at_once(dtype, new, n):
    """Several sequences to each of the layout's partial sums, and more lengths than shared memory holds;
    long sequences at the first, the last and places between."""
    g = torch.Generator().manual_seed(n)
    lens = [int(x) for x in torch.randint(0, 12, (n,), generator=g)]
    for i in (0, 100, n - 2, n - 1):
        lens[i] = 600 - i % 7
    c = make_cache(lens, 1, 128, 16, seed=n)
    q = torch.randn((n, new, 2, 128), generator=g).to(DT[dtype]).cuda()
    assert attend_check(q, c, dtype) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attend_long_split(dtype):
    """A sequence long enough to be split over blocks beside short ones, at several tokens a row: equal
    to the float64 softmax of the same cache, computed on the device."""
    lens, hk, hq, d, p, new = [40000, 3, 9001, 0, 700], 2, 8, 128, 64, 3
    c = make_cache(lens, hk, d, p, seed=77)
    q = torch.randn((5, new, hq, d), generator=torch.Generator().manual_seed(6)).to(DT[dtype]).cuda()
    o, lse = pkg.cache_attend(q, *c, want_lse=True)
    for n, length in enumerate(lens):
        if length == 0:
            assert torch.all(o[n] == 0) and torch.all(torch.isneginf(lse[n]))
            continue
        pages = c[4][n, :-(-length // p)].long()
        k, v = ((x[pages].double() * s[pages].double()[..., None, None]).transpose(0, 1).reshape(hk, -1, d)[:, :length]
                for x, s in ((c[0], c[2]), (c[1], c[3])))
        s = torch.einsum("thgd,hld->thgl", q[n].double().view(new, hk, hq // hk, d), k) / math.sqrt(d)
        ahead = torch.arange(length, device="cuda")[None] - torch.arange(new, device="cuda")[:, None] > length - new
        s = s.masked_fill(ahead[:, None, None], -math.inf)
        w = torch.softmax(s, -1)
        want, mean_v = (torch.einsum("thgl,hld->thgd", w, x).reshape(new, hq, d) for x in (v, v.abs()))
        # |scale sum q k| of these inputs stays below 64: 2 * 132 * 2^-24 * 64 + 2^-18 < 2^-9.8 relative
        rel = 2 * (2.0 ** -9.8 + WEIGHT[dtype])
        bound = rel * mean_v + U[dtype] * want.abs() + (2.0 ** -14 * mean_v if dtype == "bf16" else 0.0)
        seen = (torch.arange(new, device="cuda") + length - new >= 0)
        assert torch.all(((o[n].double() - want).abs() <= bound)[seen])
        assert torch.all((lse[n].double() - torch.logsumexp(s, -1).view(new, hq)).abs()[seen] <= 2.0 ** -9.8)


@pytest.mark.parametrize("p, d, hq, new", [(64, 128, 8, 1), (16, 64, 4, 1), (64, 128, 8, 4), (32, 64, 8, 7), (16, 128, 2, 1)])
def test_attend_long_same_answer_each_time(p, d, hq, new):
    """Blocks that go round the ring of stages many times: forty calls over caches of 200000 tokens, in
    turn, give what the first ones gave."""
    cs = [make_cache([200000 - 77 * i, 1000], 1, d, p, seed=50 + i) for i in range(2)]
    q = torch.randn((2, new, hq, d), device="cuda").bfloat16()
    first = [pkg.cache_attend(q, *c, want_lse=True) for c in cs]
    for i in range(40):
        o, lse = pkg.cache_attend(q, *cs[i % 2], want_lse=True)
        assert torch.equal(o, first[i % 2][0]) and torch.equal(lse, first[i % 2][1])
    pages = cs[0][4][0, :-(-200000 // p)].long()
    k, v = ((x[pages].double() * s[pages].double()[..., None, None]).reshape(-1, d)[:200000]
            for x, s in ((cs[0][0], cs[0][2]), (cs[0][1], cs[0][3])))
    s = (q[0, -1].double() @ k.T) / math.sqrt(d)
    w = torch.softmax(s, -1)
    # as in test_attend_long_split; the scores of these inputs stay below 64
    bound = (2 * (2.0 ** -9.8 + WEIGHT["bf16"]) + 2.0 ** -14) * (w @ v.abs()) + U["bf16"] * (w @ v).abs()
    assert torch.all((first[0][0][0, -1].double() - w @ v).abs() <= bound)


def test_attend_same_answer_each_time():
    c = make_cache([5000, 17, 900, 2600], 2, 128, 32, seed=3)
    q = torch.randn((4, 2, 16, 128), device="cuda").bfloat16()
    first = pkg.cache_attend(q, *c, want_lse=True)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda").fill_(0xff)     # a workspace full of NaN
    for _ in range(5):
        again = pkg.cache_attend(q, *c, want_lse=True, workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype, layout", [("bf16", "half"), ("fp32", "interleaved")])
def test_prompt_decode_and_verification(dtype, layout):
    """A softmax-attention layer in serving: prompts rotated and appended (packed), three decode steps, a
    verification of four tokens of which two are taken back, one more decode step.  Each call is held
    to the 64-bit one on the call's own inputs."""
    hq, hk, d, p = 8, 2, 128, 16
    prompts = [37, 1, 90, 16]
    n = len(prompts)
    c = make_cache([x + 12 for x in prompts], hk, d, p, seed=41)
    freq, amp = pkg.rope_frequencies(32, 6e6, scaling="yarn", factor=2.0, original_context=131072, device="cuda")
    kw = dict(amplitude=amp, layout=layout)
    g = torch.Generator().manual_seed(17)

    def step(count_each, lens, packed):
        total = sum(count_each)
        qkv = torch.randn((total, hq + 2 * hk, d), generator=g).to(DT[dtype]).cuda()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        pos = torch.cat([torch.arange(x - m, x) for x, m in zip(lens, count_each)]).to(torch.int32).cuda()
        qr, kr = pkg.rope(q, k, pos, freq, **kw)
        rope_check(q, qr, pos, freq, amp, layout, False, dtype)
        rope_check(k, kr, pos, freq, amp, layout, False, dtype)
        c[5].copy_(torch.tensor(lens, dtype=torch.int32))
        if packed:
            cu = torch.tensor(np.concatenate([[0], np.cumsum(count_each)]), dtype=torch.int32, device="cuda")
            assert append_check(kr, v, c, count_each, cu_seqlens=cu) == 0
            return
        m = count_each[0]
        assert append_check(kr.view(n, m, hk, d), v.unflatten(0, (n, m)), c, count_each) == 0
        assert attend_check(qr.view(n, m, hq, d), c, dtype) == 0

    lens = list(prompts)
    step(prompts, lens, True)
    for _ in range(3):
        lens = [x + 1 for x in lens]
        step([1] * n, lens, False)
    lens = [x + 4 for x in lens]
    step([4] * n, lens, False)
    lens = [x - 2 + 1 for x in lens]             # two of the four kept, then one new token over the third
    step([1] * n, lens, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_captured_decode_step(dtype):
    """Rotation, append and attention captured into a graph and replayed on new inputs and lengths equal
    the calls made one by one; two graphs that share one workspace, replayed in turn, as well."""
    hq, hk, d, p, n = 8, 2, 64, 16, 3
    start = [30, 1, 5]
    c = make_cache([x + 40 for x in start], hk, d, p, seed=14)
    eager = [x.clone() for x in c]
    freq, _ = pkg.rope_frequencies(32, device="cuda")
    qkv = torch.zeros((n, 1, hq + 2 * hk, d), dtype=DT[dtype], device="cuda")
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def one(cache, **kw):
        q, k = pkg.rope(qkv[:, :, :hq], qkv[:, :, hq:hq + hk], pos, freq)
        pkg.cache_append(k, qkv[:, :, hq + hk:], *cache, status=status)
        return pkg.cache_attend(q, *cache, want_lse=True, status=status, **kw)

    c[5].copy_(torch.tensor(start, dtype=torch.int32))
    pos.copy_(c[5] - 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        one([x.clone() for x in c], workspace=ws)
    torch.cuda.current_stream().wait_stream(stream)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = one(c, workspace=ws)
        graphs.append((graph, out))
    for i in range(6):
        lens = torch.tensor([x + 6 * i for x in start], dtype=torch.int32, device="cuda")
        qkv.copy_(torch.randn(qkv.shape, device="cuda"))
        c[5].copy_(lens)
        eager[5].copy_(lens)
        pos.copy_(lens - 1)
        graph, out = graphs[i % 2]
        graph.replay()
        want = one(eager)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        for a, b in zip(c[:4], eager[:4]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del graphs


def test_side_stream():
    """Calls run on torch's current stream: a chain on a side stream, with nothing waited for between."""
    c = make_cache([300, 200], 2, 128, 64, seed=1)
    q = torch.randn((2, 1, 8, 128), device="cuda").bfloat16()
    k = torch.randn((2, 1, 2, 128), device="cuda").bfloat16()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn((4096, 4096), device="cuda")
        for _ in range(4):
            big = big @ big                       # the calls below queue behind this
        k2 = k * 2
        pkg.cache_append(k2, k2, *c)
        o = pkg.cache_attend(q, *c)
    s.synchronize()
    want = pkg.cache_attend(q, *c)
    assert torch.equal(o, want)


def test_two_attends_at_once():
    """Two calls on two streams with a workspace each."""
    cs = [make_cache([20000, 11], 1, 128, 64, seed=s) for s in (1, 2)]
    qs = [torch.randn((2, 1, 4, 128), device="cuda").bfloat16() for _ in cs]
    want = [pkg.cache_attend(q, *c) for q, c in zip(qs, cs)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(pkg.cache_attend(qs[i], *cs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


# ---------------------------------------------------------------- failure detection

@pytest.mark.parametrize("lens, columns, new", [([600, 40], None, 1), ([300, 100], 5, 1), ([600, 40], None, 9),
                                                ([100, 128], 2, 5)])
def test_attend_waits_expire_then_recover(lens, columns, new):
    """With KDA_FLAG_TEST_EXPIRE_WAITS every bounded wait of the call gives up at its first check: the
    status word reports it, nothing faults, and the next ordinary call on the same workspace is right.
    Split items (the first case) and whole ones."""
    c = make_cache(lens, 2, 128, 64, seed=6, columns=columns)
    q = torch.randn((2, new, 8, 128), device="cuda").bfloat16()
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkg.cache_attend(q, *c, workspace=ws, status=word, flags=kda.KDA_FLAG_TEST_EXPIRE_WAITS)
    torch.cuda.synchronize()
    assert int(word) == A.KDA_STATUS_TIMEOUT_ATTEND
    assert kda.device_status(word) == kda.KDA_ERR_TIMEOUT
    assert attend_check(q, c, "bf16", workspace=ws) == 0
