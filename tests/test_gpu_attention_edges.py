"""The softmax-attention layer's operators on the GPU where they can go wrong beyond
tests/test_gpu_attention.py: rows of which one token takes almost all the weight, page scales far
apart, NaN that a row does see, batches of many tokens, other streams.

u is a type's half step (eps / 2), as there.
"""

import math

import pytest
import torch

import gated_delta_rule_70_b200 as pkg
from gated_delta_rule_70_b200 import attention as A
from gated_delta_rule_70_b200 import kda
from tests.test_gpu_attention import DT, U, WEIGHT, attend_check, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(2026)


# ---------------------------------------------------------------- the range of a weight

GAPS = (8.0, 12.0, 15.0, 16.25, 17.0, 18.0, 0.0, -3.0)


def sum_tolerance(length):
    """Relative error of the sum of a row's weights: the exponents' arguments (at most 26 + 8 + 15 in powers of two)
    take a few fp32 roundings, 2^-17; the exponential 2^-22; joins below 2^-18; and a thread adds 16 tokens' share at a
    time to its fp32 sum: at most length / 16 additions, each of which may round by 2^-24 of the sum.  (With 200000
    tokens of 2^-24.5 beside a first one of 1, pairs of 2^-23.5 all round up to 2^-23: 1041 times 2^-24.8 in one of
    twelve warps' eight lanes, 2^-14.8, so the last term is not an idle one.)"""
    return 2.0 ** -16 + -(-length // 16) * 2.0 ** -24


def weight_tolerance(dtype, length):
    """Relative error of sum w v / sum w where all v have one sign, from roundings that are all relative: the sum's
    own; the numerator's, where a tensor-core sum may truncate, 2^-23 of it for each 16 tokens that one lane takes (all
    of the sequence's at most; fp32: twice, but of a third of them); and twice the rounding of a weight."""
    return 2 * sum_tolerance(length) + 2 * -(-length // 16) * 2.0 ** -23 / (1 if dtype == "bf16" else 3) + 2 * WEIGHT[dtype]


@pytest.mark.parametrize("n, seqs", [(600, 1), (600, 160), (20000, 1), (20000, 128), (200000, 128)])
@pytest.mark.parametrize("dtype, new, d", [("bf16", 1, 128), ("bf16", 2, 64), ("bf16", 3, 128), ("bf16", 3, 64),
                                           ("fp32", 1, 64), ("fp32", 2, 128), ("fp32", 3, 128), ("fp32", 5, 64)])
def test_attend_far_below_one_large_weight(dtype, new, d, n, seqs):
    """The first token of a long sequence takes almost all of the weight with a value of 0, the others share what is
    left, up to 18 nats below it each: the output is theirs alone, and keeps its relative precision.  One sequence
    split over the blocks, and many (of the same pages) that are hardly split, so one running reference serves all."""
    p, hq = 64, len(GAPS)
    pages = -(-n // p)
    g = torch.Generator().manual_seed(n)
    k = torch.zeros((pages, 1, p, d))
    k[0, 0, 0, 0] = 1.0
    v = torch.rand((pages, 1, p, d), generator=g) + 0.5
    v[0, 0, 0] = 0.0
    c = [x.to(torch.float8_e4m3fn).cuda() for x in (k, v)]
    c += [torch.ones((pages, 1), device="cuda"), torch.full((pages, 1), 2.0 ** -7, device="cuda")]
    c += [torch.randperm(pages, generator=g).int(), torch.full((seqs,), n, dtype=torch.int32, device="cuda")]
    at = c[4].long()
    for i in range(4):                            # (tokens keep their order in the sequence)
        x = torch.empty_like(c[i].view(torch.uint8) if i < 2 else c[i])
        x[at.cuda()] = c[i].view(torch.uint8) if i < 2 else c[i]
        c[i] = x.view(torch.float8_e4m3fn) if i < 2 else x
    c[4] = c[4].cuda().expand(seqs, pages).contiguous()
    q = torch.randn((seqs, new, hq, d), generator=g).to(DT[dtype])
    q[..., 0] = torch.tensor(GAPS).to(DT[dtype])
    o, lse = pkg.cache_attend(q.cuda(), *c, scale=1.0, want_lse=True)

    values = v.to(torch.float8_e4m3fn).double().view(-1, d) * 2.0 ** -7
    gaps = q[0, 0, :, 0].double()
    for t in range(new):
        seen = n - new + t + 1
        total = torch.log(torch.exp(gaps) + (seen - 1))
        want = values[1:seen].sum(0)[None] / torch.exp(total)[:, None]
        tol = weight_tolerance(dtype, n) * want + U[dtype] * want
        assert torch.all(want > 0)
        off = (o[:, t].double().cpu() - want).abs()
        assert torch.all(off <= tol), float((off / want).max())
        assert torch.all((lse[:, t].double().cpu() - total).abs() <= sum_tolerance(n) + 2.0 ** -22 * total.abs())


@pytest.mark.parametrize("dtype, new, d", [("bf16", 1, 128), ("bf16", 2, 64), ("bf16", 3, 128), ("bf16", 3, 64),
                                           ("fp32", 1, 128), ("fp32", 2, 64), ("fp32", 3, 64), ("fp32", 5, 128)])
def test_attend_one_page_of_large_values(dtype, new, d):
    """One value of 2^20 times the others' size in one channel: its page's scale is as much larger, and the page's other
    values are zeros.  The other channels keep their relative precision."""
    n, p, hq = 500, 32, 8
    pages = -(-n // p)
    v = torch.rand((pages, 1, p, d), generator=torch.Generator().manual_seed(d)) + 0.5
    v[3] = 0.0
    v[3, 0, 5, 7] = 256.0
    k = torch.randn((pages, 1, p, d), generator=torch.Generator().manual_seed(n)) * 64
    c = [k.to(torch.float8_e4m3fn).cuda(), v.to(torch.float8_e4m3fn).cuda(),
         torch.full((pages, 1), 2.0 ** -8, device="cuda"), torch.full((pages, 1), 2.0 ** -7, device="cuda"),
         torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.full((1,), n, dtype=torch.int32, device="cuda")]
    c[3][3] = 2.0 ** 13
    q = torch.randn((1, new, hq, d), device="cuda").to(DT[dtype])
    o = pkg.cache_attend(q, *c)
    keys, values = ((x.double() * s[:, :, None, None].double()).view(-1, d) for x, s in ((c[0], c[2]), (c[1], c[3])))
    for t in range(new):
        seen = n - new + t + 1
        score = q[0, t].double() @ keys[:seen].T / math.sqrt(d)
        want = torch.softmax(score, -1) @ values[:seen]
        # a score's d products in fp32 beside the rest: these inputs' scale sum |q k| stays below 4
        tol = (2 * 2 * (d + 4) * 2.0 ** -24 * 4 + weight_tolerance(dtype, n) + U[dtype]) * want
        assert torch.all((o[0, t].double() - want).abs() <= tol)


@pytest.mark.parametrize("dtype, new, d", [("bf16", 1, 128), ("bf16", 2, 64), ("bf16", 3, 128), ("bf16", 3, 64),
                                           ("fp32", 1, 128), ("fp32", 2, 64), ("fp32", 3, 64), ("fp32", 5, 128)])
def test_attend_scores_beyond_the_digits_of_fp32(dtype, new, d):
    """Scores of +-2^10 to +-2^60, of which fp32 holds no fraction from 2^23 on: the tokens of the larger one share the
    row equally, and the lse is that score's (a few fp32 roundings off)."""
    n, p, hq = 700, 32, 8
    g = torch.Generator().manual_seed(d + new)
    side = torch.randint(0, 2, (n,), generator=g) * 2 - 1
    pages = -(-n // p)
    k = torch.zeros((pages * p, d))
    k[:n, 0] = side.float()
    v = torch.rand((pages * p, d), generator=g) + 0.5
    c = [x.view(pages, 1, p, d).to(torch.float8_e4m3fn).cuda() for x in (k, v)]
    c += [torch.ones((pages, 1), device="cuda"), torch.full((pages, 1), 2.0 ** -7, device="cuda"),
          torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.full((1,), n, dtype=torch.int32, device="cuda")]
    values = v.to(torch.float8_e4m3fn).double() * 2.0 ** -7
    for powers in ((10, 15, 19, 20, 21, 22, 23, 24), (25, 26, 27, 28, 29, 30, 40, 60)):
        size = torch.tensor([1.375 * 2.0 ** e * (-1) ** i for i, e in enumerate(powers)])
        q = torch.randn((1, new, hq, d), generator=g)
        q[..., 0] = size
        o, lse = pkg.cache_attend(q.to(DT[dtype]).cuda(), *c, scale=1.0, want_lse=True)
        for t in range(new):
            for h in range(hq):
                seen = n - new + t + 1
                mine = (side[:seen] * size[h] > 0).nonzero()[:, 0]
                want = values[mine].mean(0)
                tol = (weight_tolerance(dtype, n) + U[dtype]) * want
                assert torch.all((o[0, t, h].double().cpu() - want).abs() <= tol), (powers[h], t)
                assert abs(float(lse[0, t, h]) - float(size[h].abs()) - math.log(len(mine))) <= 2.0 ** -21 * float(size[h].abs())


@pytest.mark.parametrize("n", [5000, 60000])
@pytest.mark.parametrize("new, hq, d", [(1, 8, 128), (1, 5, 64), (2, 8, 128), (4, 8, 64), (4, 8, 128), (9, 8, 128)])
def test_attend_fp32_sums_do_not_drift(new, hq, d, n):
    """Equal weights and values of one sign in fp32, many sequences (of the same pages), so that a block takes nearly a
    whole one: the mean of the values.  Weights and their sum are exact here.  A thread adds up the share of at most
    length / 16 groups of tokens (a third or less of them: at least three warps take a row's tiles in turn); each
    addition rounds to nearest, by up to 2^-24 of the output, so without a drift the error is that of a random walk,
    eight times whose deviation is allowed.  Sums that are truncated end five to ten times further off."""
    p, seqs = 64, 160 if new < 9 else 20
    pages = -(-n // p)
    g = torch.Generator(device="cuda").manual_seed(n + d)
    v = (torch.rand((pages, 1, p, d), generator=g, device="cuda") + 0.5).to(torch.float8_e4m3fn)
    c = [torch.zeros_like(v), v, torch.ones((pages, 1), device="cuda"), torch.ones((pages, 1), device="cuda"),
         torch.arange(pages, dtype=torch.int32, device="cuda")[None].expand(seqs, pages).contiguous(),
         torch.full((seqs,), n, dtype=torch.int32, device="cuda")]
    o = pkg.cache_attend(torch.randn((seqs, new, hq, d), generator=g, device="cuda"), *c)
    values = v.double().view(-1, d)
    walk = 8 * math.sqrt(n / 16 / 3 / 3) * 2.0 ** -24
    for t in range(new):
        want = values[:n - new + t + 1].mean(0)
        assert torch.all((o[:, t].double() - want).abs() <= (walk + 2.0 ** -21) * want)


# ---------------------------------------------------------------- NaN that is seen

KINDS = [("bf16", 2, 128), ("bf16", 2, 64), ("bf16", 4, 64), ("bf16", 6, 64), ("bf16", 9, 128), ("bf16", 9, 64), ("fp32", 2, 64),
         ("fp32", 2, 128), ("fp32", 9, 128)]


@pytest.mark.parametrize("p", [16, 64])
@pytest.mark.parametrize("dtype, group, d", KINDS)
def test_attend_nan_value_scale(dtype, group, d, p):
    """A page whose value scale is NaN: rows that see one of its tokens are NaN in every channel, the others do not
    notice, and no lse does."""
    new, length = 4, 2 * p + 2                    # the last page: two tokens, which the last two rows see
    c = make_cache([length, 3 * p], 2, d, p, seed=d + group)
    q = torch.randn((2, new, 2 * group, d), device="cuda").to(DT[dtype])
    clean = pkg.cache_attend(q, *c, want_lse=True)
    keep = c[3].clone()
    last = int(c[4][0, 2])
    c[3][last, 1] = math.nan
    o, lse = pkg.cache_attend(q, *c, want_lse=True)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, 2:, group:] = True
    assert torch.equal(torch.isnan(o), hit)
    # (the page's scale changes the reference of the rows that see it, no more: two roundings of a few units)
    assert torch.equal(o[:, :2], clean[0][:, :2]) and torch.equal(o[1], clean[0][1])
    assert torch.all((lse - clean[1]).abs() <= 2.0 ** -16 + 2.0 ** -20 * clean[1].abs())
    c[3].copy_(keep)
    c[3][int(c[4][0, 0]), 0] = math.nan           # a page that every row of the first sequence sees whole
    o, lse = pkg.cache_attend(q, *c, want_lse=True)
    hit[:] = False
    hit[0, :, :group] = True
    assert torch.equal(torch.isnan(o), hit) and torch.equal(o[~hit], clean[0][~hit])
    assert torch.all((lse - clean[1]).abs() <= 2.0 ** -16 + 2.0 ** -20 * clean[1].abs())


@pytest.mark.parametrize("length", [20, 90, 700, 30000])
@pytest.mark.parametrize("dtype, group, d", KINDS)
def test_attend_nan_query(dtype, group, d, length):
    """A NaN in one query row: its output and its lse are NaN, whether the sequence is split over blocks or not, and
    no other row notices."""
    new = 4
    c = make_cache([length, 50], 2, d, 64, seed=length)
    q = torch.randn((2, new, 2 * group, d), device="cuda").to(DT[dtype])
    clean = pkg.cache_attend(q, *c, want_lse=True)
    q[0, 1, 1, 5] = math.nan
    o, lse = pkg.cache_attend(q, *c, want_lse=True)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 1, 1] = True
    assert torch.equal(torch.isnan(lse), hit)
    assert torch.equal(torch.isnan(o), hit[..., None].expand_as(o))
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("dtype, group, d", KINDS)
def test_attend_nan_keys_of_a_stretch(dtype, group, d):
    """A stretch of NaN keys as long as several blocks' shares: some parts of the row hold nothing but NaN."""
    c = make_cache([30000], 2, d, 64, seed=9)
    q = torch.randn((1, 4, 2 * group, d), device="cuda").to(DT[dtype])
    c[0].view(torch.uint8)[c[4][0, 100:300].long(), 0] = 0x7f
    o, lse = pkg.cache_attend(q, *c, want_lse=True)
    assert torch.isnan(o[:, :, :group]).all() and torch.isnan(lse[:, :, :group]).all()
    assert torch.isfinite(o[:, :, group:]).all() and torch.isfinite(lse[:, :, group:]).all()


@pytest.mark.parametrize("p", [16, 64, 128])
@pytest.mark.parametrize("new, hq, hk", [(17, 1, 1), (1, 24, 1), (5, 8, 2), (8, 4, 1), (4, 16, 2), (33, 2, 2), (11, 3, 1)])
def test_attend_17_to_33_rows_of_64_channels(new, hq, hk, p):
    """Where bf16 calls change over to the many-row kernel, at lengths around a tile's, a page's and a share's end."""
    lens = [new, new - 1, 0, 63, 64, 65, 130, 700, 511]
    c = make_cache(lens, hk, 64, p, seed=p + new)
    q = torch.randn((len(lens), new, hq, 64), device="cuda").bfloat16()
    assert attend_check(q, c, "bf16") == 0


# ---------------------------------------------------------------- rotary positions of many tokens

def rope64(x, pos, freq, amp, layout, inverse):
    """The rotation in 64 bits, and |a| + |b| of each rotated channel's pair (0 elsewhere)."""
    x, half = x.double(), freq.numel()
    angle = pos.double()[:, None] * freq[None] * (-1.0 if inverse else 1.0)
    cs, sn = (amp * angle.cos())[:, None], (amp * angle.sin())[:, None]
    ia, ib = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    a, b = x[..., ia], x[..., ib]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = a * cs - b * sn, b * cs + a * sn
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


@pytest.mark.parametrize("tokens", [4095, 4096, 4097, 80011])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hq, hk, d, layout, rot", [
    (3, 1, 64, "half", 64), (12, 4, 64, "interleaved", 64), (8, 1, 64, "half", 58), (8, 1, 64, "interleaved", 58),
    (16, 2, 128, "half", 32), (1, 0, 8, "interleaved", 2), (6, 2, 128, "interleaved", 128), (7, 0, 256, "half", 256),
    (5, 3, 40, "half", 2), (2, 1, 16, "half", 16),
])
def test_rope_many_tokens(dtype, tokens, hq, hk, d, layout, rot):
    """From 4096 tokens on heads and tokens are laid over a block's threads by another rule.  The bound is that of
    test_gpu_attention.py: positions stay below 2^20."""
    g = torch.Generator(device="cuda").manual_seed(tokens + rot)
    fused = torch.randn((tokens, hq + hk + 1, d), generator=g, device="cuda").to(DT[dtype])
    q, k = fused[:, :hq], fused[:, hq:hq + hk] if hk else None
    pos = torch.randint(-5, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    freq, _ = pkg.rope_frequencies(rot, 10000.0, device="cuda")
    out = pkg.rope(q, k, pos, freq, amplitude=1.25, layout=layout, inverse=tokens % 2 == 1)
    for x, y in zip((q, k), out):
        if x is None:
            continue
        want, size = rope64(x, pos, freq, 1.25, layout, tokens % 2 == 1)
        bound = 1.25 * size * 2.0 ** -21 + U[dtype] * want.abs() * (size > 0) + 1e-38
        assert torch.all((y.double() - want).abs() <= bound)
        assert torch.equal(y[..., rot:], x[..., rot:])
    rest = fused[:, hq + hk:].clone()
    pkg.rope(q, k, pos, freq, amplitude=1.25, layout=layout, inverse=tokens % 2 == 1, out=(q, k))
    assert torch.equal(q, out[0]) and (k is None or torch.equal(k, out[1]))
    assert torch.equal(fused[:, hq + hk:], rest)


# ---------------------------------------------------------------- streams

def test_side_stream_against_a_run_before():
    """A chain on a side stream whose input is written there, behind other work, after the calls are made: what it
    leaves is what the same chain left on the default stream before.  Calls on another stream would have read the
    input's earlier values."""
    c = make_cache([300, 200], 2, 128, 64, seed=1)
    q = torch.randn((2, 1, 8, 128), device="cuda").bfloat16()
    k = torch.randn((2, 1, 2, 128), device="cuda").bfloat16()
    other = [x.clone() for x in c]
    pkg.cache_append(k * 2, k * 4, *other)
    want = pkg.cache_attend(q, *other)
    k2, v2 = torch.full_like(k, 100.0), torch.full_like(k, -100.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn((8192, 8192), device="cuda")
        for _ in range(8):
            big = big @ big                       # the writes below queue behind this
        torch.mul(k, 2, out=k2)
        torch.mul(k, 4, out=v2)
        pkg.cache_append(k2, v2, *c)
        o = pkg.cache_attend(q, *c)
    s.synchronize()
    assert torch.equal(o, want)
    for a, b in zip(c[:2], other[:2]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(c[2], other[2]) and torch.equal(c[3], other[3])


def test_equal_inputs_give_equal_bits():
    """Each kind of call, repeated between other calls: the same codes of the outputs."""
    for dtype, new, group, d in (("bf16", 1, 8, 128), ("bf16", 4, 8, 128), ("fp32", 1, 1, 64), ("fp32", 4, 8, 64)):
        c = make_cache([4000 - 31 * i for i in range(40)], 2, d, 16, seed=new + d)
        q = torch.randn((40, new, 2 * group, d), device="cuda").to(DT[dtype])
        first = pkg.cache_attend(q, *c, want_lse=True)
        for _ in range(20):
            pkg.cache_attend(-q, *c)
            again = pkg.cache_attend(q, *c, want_lse=True)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


# ---------------------------------------------------------------- failure detection

@pytest.mark.parametrize("lens, columns", [([200000, 1000], None), ([5000] * 40, None), ([3, 300, 70], 6)])
@pytest.mark.parametrize("dtype, new, group, d, p", [("bf16", 1, 4, 128, 64), ("bf16", 1, 4, 64, 16), ("bf16", 2, 8, 128, 16),
                                                     ("fp32", 1, 4, 64, 16), ("fp32", 5, 8, 128, 32), ("bf16", 5, 8, 128, 16),
                                                     ("bf16", 5, 8, 64, 64), ("bf16", 3, 8, 64, 16)])
def test_attend_waits_run_out_with_work_in_flight(dtype, new, group, d, p, lens, columns):
    """With KDA_FLAG_TEST_EXPIRE_WAITS one reader of each block gives up before its first tile: the ring fills up
    behind it, and the others' waits run out in the middle of a turn, with copies and products under way.  The call
    ends soon (a drain that waited for the wrong phase would take 2^22 polls for each stage), reports the time-out,
    and the next call on the same workspace is right."""
    c = make_cache(lens, 2, d, p, seed=19, columns=None if columns is None else columns * 64 // p)
    q = torch.randn((len(lens), new, 2 * group, d), device="cuda").to(DT[dtype])
    want = pkg.cache_attend(q, *c, want_lse=True)
    ws = torch.full((1 << 25,), 0xff, dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    pkg.cache_attend(q, *c, workspace=ws, status=word, flags=kda.KDA_FLAG_TEST_EXPIRE_WAITS)
    end.record()
    torch.cuda.synchronize()
    assert int(word) == A.KDA_STATUS_TIMEOUT_ATTEND
    assert begin.elapsed_time(end) < 500
    o, lse = pkg.cache_attend(q, *c, want_lse=True, workspace=ws, status=word)
    assert int(word) == 0 and torch.equal(o, want[0]) and torch.equal(lse, want[1])
