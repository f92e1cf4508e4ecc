"""Host-side checks of rotary positions, the cache append and the cache attention: refused before
any launch, so no GPU is needed.  And the rotary frequencies, which are a host call."""

import ctypes
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_70_b200 as pkg
from gated_delta_rule_70_b200 import attention as A
from gated_delta_rule_70_b200 import build, kda
from tests import attention_ref as ref

INVALID, UNSUPPORTED, WORKSPACE = (kda.KDA_ERR_INVALID_ARGUMENT, kda.KDA_ERR_UNSUPPORTED,
                                   kda.KDA_ERR_WORKSPACE)
P256 = 256      # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return kda.load_library()


# ---------------------------------------------------------------- the reference's own 8-bit format

def test_reference_e4m3_against_torch():
    x = np.concatenate([np.linspace(-500, 500, 40001), np.ldexp(np.linspace(-2, 2, 4001), -7),
                        [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -10, 464.0, np.nan]]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_encode(x), want)
    codes = np.arange(256, dtype=np.uint8)
    values = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_decode(codes), values, equal_nan=True)


# ---------------------------------------------------------------- frequencies

def test_frequencies_unscaled_linear_ntk():
    f, amp = pkg.rope_frequencies(64, 10000.0)
    want = 10000.0 ** (-2.0 * np.arange(32) / 64)
    # one pow and one product in fp64: a few units in the last place
    assert np.allclose(f.numpy(), want, rtol=8 * 2.0 ** -53, atol=0) and amp == 1.0
    g, amp = pkg.rope_frequencies(64, 10000.0, scaling="linear", factor=4.0)
    assert np.allclose(g.numpy(), want / 4, rtol=8 * 2.0 ** -53, atol=0) and amp == 1.0
    h, _ = pkg.rope_frequencies(64, 10000.0, scaling="ntk", factor=4.0)
    # the rule's own property: the first pair turns as before, the last one factor times slower
    assert h[0] == 1.0 and abs(h[-1] * 4 / want[-1] - 1) < 1e-12


def test_frequencies_yarn():
    rot, base, factor, ctx = 32, 6e6, 2.0, 131072.0
    f, amp = pkg.rope_frequencies(rot, base, scaling="yarn", factor=factor, original_context=ctx)
    plain = base ** (-2.0 * np.arange(rot // 2) / rot)
    turns = ctx * plain / (2 * math.pi)
    f = f.numpy()
    assert abs(amp - (0.1 * math.log(2) + 1)) < 2.0 ** -23
    # pairs that turn often keep their frequency, those that hardly turn are interpolated
    assert np.allclose(f[turns > 32 * 3], plain[turns > 32 * 3], rtol=1e-12)
    assert np.allclose(f[turns < 1 / 3], plain[turns < 1 / 3] / factor, rtol=1e-12)
    assert np.all((f <= plain * (1 + 1e-12)) & (f >= plain / factor * (1 - 1e-12)))
    assert np.all(np.diff(f) < 0)
    same, amp = pkg.rope_frequencies(rot, base, scaling="yarn", factor=1.0, original_context=ctx)
    assert np.allclose(same.numpy(), plain, rtol=1e-12) and amp == 1.0


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=258), dict(base=1.0),
                                dict(base=float("nan")), dict(scaling="linear", factor=0.5),
                                dict(scaling="ntk", factor=2.0, rot_dim=2),
                                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=float("inf"),
                                                                       original_context=100.0),
                                dict(scaling="yarn", factor=2.0, original_context=100.0, beta_fast=1.0)])
def test_frequencies_refuse(lib, kw):
    with pytest.raises(kda.KdaError) as e:
        pkg.rope_frequencies(**{"rot_dim": 64, **kw})
    assert e.value.status == INVALID


def test_frequencies_unknown_rule():
    with pytest.raises(ValueError):
        pkg.rope_frequencies(64, scaling="cubic")


# ---------------------------------------------------------------- kda_rope

def _rope_args(**kw):
    a = dict(num_tokens=4, q_heads=2, k_heads=1, head_dim=64, rot_dim=64, layout=0, inverse=0, io_dtype=0,
             amplitude=1.0, q=P256, k=P256, q_out=P256, k_out=P256, q_stride=128, k_stride=64,
             q_out_stride=128, k_out_stride=64, positions=P256, frequencies=P256)
    a.update(kw)
    return A.RopeArgs(*[a[n] for n, _ in A.RopeArgs._fields_])


@pytest.mark.parametrize("kw, want", [
    (dict(io_dtype=2), INVALID), (dict(num_tokens=-1), INVALID), (dict(layout=2), INVALID),
    (dict(q_heads=0), INVALID), (dict(k_heads=-1), INVALID), (dict(rot_dim=66), INVALID),
    (dict(rot_dim=63), INVALID), (dict(rot_dim=0), INVALID), (dict(amplitude=float("nan")), INVALID),
    (dict(head_dim=60, rot_dim=60), UNSUPPORTED), (dict(head_dim=264), UNSUPPORTED),
    (dict(q_heads=257, q_stride=1 << 20, q_out_stride=1 << 20), UNSUPPORTED),
    (dict(num_tokens=1 << 31), UNSUPPORTED), (dict(q_stride=120), INVALID), (dict(q_stride=132), INVALID),
    (dict(k_out_stride=56), INVALID), (dict(q_out_stride=256), INVALID), (dict(q=None), INVALID),
    (dict(q=P256 + 8), INVALID), (dict(k=None), INVALID), (dict(k_out=P256 + 2), INVALID),
    (dict(positions=None), INVALID), (dict(positions=P256 + 2), INVALID), (dict(frequencies=P256 + 4), INVALID),
])
def test_rope_refuses(lib, kw, want):
    assert lib.kda_rope(ctypes.byref(_rope_args(**kw)), None) == want


def test_rope_nothing_to_do(lib):
    assert lib.kda_rope(None, None) == INVALID
    assert lib.kda_rope(ctypes.byref(_rope_args(num_tokens=0, q=None, k=None)), None) == kda.KDA_OK


# ---------------------------------------------------------------- the cache

def _cache(**kw):
    c = dict(num_seqs=2, num_kv_heads=2, head_dim=128, page_tokens=64, num_pages=8, max_pages=4, k_cache=P256,
             v_cache=P256, k_scale=P256, v_scale=P256, block_table=P256, seq_lens=P256)
    c.update(kw)
    return A.Cache(*[c[n] for n, _ in A.Cache._fields_])


def _append_args(**kw):
    a = dict(k=P256, v=P256, k_stride=256, v_stride=256, num_new=3, io_dtype=0, cu_seqlens=None, status=None)
    a.update(kw)
    return A.CacheAppendArgs(*[a[n] for n, _ in A.CacheAppendArgs._fields_])


def _attend_args(**kw):
    a = dict(q=P256, q_stride=1024, num_new=1, num_heads=8, io_dtype=0, flags=0, scale=1.0, o=P256, lse=None,
             status=None)
    a.update(kw)
    return A.CacheAttendArgs(*[a[n] for n, _ in A.CacheAttendArgs._fields_])


CACHE_BAD = [
    (dict(num_seqs=-1), INVALID), (dict(num_kv_heads=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(page_tokens=48), UNSUPPORTED),
    (dict(page_tokens=256), UNSUPPORTED), (dict(num_pages=1 << 24), UNSUPPORTED),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(k_cache=None), INVALID), (dict(v_cache=P256 + 4), INVALID),
    (dict(k_scale=None), INVALID), (dict(v_scale=P256 + 1), INVALID), (dict(block_table=None), INVALID),
    (dict(seq_lens=None), INVALID),
]


@pytest.mark.parametrize("kw, want", CACHE_BAD + [(dict(num_kv_heads=65), UNSUPPORTED)])
def test_append_refuses_cache(lib, kw, want):
    a = _append_args(k_stride=1 << 20, v_stride=1 << 20)
    assert lib.kda_cache_append(ctypes.byref(_cache(**kw)), ctypes.byref(a), None) == want


@pytest.mark.parametrize("kw, want", [
    (dict(io_dtype=5), INVALID), (dict(num_new=-1), INVALID), (dict(k_stride=248), INVALID),
    (dict(v_stride=260), INVALID), (dict(k=None), INVALID), (dict(v=P256 + 2), INVALID),
    (dict(cu_seqlens=P256 + 2), INVALID), (dict(status=P256 + 2), INVALID),
    (dict(num_new=1 << 30), UNSUPPORTED), (dict(num_new=(1 << 31) - 1, cu_seqlens=P256), UNSUPPORTED),
])
def test_append_refuses(lib, kw, want):
    assert lib.kda_cache_append(ctypes.byref(_cache()), ctypes.byref(_append_args(**kw)), None) == want


def test_append_nothing_to_do(lib):
    assert lib.kda_cache_append(ctypes.byref(_cache()), ctypes.byref(_append_args(num_new=0, k=None)), None) == kda.KDA_OK
    assert lib.kda_cache_append(ctypes.byref(_cache(num_seqs=0)), ctypes.byref(_append_args()), None) == kda.KDA_OK
    assert lib.kda_cache_append(None, ctypes.byref(_append_args()), None) == INVALID
    assert lib.kda_cache_append(ctypes.byref(_cache()), None, None) == INVALID


def _attend(lib, c, a, ws=P256 * 16, ws_bytes=1 << 40):
    return lib.kda_cache_attend(ctypes.byref(c), ctypes.byref(a), ws, ws_bytes, None)


@pytest.mark.parametrize("kw, want", CACHE_BAD)
def test_attend_refuses_cache(lib, kw, want):
    assert _attend(lib, _cache(**kw), _attend_args()) == want


@pytest.mark.parametrize("kw, want", [
    (dict(io_dtype=-1), INVALID), (dict(num_new=0), INVALID), (dict(num_heads=0), INVALID),
    (dict(num_heads=7), INVALID), (dict(scale=float("inf")), INVALID), (dict(flags=1), INVALID),
    (dict(num_heads=258, q_stride=1 << 20), UNSUPPORTED), (dict(num_new=1 << 28), UNSUPPORTED),
    (dict(q_stride=1016), INVALID), (dict(q_stride=1028), INVALID), (dict(q=None), INVALID),
    (dict(q=P256 + 8), INVALID), (dict(o=None), INVALID), (dict(lse=P256 + 2), INVALID),
    (dict(status=P256 + 1), INVALID),
])
def test_attend_refuses(lib, kw, want):
    assert _attend(lib, _cache(), _attend_args(**kw)) == want


def test_attend_workspace(lib):
    c, a = _cache(max_pages=40), _attend_args()
    need = A.cache_attend_workspace_size(c, a)
    assert need > 0
    assert _attend(lib, c, a, ws=None) == WORKSPACE
    assert _attend(lib, c, a, ws=P256 + 16) == WORKSPACE
    assert _attend(lib, c, a, ws_bytes=need - 1) == WORKSPACE
    assert A.cache_attend_workspace_size(_cache(head_dim=80), a) == 0
    assert _attend(lib, _cache(num_seqs=0), a, ws=None) == kda.KDA_OK


@pytest.mark.parametrize("new, dtype, columns", [(1, 0, 6), (4, 0, 6), (5, 0, 2), (1, 1, 6), (5, 1, 3), (9, 1, 1)])
def test_attend_needs_no_workspace_for_short_tables(lib, new, dtype, columns):
    """Up to as many tiles as a block takes at a time (12 of 32 tokens; 6 and 3 with more rows in fp32; one of 128
    for many rows in bf16) an item is never split; with one page more it may be."""
    a = _attend_args(num_new=new, io_dtype=dtype)
    assert A.cache_attend_workspace_size(_cache(max_pages=columns), a) == 0
    assert A.cache_attend_workspace_size(_cache(max_pages=columns + 1), a) > 0


# ---------------------------------------------------------------- the binding's own checks

def _cpu_cache(n=2, hk=2, d=64, p=16, pages=8, columns=4):
    f8 = lambda: torch.zeros((pages, hk, p, d), dtype=torch.float8_e4m3fn)  # noqa: E731
    sc = lambda: torch.ones((pages, hk))  # noqa: E731
    return [f8(), f8(), sc(), sc(), torch.zeros((n, columns), dtype=torch.int32), torch.zeros(n, dtype=torch.int32)]


def test_binding_refuses(lib):
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16)
    c = _cpu_cache()
    with pytest.raises(ValueError, match="CUDA"):
        pkg.cache_attend(q, *c)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.cache_append(k, k, *c)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rope(q, k, torch.zeros(2, dtype=torch.int32), torch.ones(32, dtype=torch.float64))
    for i, bad in ((0, c[0].view(torch.uint8)), (1, c[1][:4]), (2, c[2].double()), (3, c[3][:, :1]),
                   (4, c[4].long()), (4, c[4][:1]), (5, c[5][:1])):
        with pytest.raises(ValueError):
            pkg.cache_attend(q, *[bad if j == i else x for j, x in enumerate(c)])
    with pytest.raises(ValueError):
        pkg.cache_attend(q.half(), *c)
    with pytest.raises(ValueError):
        pkg.cache_attend(q[:, :0], *c)
    with pytest.raises(ValueError):
        pkg.cache_attend(q, *c, out=torch.zeros((2, 1, 4, 64)))
    with pytest.raises(ValueError):
        pkg.cache_attend(q, *c, lse=torch.zeros((2, 4)))
    with pytest.raises(ValueError):
        pkg.cache_append(k, k[:1], *c)
    with pytest.raises(ValueError):
        pkg.cache_append(torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros((3, 2, 64), dtype=torch.bfloat16), *c)
    with pytest.raises(ValueError):
        pkg.cache_append(k, k, *c, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    pos, f = torch.zeros(2, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:1]), dict(frequencies=f.float()),
                dict(k=k[:1]), dict(layout="pairs"), dict(q=q.transpose(2, 3))):
        with pytest.raises(ValueError):
            pkg.rope(**{**dict(q=q, k=k, positions=pos, frequencies=f), **bad})


def test_token_strides():
    dev = torch.device("cpu")
    fused = torch.zeros((3, 5, 8, 64))
    take = lambda t, h: A._tokens(t, "x", torch.float32, dev, h, 64)  # noqa: E731
    assert take(fused[:, :, :4], 4) == (15, 512)
    assert take(fused[:, :, 4:6], 2) == (15, 512)
    assert take(fused, 8) == (15, 512)
    assert take(fused[:1, :1], 8) == (1, 512)
    assert take(fused[:, :1, :2], 2) == (3, 5 * 512)
    assert take(fused[:0], 8)[0] == 0
    for bad, h in ((fused[:, :4], 8), (fused[..., ::2], 8), (fused.transpose(0, 1), 8), (fused.transpose(1, 2), 5),
                   (fused[:, :1].expand(3, 5, 8, 64), 8)):
        with pytest.raises(ValueError):
            take(bad, h)


# ---------------------------------------------------------------- sizes at the end of 32 bits

@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_tables_leave_room_for_the_last_tiles(lib, page):
    """A row of the table as long as 2^31 - 4096 tokens is accepted, a page more is not: the kernels count token
    positions in 32 bits, those of a batch of tiles behind the last token among them."""
    most = (2 ** 31 - 4096) // page
    for pages, ok in ((most, True), (most + 1, False), (2 ** 31 // page - 1, False)):
        c, a = _cache(page_tokens=page, max_pages=pages), _attend_args()
        # (accepted: the call goes on to ask for its workspace)
        assert _attend(lib, c, a, ws=None) == (WORKSPACE if ok else UNSUPPORTED)
        assert (A.cache_attend_workspace_size(c, a) > 0) == ok
        n = _append_args(num_new=0)
        assert lib.kda_cache_append(ctypes.byref(c), ctypes.byref(n), None) == (kda.KDA_OK if ok else UNSUPPORTED)


@pytest.mark.parametrize("seqs, new, cu", [(1 << 24, 1, None), (1 << 23, 1, P256), (1, (1 << 31) - 200, None),
                                           (1, (1 << 31) - 200, P256)])
def test_append_refuses_more_units_than_32_bits_count(lib, seqs, new, cu):
    """(page, head, tensor) units of a call: the kernel counts them in 32 bits, so a call that may have more is refused
    before anything is enqueued."""
    c = _cache(num_seqs=seqs, num_kv_heads=64, num_pages=1, page_tokens=16)
    a = _append_args(num_new=new, cu_seqlens=cu, k_stride=1 << 20, v_stride=1 << 20, status=P256 * 4)
    assert lib.kda_cache_append(ctypes.byref(c), ctypes.byref(a), None) == UNSUPPORTED


@pytest.mark.parametrize("d, new, dtype, rows", [(64, 4, 0, 16), (64, 5, 0, 32), (64, 8, 0, 32), (64, 9, 0, 128),
                                                 (128, 4, 0, 16), (128, 5, 0, 128), (64, 5, 1, 32), (64, 9, 1, 64)])
def test_attend_rows_of_an_item(lib, d, new, dtype, rows):
    """The workspace holds for each of 148 blocks a record and two parts of the item's rows: outputs, maximum and sum.
    With 4 query heads to a key / value head, bf16 rows go up to 32 (heads of 64) or 16 before items have 128."""
    a = _attend_args(num_new=new, io_dtype=dtype)
    want = 148 * 16 + 148 * 2 * (rows * d + 2 * rows) * 4
    assert A.cache_attend_workspace_size(_cache(head_dim=d, max_pages=100), a) == -(-want // 256) * 256
